/*
 * mta_ops.h -- the operators that make a mixed-precision step's gradients, for
 * AMD Instinct MI355X (gfx950), in the library of mta.h and under its
 * conventions: plain pointers and sizes, work enqueued on the caller's stream,
 * negative mta_status on failure with nothing enqueued, mta_last_error().
 *
 *   mta_ckpt_pack           activations kept for the backward pass in 8 bits
 *                           (a "checkpoint"), optionally with the activation
 *                           function's value written in the same pass
 *   mta_ckpt_unpack         the kept values back in 16 or 32 bits
 *   mta_ckpt_act_backward   an activation function's gradient from the
 *                           checkpoint of its input
 *   mta_ckpt_wgrad          a linear layer's weight and bias gradient from the
 *                           checkpoint of its input, written or added into the
 *                           gradient buffers that mta_clip_norm and mta_step
 *                           read
 *   mta_policy_loss         a clipped policy loss with a KL term straight from
 *                           the logits, optionally with its gradient times the
 *                           loss scale that mta_amp_* divides out again
 *   mta_policy_loss_backward  that gradient in a second call
 *
 * No call allocates, waits or keeps anything between calls, so all of them may
 * be captured into a HIP graph and calls on different streams are independent
 * as long as their buffers (workspaces included) are.  The same inputs give
 * the same bits on the same device: no result depends on the order of atomics.
 * Element types are those of mta_gtype (MTA_F32, MTA_BF16, MTA_F16).  Buffers
 * are aligned to their element size (checkpoint codes to 16 bytes); more
 * alignment is not required.  A buffer that is written overlaps no other
 * buffer of its call, except where an entry allows it (MTA_EINVAL).
 *
 * The checkpoint format.  A tensor x[rows, cols] is kept as codes and scales:
 *   codes   one byte (e4m3: 1 sign, 4 exponent, 3 mantissa bits, largest 448,
 *           0x7F / 0xFF NaN, no infinity) per element, rows of ldq =
 *           cols rounded up to 32 bytes, the padding codes 0;
 *   scales  one byte per 32 consecutive columns of a row, rows of ldq / 32
 *           bytes: the biased exponent k + 127 of a power of two.
 * The value kept is code * 2^k, where k is the smallest integer >= -117 with
 * max|x| <= 448 * 2^k over the block's finite elements, and the code is
 * x * 2^-k rounded to nearest-even.  Finite values are first clamped to the
 * largest 4-significant-bit value of x's type, 1.875*2^15 (MTA_F16) or
 * 1.875*2^127, so that no kept value overflows that type; NaN and infinities
 * are kept as NaN and leave the block's scale alone.  A kept value differs
 * from x by at most 2^-4 |x| or 2^(k-10), whichever is larger, and is exact
 * in float32 and bfloat16.
 */
#ifndef MTA_OPS_H
#define MTA_OPS_H

#include "mta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 1: the first version. */
#define MTA_OPS_VERSION 1

/* Columns that share one scale. */
#define MTA_CKPT_BLOCK 32

typedef enum {
  MTA_ACT_NONE = 0,
  MTA_ACT_RELU = 1,     /* x > 0 ? x : 0 */
  MTA_ACT_SILU = 2,     /* x / (1 + exp(-x)) */
  MTA_ACT_GELU = 3,     /* x/2 (1 + erf(x / sqrt 2)) */
  MTA_ACT_GELU_TANH = 4 /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
} mta_act;

/* One tensor of a list call.  rows * cols may be 0 (skipped). */
typedef struct {
  const void *x;   /* input, rows of ldx elements                          */
  void *y;         /* output, rows of ldy elements                         */
  uint8_t *q;      /* codes, rows of cols rounded up to 32 bytes           */
  uint8_t *scale;  /* scales, rows of (cols rounded up to 32) / 32 bytes   */
  int64_t rows, cols;
  int64_t ldx, ldy; /* >= cols where the buffer is used                    */
} mta_ckpt_tensor;

/* Keep x (elements of type `type`) of each of the `count` tensors: writes q
 * and scale, padding codes included.  act != MTA_ACT_NONE also writes
 * y = act(x), computed from x itself in float32 and rounded once to `type`; y
 * is then required and may be x itself (with ldy == ldx).  Otherwise y is
 * not looked at.  One launch per 32 tensors.  (A 16-bit result's exponentials
 * are the hardware's, off by |u| 2^-24 of themselves.  gelu's 1 + erf is off
 * by 2^-24 of 1: its values for x far below 0 have fewer digits.) */
int mta_ckpt_pack(const mta_ckpt_tensor *tensors, int64_t count, int type,
                  int act, void *stream);

/* y = the kept values in `type` (rounded to nearest-even for MTA_F16, where
 * a magnitude of 65520 or more becomes 65504 with its sign: a finite value
 * stays finite); x is not looked at.  One launch per 32 tensors. */
int mta_ckpt_unpack(const mta_ckpt_tensor *tensors, int64_t count, int type,
                    void *stream);

/* y = x * act'(kept value), in float32 and rounded once to `type`, where x is
 * the gradient of act's output; y may be x itself (with ldy == ldx).  relu's
 * slope at 0 is 0.  act is not MTA_ACT_NONE.  One launch per 32 tensors. */
int mta_ckpt_act_backward(const mta_ckpt_tensor *tensors, int64_t count,
                          int type, int act, void *stream);

/* The weight gradient of y = x W^T + b from x's checkpoint:
 *   dw[o][i] (+)= sum over tokens t of dy[t][o] * kept[t][i]
 *   db[o]    (+)= sum over tokens t of dy[t][o]
 * Products of bfloat16 dy are exact and summed in float32, and so are those of
 * float16 dy where every kept value is a float16 value, as those of a float16
 * tensor are.  With any kept value that is not (it is smaller or larger than
 * float16 holds) a float16 dy is taken as the exact sum of two bfloat16 values,
 * at twice the matrix work: the time depends on the checkpoint's contents.  A
 * float32 dy is taken as the sum of three, at three times the work: exact for
 * |dy| >= 2^-117, less by below 2^-133 under that.  The sum, and with `accumulate` the old value, are
 * added in float32 and rounded once to gtype. */
typedef struct {
  const uint8_t *q;     /* codes of x[tokens, fin] */
  const uint8_t *scale; /* scales */
  const void *dy;       /* [tokens, fout], rows of lddy elements */
  void *dw;             /* [fout, fin], rows of lddw elements */
  void *db;             /* [fout], or NULL */
  void *workspace;      /* mta_ckpt_wgrad_workspace bytes, 16-byte aligned
                           (NULL when that is 0); contents need not be kept */
  int64_t workspace_bytes;
  int64_t tokens, fin, fout; /* tokens may be 0: the sums are then 0 */
  int64_t lddy, lddw;
  int32_t type;         /* of dy */
  int32_t gtype;        /* of dw and db */
  int32_t accumulate;   /* 0: overwrite, 1: add to what is there */
  int32_t reserved;     /* 0 */
} mta_ckpt_wgrad_args;

int mta_ckpt_wgrad(const mta_ckpt_wgrad_args *args, void *stream);

/* Host only: workspace bytes of mta_ckpt_wgrad for these sizes and dy type on
 * a device of `cus` compute units (0: the current device's) in *bytes. */
int mta_ckpt_wgrad_workspace(int64_t tokens, int64_t fin, int64_t fout,
                             int type, int32_t cus, int64_t *bytes);

/* What the forward keeps of a row for mta_policy_loss_backward of the same
 * library, which alone needs to know its fields: softmax(z)[j] is
 * exp(z[j] - top) / total.  (The log of the sum as one number would not do:
 * beside a top of 2^53 nothing is left of log(total).)  All 0 in a row of
 * weight 0. */
typedef struct {
  float top;   /* the row's largest logit */
  float total; /* the sum of exp(logits - top) */
  float coef;  /* d loss / d logp of the row, weight included */
  float rest;  /* 1 - softmax(logits)[action], with all its digits near 0 */
} mta_policy_row;

/* Clipped policy loss with a KL term, summed over the rows (tokens) with
 * weights w:
 *   logp = logits[action] - log sum exp(logits)
 *   r = exp(logp - old_logp),  c = min(max(r, 1 - clip_low), 1 + clip_high)
 *   d = ref_logp - logp,       kl = exp(d) - d - 1
 *   loss = sum w (-min(r A, c A) + kl_coef kl)
 * and its gradient with respect to the logits,
 *   dlogits[j] = S w (d loss/d logp) ([j == action] - softmax(logits)[j]),
 *   d loss/d logp = (r A <= c A ? -r A : 0) + kl_coef (1 - exp(d)),
 * S = *d_grad_scale (1 when NULL).  A row of weight 0 is not read: its logp is
 * 0 and its gradient +0, whatever its other inputs hold.  An action outside
 * [0, vocab) in a row of other weight reads nothing out of range and makes
 * logp, the loss and the row's gradient NaN. */
typedef struct {
  const void *logits;       /* [rows, vocab], rows of ld elements */
  const int64_t *actions;   /* [rows] */
  const float *old_logp;    /* [rows] */
  const float *advantages;  /* [rows] */
  const float *weights;     /* [rows], or NULL: 1 / rows each */
  const float *ref_logp;    /* [rows], or NULL: no KL term (kl_coef 0) */
  const float *d_grad_scale; /* device float, or NULL: 1 */
  void *dlogits;            /* [rows, vocab], rows of ldd elements, logits'
                               type; NULL: the loss alone; may be logits
                               itself (with ldd == ld) */
  mta_policy_row *saved;    /* [rows], or NULL */
  float *logp;              /* [rows], or NULL */
  float *stats;             /* [3]: loss, sum w kl, sum w [r A > c A] */
  void *workspace;          /* mta_policy_loss_workspace bytes, 8-byte aligned */
  int64_t workspace_bytes;
  int64_t rows, vocab, ld, ldd; /* rows may be 0; vocab in
                                     [1, 2^28] */
  double clip_low;          /* in [0, 1] */
  double clip_high;         /* finite, >= 0 */
  double kl_coef;           /* finite, >= 0 */
  int32_t type;
  int32_t reserved;         /* 0 */
} mta_policy_args;

int mta_policy_loss(const mta_policy_args *args, void *stream);

/* Host only: workspace bytes of mta_policy_loss for this many rows. */
int mta_policy_loss_workspace(int64_t rows, int64_t *bytes);

/* The gradient from what mta_policy_loss saved: reads logits, actions, saved
 * and d_grad_scale, writes dlogits (which may be logits itself with
 * ldd == ld).  The other fields are not looked at. */
int mta_policy_loss_backward(const mta_policy_args *args, void *stream);

/* MTA_OPS_VERSION of the built library. */
int mta_ops_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MTA_OPS_H */
