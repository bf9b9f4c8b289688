/*
 * mta_matrix.h -- operators whose work is matrix products, for AMD Instinct
 * MI355X (gfx950), in the library of mta.h and under its conventions: plain
 * pointers and sizes, work enqueued on the caller's stream, negative
 * mta_status on failure with nothing enqueued, mta_last_error().
 *
 *   mta_orthogonalize     the orthogonalised update of the Muon rule for a
 *                         list of matrices: momentum, Newton-Schulz steps, and
 *                         the result written out or applied to the weights
 *   mta_linear_loss       the cross entropy of a linear output layer from its
 *                         input and weights, without keeping the logits, and
 *                         its gradients with respect to both
 *   mta_linear_loss_backward
 *                         those gradients in a second call
 *
 * No call allocates, waits or keeps anything between calls, so all of them may
 * be captured into a HIP graph and calls on different streams are independent
 * as long as their buffers (workspaces included) are.  The same inputs give
 * the same bits on the same device: no result depends on the order of atomics.
 * Element types are those of mta_gtype (MTA_F32, MTA_BF16, MTA_F16).  Buffers
 * are aligned to their element size, workspaces to 256 bytes.  A buffer that
 * is written overlaps no other buffer of its call (MTA_EINVAL).
 */
#ifndef MTA_MATRIX_H
#define MTA_MATRIX_H

#include "mta.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 1: the first version. */
#define MTA_MATRIX_VERSION 1

/* Rows and columns of a matrix, at most; steps of one call, at most. */
#define MTA_ORTHO_MOST 1048576
#define MTA_ORTHO_STEPS 16

/* One matrix of a call.  rows * cols may be 0 (skipped). */
typedef struct {
  const void *g; /* gradient, or the matrix itself; rows of ldg elements */
  float *m;      /* momentum, rows of cols elements, read and written; NULL:
                    none */
  void *out;     /* the result in out_type, rows of ldout elements, or NULL */
  float *w;      /* weights, rows of cols elements, updated; or NULL */
  void *w16;     /* the new weights in copy_type, rows of cols elements, or
                    NULL */
  int64_t rows, cols, ldg, ldout;
  double scale;  /* factor of the result, finite */
} mta_ortho_matrix;

/* For each matrix, with s the unscale factor float32(1 / float64(scale)) of
 * d_amp (1 when NULL) and c = *d_coef (1 when NULL):
 *   g' = (g s) c                              each product rounded to float32
 *   m = m mu + g',   u = nesterov ? g' + mu m : m     (u = g' without m)
 *   X = u / (|u| + eps)         |u| the square root of the sum of squares, in
 *                               float64; of the transpose if rows > cols
 *   `steps` times, with the step's coefficients a, b, c:
 *     A = X X^T,  B = b A + c A A,  X = a X + B X
 *   out = scale X        (transposed back), rounded once to out_type
 *   w = w f32(1 - lr weight_decay) + f32(-lr scale) X,  w16 its rounding
 * With d_amp->found_inf set m, w and w16 stay as they were and out is
 * unspecified.  A matrix with a NaN or infinity comes out all NaN and leaves
 * the others alone; one of zeros comes out zero.
 *
 * Matrices are taken up to forty at a time, those of up to 64 rows or columns
 * apart, and by 4 GiB of workspace; one such group follows the other.
 *
 * A matrix of up to 64 rows or columns is computed in float64.  Otherwise X is
 * kept as a float16 value and a second one for what it leaves (22 bits), times a
 * power of two as long as it is far below 1 (|u| far below eps); the
 * symmetric matrices as such values and their diagonals in float32; sums are
 * float32, and two steps may be taken as one product (Q' Q) X.  With `precise`
 * all products are those of 22 bits, three float16 products each.  Without,
 * products are of the first values alone, one product each, the diagonals apart:
 * off by 2e-4 to 1.1e-3 of the result's root mean square, up to 2.5e-3 where the
 * singular values span five decades.
 * The coefficients have to keep every singular value in [0, 1] below 7 from
 * step to step and may not let one grow to 100 times itself in a step, or to
 * more than 2^18 times in all (MTA_EINVAL). */
typedef struct {
  const mta_ortho_matrix *matrices;
  int64_t count;
  void *workspace; /* mta_orthogonalize_workspace bytes */
  int64_t workspace_bytes;
  const double *coefficients;  /* host: a, b, c of each step */
  const float *d_coef;         /* device float, or NULL */
  const mta_amp_state *d_amp;  /* or NULL */
  double eps;                  /* finite, >= 0 */
  double momentum;             /* finite, >= 0 */
  double lr, weight_decay;     /* finite, >= 0; used where there is a w */
  int32_t steps;               /* 1 .. MTA_ORTHO_STEPS */
  int32_t type;                /* of g */
  int32_t out_type;
  int32_t copy_type;           /* of w16: MTA_BF16 or MTA_F16 */
  int32_t nesterov;            /* 0 or 1 */
  int32_t precise;             /* 0 or 1 */
} mta_ortho_args;

int mta_orthogonalize(const mta_ortho_args *args, void *stream);

/* Host only: workspace bytes of mta_orthogonalize for these arguments, of
 * which it looks at the matrices' sizes and at `precise`. */
int mta_orthogonalize_workspace(const mta_ortho_args *args, int64_t *bytes);

/* What the forward keeps of a row for mta_linear_loss_backward of the same
 * library: softmax(z)[j] is exp(z[j] - top) / total.  All 0 in a row of weight
 * 0. */
typedef struct {
  float top;    /* the row's largest logit */
  float total;  /* the sum of exp(z - top) */
  float weight; /* of the row in the loss */
  float rest;   /* 1 - softmax(z)[target], with all its digits near 0 */
} mta_linear_row;

/* The cross entropy of a linear output layer, z = h w^T, summed over the rows
 * (tokens) with weights:
 *   loss = sum over rows of weight (-logp),  logp = log softmax(z)[target]
 * and its gradients, times S = *d_grad_scale (1 when NULL):
 *   dz[j] = S weight (softmax(z)[j] - [j == target])
 *   dh = dz w,   dw (+)= dz^T h
 * The logits are never stored: the gradients' half makes them a second time,
 * in pieces of the vocabulary, and keeps one piece of dz, in h's type.
 * A row whose target is ignore_index or whose weight is 0 is left out: its h
 * is not read, its logp is 0 and its dh +0.  Without weights every other row
 * has 1 / their number; a call without such rows has loss 0.  Another target
 * outside [0, vocab) reads nothing out of range and makes the row's logp and
 * dh, the loss and dw NaN.  So does a largest logit that is infinite (of either
 * sign) or, for 16-bit elements, beyond +-2.35e38 (2^128 / log2(e)).
 * Products of 16-bit elements are exact, those of float32 elements are taken as
 * the six largest of nine products of three bfloat16 values; sums are float32.
 * dz is rounded once to the 16-bit type (float32: to three bfloat16 values)
 * before dh and dw are made of it, scaled so that its largest finite weight is 1
 * (float16: 2^14): neither S nor weights that are all small cost digits.  Float16
 * has 11 bits down to 2^-28 of the largest weight and none below 2^-39: a row
 * whose own weight is 1e-6 of the largest has its target's digits, and those of
 * probabilities of 1 / 50257 to 9%. */
typedef struct {
  const void *h;              /* [rows, width], rows of ldh elements */
  const void *w;              /* [vocab, width], rows of ldw elements */
  const int64_t *targets;     /* [rows] */
  const float *weights;       /* [rows], or NULL */
  const float *d_grad_scale;  /* device float, or NULL: 1 */
  void *dh;                   /* [rows, width], rows of lddh, or NULL */
  void *dw;                   /* [vocab, width], rows of lddw, or NULL */
  mta_linear_row *saved;      /* [rows], or NULL */
  float *logp;                /* [rows], or NULL */
  float *loss;                /* [1] */
  void *workspace;            /* mta_linear_loss_workspace bytes */
  int64_t workspace_bytes;
  int64_t rows, vocab, width; /* rows may be 0; vocab >= 1, width >= 1 */
  int64_t ldh, ldw, lddh, lddw;
  int64_t ignore_index;
  int32_t type;               /* of h, w and dh */
  int32_t dw_type;
  int32_t accumulate;         /* 0: overwrite dw, 1: add to what is there */
  int32_t reserved;           /* 0 */
} mta_linear_loss_args;

/* The loss, and with dh or dw their gradients (saved may then be NULL too). */
int mta_linear_loss(const mta_linear_loss_args *args, void *stream);

/* The gradients from what mta_linear_loss saved for the same h, w and targets:
 * reads h, w, targets, saved and d_grad_scale, writes dh and dw, one of which
 * may be NULL.  weights, logp and loss are not looked at. */
int mta_linear_loss_backward(const mta_linear_loss_args *args, void *stream);

/* Host only: workspace bytes of either call for these arguments, of which it
 * looks at the sizes and types, at w's address and pitch and at which of dh
 * and dw are there, on a device of `cus` compute units (0: the current
 * device's). */
int mta_linear_loss_workspace(const mta_linear_loss_args *args, int32_t cus,
                              int64_t *bytes);

/* MTA_MATRIX_VERSION of the built library. */
int mta_matrix_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MTA_MATRIX_H */
