/*
 * mta_matrix.h -- operators whose work is matrix products, for AMD Instinct
 * MI355X (gfx950), in the library of mta.h and under its conventions: plain
 * pointers and sizes, work enqueued on the caller's stream, negative
 * mta_status on failure with nothing enqueued, mta_last_error().
 *
 *   mta_orthogonalize     the orthogonalised update of the Muon rule for a
 *                         list of matrices: momentum, Newton-Schulz steps, and
 *                         the result written out or applied to the weights
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
 * X and A are kept as a float16 value and a second one for what it leaves (22
 * bits), B as one such value and its diagonal in float32; sums are float32.
 * With `precise`, and for a matrix of fewer than 16 rows or columns, all
 * products are those of 22 bits, three float16 products each.  Without,
 * products are of the first values alone, one product each, the diagonals
 * apart: off by 2e-4 to 1.1e-3 of the result's root mean square.
 * The coefficients have to keep every singular value in [0, 1] below 7 from
 * step to step (MTA_EINVAL). */
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

/* MTA_MATRIX_VERSION of the built library. */
int mta_matrix_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MTA_MATRIX_H */
