/* san_matrix.c -- drives the host side of include/mta_matrix.h under
 * AddressSanitizer and UndefinedBehaviorSanitizer, with no device: refusals
 * over random and extreme arguments, and the workspace sizes of a sweep of
 * shapes.  Exits 0 and prints "clean" when every call answers as it must. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "mta_matrix.h"

#define CHECK(c, ...)                     \
  do {                                    \
    if (!(c)) {                           \
      fprintf(stderr, "line %d: ", __LINE__); \
      fprintf(stderr, __VA_ARGS__);       \
      fprintf(stderr, "\n");              \
      return 1;                           \
    }                                     \
  } while (0)

static uint64_t state = 88172645463325252ull;
static uint64_t rnd(void) {
  state ^= state << 13;
  state ^= state >> 7;
  state ^= state << 17;
  return state;
}

/* a size: small, odd, large or out of any range */
static int64_t size(void) {
  switch (rnd() % 6) {
    case 0: return (int64_t)(rnd() % 4);
    case 1: return (int64_t)(rnd() % 5000);
    case 2: return (int64_t)1 << (rnd() % 62);
    case 3: return INT64_MAX - (int64_t)(rnd() % 100);
    case 4: return -(int64_t)(rnd() % 100);
    default: return (int64_t)(rnd() >> (rnd() % 63));
  }
}

static void *at(void) {
  return rnd() % 4 ? (void *)(uintptr_t)(rnd() >> (rnd() % 60)) : NULL;
}

static double number(void) {
  static const double odd[6] = {0.0, -1.0, 1e300, -1e300, 1e-300, 3.4445};
  return rnd() % 2 ? odd[rnd() % 6] : (double)(int64_t)(rnd() % 2001) / 100 - 10;
}

int main(void) {
  int64_t bytes = -1;
  CHECK(mta_matrix_version() == MTA_MATRIX_VERSION, "version");

  /* every list here holds a matrix that is refused */
  for (int n = 0; n < 20000; ++n) {
    mta_ortho_matrix m[5];
    double co[3 * MTA_ORTHO_STEPS];
    mta_ortho_args a;
    memset(&a, 0, sizeof a);
    const int count = 1 + (int)(rnd() % 5);
    for (int i = 0; i < count; ++i) {
      m[i].g = at();
      m[i].m = (float *)at();
      m[i].out = at();
      m[i].w = (float *)at();
      m[i].w16 = at();
      m[i].rows = size();
      m[i].cols = size();
      m[i].ldg = size();
      m[i].ldout = size();
      m[i].scale = number();
    }
    m[count - 1].rows = 2;
    m[count - 1].cols = 40;
    m[count - 1].g = NULL;
    for (int i = 0; i < 3 * MTA_ORTHO_STEPS; ++i) co[i] = number();
    a.matrices = m;
    a.count = count;
    a.workspace = at();
    a.workspace_bytes = size();
    a.coefficients = rnd() % 8 ? co : NULL;
    a.d_coef = (const float *)at();
    a.eps = number();
    a.momentum = number();
    a.lr = number();
    a.weight_decay = number();
    a.steps = (int)(rnd() % 20) - 1;
    a.type = (int)(rnd() % 4);
    a.out_type = (int)(rnd() % 4);
    a.copy_type = (int)(rnd() % 4);
    a.nesterov = (int)(rnd() % 3);
    a.precise = (int)(rnd() % 3);
    CHECK(mta_orthogonalize(&a, NULL) < 0, "orthogonalize");
    CHECK(mta_last_error()[0], "a refusal has a message");
    bytes = -1;
    if (mta_orthogonalize_workspace(&a, &bytes) == 0)
      CHECK(bytes >= 0 && bytes % 256 == 0, "%lld bytes", (long long)bytes);
    else
      CHECK(bytes == 0, "a refusal says no size");
  }
  CHECK(mta_orthogonalize(NULL, NULL) < 0, "no arguments");
  CHECK(mta_orthogonalize_workspace(NULL, &bytes) < 0, "no arguments");

  /* more matrices never need less than each of them */
  for (int n = 0; n < 2000; ++n) {
    mta_ortho_matrix m[100];
    mta_ortho_args a;
    memset(&a, 0, sizeof a);
    memset(m, 0, sizeof m);
    const int count = 1 + (int)(rnd() % 100);
    for (int i = 0; i < count; ++i) {
      m[i].rows = (int64_t)(rnd() % (rnd() % 8 ? 700 : MTA_ORTHO_MOST + 1));
      m[i].cols = (int64_t)(rnd() % 700);
    }
    a.matrices = m;
    a.count = count;
    a.precise = (int)(rnd() % 2);
    CHECK(mta_orthogonalize_workspace(&a, &bytes) == 0, "sizes");
    for (int i = 0; i < count; ++i) {
      int64_t one = -1;
      mta_ortho_args b = a;
      b.matrices = m + i;
      b.count = 1;
      CHECK(mta_orthogonalize_workspace(&b, &one) == 0, "one");
      /* X alone: two buffers of two planes of 16 bits */
      if (m[i].rows > 64 && m[i].cols > 64)
        CHECK(one >= 8 * m[i].rows * m[i].cols &&
                  bytes >= 8 * m[i].rows * m[i].cols,
              "%lld x %lld", (long long)m[i].rows, (long long)m[i].cols);
    }
  }

  for (int n = 0; n < 20000; ++n) {
    mta_linear_loss_args a;
    memset(&a, 0, sizeof a);
    a.h = at();
    a.w = at();
    a.targets = (const int64_t *)at();
    a.weights = (const float *)at();
    a.d_grad_scale = (const float *)at();
    a.dh = at();
    a.dw = at();
    a.saved = (mta_linear_row *)at();
    a.logp = (float *)at();
    a.loss = (float *)at();
    a.workspace = NULL;
    a.workspace_bytes = size();
    a.rows = size();
    a.vocab = size();
    a.width = size();
    a.ldh = size();
    a.ldw = size();
    a.lddh = size();
    a.lddw = size();
    a.ignore_index = size();
    a.type = (int)(rnd() % 4);
    a.dw_type = (int)(rnd() % 4);
    a.accumulate = (int)(rnd() % 3);
    a.reserved = (int)(rnd() % 2);
    CHECK(mta_linear_loss(&a, NULL) < 0, "loss");
    CHECK(mta_last_error()[0], "a refusal has a message");
    CHECK(mta_linear_loss_backward(&a, NULL) < 0, "backward");
    bytes = -1;
    if (mta_linear_loss_workspace(&a, 1 + (int32_t)(rnd() % 400), &bytes) == 0)
      CHECK(bytes > 0 && bytes % 256 == 0, "%lld bytes", (long long)bytes);
    else
      CHECK(bytes == 0, "a refusal says no size");
  }
  CHECK(mta_linear_loss(NULL, NULL) < 0, "no arguments");

  /* the largest of each size, alone and together with others */
  static const int64_t rows[4] = {0, 1, 70000, (int64_t)1 << 30};
  static const int64_t vocab[4] = {1, 2, 70001, (int64_t)1 << 28};
  static const int64_t width[4] = {1, 100, 16384, (int64_t)1 << 20};
  for (int n = 0; n < 4 * 4 * 4 * 3 * 4; ++n) {
    mta_linear_loss_args a;
    memset(&a, 0, sizeof a);
    a.rows = rows[n % 4];
    a.vocab = vocab[n / 4 % 4];
    a.width = width[n / 16 % 4];
    a.ldh = a.ldw = a.lddh = a.lddw = a.width;
    a.type = n / 64 % 3;
    a.dh = n / 192 & 1 ? (void *)256 : NULL;
    a.dw = n / 192 & 2 ? (void *)256 : NULL;
    a.w = (const void *)256;
    if (mta_linear_loss_workspace(&a, 256, &bytes) == 0)
      CHECK(bytes > 0 && bytes / 2 >= a.rows * a.width &&
                bytes < INT64_MAX / 4,
            "%lld x %lld x %lld", (long long)a.rows, (long long)a.vocab,
            (long long)a.width);
    else
      CHECK(mta_last_error()[0], "a refusal has a message");
  }
  puts("clean");
  return 0;
}
