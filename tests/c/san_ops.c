/* san_ops.c -- drives the host side of include/mta_ops.h under
 * AddressSanitizer and UndefinedBehaviorSanitizer, with no device: refusals
 * over random and extreme arguments, and the workspace sizes of a sweep of
 * shapes.  Exits 0 and prints "clean" when every call answers as it must. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "mta_ops.h"

#define CHECK(c, ...)                     \
  do {                                    \
    if (!(c)) {                           \
      fprintf(stderr, "line %d: ", __LINE__); \
      fprintf(stderr, __VA_ARGS__);       \
      fprintf(stderr, "\n");              \
      return 1;                           \
    }                                     \
  } while (0)

int san_wgrad_grid(int64_t tokens, int64_t fin, int64_t fout, int type,
                   int cus);

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

int main(void) {
  int64_t bytes = -1;
  CHECK(mta_ops_version() == MTA_OPS_VERSION, "version");

  /* every list here holds a tensor that is refused */
  for (int n = 0; n < 20000; ++n) {
    mta_ckpt_tensor t[5];
    const int count = 1 + (int)(rnd() % 5);
    for (int i = 0; i < count; ++i) {
      t[i].x = at();
      t[i].y = at();
      t[i].q = at();
      t[i].scale = at();
      t[i].rows = size();
      t[i].cols = size();
      t[i].ldx = size();
      t[i].ldy = size();
    }
    t[count - 1].rows = 2;
    t[count - 1].cols = 40;
    t[count - 1].q = NULL;
    const int act = 1 + (int)(rnd() % 4);
    CHECK(mta_ckpt_pack(t, count, (int)(rnd() % 3), act, NULL) < 0, "pack");
    CHECK(mta_last_error()[0], "a refusal has a message");
    CHECK(mta_ckpt_unpack(t, count, (int)(rnd() % 3), NULL) < 0, "unpack");
    CHECK(mta_ckpt_act_backward(t, count, (int)(rnd() % 3), act, NULL) < 0,
          "backward");
  }
  CHECK(mta_ckpt_pack(NULL, 0, 0, 0, NULL) == 0, "no tensors");

  for (int n = 0; n < 20000; ++n) {
    mta_ckpt_wgrad_args a;
    memset(&a, 0, sizeof a);
    a.q = at();
    a.scale = at();
    a.dy = at();
    a.dw = at();
    a.db = at();
    a.tokens = size();
    a.fin = size();
    a.fout = size();
    a.lddy = size();
    a.lddw = size();
    a.type = (int)(rnd() % 4);
    a.gtype = (int)(rnd() % 4);
    a.accumulate = (int)(rnd() % 3);
    /* with a reserved field set it is refused whatever the rest is */
    a.reserved = 1;
    CHECK(mta_ckpt_wgrad(&a, NULL) < 0, "wgrad");
    bytes = -1;
    const int rc = mta_ckpt_wgrad_workspace(a.tokens, a.fin, a.fout, a.type,
                                            256, &bytes);
    CHECK(rc == 0 ? bytes >= 0 : rc < 0 && bytes == 0, "workspace");
  }
  /* shapes that are taken: their workspace, and their grid */
  for (int64_t t = 0; t < 300000; t = t * 3 + 1 + (int64_t)(rnd() % 2))
    for (int64_t i = 0; i < 9000; i = i * 2 + 5)
      for (int64_t o = 1; o < 60000; o = o * 2 + 3)
        for (int type = 0; type < 3; ++type) {
          const int cus = rnd() % 2 ? 256 : 1 + (int)(rnd() % 400);
          const int bad = san_wgrad_grid(t, i, o, type, cus);
          CHECK(mta_ckpt_wgrad_workspace(t, i, o, type, cus, &bytes) == 0 &&
                    bytes % 16 == 0 && bad == 0,
                "%lld %lld %lld on %d: %d", (long long)t, (long long)i,
                (long long)o, cus, bad);
        }

  for (int n = 0; n < 20000; ++n) {
    mta_policy_args a;
    memset(&a, 0, sizeof a);
    a.logits = at();
    a.actions = at();
    a.old_logp = at();
    a.advantages = at();
    a.weights = at();
    a.ref_logp = at();
    a.d_grad_scale = at();
    a.dlogits = at();
    a.saved = at();
    a.logp = at();
    a.stats = at();
    a.workspace = at();
    a.workspace_bytes = size();
    a.rows = size();
    a.vocab = size();
    a.ld = size();
    a.ldd = size();
    a.clip_low = 0.2;
    a.type = (int)(rnd() % 4);
    a.reserved = 1;
    CHECK(mta_policy_loss(&a, NULL) < 0, "policy");
    CHECK(mta_policy_loss_backward(&a, NULL) < 0, "policy backward");
    const int rc = mta_policy_loss_workspace(a.rows, &bytes);
    CHECK(rc == 0 ? bytes >= 0 : bytes == 0, "policy workspace");
    /* past the reserved field: a gradient shifted against the logits */
    a.reserved = 0;
    a.type = 1;
    a.rows = 1 + (int64_t)(rnd() % 1000);
    a.vocab = 2 + (int64_t)(rnd() % 1000);
    a.ld = a.ldd = a.vocab;
    a.logits = (void *)(uintptr_t)0x10000000;
    a.dlogits = (void *)(uintptr_t)(
        0x10000000 + 2 * (1 + rnd() % (uint64_t)(a.vocab - 1)));
    a.actions = (void *)(uintptr_t)0x20000000;
    a.saved = (void *)(uintptr_t)0x30000000;
    a.d_grad_scale = NULL;
    CHECK(mta_policy_loss_backward(&a, NULL) < 0, "a shifted gradient");
  }
  printf("clean\n");
  return 0;
}
