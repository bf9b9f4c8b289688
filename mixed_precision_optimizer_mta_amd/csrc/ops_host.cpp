// ops_host.cpp -- host side and C ABI of the operators of include/mta_ops.h:
// argument checks, launch shapes, workspace sizes.  No C++ exception crosses
// the ABI.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <vector>

#include "ops_internal.h"

static_assert(sizeof(mta_ckpt_tensor) == 64, "mta_ckpt_tensor layout");
static_assert(sizeof(mta_ckpt_wgrad_args) == 112,
              "mta_ckpt_wgrad_args layout");
static_assert(sizeof(mta_policy_args) == 168, "mta_policy_args layout");

namespace {

int fail(int code, const char *fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return mta::report(code, msg);
}

int ok() { return mta::report(MTA_OK, ""); }

bool known_type(int t) {
  return t == MTA_F32 || t == MTA_BF16 || t == MTA_F16;
}

int64_t size_of(int type) { return type == MTA_F32 ? 4 : 2; }

bool aligned(const void *p, int64_t a) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(a - 1)) == 0;
}

// Sizes beyond this would overflow 64-bit byte offsets.
constexpr int64_t kMostBytes = int64_t{1} << 60;

// rows * pitch * size fits.
bool fits(int64_t rows, int64_t pitch, int64_t size) {
  return rows == 0 || pitch == 0 || rows <= kMostBytes / size / pitch;
}

// A buffer of `rows` runs of `width` bytes, `pitch` bytes apart.
struct Region {
  uintptr_t lo, hi;  // first byte, one past the last
  uintptr_t pitch, width;
  const char *name;
  int64_t tensor;  // of a list, or -1
  bool written;
  const void *pair;  // a buffer that this one may be, element for element
};

Region region(const void *p, int64_t rows, int64_t pitch, int64_t width,
              const char *name, int64_t tensor, bool written,
              const void *pair = nullptr) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  const uintptr_t bytes =
      rows > 0 && width > 0
          ? static_cast<uintptr_t>((rows - 1) * pitch + width)
          : 0;
  return Region{lo,     lo + bytes, static_cast<uintptr_t>(pitch),
                static_cast<uintptr_t>(width), name, tensor, written, pair};
}

// Whether two buffers share a byte.  Column slices of one wide buffer lie
// between each other's rows without doing so.
bool shares(const Region &a, const Region &b) {  // a.lo <= b.lo
  if (a.lo == a.hi || b.lo == b.hi || b.lo >= a.hi) return false;
  if (a.pitch != b.pitch || a.pitch == 0) return true;
  const uintptr_t d = (b.lo - a.lo) % a.pitch;
  return !(d >= a.width && d + b.width <= a.pitch);
}

int check_regions(std::vector<Region> *r) {
  std::sort(r->begin(), r->end(),
            [](const Region &a, const Region &b) { return a.lo < b.lo; });
  for (size_t i = 0; i < r->size(); ++i)
    for (size_t j = i + 1; j < r->size() && (*r)[j].lo < (*r)[i].hi; ++j) {
      const Region &a = (*r)[i], &b = (*r)[j];
      if (!a.written && !b.written) continue;
      // in place: the same elements of the same tensor
      if (a.lo == b.lo && a.hi == b.hi && a.pitch == b.pitch &&
          a.tensor == b.tensor &&
          (a.pair == reinterpret_cast<const void *>(b.lo) ||
           b.pair == reinterpret_cast<const void *>(a.lo)))
        continue;
      if (!shares(a, b)) continue;
      if (a.tensor < 0)
        return fail(MTA_EINVAL, "buffers overlap: %s and %s", a.name, b.name);
      return fail(MTA_EINVAL,
                  "buffers overlap: tensor %lld %s and tensor %lld %s",
                  static_cast<long long>(a.tensor), a.name,
                  static_cast<long long>(b.tensor), b.name);
    }
  return MTA_OK;
}

int64_t blocks_of(int64_t cols) {
  return (cols + MTA_CKPT_BLOCK - 1) / MTA_CKPT_BLOCK;
}

// Columns of a checkpoint row: positions within a row are 32-bit on the
// device.
constexpr int64_t kMostCols = int64_t{1} << 30;

int check_ckpt(const mta_ckpt_tensor *ts, int64_t count, int mode, int type,
               int act) {
  if (count < 0) return fail(MTA_EINVAL, "count must be >= 0");
  if (count > 0 && !ts) return fail(MTA_EINVAL, "tensors is NULL");
  if (!known_type(type)) return fail(MTA_EDTYPE, "unknown type %d", type);
  if (act < MTA_ACT_NONE || act > MTA_ACT_GELU_TANH)
    return fail(MTA_EINVAL, "unknown activation %d", act);
  if (mode == mta::kCkptBackward && act == MTA_ACT_NONE)
    return fail(MTA_EINVAL, "a backward needs an activation");
  const bool has_x = mode != mta::kCkptUnpack;
  const bool has_y = mode != mta::kCkptPack || act != MTA_ACT_NONE;
  const bool fills = mode == mta::kCkptPack;
  const int64_t sz = size_of(type);
  std::vector<Region> regions;
  regions.reserve(static_cast<size_t>(count) * 4);
  for (int64_t i = 0; i < count; ++i) {
    const mta_ckpt_tensor &t = ts[i];
    const long long n = static_cast<long long>(i);
    if (t.rows < 0 || t.cols < 0)
      return fail(MTA_EINVAL, "tensor %lld: rows or cols < 0", n);
    if (t.rows == 0 || t.cols == 0) continue;
    if (t.cols > kMostCols)
      return fail(MTA_EINVAL, "tensor %lld: more than 2^30 columns", n);
    if ((has_x && !t.x) || (has_y && !t.y) || !t.q || !t.scale)
      return fail(MTA_EINVAL, "tensor %lld: a buffer is NULL", n);
    if ((has_x && t.ldx < t.cols) || (has_y && t.ldy < t.cols))
      return fail(MTA_EINVAL, "tensor %lld: a row pitch is below cols", n);
    const int64_t nb = blocks_of(t.cols);
    if ((has_x && !fits(t.rows, t.ldx, sz)) ||
        (has_y && !fits(t.rows, t.ldy, sz)) ||
        !fits(t.rows, nb * MTA_CKPT_BLOCK, 1))
      return fail(MTA_EINVAL, "tensor %lld: too large", n);
    if ((has_x && !aligned(t.x, sz)) || (has_y && !aligned(t.y, sz)))
      return fail(MTA_EALIGN,
                  "tensor %lld: a buffer is not aligned to its element size",
                  n);
    if (!aligned(t.q, 16))
      return fail(MTA_EALIGN, "tensor %lld: q is not 16-byte aligned", n);
    if (has_x)
      regions.push_back(region(t.x, t.rows, t.ldx * sz, t.cols * sz, "x", i,
                               false, has_y ? t.y : nullptr));
    if (has_y)
      regions.push_back(
          region(t.y, t.rows, t.ldy * sz, t.cols * sz, "y", i, true));
    const int64_t qb = t.rows * nb * MTA_CKPT_BLOCK;
    regions.push_back(region(t.q, 1, qb, qb, "q", i, fills));
    regions.push_back(
        region(t.scale, 1, t.rows * nb, t.rows * nb, "scale", i, fills));
  }
  return check_regions(&regions);
}

// Units a workgroup handles at a time: as many as keep 1024 workgroups, four a
// lane at most.  Against four always, silu and its kept input of 512 x 768
// bfloat16 take 4.3 us instead of 6.4, of 517 x 1601 float16 5.5 instead of
// 7.8 and of 4096 x 1600 11.2 instead of 11.7; large tensors the same.
uint32_t ckpt_chunk(uint64_t units) {
  const uint64_t each = units / (mta::kCkptThreads * 1024);
  return mta::kCkptThreads *
         static_cast<uint32_t>(std::clamp<uint64_t>(each, 1, mta::kCkptUnroll));
}

int run_ckpt(const mta_ckpt_tensor *ts, int64_t count, int mode, int type,
             int act, void *stream, const char *what) {
  try {
    const int rc = check_ckpt(ts, count, mode, type, act);
    if (rc) return rc;
  } catch (const std::bad_alloc &) {
    return fail(MTA_ENOMEM, "host allocation failed");
  }
  const bool has_x = mode != mta::kCkptUnpack;
  const bool has_y = mode != mta::kCkptPack || act != MTA_ACT_NONE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  mta::CkptList list;
  list.count = 0;
  list.first[0] = 0;
  hipError_t e = hipSuccess;
  for (int64_t i = 0; i < count && e == hipSuccess; ++i) {
    const mta_ckpt_tensor &t = ts[i];
    if (t.rows > 0 && t.cols > 0) {
      const uint32_t k = list.count++;
      mta::CkptItem &it = list.item[k];
      it.x = t.x;
      it.y = t.y;
      it.q = t.q;
      it.scale = t.scale;
      it.ldx = has_x ? t.ldx : t.cols;
      it.ldy = has_y ? t.ldy : t.cols;
      it.cols = static_cast<uint32_t>(t.cols);
      it.row_units = static_cast<uint32_t>(
          blocks_of(t.cols) * (MTA_CKPT_BLOCK / mta::ckpt_unit(type)));
      it.units = static_cast<uint64_t>(t.rows) * it.row_units;
      if (t.cols % MTA_CKPT_BLOCK == 0 &&
          (t.rows == 1 || (it.ldx == t.cols && it.ldy == t.cols)))
        it.row_units = 0;
      it.chunk = ckpt_chunk(it.units);
      // 32 tensors of 2^18 workgroups of 2^8 threads stay below 2^32
      const uint64_t groups = (it.units + it.chunk - 1) / it.chunk;
      list.first[k + 1] =
          list.first[k] +
          static_cast<uint32_t>(std::min<uint64_t>(groups, 1u << 18));
    }
    if (list.count == mta::kCkptTensors || (i == count - 1 && list.count)) {
      e = mta::launch_ckpt(mode, type, act, list, s);
      list.count = 0;
    }
  }
  return mta::report_launch(e, s, what);
}

// Compute units of the current device.
int current_cus(int *cus) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess)
    e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess || *cus <= 0)
    return fail(MTA_EHIP, "cannot read the compute-unit count: %s",
                hipGetErrorString(e));
  return MTA_OK;
}

int check_wgrad_sizes(int64_t tokens, int64_t fin, int64_t fout, int type) {
  if (tokens < 0 || fin < 0 || fout < 0)
    return fail(MTA_EINVAL, "tokens, fin or fout < 0");
  if (!known_type(type)) return fail(MTA_EDTYPE, "unknown type %d", type);
  // (31 rows of codes are a 32-bit offset on the device)
  if (fin > kMostCols / 16 || fout > kMostCols ||
      !fits(tokens, fin + MTA_CKPT_BLOCK, 1) || !fits(tokens, fout, 4) ||
      !fits(fout, fin, 4096))
    return fail(MTA_EINVAL, "too large");
  return MTA_OK;
}

// Workgroups of one launch: below 2^32 threads of up to 512 to a workgroup.
constexpr int64_t kMostGroups = int64_t{1} << 22;

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

// What lies in the workspace, and where.
struct WgradSpace {
  int64_t part_db, range, bytes;  // the tiles' parts come first
};

WgradSpace wgrad_space(const mta::WgradGrid &g, int64_t fout) {
  const int64_t tile = int64_t{mta::kWgradTile} * mta::kWgradTile;
  WgradSpace s;
  s.part_db = g.cut * g.parts * tile * 4;
  s.range = s.part_db + (g.cut > 0 ? round16(g.parts * fout * 4) : 0);
  s.bytes = s.range + round16(g.ranges * 4);
  return s;
}

// Positions within a row are 32-bit byte offsets on the device.
constexpr int64_t kMostVocab = int64_t{1} << 28;

int check_policy(const mta_policy_args *a, bool backward,
                 std::vector<Region> *regions) {
  if (!a) return fail(MTA_EINVAL, "args is NULL");
  if (a->rows < 0) return fail(MTA_EINVAL, "rows < 0");
  if (a->vocab < 1 || a->vocab > kMostVocab)
    return fail(MTA_EINVAL, "vocab must be in [1, 2^28] (got %lld)",
                static_cast<long long>(a->vocab));
  if (!known_type(a->type)) return fail(MTA_EDTYPE, "unknown type %d", a->type);
  if (a->reserved) return fail(MTA_EINVAL, "reserved must be 0");
  const int64_t sz = size_of(a->type);
  const bool grad = a->dlogits != nullptr;
  if (!backward) {
    if (!(a->clip_low >= 0.0 && a->clip_low <= 1.0))
      return fail(MTA_EINVAL, "clip_low must be in [0, 1] (got %g)",
                  a->clip_low);
    if (!(std::isfinite(a->clip_high) && a->clip_high >= 0.0))
      return fail(MTA_EINVAL, "clip_high must be finite and >= 0 (got %g)",
                  a->clip_high);
    if (!(std::isfinite(a->kl_coef) && a->kl_coef >= 0.0))
      return fail(MTA_EINVAL, "kl_coef must be finite and >= 0 (got %g)",
                  a->kl_coef);
    if (a->kl_coef != 0.0 && !a->ref_logp)
      return fail(MTA_EINVAL, "a KL term needs ref_logp");
    if (!a->stats) return fail(MTA_EINVAL, "stats is NULL");
    if (!aligned(a->stats, 4))
      return fail(MTA_EALIGN, "stats must be 4-byte aligned");
    regions->push_back(region(a->stats, 1, 12, 12, "stats", -1, true));
    int64_t need = 0;
    const int rc = mta_policy_loss_workspace(a->rows, &need);
    if (rc) return rc;
    if (need > 0 && !a->workspace)
      return fail(MTA_EINVAL, "workspace is NULL");
    if (a->workspace_bytes < need)
      return fail(MTA_EINVAL, "workspace has %lld bytes, %lld are needed",
                  static_cast<long long>(a->workspace_bytes),
                  static_cast<long long>(need));
    if (!aligned(a->workspace, 8))
      return fail(MTA_EALIGN, "workspace must be 8-byte aligned");
    regions->push_back(
        region(a->workspace, 1, need, need, "workspace", -1, true));
  }
  if (!aligned(a->d_grad_scale, 4))
    return fail(MTA_EALIGN, "d_grad_scale must be 4-byte aligned");
  if (a->d_grad_scale)
    regions->push_back(
        region(a->d_grad_scale, 1, 4, 4, "d_grad_scale", -1, false));
  if (a->rows == 0) return check_regions(regions);
  if (!a->logits || !a->actions)
    return fail(MTA_EINVAL, "logits or actions is NULL");
  if (!backward && (!a->old_logp || !a->advantages))
    return fail(MTA_EINVAL, "old_logp or advantages is NULL");
  if (backward && (!grad || !a->saved))
    return fail(MTA_EINVAL, "dlogits or saved is NULL");
  if (a->ld < a->vocab || (grad && a->ldd < a->vocab))
    return fail(MTA_EINVAL, "a row pitch is below vocab");
  if (!fits(a->rows, a->ld, sz) || (grad && !fits(a->rows, a->ldd, sz)) ||
      !fits(a->rows, 16, 1))
    return fail(MTA_EINVAL, "too large");
  if (!aligned(a->logits, sz) || !aligned(a->dlogits, sz) ||
      !aligned(a->actions, 8) || !aligned(a->saved, 8))
    return fail(MTA_EALIGN, "a buffer is not aligned to its element size");
  regions->push_back(region(a->logits, a->rows, a->ld * sz, a->vocab * sz,
                            "logits", -1, false, a->dlogits));
  if (grad)
    regions->push_back(region(a->dlogits, a->rows, a->ldd * sz,
                              a->vocab * sz, "dlogits", -1, true));
  const auto flat = [&](const void *p, int64_t size, const char *name,
                        bool written) {
    if (p)
      regions->push_back(region(p, 1, a->rows * size, a->rows * size, name, -1,
                                written));
  };
  flat(a->actions, 8, "actions", false);
  flat(a->saved, 16, "saved", !backward);
  if (!backward) {
    if (!aligned(a->old_logp, 4) || !aligned(a->advantages, 4) ||
        !aligned(a->weights, 4) || !aligned(a->ref_logp, 4) ||
        !aligned(a->logp, 4))
      return fail(MTA_EALIGN, "a buffer is not aligned to its element size");
    flat(a->old_logp, 4, "old_logp", false);
    flat(a->advantages, 4, "advantages", false);
    flat(a->weights, 4, "weights", false);
    flat(a->ref_logp, 4, "ref_logp", false);
    flat(a->logp, 4, "logp", true);
  }
  return check_regions(regions);
}

int run_policy(const mta_policy_args *a, bool backward, void *stream,
               const char *what) {
  try {
    std::vector<Region> regions;
    regions.reserve(16);
    const int rc = check_policy(a, backward, &regions);
    if (rc) return rc;
  } catch (const std::bad_alloc &) {
    return fail(MTA_ENOMEM, "host allocation failed");
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = backward ? mta::launch_policy_backward(*a, s)
                                : mta::launch_policy(*a, s);
  return mta::report_launch(e, s, what);
}

}  // namespace

// Output tiles are dealt in rounds of one to a CU.  Whole rounds take their
// tiles over all tokens; the tiles of a last, partial round (all of them, when
// there are fewer than CUs) may be cut along the tokens into parts, whose sums
// a second kernel joins, and when no CU gets more than one, a workgroup may
// bring as many groups of waves as a CU holds, each with a share of the
// tokens.  Taken is what these times, measured here, say is the shortest, in
// us: 7 for a workgroup to start and end and 4 more to join its groups; a step
// of a tile 0.37 of a CU that holds one workgroup, 0.285 with two, 0.27 with
// more and 0.265 with groups (float32 dY: 1.1, 0.85, 0.85 and 0.75); 5 for the
// second kernel and 0.015 a part for its bytes.  Against whole tiles by single
// groups, in bfloat16: 404 us instead of 423 for 1600 x 6400 outputs (2.5
// rounds) over 16384 tokens, 68 instead of 91 for 1600 x 1600 over 8192, 56
// instead of 338 for 768 x 768 over 32768 (58 with parts alone), and 28
// instead of 40 for 768 x 2304 over 1024 tokens of float32 dY (32).
mta::WgradGrid mta::wgrad_grid(int64_t tokens, int64_t fin, int64_t fout,
                               int type, int cus) {
  static constexpr double kStepUs[2][4] = {{0.37, 0.285, 0.27, 0.265},
                                           {1.1, 0.85, 0.85, 0.75}};
  const double *step_us = kStepUs[type == MTA_F32];
  WgradGrid g{};
  g.tiles_o = (fout + kWgradTile - 1) / kWgradTile;
  // no input features: the bias gradient alone still takes a column of tiles
  g.tiles_i = fin > 0 ? (fin + kWgradTile - 1) / kWgradTile : 1;
  const int64_t tiles = g.tiles_o * g.tiles_i;
  const int64_t steps = (tokens + kWgradStep - 1) / kWgradStep;
  g.whole = tiles / cus * cus;
  g.cut = tiles - g.whole;
  g.parts = 1;
  double best = 0.0;
  for (int64_t p = 1; g.cut > 0 && p <= 64 && (p == 1 || p * 4 <= steps);
       ++p) {
    const int64_t groups = g.whole + g.cut * p;
    const int64_t held = std::min<int64_t>((groups + cus - 1) / cus, 3);
    const int64_t each = (steps + p - 1) / p;
    const double taken = static_cast<double>(
        g.whole / cus * steps + (g.cut * p + cus - 1) / cus * each);
    const double join =
        p > 1 ? 5.0 + 0.015 * static_cast<double>(g.cut * p) : 0.0;
    for (int grouped = 0; grouped <= (groups <= cus ? 1 : 0); ++grouped) {
      const double us = (grouped ? 11.0 : 7.0) + join +
                        step_us[grouped ? 3 : held - 1] * taken;
      if ((p > 1 || grouped) && us >= best) continue;
      best = us;
      g.parts = static_cast<int>(p);
      g.grouped = grouped;
    }
  }
  if (g.parts == 1) {
    g.whole = tiles;
    g.cut = 0;
  }
  const int64_t each = (steps + g.parts - 1) / g.parts;
  g.part_tokens = each * kWgradStep;
  // (a part that would be empty is none)
  if (g.cut > 0 && each > 0)
    g.parts = static_cast<int>((steps + each - 1) / each);
  if (type == MTA_F16) {
    const int64_t blocks = tokens * blocks_of(fin);
    g.ranges = static_cast<int>(
        std::min<int64_t>((blocks + 1023) / 1024, kWgradRanges));
  }
  return g;
}

extern "C" {

int mta_ops_version(void) { return MTA_OPS_VERSION; }

int mta_ckpt_pack(const mta_ckpt_tensor *tensors, int64_t count, int type,
                  int act, void *stream) {
  return run_ckpt(tensors, count, mta::kCkptPack, type, act, stream,
                  "mta_ckpt_pack");
}

int mta_ckpt_unpack(const mta_ckpt_tensor *tensors, int64_t count, int type,
                    void *stream) {
  return run_ckpt(tensors, count, mta::kCkptUnpack, type, MTA_ACT_NONE, stream,
                  "mta_ckpt_unpack");
}

int mta_ckpt_act_backward(const mta_ckpt_tensor *tensors, int64_t count,
                          int type, int act, void *stream) {
  return run_ckpt(tensors, count, mta::kCkptBackward, type, act, stream,
                  "mta_ckpt_act_backward");
}

int mta_ckpt_wgrad_workspace(int64_t tokens, int64_t fin, int64_t fout,
                             int type, int32_t cus, int64_t *bytes) {
  if (!bytes) return fail(MTA_EINVAL, "bytes is NULL");
  *bytes = 0;
  int rc = check_wgrad_sizes(tokens, fin, fout, type);
  if (rc) return rc;
  if (cus < 0) return fail(MTA_EINVAL, "cus must be >= 0");
  int n = cus;
  if (n == 0 && (rc = current_cus(&n))) return rc;
  *bytes = wgrad_space(mta::wgrad_grid(tokens, fin, fout, type, n), fout).bytes;
  return ok();
}

int mta_ckpt_wgrad(const mta_ckpt_wgrad_args *a, void *stream) {
  if (!a) return fail(MTA_EINVAL, "args is NULL");
  int rc = check_wgrad_sizes(a->tokens, a->fin, a->fout, a->type);
  if (rc) return rc;
  if (!known_type(a->gtype))
    return fail(MTA_EDTYPE, "unknown gradient type %d", a->gtype);
  if (a->accumulate != 0 && a->accumulate != 1)
    return fail(MTA_EINVAL, "accumulate must be 0 or 1");
  if (a->reserved) return fail(MTA_EINVAL, "reserved must be 0");
  const int64_t sz = size_of(a->type), gsz = size_of(a->gtype);
  if (a->fout > 0 && a->fin > 0 && !a->dw)
    return fail(MTA_EINVAL, "dw is NULL");
  if (a->fin > 0 && a->fout > 0 && a->lddw < a->fin)
    return fail(MTA_EINVAL, "lddw is below fin");
  if (a->tokens > 0 && a->fout > 0) {
    if (!a->dy) return fail(MTA_EINVAL, "dy is NULL");
    if (a->lddy < a->fout) return fail(MTA_EINVAL, "lddy is below fout");
    if (a->fin > 0 && (!a->q || !a->scale))
      return fail(MTA_EINVAL, "q or scale is NULL");
  }
  if (!fits(a->tokens, a->lddy, sz) || !fits(a->fout, a->lddw, gsz))
    return fail(MTA_EINVAL, "too large");
  if (!aligned(a->dy, sz) || !aligned(a->dw, gsz) || !aligned(a->db, gsz))
    return fail(MTA_EALIGN, "a buffer is not aligned to its element size");
  if (!aligned(a->q, 16) || !aligned(a->workspace, 16))
    return fail(MTA_EALIGN, "q and workspace must be 16-byte aligned");
  const int64_t nb = blocks_of(a->fin);
  const int64_t ldq = nb * MTA_CKPT_BLOCK;
  int64_t need = 0;
  mta::WgradGrid grid{};
  WgradSpace space{};
  try {
    std::vector<Region> r;
    r.reserve(8);
    if (a->tokens > 0) {
      r.push_back(region(a->q, 1, a->tokens * ldq, a->tokens * ldq, "q", -1,
                         false));
      r.push_back(region(a->scale, 1, a->tokens * nb, a->tokens * nb, "scale",
                         -1, false));
      r.push_back(region(a->dy, a->tokens, a->lddy * sz, a->fout * sz, "dy",
                         -1, false));
    }
    r.push_back(region(a->dw, a->fout, a->lddw * gsz, a->fin * gsz, "dw", -1,
                       true));
    if (a->db)
      r.push_back(region(a->db, 1, a->fout * gsz, a->fout * gsz, "db", -1,
                         true));
    if ((rc = check_regions(&r))) return rc;
    if (a->fout == 0 || (a->fin == 0 && !a->db)) return ok();
    int cus = 0;
    if ((rc = current_cus(&cus))) return rc;
    grid = mta::wgrad_grid(a->tokens, a->fin, a->fout, a->type, cus);
    if (grid.whole + grid.cut * grid.parts > kMostGroups)
      return fail(MTA_EINVAL, "too large: %lld output tiles",
                  static_cast<long long>(grid.whole + grid.cut));
    space = wgrad_space(grid, a->fout);
    need = space.bytes;
    if (need > 0 && !a->workspace)
      return fail(MTA_EINVAL, "workspace is NULL");
    if (a->workspace_bytes < need)
      return fail(MTA_EINVAL, "workspace has %lld bytes, %lld are needed",
                  static_cast<long long>(a->workspace_bytes),
                  static_cast<long long>(need));
    if (need > 0) {
      r.push_back(region(a->workspace, 1, need, need, "workspace", -1, true));
      if ((rc = check_regions(&r))) return rc;
    }
  } catch (const std::bad_alloc &) {
    return fail(MTA_ENOMEM, "host allocation failed");
  }
  mta::WgradArgs w{};
  w.q = a->q;
  w.scale = a->scale;
  w.dy = a->dy;
  w.dw = a->dw;
  w.db = a->db;
  char *base = static_cast<char *>(a->workspace);
  w.part = reinterpret_cast<float *>(base);
  w.part_db = reinterpret_cast<float *>(base + space.part_db);
  w.range = reinterpret_cast<int *>(base + space.range);
  w.tokens = a->tokens;
  w.fin = a->fin;
  w.fout = a->fout;
  w.lddy = a->lddy;
  w.lddw = a->lddw;
  w.ldq = ldq;
  w.type = a->type;
  w.gtype = a->gtype;
  w.accumulate = a->accumulate;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return mta::report_launch(mta::launch_wgrad(w, grid, s), s,
                            "mta_ckpt_wgrad");
}

int mta_policy_loss_workspace(int64_t rows, int64_t *bytes) {
  if (!bytes) return fail(MTA_EINVAL, "bytes is NULL");
  *bytes = 0;
  if (rows < 0) return fail(MTA_EINVAL, "rows < 0");
  if (!fits(rows, 64, 1)) return fail(MTA_EINVAL, "too large");
  // a row's terms, and those of the stretches that many rows are joined in
  *bytes = (rows + (rows > mta::kPolicyJoin ? mta::kPolicyJoin : 0)) *
           mta::kPolicySums * 8;
  return ok();
}

int mta_policy_loss(const mta_policy_args *args, void *stream) {
  return run_policy(args, false, stream, "mta_policy_loss");
}

int mta_policy_loss_backward(const mta_policy_args *args, void *stream) {
  return run_policy(args, true, stream, "mta_policy_loss_backward");
}

}  // extern "C"
