// matrix_host.cpp -- host side and C ABI of the operators of
// include/mta_matrix.h: argument checks, launch shapes, workspace sizes.  No
// C++ exception crosses the ABI.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "matrix_internal.h"
#include "ops_check.h"

static_assert(sizeof(mta_ortho_matrix) == 80, "mta_ortho_matrix layout");
static_assert(sizeof(mta_ortho_args) == 112, "mta_ortho_args layout");
static_assert(sizeof(mta_linear_loss_args) == 176,
              "mta_linear_loss_args layout");

namespace {

using namespace mta::check;

long long ll(int64_t x) { return static_cast<long long>(x); }

int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Times of workgroups in us, measured here: a step of 64 of k takes the large
// tile 1.75, two of 128 that share a CU 1.1 and one alone 0.58, two of 64 0.5 and
// one alone 0.3; a workgroup's start and end 6, 4 and 3.
// Tiles of 64 read each operand twice as often: they are taken only where all of
// them run at once.
constexpr int kTiles[3] = {256, 128, 64};
bool too_many(int tile, int64_t groups, int64_t cus) {
  return tile == 64 && groups > 2 * cus;
}
struct TileTime {
  double step, ends;
  int64_t slots;  // workgroups at a time
};
TileTime tile_time(int tile, int64_t groups, int64_t cus) {
  const bool shared = groups > cus;
  if (tile == 256) return TileTime{1.75, 6.0, cus};
  if (tile == 128)
    return TileTime{shared ? 1.1 : 0.58, 4.0, shared ? 2 * cus : cus};
  return TileTime{shared ? 0.5 : 0.3, 3.0, shared ? 2 * cus : cus};
}

// ---- orthogonalised updates ---------------------------------------------

int check_ortho_sizes(const mta_ortho_args *a) {
  if (!a) return fail(MTA_EINVAL, "args is NULL");
  if (a->count < 0) return fail(MTA_EINVAL, "count must be >= 0");
  if (a->count > 0 && !a->matrices)
    return fail(MTA_EINVAL, "matrices is NULL");
  if (a->precise != 0 && a->precise != 1)
    return fail(MTA_EINVAL, "precise must be 0 or 1");
  for (int64_t i = 0; i < a->count; ++i) {
    const mta_ortho_matrix &m = a->matrices[i];
    if (m.rows < 0 || m.cols < 0)
      return fail(MTA_EINVAL, "matrix %lld: rows or cols < 0", ll(i));
    if (m.rows > MTA_ORTHO_MOST || m.cols > MTA_ORTHO_MOST)
      return fail(MTA_EINVAL, "matrix %lld: more than 2^20 rows or columns",
                  ll(i));
  }
  return MTA_OK;
}

// Whether every singular value of [0, 1] stays below 7 over the steps and grows
// to less than 100 times itself in one, so that what is kept in float16 stays
// finite; *pairs: in two of them, too.  And whether the smallest grow to at most
// 2^18 times themselves in all (ten usual steps): 2^-22 of X is what its two
// float16 values leave, and 2^-52 what rounding leaves in place of an eigenvalue
// of 0 beside the matrices of the small, which grows by the square.  grown[k]: what
// one of them is after any of the first k steps over what it was, at most.
bool bounded(const double *c, int steps, bool *pairs, double *grown) {
  double slope = 1.0;
  for (int k = 0; k < 3 * steps; ++k) {
    if (!std::isfinite(c[k])) return false;
    if (k % 3 == 0) slope *= std::max(1.0, std::fabs(c[k]));
  }
  if (!(slope <= 262144.0)) return false;
  // (those that are usual, without another look)
  constexpr double kUsual[3] = {3.4445, -4.7750, 2.0315};
  bool usual = true;
  for (int k = 0; k < 3 * steps; ++k) usual = usual && c[k] == kUsual[k % 3];
  *pairs = true;
  grown[0] = 1.0;
  if (usual) {
    // (the slope at 0)
    for (int s = 0; s < steps; ++s) grown[s + 1] = grown[s] * kUsual[0];
    return true;
  }
  std::fill(grown + 1, grown + steps + 1, 1.0);
  // evenly, and down to 2^-32, 16 points an octave: the smallest ones come to
  // any place in later steps
  constexpr int kEven = 512, kFine = 512;
  for (int i = 0; i <= kEven + kFine; ++i) {
    double x = i <= kEven ? static_cast<double>(i) / kEven
                          : std::exp2((kEven - i) / 16.0);
    double before = 1.0, all = 1.0;
    for (int s = 0; s < steps; ++s) {
      const double q = x * x;
      const double f = c[3 * s] + q * (c[3 * s + 1] + q * c[3 * s + 2]);
      x *= f;
      all *= f;
      grown[s + 1] = std::max(grown[s + 1], std::fabs(all));
      if (!(std::fabs(x) < 7.0) || !(std::fabs(f) < 100.0)) return false;
      if (s % 2 && !(std::fabs(f * before) < 100.0)) *pairs = false;
      before = f;
    }
  }
  for (int s = 0; s < steps; ++s) grown[s + 1] = std::max(grown[s + 1], grown[s]);
  return true;
}

// What check_ortho finds out about the coefficients.
struct OrthoCourse {
  bool pairs;
  double grown[MTA_ORTHO_STEPS + 1];
};

int check_ortho(const mta_ortho_args *a, OrthoCourse *course) {
  int rc = check_ortho_sizes(a);
  if (rc) return rc;
  if (!known_type(a->type) || !known_type(a->out_type))
    return fail(MTA_EDTYPE, "unknown type %d or %d", a->type, a->out_type);
  if (a->steps < 1 || a->steps > MTA_ORTHO_STEPS)
    return fail(MTA_EINVAL, "steps must be in [1, %d]", MTA_ORTHO_STEPS);
  if (!a->coefficients) return fail(MTA_EINVAL, "coefficients is NULL");
  if (!bounded(a->coefficients, a->steps, &course->pairs, course->grown))
    return fail(MTA_EINVAL,
                "the coefficients let a singular value of [0, 1] grow to 7, to "
                "100 times itself in a step, or to 2^18 times in all");
  if (!std::isfinite(a->eps) || a->eps < 0.0)
    return fail(MTA_EINVAL, "eps must be finite and >= 0 (got %g)", a->eps);
  if (a->nesterov != 0 && a->nesterov != 1)
    return fail(MTA_EINVAL, "nesterov must be 0 or 1");
  if (!aligned(a->d_coef, 4) || !aligned(a->d_amp, 8))
    return fail(MTA_EALIGN, "d_coef or d_amp is misaligned");
  const int64_t sz = size_of(a->type), osz = size_of(a->out_type);
  std::vector<Region> r;
  r.reserve(static_cast<size_t>(a->count) * 5 + 3);
  for (int64_t i = 0; i < a->count; ++i) {
    const mta_ortho_matrix &m = a->matrices[i];
    if (m.rows == 0 || m.cols == 0) continue;
    if (!m.g) return fail(MTA_EINVAL, "matrix %lld: g is NULL", ll(i));
    if (!m.out && !m.w)
      return fail(MTA_EINVAL, "matrix %lld: neither out nor w", ll(i));
    if (m.w16 && !m.w)
      return fail(MTA_EINVAL, "matrix %lld: w16 without w", ll(i));
    if (!std::isfinite(m.scale))
      return fail(MTA_EINVAL, "matrix %lld: scale is not finite", ll(i));
    if (m.ldg < m.cols || (m.out && m.ldout < m.cols))
      return fail(MTA_EINVAL, "matrix %lld: a row pitch is below cols", ll(i));
    if (!fits(m.rows, m.ldg, sz) || (m.out && !fits(m.rows, m.ldout, osz)))
      return fail(MTA_EINVAL, "matrix %lld: too large", ll(i));
    if (!aligned(m.g, sz) || !aligned(m.out, osz) || !aligned(m.m, 4) ||
        !aligned(m.w, 4) || !aligned(m.w16, 2))
      return fail(MTA_EALIGN,
                  "matrix %lld: a buffer is not aligned to its element size",
                  ll(i));
    if (m.m && (!std::isfinite(a->momentum) || a->momentum < 0.0))
      return fail(MTA_EINVAL, "momentum must be finite and >= 0 (got %g)",
                  a->momentum);
    if (m.w && (!std::isfinite(a->lr) || a->lr < 0.0 ||
                !std::isfinite(a->weight_decay) || a->weight_decay < 0.0))
      return fail(MTA_EINVAL, "lr and weight_decay must be finite and >= 0");
    if (m.w16 && a->copy_type != MTA_BF16 && a->copy_type != MTA_F16)
      return fail(MTA_EDTYPE, "copy_type must be MTA_BF16 or MTA_F16");
    const int64_t flat = m.rows * m.cols;
    r.push_back(region(m.g, m.rows, m.ldg * sz, m.cols * sz, "g", i, false));
    if (m.out)
      r.push_back(
          region(m.out, m.rows, m.ldout * osz, m.cols * osz, "out", i, true));
    if (m.m) r.push_back(region(m.m, 1, flat * 4, flat * 4, "m", i, true));
    if (m.w) r.push_back(region(m.w, 1, flat * 4, flat * 4, "w", i, true));
    if (m.w16)
      r.push_back(region(m.w16, 1, flat * 2, flat * 2, "w16", i, true));
  }
  if (a->d_coef)
    r.push_back(region(a->d_coef, 1, 4, 4, "d_coef", -1, false));
  if (a->d_amp) r.push_back(region(a->d_amp, 1, 24, 24, "d_amp", -1, false));
  int64_t need = 0;
  if ((rc = mta_orthogonalize_workspace(a, &need))) return rc;
  if (need > 0) {
    if (!a->workspace) return fail(MTA_EINVAL, "workspace is NULL");
    if (a->workspace_bytes < need)
      return fail(MTA_EINVAL, "workspace has %lld bytes, %lld are needed",
                  ll(a->workspace_bytes), ll(need));
    if (!aligned(a->workspace, 256))
      return fail(MTA_EALIGN, "workspace must be 256-byte aligned");
    r.push_back(region(a->workspace, 1, need, need, "workspace", -1, true));
  }
  return check_regions(&r);
}

// Output tiles of a matrix in one product.
int64_t ortho_tiles(int step, int64_t rows, int64_t cols, int64_t tile) {
  const int64_t m = up(std::min(rows, cols), tile);
  const int64_t n = up(std::max(rows, cols), tile);
  return step == mta::kOrthoGram || step == mta::kOrthoTimes ? m * (m + 1) / 2
                                                              : m * n;
}

// The matrices of a call in groups of a launch each, the small ones apart, and
// longest products first, so that the last workgroups to start are short ones.
struct OrthoGroup {
  std::vector<int64_t> index;
  int64_t bytes = 0;
  bool small = false;
  int cuts = 1;
};

// A group's workspace, at most, unless one matrix alone needs more.
constexpr int64_t kOrthoGroupBytes = int64_t{4} << 30;

int64_t ortho_bytes(const mta_ortho_matrix &m, int precise, int cuts = 1) {
  const int64_t b =
      mta::ortho_is_small(m.rows, m.cols)
          ? mta::ortho_small_space(m.rows, m.cols).bytes
          : mta::ortho_space(m.rows, m.cols, precise ? 2 : 1, cuts).bytes;
  return up(b, 256) * 256;
}

std::vector<OrthoGroup> ortho_groups(const mta_ortho_args *a) {
  std::vector<int64_t> order;
  order.reserve(static_cast<size_t>(a->count));
  for (int64_t i = 0; i < a->count; ++i)
    if (a->matrices[i].rows > 0 && a->matrices[i].cols > 0)
      order.push_back(i);
  const auto small = [&](int64_t i) {
    return mta::ortho_is_small(a->matrices[i].rows, a->matrices[i].cols);
  };
  std::stable_sort(order.begin(), order.end(), [&](int64_t x, int64_t y) {
    const mta_ortho_matrix &p = a->matrices[x], &q = a->matrices[y];
    if (small(x) != small(y)) return small(y);
    return std::max(p.rows, p.cols) > std::max(q.rows, q.cols);
  });
  std::vector<OrthoGroup> groups;
  for (int64_t i : order) {
    const int64_t bytes = ortho_bytes(a->matrices[i], a->precise);
    if (groups.empty() || groups.back().small != small(i) ||
        static_cast<int>(groups.back().index.size()) == mta::kOrthoItems ||
        groups.back().bytes + bytes > kOrthoGroupBytes) {
      groups.emplace_back();
      groups.back().small = small(i);
    }
    groups.back().index.push_back(i);
    groups.back().bytes += bytes;
  }
  // Few tiles of A with long sums are cut along k, eight steps of 64 a part at
  // least, to about one workgroup for each of 256 compute units (the workspace
  // does not depend on the device): 256 x 6400 79 us a product, now 12 and 5
  // for the joining of its parts.  Two for each were slower: an update of
  // matrices with 252 tiles of A takes 601 us so and 575 uncut.
  for (OrthoGroup &g : groups) {
    if (g.small) continue;
    int64_t tiles = 0, steps = 0;
    for (int64_t i : g.index) {
      const mta_ortho_matrix &m = a->matrices[i];
      tiles += ortho_tiles(mta::kOrthoGram, m.rows, m.cols, 128);
      steps = std::max(steps, up(std::max(m.rows, m.cols), 64));
    }
    g.cuts = static_cast<int>(std::clamp<int64_t>(
        std::min(256 / tiles, steps * (a->precise ? 3 : 1) / 8), 1, 32));
    if (g.cuts == 1) continue;
    g.bytes = 0;
    for (int64_t i : g.index)
      g.bytes += ortho_bytes(a->matrices[i], a->precise, g.cuts);
  }
  return groups;
}

hipError_t run_ortho(const mta_ortho_args *a,
                     const std::vector<OrthoGroup> &groups,
                     const OrthoCourse &course, int cus, hipStream_t s) {
  hipError_t e = hipSuccess;
  mta::OrthoCall c{};
  c.d_coef = a->d_coef;
  c.amp = a->d_amp;
  c.eps = a->eps;
  c.mu = static_cast<float>(a->momentum);
  c.decay = static_cast<float>(1.0 - a->lr * a->weight_decay);
  c.type = a->type;
  c.out_type = a->out_type;
  c.copy_type = a->copy_type;
  c.nesterov = a->nesterov;
  c.planes = a->precise ? 2 : 1;
  for (const OrthoGroup &g : groups) {
    c.cuts = g.cuts;
    mta::OrthoList l;
    l.count = static_cast<uint32_t>(g.index.size());
    uint8_t *ws = static_cast<uint8_t *>(a->workspace);
    for (uint32_t k = 0; k < l.count; ++k) {
      const mta_ortho_matrix &m = a->matrices[g.index[k]];
      l.item[k] = {m.g,
                   m.m,
                   m.out,
                   m.w,
                   m.w16,
                   ws,
                   m.ldg,
                   m.ldout,
                   static_cast<uint32_t>(m.rows),
                   static_cast<uint32_t>(m.cols),
                   static_cast<float>(m.scale),
                   static_cast<float>(-(a->lr * m.scale))};
      ws += ortho_bytes(m, a->precise, g.cuts);
    }
    const auto deal = [&](auto &&of) {
      l.first[0] = 0;
      for (uint32_t k = 0; k < l.count; ++k)
        l.first[k + 1] = l.first[k] + static_cast<uint32_t>(of(
                                          int64_t{l.item[k].rows},
                                          int64_t{l.item[k].cols}));
    };
    if (g.small) {
      mta::OrthoCoefficients co{};
      co.steps = a->steps;
      for (int k = 0; k < a->steps; ++k)
        for (int i = 0; i < 3; ++i) co.v[k][i] = a->coefficients[3 * k + i];
      deal([](int64_t r, int64_t n) {
        return mta::ortho_small_space(r, n).parts;
      });
      if ((e = mta::launch_ortho_small_gram(l, c, s)) != hipSuccess) return e;
      if ((e = mta::launch_ortho_small_factor(l, c, co, s)) != hipSuccess)
        return e;
      deal([](int64_t r, int64_t n) { return up(std::max(r, n), 64); });
      if ((e = mta::launch_ortho_small_apply(l, c, s)) != hipSuccess) return e;
      continue;
    }
    // Each kind of product's tile, and its time in us.
    const int runs = mta::pair_count(c.planes);
    int tile[4];
    double us[4];
    for (int step = 0; step < 4; ++step) {
      us[step] = 0.0;
      for (int t : kTiles) {
        const int cuts = step == mta::kOrthoGram ? g.cuts : 1;
        if (cuts > 1 && t != 128) continue;
        int64_t groups = 0;
        for (uint32_t k = 0; k < l.count; ++k)
          groups += ortho_tiles(step, l.item[k].rows, l.item[k].cols, t) * cuts;
        if (too_many(t, groups, cus)) continue;
        TileTime x = tile_time(t, groups, cus);
        // X is read and written at a tile's end, beside the products of the
        // workgroup that shares the CU with a tile of 128 (768 deep: 69 us, and 75
        // in tiles of 256; 1600 deep 410 and 350)
        if (t == 256 && step >= mta::kOrthoNext) x.ends += 4.0;
        double longest = 0.0, work = 0.0;
        for (uint32_t k = 0; k < l.count; ++k) {
          const int64_t rows = l.item[k].rows, cols = l.item[k].cols;
          const int64_t deep = step == mta::kOrthoGram ? std::max(rows, cols)
                                                       : std::min(rows, cols);
          const double one =
              static_cast<double>(up(up(deep, 64), cuts) * runs) * x.step +
              x.ends + (cuts > 1 ? 6.0 : 0.0);
          work += static_cast<double>(ortho_tiles(step, rows, cols, t) * cuts) *
                  one;
          longest = std::max(longest, one);
        }
        const double all =
            groups <= x.slots
                ? longest
                : std::max(work / static_cast<double>(x.slots) + longest / 2,
                           longest);
        if (us[step] > 0.0 && all >= us[step]) continue;
        us[step] = all;
        tile[step] = t;
      }
    }
    const auto product = [&](int step) {
      const int t = tile[step];
      if (step == mta::kOrthoGram && g.cuts > 1) {
        deal([&](int64_t r, int64_t m) {
          return ortho_tiles(step, r, m, 128) * g.cuts;
        });
        const hipError_t x = mta::launch_ortho_product(
            step, 128, l.first[l.count] <= static_cast<uint32_t>(cus), l, c, s);
        if (x != hipSuccess) return x;
        deal([&](int64_t r, int64_t m) { return ortho_tiles(step, r, m, 64); });
        return mta::launch_ortho_join(l, c, s);
      }
      deal([&](int64_t r, int64_t m) { return ortho_tiles(step, r, m, t); });
      return mta::launch_ortho_product(
          step, t, l.first[l.count] <= static_cast<uint32_t>(cus), l, c, s);
    };
    // buffer `out` = P Q, or a + b P + c P P with a step's coefficients
    const auto times = [&](int p, int q, int out, const double *of) {
      c.p = p;
      c.q = q;
      c.out = out;
      c.steps_of = of != nullptr;
      c.e0 = of ? static_cast<float>(of[2]) : 1.0f;
      c.e1 = of ? static_cast<float>(of[1]) : 0.0f;
      c.e2 = of ? static_cast<float>(of[0]) : 0.0f;
      return product(mta::kOrthoTimes);
    };
    // Two steps at once where that takes less: one product over the columns of
    // either kind less and three of small matrices more (and a launch).
    const bool by_two =
        course.pairs && us[mta::kOrthoGram] + us[mta::kOrthoNext] >
                            3.0 * us[mta::kOrthoTimes] + 5.0;
    const int blocks = by_two ? (a->steps + 1) / 2 : a->steps;
    // the step behind those that are taken together with step k, and what
    // singular values have grown by there (0: there is no step k)
    const auto behind = [&](int k) {
      return by_two ? std::min(k + 2, a->steps) : k + 1;
    };
    const auto grown = [&](int k) {
      return k < a->steps ? static_cast<float>(course.grown[behind(k)]) : 0.0f;
    };
    c.grown = grown(0);
    deal([](int64_t r, int64_t n) { return mta::ortho_parts(r, n); });
    if ((e = mta::launch_ortho_norm(l, c, s)) != hipSuccess) return e;
    deal([](int64_t r, int64_t n) {
      return up(std::min(r, n), mta::kOrthoLoadTile) *
             up(mta::plane_pitch(std::max(r, n)), mta::kOrthoLoadTile);
    });
    if ((e = mta::launch_ortho_load(l, c, s)) != hipSuccess) return e;
    c.which = 0;
    for (int k = 0, block = 0; k < a->steps; ++block) {
      const double *co = a->coefficients + 3 * k;
      const bool two = behind(k) == k + 2;
      c.grown = grown(k);
      c.grows = grown(behind(k));
      if ((e = product(mta::kOrthoGram)) != hipSuccess) return e;
      if ((e = times(0, 0, 1, co)) != hipSuccess) return e;
      double rest = co[0];
      if (two) {
        if ((e = times(0, 1, 2, nullptr)) != hipSuccess) return e;
        if ((e = times(2, 1, 0, nullptr)) != hipSuccess) return e;
        if ((e = times(0, 0, 2, co + 3)) != hipSuccess) return e;
        if ((e = times(2, 1, 0, nullptr)) != hipSuccess) return e;
        rest *= co[3];
      }
      k = behind(k);
      c.out = two ? 0 : 1;
      c.rest = static_cast<float>(rest);
      c.whole = block + 2 >= blocks;
      const int step = k < a->steps ? mta::kOrthoNext : mta::kOrthoLast;
      if ((e = product(step)) != hipSuccess) return e;
      c.which = 1 - c.which;
    }
  }
  return e;
}

// ---- cross entropy of a linear output layer -----------------------------

constexpr int64_t kMostVocab = int64_t{1} << 28;
// (255 rows of an operand are a 32-bit offset on the device)
constexpr int64_t kMostWidth = int64_t{1} << 20;
constexpr int64_t kMostPitch = int64_t{1} << 22;
constexpr int64_t kMostRows = int64_t{1} << 30;
// Workgroups of a launch, for each of its parts (of 128 x 128 at least: smaller
// ones are taken where there are few).
constexpr int64_t kMostGroups = int64_t{1} << 22;
// A plane of dz of a piece of the vocabulary, at most, unless 256 columns need
// more; there are two pieces.  (With twice as much 8192 x 1600 x 50257 takes 1.3%
// longer: dz is then read from farther away.)
constexpr int64_t kPieceBytes = int64_t{160} << 20;

// Whether the products can read w where it is.
bool lies_well(const mta_linear_loss_args *a) {
  return a->type != MTA_F32 && a->width % 64 == 0 && a->ldw % 8 == 0 &&
         a->ldw <= kMostPitch && aligned(a->w, 16);
}

// The tile of a product that is a launch of its own.
int lone_tile(int64_t m, int64_t n, int64_t k, int runs, int cus) {
  int best = 0;
  double best_us = 0.0;
  for (int tile : kTiles) {
    const int64_t groups = up(m, tile) * up(n, tile);
    if (too_many(tile, groups, cus)) continue;
    const TileTime x = tile_time(tile, groups, cus);
    const double us = static_cast<double>(up(groups, x.slots)) *
                      (x.step * static_cast<double>(up(k, 64) * runs) + x.ends);
    if (best && us >= best_us) continue;
    best = tile;
    best_us = us;
  }
  return best;
}

// Pieces, tile and parts of the gradients' launches.  A launch has dh and dw of a
// piece and dz of the next: it takes as long as its work on all CUs and, behind
// that, about half of its longest workgroup, or as that one alone; held sums cost
// their bytes at 4 TB/s.
void plan_back(const mta_linear_loss_args *a, int runs, int64_t cus,
               mta::LinearPlan *p) {
  const auto real = [](int64_t x) { return static_cast<double>(x); };
  const int64_t column = std::max<int64_t>(64, p->deep_rows) * 2;
  const int64_t most = std::max<int64_t>(256, kPieceBytes / column / 256 * 256);
  const int64_t least = up(a->vocab, most);
  double best = 0.0;
  for (int64_t n = least; n <= least + (least > 1 ? 2 : 0); ++n) {
    const int64_t piece = n == 1 ? a->vocab : up(up(a->vocab, n), 256) * 256;
    const int64_t pieces = up(a->vocab, piece);
    for (int tile : kTiles) {
      const int64_t rows = up(a->rows, tile), cols = up(a->width, tile);
      const int64_t high = up(piece, tile);
      for (int hp : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
        if (hp > 1 && (!a->dh || hp * 4 > up(piece, 64))) break;
        for (int wp : {1, 2, 4, 8, 16, 32}) {
          if (wp > 1 && (!a->dw || wp * 4 > up(a->rows, 64))) break;
          const int64_t groups = rows * (a->dh ? cols * hp : 0) + rows * high +
                                 (a->dw ? high * cols * wp : 0);
          if (too_many(tile, groups, cus)) break;
          const TileTime x = tile_time(tile, groups, cus);
          const double dz = real(up(a->width, 64) * runs) * x.step + x.ends;
          const double dh =
              a->dh ? real(up(up(piece, 64), hp) * runs) * x.step + x.ends
                    : 0.0;
          const double dw =
              a->dw ? real(up(up(a->rows, 64), wp) * runs) * x.step + x.ends
                    : 0.0;
          const double longest = std::max(std::max(dh, dw), dz);
          const double work = real(rows * cols * hp) * dh +
                              real(high * cols * wp) * dw +
                              real(rows * high) * dz;
          double us =
              groups <= x.slots
                  ? longest
                  : std::max(work / real(x.slots) + longest / 2, longest);
          const bool hold_h = a->dh && (pieces > 1 || hp > 1);
          if (hold_h) us += real(hp * a->rows * p->pitch) * 8.0 / 4e6;
          if (wp > 1) us += 5.0 + real(wp * piece * p->pitch) * 8.0 / 4e6;
          us = us * real(pieces) + (hold_h ? 5.0 : 0.0);
          if (best > 0.0 && us >= best) continue;
          best = us;
          p->piece = piece;
          p->pieces = pieces;
          p->back_tile = tile;
          p->dh_parts = hp;
          p->dw_parts = wp;
        }
      }
    }
  }
  p->pitch_z = mta::plane_pitch(p->piece);
  p->hold_dh = a->dh && (p->pieces > 1 || p->dh_parts > 1);
  p->hold_dw = a->dw && p->dw_parts > 1;
}

mta::LinearPlan linear_plan(const mta_linear_loss_args *a, bool copy_w,
                            int cus) {
  mta::LinearPlan p{};
  p.planes = a->type == MTA_F32 ? 3 : 1;
  const int runs = mta::pair_count(p.planes);
  p.copy_w = copy_w;
  p.pitch = mta::plane_pitch(a->width);
  p.deep_rows = up(a->rows, 64) * 64;
  const bool grad = a->dh || a->dw;
  p.tile = lone_tile(a->rows, a->vocab, a->width, runs, cus);
  if (grad) plan_back(a, runs, cus, &p);
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up(bytes, 256) * 256;
    return here;
  };
  const int64_t z = grad ? p.deep_rows * p.pitch_z * 2 * p.planes : 0;
  p.active = take(4);
  p.scalars = take(8);
  p.index = take(a->rows * 4);
  p.info = take(grad ? p.deep_rows * 16 : 0);
  p.terms = take(a->rows * 8);
  p.rows = take(a->rows * 16);
  p.z_target = take(a->rows * 4);
  p.partial = take(up(a->vocab, p.tile) * a->rows * 8);
  p.h = take(a->rows * p.pitch * 2 * p.planes);
  p.w = take(copy_w ? a->vocab * p.pitch * 2 * p.planes : 0);
  p.z[0] = take(z);
  p.z[1] = p.pieces > 1 ? take(z) : p.z[0];
  p.sum_h = take(p.hold_dh ? p.dh_parts * a->rows * p.pitch * 4 : 0);
  p.sum_w = take(p.hold_dw ? p.dw_parts * p.piece * p.pitch * 4 : 0);
  p.bytes = at;
  return p;
}

int check_linear_sizes(const mta_linear_loss_args *a) {
  if (!a) return fail(MTA_EINVAL, "args is NULL");
  if (a->rows < 0 || a->rows > kMostRows)
    return fail(MTA_EINVAL, "rows must be in [0, 2^30]");
  if (a->vocab < 1 || a->vocab > kMostVocab)
    return fail(MTA_EINVAL, "vocab must be in [1, 2^28] (got %lld)",
                ll(a->vocab));
  if (a->width < 1 || a->width > kMostWidth)
    return fail(MTA_EINVAL, "width must be in [1, 2^20] (got %lld)",
                ll(a->width));
  if (!known_type(a->type)) return fail(MTA_EDTYPE, "unknown type %d", a->type);
  if (up(a->rows, 128) * up(a->vocab, 128) > kMostGroups ||
      up(a->vocab, 128) * up(a->width, 128) > kMostGroups ||
      up(a->rows, 128) * up(a->width, 128) > kMostGroups)
    return fail(MTA_EINVAL, "too large");
  return MTA_OK;
}

int check_linear(const mta_linear_loss_args *a, bool backward,
                 mta::LinearPlan *plan) {
  int rc = check_linear_sizes(a);
  if (rc) return rc;
  if (!known_type(a->dw_type))
    return fail(MTA_EDTYPE, "unknown type %d", a->dw_type);
  if (a->accumulate != 0 && a->accumulate != 1)
    return fail(MTA_EINVAL, "accumulate must be 0 or 1");
  if (a->reserved) return fail(MTA_EINVAL, "reserved must be 0");
  const int64_t sz = size_of(a->type), wsz = size_of(a->dw_type);
  if (!a->w) return fail(MTA_EINVAL, "w is NULL");
  if (a->rows > 0 && (!a->h || !a->targets))
    return fail(MTA_EINVAL, "h or targets is NULL");
  if (backward && a->rows > 0 && !a->saved)
    return fail(MTA_EINVAL, "saved is NULL");
  if (backward && !a->dh && !a->dw)
    return fail(MTA_EINVAL, "neither dh nor dw");
  if (!backward && !a->loss) return fail(MTA_EINVAL, "loss is NULL");
  if (a->ldh < a->width || a->ldw < a->width ||
      (a->dh && a->lddh < a->width) || (a->dw && a->lddw < a->width))
    return fail(MTA_EINVAL, "a row pitch is below width");
  if (!fits(a->rows, a->ldh, 4) || !fits(a->vocab, a->ldw, 4) ||
      (a->dh && !fits(a->rows, a->lddh, 4)) ||
      (a->dw && !fits(a->vocab, a->lddw, 4)))
    return fail(MTA_EINVAL, "too large");
  if (!aligned(a->h, sz) || !aligned(a->w, sz) || !aligned(a->dh, sz) ||
      !aligned(a->dw, wsz) || !aligned(a->targets, 8) ||
      !aligned(a->weights, 4) || !aligned(a->d_grad_scale, 4) ||
      !aligned(a->saved, 16) || !aligned(a->logp, 4) || !aligned(a->loss, 4))
    return fail(MTA_EALIGN, "a buffer is not aligned to its element size");
  std::vector<Region> r;
  r.reserve(16);
  const auto flat = [&](const void *p, int64_t bytes, const char *name,
                        bool written) {
    if (p && bytes > 0)
      r.push_back(region(p, 1, bytes, bytes, name, -1, written));
  };
  const auto rows = [&](const void *p, int64_t n, int64_t ld, int64_t size,
                        const char *name, bool written) {
    if (p)
      r.push_back(region(p, n, ld * size, a->width * size, name, -1, written));
  };
  rows(a->h, a->rows, a->ldh, sz, "h", false);
  rows(a->w, a->vocab, a->ldw, sz, "w", false);
  rows(a->dh, a->rows, a->lddh, sz, "dh", true);
  rows(a->dw, a->vocab, a->lddw, wsz, "dw", true);
  flat(a->targets, a->rows * 8, "targets", false);
  flat(a->d_grad_scale, 4, "d_grad_scale", false);
  flat(a->saved, a->rows * 16, "saved", !backward);
  if (!backward) {
    flat(a->weights, a->rows * 4, "weights", false);
    flat(a->logp, a->rows * 4, "logp", true);
    flat(a->loss, 4, "loss", true);
  }
  if ((rc = check_regions(&r))) return rc;
  int cus = 0;
  if ((rc = current_cus(&cus))) return rc;
  *plan = linear_plan(a, !lies_well(a), cus);
  const int64_t need = plan->bytes;
  if (!a->workspace) return fail(MTA_EINVAL, "workspace is NULL");
  if (a->workspace_bytes < need)
    return fail(MTA_EINVAL, "workspace has %lld bytes, %lld are needed",
                ll(a->workspace_bytes), ll(need));
  if (!aligned(a->workspace, 256))
    return fail(MTA_EALIGN, "workspace must be 256-byte aligned");
  flat(a->workspace, need, "workspace", true);
  return check_regions(&r);
}

hipError_t run_linear(const mta_linear_loss_args *a, const mta::LinearPlan &p,
                      bool backward, hipStream_t s) {
  uint8_t *ws = static_cast<uint8_t *>(a->workspace);
  mta::LinearArgs l{};
  l.a = *a;
  l.rows = a->saved ? a->saved
                    : reinterpret_cast<mta_linear_row *>(ws + p.rows);
  l.scalars = reinterpret_cast<float *>(ws + p.scalars);
  l.active = reinterpret_cast<int *>(ws + p.active);
  l.index = reinterpret_cast<int *>(ws + p.index);
  l.info = reinterpret_cast<mta::LinearInfo *>(ws + p.info);
  l.terms = reinterpret_cast<double *>(ws + p.terms);
  l.z_target = reinterpret_cast<float *>(ws + p.z_target);
  l.partial = reinterpret_cast<float2 *>(ws + p.partial);
  l.h = reinterpret_cast<uint16_t *>(ws + p.h);
  l.sum_h = reinterpret_cast<float *>(ws + p.sum_h);
  l.sum_w = reinterpret_cast<float *>(ws + p.sum_w);
  l.planes = p.planes;
  l.backward = backward;
  l.pitch = p.pitch;
  l.pitch_z = p.pitch_z;
  l.h_plane = a->rows * p.pitch;
  l.z_plane = p.deep_rows * p.pitch_z;
  l.tiles = up(a->vocab, p.tile);
  hipError_t e;
  const auto ok = [&](hipError_t x) { return (e = x) == hipSuccess; };
  if (!ok(mta::launch_linear_rows_in(l, s))) return e;
  if (a->rows > 0) {
    if (p.copy_w) {
      uint16_t *to = reinterpret_cast<uint16_t *>(ws + p.w);
      l.w = to;
      l.w_pitch = p.pitch;
      l.w_plane = a->vocab * p.pitch;
      if (!ok(mta::launch_linear_pack_w(l, to, s))) return e;
    } else {
      l.w = static_cast<const uint16_t *>(a->w);
      l.w_pitch = a->ldw;
    }
  }
  if (!backward) {
    if (a->rows > 0 && !ok(mta::launch_linear_logits(l, p.tile, s))) return e;
    if (!ok(mta::launch_linear_rows(l, s))) return e;
  }
  if (!a->dh && !a->dw) return e;
  if (a->rows == 0) return a->dw ? mta::launch_linear_none(l, s) : e;
  if (!ok(mta::launch_linear_info(l, s))) return e;
  const auto piece = [&](int64_t k) {
    const int64_t first = k * p.piece;
    return mta::LinearPiece{first, std::min(p.piece, a->vocab - first),
                            reinterpret_cast<uint16_t *>(ws + p.z[k % 2])};
  };
  const mta::LinearBack back{p.dh_parts, p.dw_parts, p.hold_dh, p.hold_dw, 0,
                             0};
  mta::LinearPiece here, next = piece(0);
  if (!ok(mta::launch_linear_back(l, p.back_tile, nullptr, &next, back, s)))
    return e;
  for (int64_t k = 0; k < p.pieces; ++k) {
    here = next;
    const bool more = k + 1 < p.pieces;
    if (more) next = piece(k + 1);
    if (!ok(mta::launch_linear_back(l, p.back_tile, &here,
                                    more ? &next : nullptr, back, s)))
      return e;
    if (p.hold_dw &&
        !ok(mta::launch_linear_out(l, here, false, p.dw_parts, s)))
      return e;
  }
  if (p.hold_dh) e = mta::launch_linear_out(l, here, true, p.dh_parts, s);
  return e;
}

int call_linear(const mta_linear_loss_args *a, bool backward, void *stream,
                const char *what) {
  mta::LinearPlan plan{};
  try {
    const int rc = check_linear(a, backward, &plan);
    if (rc) return rc;
  } catch (const std::bad_alloc &) {
    return fail(MTA_ENOMEM, "host allocation failed");
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  return mta::report_launch(run_linear(a, plan, backward, s), s, what);
}

}  // namespace

extern "C" {

int mta_linear_loss_workspace(const mta_linear_loss_args *a, int32_t cus,
                              int64_t *bytes) {
  if (!bytes) return fail(MTA_EINVAL, "bytes is NULL");
  *bytes = 0;
  int rc = check_linear_sizes(a);
  if (rc) return rc;
  if (cus < 0) return fail(MTA_EINVAL, "cus must be >= 0");
  int n = cus;
  if (n == 0 && (rc = current_cus(&n))) return rc;
  *bytes = linear_plan(a, !lies_well(a), n).bytes;
  return ok();
}

int mta_linear_loss(const mta_linear_loss_args *args, void *stream) {
  return call_linear(args, false, stream, "mta_linear_loss");
}

int mta_linear_loss_backward(const mta_linear_loss_args *args, void *stream) {
  return call_linear(args, true, stream, "mta_linear_loss_backward");
}

int mta_matrix_version(void) { return MTA_MATRIX_VERSION; }

int mta_orthogonalize_workspace(const mta_ortho_args *a, int64_t *bytes) {
  if (!bytes) return fail(MTA_EINVAL, "bytes is NULL");
  *bytes = 0;
  const int rc = check_ortho_sizes(a);
  if (rc) return rc;
  try {
    for (const OrthoGroup &g : ortho_groups(a))
      *bytes = std::max(*bytes, g.bytes);
  } catch (const std::bad_alloc &) {
    return fail(MTA_ENOMEM, "host allocation failed");
  }
  return ok();
}

int mta_orthogonalize(const mta_ortho_args *a, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  try {
    OrthoCourse course;
    int rc = check_ortho(a, &course);
    if (rc) return rc;
    const std::vector<OrthoGroup> groups = ortho_groups(a);
    if (groups.empty()) return ok();
    int cus = 0;
    if ((rc = current_cus(&cus))) return rc;
    e = run_ortho(a, groups, course, cus, s);
  } catch (const std::bad_alloc &) {
    return fail(MTA_ENOMEM, "host allocation failed");
  }
  return mta::report_launch(e, s, "mta_orthogonalize");
}

}  // extern "C"
