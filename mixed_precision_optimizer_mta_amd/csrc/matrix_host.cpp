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

namespace {

using namespace mta::check;

long long ll(int64_t x) { return static_cast<long long>(x); }

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

// Whether every singular value of [0, 1] stays below 7 over the steps, so that
// what is kept in float16 stays finite.
bool bounded(const double *c, int steps) {
  for (int k = 0; k < 3 * steps; ++k)
    if (!std::isfinite(c[k])) return false;
  constexpr int kPoints = 512;
  for (int i = 1; i <= kPoints; ++i) {
    double x = static_cast<double>(i) / kPoints;
    for (int s = 0; s < steps; ++s) {
      const double q = x * x;
      x *= c[3 * s] + q * (c[3 * s + 1] + q * c[3 * s + 2]);
      if (!(std::fabs(x) < 7.0)) return false;
    }
  }
  return true;
}

int check_ortho(const mta_ortho_args *a) {
  int rc = check_ortho_sizes(a);
  if (rc) return rc;
  if (!known_type(a->type) || !known_type(a->out_type))
    return fail(MTA_EDTYPE, "unknown type %d or %d", a->type, a->out_type);
  if (a->steps < 1 || a->steps > MTA_ORTHO_STEPS)
    return fail(MTA_EINVAL, "steps must be in [1, %d]", MTA_ORTHO_STEPS);
  if (!a->coefficients) return fail(MTA_EINVAL, "coefficients is NULL");
  if (!bounded(a->coefficients, a->steps))
    return fail(MTA_EINVAL,
                "the coefficients let a singular value of [0, 1] grow to 7");
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

// The matrices of a call in groups of a launch each, longest products first,
// so that the last workgroups to start are short ones.
struct OrthoGroup {
  std::vector<int64_t> index;
  int64_t bytes = 0;
};

// A group's workspace, at most, unless one matrix alone needs more.
constexpr int64_t kOrthoGroupBytes = int64_t{4} << 30;

int64_t ortho_bytes(const mta_ortho_matrix &m, int precise) {
  const int64_t b =
      mta::ortho_space(m.rows, m.cols,
                       mta::ortho_planes(m.rows, m.cols, precise))
          .bytes;
  return (b + 255) / 256 * 256;
}

std::vector<OrthoGroup> ortho_groups(const mta_ortho_args *a) {
  std::vector<int64_t> order;
  order.reserve(static_cast<size_t>(a->count));
  for (int64_t i = 0; i < a->count; ++i)
    if (a->matrices[i].rows > 0 && a->matrices[i].cols > 0)
      order.push_back(i);
  std::stable_sort(order.begin(), order.end(), [&](int64_t x, int64_t y) {
    const mta_ortho_matrix &p = a->matrices[x], &q = a->matrices[y];
    return std::max(p.rows, p.cols) > std::max(q.rows, q.cols);
  });
  std::vector<OrthoGroup> groups;
  for (int64_t i : order) {
    const int64_t bytes = ortho_bytes(a->matrices[i], a->precise);
    if (groups.empty() ||
        static_cast<int>(groups.back().index.size()) == mta::kOrthoItems ||
        groups.back().bytes + bytes > kOrthoGroupBytes)
      groups.emplace_back();
    groups.back().index.push_back(i);
    groups.back().bytes += bytes;
  }
  return groups;
}

int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

// Output tiles of a matrix in one product.
int64_t ortho_tiles(int step, int64_t rows, int64_t cols, int64_t tile) {
  const int64_t m = up(std::min(rows, cols), tile);
  const int64_t n = up(std::max(rows, cols), tile);
  return step == mta::kOrthoGram || step == mta::kOrthoSquare ? m * (m + 1) / 2
                                                              : m * n;
}

hipError_t run_ortho(const mta_ortho_args *a,
                     const std::vector<OrthoGroup> &groups, int cus,
                     hipStream_t s) {
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
  for (const OrthoGroup &g : groups) {
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
                   mta::ortho_planes(m.rows, m.cols, a->precise),
                   static_cast<float>(m.scale),
                   static_cast<float>(-(a->lr * m.scale))};
      ws += ortho_bytes(m, a->precise);
    }
    const auto deal = [&](auto &&of) {
      l.first[0] = 0;
      for (uint32_t k = 0; k < l.count; ++k)
        l.first[k + 1] = l.first[k] + static_cast<uint32_t>(of(
                                          int64_t{l.item[k].rows},
                                          int64_t{l.item[k].cols}));
    };
    deal([](int64_t r, int64_t n) { return mta::ortho_parts(r, n); });
    if ((e = mta::launch_ortho_norm(l, c, s)) != hipSuccess) return e;
    deal([](int64_t r, int64_t n) {
      return up(std::min(r, n), mta::kOrthoLoadTile) *
             up(mta::plane_pitch(std::max(r, n)), mta::kOrthoLoadTile);
    });
    if ((e = mta::launch_ortho_load(l, c, s)) != hipSuccess) return e;
    const auto product = [&](int step) {
      // The large tile takes a CU for as long as 1.8 small ones, two of which
      // share one: whichever needs less.
      int64_t n[2] = {0, 0};
      for (uint32_t k = 0; k < l.count; ++k)
        for (int t = 0; t < 2; ++t)
          n[t] += ortho_tiles(step, l.item[k].rows, l.item[k].cols,
                              t ? 256 : 128);
      const int tile =
          up(n[1], cus) * 18 <= up(n[0], 2 * cus) * 10 ? 256 : 128;
      deal([&](int64_t r, int64_t m) { return ortho_tiles(step, r, m, tile); });
      return mta::launch_ortho_product(step, tile, l, c, s);
    };
    c.which = 0;
    for (int k = 0; k < a->steps; ++k) {
      c.a = static_cast<float>(a->coefficients[3 * k]);
      c.b = static_cast<float>(a->coefficients[3 * k + 1]);
      c.c = static_cast<float>(a->coefficients[3 * k + 2]);
      const bool last = k + 1 == a->steps;
      c.whole = k + 2 >= a->steps;
      if ((e = product(mta::kOrthoGram)) != hipSuccess) return e;
      if ((e = product(mta::kOrthoSquare)) != hipSuccess) return e;
      if ((e = product(last ? mta::kOrthoLast : mta::kOrthoNext)) !=
          hipSuccess)
        return e;
      c.which = 1 - c.which;
    }
  }
  return e;
}

}  // namespace

extern "C" {

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
    int rc = check_ortho(a);
    if (rc) return rc;
    const std::vector<OrthoGroup> groups = ortho_groups(a);
    if (groups.empty()) return ok();
    int cus = 0;
    if ((rc = current_cus(&cus))) return rc;
    e = run_ortho(a, groups, cus, s);
  } catch (const std::bad_alloc &) {
    return fail(MTA_ENOMEM, "host allocation failed");
  }
  return mta::report_launch(e, s, "mta_orthogonalize");
}

}  // extern "C"
