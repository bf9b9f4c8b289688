// ortho_kernels.hip -- the orthogonalised update of the Muon rule on the matrix
// cores of gfx950, for the matrices of a list together.
//
//   X = u / (|u| + eps);  steps times  X = Q X,  Q = a + b R + c R R,  R = X X^T
//
// u is the gradient or its momentum, X the one with fewer rows than columns of
// u and its transpose.  One launch a product, over the tiles of all matrices;
// those of symmetric matrices are computed on and right of the diagonal and
// copied.  X of many columns is read and written once for two steps: the second
// one's R is Q R Q, and (Q' Q) X its result, five products of small matrices in
// the place of one of each kind over the columns.  (Three steps at once, or all
// of them, would not do in 16 bits: an eigenvalue of R that rounding has made
// negative grows by a^2 = 12 a step.)
//
// Which digits are kept.  Small singular values grow by a = 3.4 in a step and
// gradients have many: with X in bfloat16 the result is off by 1.3% of its norm
// for normal entries and by 32% where four directions stand out a thousandfold,
// whatever the products' sums.  X is therefore kept in 22 bits, as the sum of
// two float16 values (scaled by 2^13, so that 1/sqrt(rows cols) and its rest are
// normal numbers; by more for a matrix whose norm is far below eps, until it has
// grown).  The products take the first values alone.  What hurts then
// is that Q's diagonal, 1 of rows that have converged but -2.6 + 3.4, is rounded
// with the rest: diagonals are kept in float32 apart and enter as d_i X_i, and
// the error falls from 2.9e-3 to 4.5e-4 (512 x 2048 normal entries).  In the
// first steps the diagonal's part of R multiplies the rounded X that R was made
// from, so that small directions cancel as they do in R (from 3.3e-3 to 6.8e-4
// where eight directions stand out); in the last two products the whole X.  With
// `precise` every product is of both values: 4e-7.
//
// Large matrices are bound by the matrix pipes at the clock that this card's power
// allows: four of 6400 x 1600 and four of 1600 x 6400 take 2.22 ms for the 1.54
// TFLOP of a (2, 2, 1) course, and a library product of that size would take 1.25.
// Small ones are bound by launches of which each waits for the one before: twelve
// of 768 x 768 take 0.30 to 0.35 ms in 17 launches, of whose products' 17 to 23 us
// (under a tracer) 12 steps along k are 7, what comes before the first and after
// the last the rest.
#include "gemm_device.h"
#include "ortho_device.h"

namespace mta {
namespace {

// Powers of two that the float16 values are multiplied by: room for singular
// values of 7 in X and of 100 in the symmetric matrices.
constexpr float kScaleX = 8192.0f, kScaleA = 512.0f;

// Eight values as float16, and with Two what their roundings leave as a second
// eight (an infinity leaves a NaN: its matrix is lost anyway).
template <bool Two>
__device__ __forceinline__ void store_planes(uint16_t *hi_at, int64_t plane,
                                             const float (&x)[8]) {
  u32x4 hi, lo;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    hi[k] = narrow2<MTA_F16>(x[2 * k], x[2 * k + 1]);
    if constexpr (Two)
      lo[k] = narrow2<MTA_F16>(x[2 * k] - widen<MTA_F16>(hi[k] & 0xFFFFu),
                               x[2 * k + 1] - widen<MTA_F16>(hi[k] >> 16));
  }
  *(MTA_GLOBAL u32x4 *)hi_at = hi;
  if constexpr (Two) *(MTA_GLOBAL u32x4 *)(hi_at + plane) = lo;
}

// The momentum takes the gradient in, and the squares of u are summed: partial
// sums of a matrix by workgroup, each lane's in order.  Bound by memory: a
// gradient is read once, a momentum read and written.
template <int D>
__global__ __launch_bounds__(256) void k_ortho_norm(const OrthoList l,
                                                    const OrthoCall c) {
  const int k = item_of(l, blockIdx.x);
  const OrthoItem &it = l.item[k];
  const int64_t part = blockIdx.x - l.first[k];
  const int64_t parts = l.first[k + 1] - l.first[k];
  const Look look = look_of(c);
  const bool skip = c.amp && c.amp->found_inf != 0.0f;
  // a matrix without gaps is one row
  const bool flat = it.ldg == it.cols || it.rows == 1;
  const int64_t cols = flat ? int64_t{it.rows} * it.cols : it.cols;
  const int64_t rows = flat ? 1 : it.rows;
  const int64_t runs = (cols + 7) / 8;
  double sum = 0.0;
  for (int64_t q = part * 256 + threadIdx.x; q < rows * runs;
       q += parts * 256) {
    const int64_t r = flat ? 0 : q / runs;
    const int64_t i = (flat ? q : q - r * runs) * 8;
    const int n = static_cast<int>(min(int64_t{8}, cols - i));
    const Raw8<D> g = n == 8 ? load8<D, false>(it.g, r * it.ldg + i)
                             : load8_part<D>(it.g, r * it.ldg + i, n, 0);
    if (it.m) {
      const int64_t at = r * it.cols + i;
      const Raw8<MTA_F32> m = n == 8 ? load8<MTA_F32, false>(it.m, at)
                                     : load8_part<MTA_F32>(it.m, at, n, 0);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = look.gradient(g[e]);
        y[e] = look.next(m[e], x);
        const double u = look.ahead(y[e], x);
        if (e < n) sum = __builtin_fma(u, u, sum);
      }
      if (!skip) {
        if (n == 8) {
          store8<MTA_F32, false>(it.m, at, y);
        } else {
          for (int e = 0; e < n; ++e) it.m[at + e] = y[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double u = look.gradient(g[e]);
        if (e < n) sum = __builtin_fma(u, u, sum);
      }
    }
  }
  __shared__ double four[4];
  sum = sum256(sum, four);
  const OrthoSpace sp = ortho_space(it.rows, it.cols, c.planes, c.cuts);
  if (threadIdx.x == 0)
    reinterpret_cast<double *>(it.ws + sp.part)[part] = sum;
}

// X from u: a workgroup takes 64 x 64 of X, turned through LDS where u has more
// rows than columns.
template <int D>
__global__ __launch_bounds__(256) void k_ortho_load(const OrthoList l,
                                                    const OrthoCall c) {
  constexpr int kT = kOrthoLoadTile;
  const int k = item_of(l, blockIdx.x);
  const OrthoItem &it = l.item[k];
  const OrthoSpace sp = ortho_space(it.rows, it.cols, c.planes, c.cuts);
  __shared__ double four[4];
  __shared__ float tile[kT][kT + 1];
  const int64_t parts = ortho_parts(it.rows, it.cols);
  const double mine =
      threadIdx.x < parts
          ? reinterpret_cast<const double *>(it.ws + sp.part)[threadIdx.x]
          : 0.0;
  const double size = sqrt(sum256(mine, four)), norm = size + c.eps;
  // (zeros stay zeros, however small eps is)
  const float begin = size == 0.0 ? 0.0f : static_cast<float>(size / norm);
  const double factor =
      size == 0.0 ? 0.0
                  : ldexp(kScaleX / norm, lift_of(begin, c.grown));
  const Look look = look_of(c);
  const bool skip = c.amp && c.amp->found_inf != 0.0f;
  const bool tall = it.rows > it.cols;
  if (blockIdx.x == l.first[k]) {
    for (int n = 0; n < kOrthoSquares; ++n)
      for (int64_t i = sp.small + threadIdx.x; i < sp.pitch_a; i += 256)
        reinterpret_cast<float *>(it.ws + sp.diag + n * sp.next_diag)[i] = 0.0f;
    if (threadIdx.x == 0) *reinterpret_cast<float *>(it.ws + sp.norm) = begin;
  }
  const uint32_t t = blockIdx.x - l.first[k];
  const uint32_t wide = static_cast<uint32_t>(sp.pitch_x) / kT;
  const int64_t m0 = int64_t{t / wide} * kT, n0 = int64_t{t % wide} * kT;
  // the place in u: rows r0 .., columns c0 ..
  const int64_t r0 = tall ? n0 : m0, c0 = tall ? m0 : n0;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int y = p * 32 + threadIdx.x / 8, x = threadIdx.x % 8 * 8;
    const int64_t r = r0 + y, col = c0 + x;
    const int n = r < it.rows && col < it.cols
                      ? static_cast<int>(min(int64_t{8}, it.cols - col))
                      : 0;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0) {
      const int64_t ag = r * it.ldg + col, am = r * it.cols + col;
      const Raw8<D> g = n == 8 ? load8<D, false>(it.g, ag)
                               : load8_part<D>(it.g, ag, n, 0);
      if (it.m) {
        const Raw8<MTA_F32> m = n == 8 ? load8<MTA_F32, false>(it.m, am)
                                       : load8_part<MTA_F32>(it.m, am, n, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gr = look.gradient(g[e]);
          // (skipped: m is still the old one)
          const float now = skip ? look.next(m[e], gr) : m[e];
          v[e] = look.ahead(now, gr);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = look.gradient(g[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = e < n ? static_cast<float>(v[e] * factor) : 0.0f;
    }
    if (tall) {
#pragma unroll
      for (int e = 0; e < 8; ++e) tile[x + e][y] = v[e];
    } else if (r < sp.small && col < sp.pitch_x) {
      auto *hi = reinterpret_cast<uint16_t *>(it.ws + sp.x) +
                 r * sp.pitch_x + col;
      store_planes<true>(hi, sp.plane_x, v);
    }
  }
  if (!tall) return;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int y = p * 32 + threadIdx.x / 8, x = threadIdx.x % 8 * 8;
    const int64_t m = m0 + y, n = n0 + x;
    if (m >= sp.small || n >= sp.pitch_x) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[y][x + e];
    auto *hi =
        reinterpret_cast<uint16_t *>(it.ws + sp.x) + m * sp.pitch_x + n;
    store_planes<true>(hi, sp.plane_x, v);
  }
}

// The diagonal's value among eight of a row, if it is there, goes to its own
// array and leaves a zero; so do the values behind the last column.
__device__ __forceinline__ void take_diagonal(float *diag, int64_t row,
                                              int64_t col, int64_t small,
                                              float (&v)[8]) {
  const int64_t own = row - col, left = small - col;
  float d = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    d = e == own ? v[e] : d;
    v[e] = e == own || e >= left ? 0.0f : v[e];
  }
  if (own >= 0 && own < 8) diag[row] = d;
}

// A's parts joined in order: a workgroup takes 64 x 64 on or right of the
// diagonal and writes its mirror image too.
__global__ __launch_bounds__(256) void k_ortho_join(const OrthoList l,
                                                    const OrthoCall c) {
  __shared__ float tile[64][65];
  const int k = item_of(l, blockIdx.x);
  const OrthoItem &it = l.item[k];
  const OrthoSpace sp = ortho_space(it.rows, it.cols, c.planes, c.cuts);
  const uint32_t side = static_cast<uint32_t>(sp.small + 63) / 64;
  uint32_t tn = blockIdx.x - l.first[k], tm = 0;
  while (tn >= side - tm) tn -= side - tm++;
  tn += tm;
  auto *to = reinterpret_cast<uint16_t *>(it.ws + sp.a);
  auto *diag = reinterpret_cast<float *>(it.ws + sp.diag);
  const auto *from = reinterpret_cast<const float *>(it.ws + sp.cut);
  const int y = threadIdx.x / 8, x = threadIdx.x % 8 * 8;
  const auto put = [&](int64_t row, int64_t col, float (&v)[8]) {
    if (tm == tn || tn + 1 == side) take_diagonal(diag, row, col, sp.small, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= kScaleA;
    auto *at = to + row * sp.pitch_a + col;
    if (c.planes > 1) store_planes<true>(at, sp.plane_a, v);
    else store_planes<false>(at, 0, v);
  };
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int64_t row = tm * 64 + p * 32 + y, col = tn * 64 + x;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row < sp.small) {
#pragma unroll 4
      for (int q = 0; q < c.cuts; ++q) {
        const Raw8<MTA_F32> u = load8<MTA_F32, false>(
            from, q * sp.plane_a + row * sp.pitch_a + col);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += u[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) tile[x + e][p * 32 + y] = v[e];
      put(row, col, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) tile[x + e][p * 32 + y] = 0.0f;
    }
  }
  if (tm == tn) return;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int64_t row = tn * 64 + p * 32 + y, col = tm * 64 + x;
    if (row >= sp.small) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tile[p * 32 + y][x + e];
    put(row, col, v);
  }
}

// One tile of a step's product.
template <class C, int Step, int Planes>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_ortho_product(const OrthoList l, const OrthoCall c) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  const uint32_t block = beside(blockIdx.x, gridDim.x);
  const int k = item_of(l, block);
  const OrthoItem &it = l.item[k];
  const OrthoSpace sp = ortho_space(it.rows, it.cols, Planes, c.cuts);
  const uint32_t t = block - l.first[k];
  constexpr bool kSym = Step == kOrthoGram || Step == kOrthoTimes;
  constexpr bool kTwo = Planes > 1;
  const uint32_t side = static_cast<uint32_t>(sp.small + C::kBM - 1) / C::kBM;
  const uint32_t part = Step == kOrthoGram ? t % c.cuts : 0;
  uint32_t tm, tn;
  if constexpr (kSym) {
    // tiles on and right of the diagonal, row by row
    uint32_t left = Step == kOrthoGram ? t / c.cuts : t;
    tm = 0;
    while (left >= side - tm) left -= side - tm++;
    tn = tm + left;
  } else {
    banded(t, side, static_cast<uint32_t>(sp.large + C::kBN - 1) / C::kBN, tm,
           tn);
  }
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  auto *x_old =
      reinterpret_cast<uint16_t *>(it.ws + sp.x + c.which * sp.next_x);
  const auto square = [&](int n) {
    return reinterpret_cast<uint16_t *>(it.ws + sp.a + n * sp.next_a);
  };
  const auto diagonal = [&](int n) {
    return reinterpret_cast<float *>(it.ws + sp.diag + n * sp.next_diag);
  };
  const Pairs pairs = pairs_of(Planes);
  const int64_t deep_x = (sp.large + 63) / 64 * 64;
  const int64_t deep_a = (sp.small + 63) / 64 * 64;
  // rows that are there, from the tile's first
  const int rows = static_cast<int>(min(sp.small - m0, int64_t{C::kBM}));
  // (on its way until the sums are there)
  const float begin = *reinterpret_cast<const float *>(it.ws + sp.norm);
  f32x16 acc[C::kRM][C::kRN];

  if constexpr (kSym) {
    if constexpr (Step == kOrthoGram) {
      const Operand x{x_old, sp.plane_x, sp.pitch_x, sp.small, sp.small};
      const int64_t each = (deep_x / 64 + c.cuts - 1) / c.cuts * 64;
      const int64_t k0 = min(deep_x, part * each);
      tile_product<C, true, kAlong, kAlong>(x, x, pairs, m0, n0, k0,
                                            min(deep_x, k0 + each), lds, acc);
    } else {
      const Operand p{square(c.p), sp.plane_a, sp.pitch_a, sp.small, sp.small};
      const Operand q{square(c.q), sp.plane_a, sp.pitch_a, sp.small, sp.small};
      tile_product<C, true, kAlong, kAlong>(p, q, pairs, m0, n0, 0, deep_a, lds,
                                            acc);
    }
    float *cut = Step == kOrthoGram && c.cuts > 1
                     ? reinterpret_cast<float *>(it.ws + sp.cut) +
                           part * sp.plane_a + m0 * sp.pitch_a + n0
                     : nullptr;
    // from the tile's corner, and from its mirror image's, in 32 bits a lane
    const uint32_t pitch = static_cast<uint32_t>(sp.pitch_a);
    const int cols = static_cast<int>(min(sp.pitch_a - n0, int64_t{C::kBN}));
    const int out = Step == kOrthoGram ? 0 : c.out;
    uint16_t *to = square(out);
    float *diag = diagonal(out);
    const int64_t corner = m0 * sp.pitch_a + n0;
    uint16_t *here = to + corner, *there = to + n0 * sp.pitch_a + m0;
    const uint16_t *at_p = square(c.p) + corner, *at_q = square(c.q) + corner;
    const float *diag_p = diagonal(c.p), *diag_q = diagonal(c.q);
    // A is that of the lifted X
    const int lift = lift_of(begin, c.grown);
    const float e1 = scalar(c.steps_of ? ldexpf(c.e1, -2 * lift) : c.e1);
    const float e0 = scalar(c.steps_of ? ldexpf(c.e0, -4 * lift) : c.e0);
    // the tile holds a part of the diagonal, or a last column
    const bool edge = tm == tn || tn + 1 == side;
    struct Seen {
      Raw8<MTA_F16> p, q, p_lo, q_lo;
      float row;
      Raw8<MTA_F32> col;
    };
    // With P = D + O, Q = E + N and D, E their diagonals:
    // P Q = O N + D N + O E + D E, in units of kScaleA
    tile_out<C, true>(
        lds, acc, true, tm != tn && !cut,
        [&](int m, int n) {
          Seen x;
          if constexpr (Step == kOrthoTimes) {
            m = min(m, rows - 1);
            n = min(n, cols - 8);
            const uint32_t at = static_cast<uint32_t>(m) * pitch + n;
            x.p = load8<MTA_F16, false>(at_p + at, 0);
            x.q = load8<MTA_F16, false>(at_q + at, 0);
            if constexpr (kTwo) {
              x.p_lo = load8<MTA_F16, false>(at_p + at + sp.plane_a, 0);
              x.q_lo = load8<MTA_F16, false>(at_q + at + sp.plane_a, 0);
            }
            x.row = diag_p[m0 + m];
            x.col = load8<MTA_F32, false>(diag_q + n0, n);
          }
          return x;
        },
        [&](int m, int n, float (&v)[8], const Seen &x) {
          if (m >= rows || n >= cols) return;
          const uint32_t at = static_cast<uint32_t>(m) * pitch + n;
          if constexpr (Step == kOrthoGram) {
            if (cut) {
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] *= 1.0f / (kScaleX * kScaleX);
              auto *p = (MTA_GLOBAL f32x4 *)(cut + at);
              p[0] = f32x4{v[0], v[1], v[2], v[3]};
              p[1] = f32x4{v[4], v[5], v[6], v[7]};
              return;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[e] *= kScaleA / (kScaleX * kScaleX);
          } else {
            const float of_q = e0 * x.row;
            const int64_t own = m0 + m - (n0 + n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float o = x.p[e], r = x.q[e];
              if constexpr (kTwo) {
                o += x.p_lo[e];
                r += x.q_lo[e];
              }
              const float of_p = __builtin_fmaf(e0, x.col[e], e1);
              float y = __builtin_fmaf(
                  of_p, o,
                  __builtin_fmaf(of_q, r, v[e] * (e0 / kScaleA)));
              // (O and N are 0 there)
              if (edge && e == own)
                y += kScaleA * __builtin_fmaf(of_p, x.row, c.e2);
              v[e] = y;
            }
          }
          if (edge) {
            const int64_t own = m0 + m - (n0 + n);
            const int64_t left = sp.small - (n0 + n);
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              d = e == own ? v[e] : d;
              v[e] = e == own || e >= left ? 0.0f : v[e];
            }
            if (own >= 0 && own < 8) diag[m0 + m] = d * (1.0f / kScaleA);
          }
          store_planes<kTwo>(here + at, sp.plane_a, v);
        },
        [](int, int) { return 0; },
        [&](int n, int m, float (&v)[8], int) {
          // (rows of the mirror image are the columns; all of its columns are)
          if (n0 + n >= sp.small) return;
          const uint32_t at = static_cast<uint32_t>(n) * pitch + m;
          store_planes<kTwo>(there + at, sp.plane_a, v);
        });
  } else {
    const Operand b{square(c.out), sp.plane_a, sp.pitch_a, sp.small, sp.small};
    const float *diag = diagonal(c.out);
    tile_product<C, true, kAlong, kAcross>(
        b, Operand{x_old, sp.plane_x, sp.pitch_x, sp.pitch_x, sp.small}, pairs,
        m0, n0, 0, deep_a, lds, acc);
    const bool tall = it.rows > it.cols;
    const bool skip = c.amp && c.amp->found_inf != 0.0f;
    const uint32_t pitch = static_cast<uint32_t>(sp.pitch_x);
    const int cols = static_cast<int>(min(sp.pitch_x - n0, int64_t{C::kBN}));
    const uint16_t *from = x_old + m0 * sp.pitch_x + n0;
    uint16_t *to = reinterpret_cast<uint16_t *>(
                       it.ws + sp.x + (1 - c.which) * sp.next_x) +
                   m0 * sp.pitch_x + n0;
    // kept: times kScaleX and what the next steps leave of the lift; handed out:
    // as it is
    const float to_next =
        scalar(ldexpf(Step == kOrthoLast ? 1.0f / kScaleX : 1.0f,
                      lift_of(begin, c.grows) - lift_of(begin, c.grown)));
    struct Seen {
      Raw8<MTA_F16> hi, lo;
      float diag;
    };
    tile_out<C, Step == kOrthoLast>(
        lds, acc, true, Step == kOrthoLast && tall,
        [&](int m, int n) {
          m = min(m, rows - 1);
          n = min(n, cols - 8);
          const uint32_t at = static_cast<uint32_t>(m) * pitch + n;
          return Seen{load8<MTA_F16, false>(from + at, 0),
                      load8<MTA_F16, false>(from + at + sp.plane_x, 0),
                      diag[m0 + m]};
        },
        [&](int m, int n, float (&v)[8], const Seen &x) {
          if (m >= rows || n >= cols) return;
          const float of_hi = x.diag * to_next;
          const float of_lo = kTwo || c.whole ? of_hi : c.rest * to_next;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = __builtin_fmaf(
                of_hi, x.hi[e],
                __builtin_fmaf(of_lo, x.lo[e], v[e] * (to_next / kScaleA)));
          if constexpr (Step == kOrthoNext)
            store_planes<true>(to + static_cast<uint32_t>(m) * pitch + n,
                               sp.plane_x, v);
          else if (!tall)
            put_result(it, c, m0 + m, n0 + n, v, skip);
        },
        [](int, int) { return 0; },
        [&](int n, int m, float (&v)[8], int) {
          if constexpr (Step == kOrthoLast)
            put_result(it, c, n0 + n, m0 + m, v, skip);
        });
  }
}

template <class C, int Planes>
hipError_t start(int step, const OrthoList &l, const OrthoCall &c,
                 hipStream_t s) {
  const auto go = [&](auto which) {
    k_ortho_product<C, decltype(which)::value, Planes>
        <<<l.first[l.count], C::kThreads, 0, s>>>(l, c);
    return hipGetLastError();
  };
  switch (step) {
    case kOrthoGram: return go(std::integral_constant<int, kOrthoGram>{});
    case kOrthoTimes: return go(std::integral_constant<int, kOrthoTimes>{});
    case kOrthoNext: return go(std::integral_constant<int, kOrthoNext>{});
    default: return go(std::integral_constant<int, kOrthoLast>{});
  }
}

template <class C>
hipError_t start(int step, const OrthoList &l, const OrthoCall &c,
                 hipStream_t s) {
  return c.planes > 1 ? start<C, 2>(step, l, c, s) : start<C, 1>(step, l, c, s);
}

}  // namespace

hipError_t launch_ortho_norm(const OrthoList &l, const OrthoCall &c,
                             hipStream_t s) {
  with_type(c.type, [&](auto type) {
    k_ortho_norm<decltype(type)::value>
        <<<l.first[l.count], 256, 0, s>>>(l, c);
  });
  return hipGetLastError();
}

hipError_t launch_ortho_load(const OrthoList &l, const OrthoCall &c,
                             hipStream_t s) {
  with_type(c.type, [&](auto type) {
    k_ortho_load<decltype(type)::value>
        <<<l.first[l.count], 256, 0, s>>>(l, c);
  });
  return hipGetLastError();
}

hipError_t launch_ortho_join(const OrthoList &l, const OrthoCall &c,
                             hipStream_t s) {
  k_ortho_join<<<l.first[l.count], 256, 0, s>>>(l, c);
  return hipGetLastError();
}

hipError_t launch_ortho_product(int step, int tile, bool deep,
                                const OrthoList &l, const OrthoCall &c,
                                hipStream_t s) {
  if (tile == 256) return start<Tile256>(step, l, c, s);
  if (tile == 64) return start<Tile64>(step, l, c, s);
  return deep ? start<TileDeep>(step, l, c, s) : start<Tile128>(step, l, c, s);
}

}  // namespace mta
