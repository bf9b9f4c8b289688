// ortho_kernels.hip -- the orthogonalised update of the Muon rule on the matrix
// cores of gfx950, for the matrices of a list together.
//
//   X = u / (|u| + eps);  steps times  A = X X^T,  B = b A + c A A,  X = a X + B X
//
// u is the gradient or its momentum, X the one with fewer rows than columns of
// u and its transpose.  Each step is three products, one launch each over the
// tiles of all matrices: A and A A are symmetric, so tiles below the diagonal
// are copies.
//
// Which digits are kept.  Small singular values grow by a = 3.4 in a step and
// gradients have many: with X in bfloat16 the result is off by 1.3% of its norm
// for normal entries and by 32% where four directions stand out a thousandfold,
// whatever the products' sums.  X is therefore kept in 22 bits, as the sum of
// two float16 values (scaled by 2^13, so that 1/sqrt(rows cols) and its rest are
// normal numbers), and the term a X uses them all.  The products take the first
// values alone.  What hurts then is that B's diagonal, -2.6 of rows that have
// converged, is rounded with the rest of it: diagonals are kept in float32 apart
// and enter as e_i X_i, and the error falls from 2.9e-3 to 4.5e-4 (512 x 2048
// normal entries).  In the first steps e_i multiplies the rounded X that A was
// made from, so that small directions cancel as they do in A (from 3.3e-3 to
// 6.8e-4 where eight directions stand out); in the last two the whole X.  With
// `precise` every product is of both values: 4e-7.
#include "gemm_device.h"
#include "matrix_internal.h"

namespace mta {
namespace {

// Powers of two that the float16 values are multiplied by: room for singular
// values of 7 in X, of 49 in A and a multiple of that in B.
constexpr float kScaleX = 8192.0f, kScaleA = 1024.0f, kScaleB = 512.0f;

__device__ __forceinline__ float unscale_of(const OrthoCall &c) {
  return c.amp ? static_cast<float>(1.0 / static_cast<double>(c.amp->scale))
               : 1.0f;
}

__device__ __forceinline__ int item_of(const OrthoList &l, uint32_t block) {
  int k = 0;
  while (k + 1 < static_cast<int>(l.count) && block >= l.first[k + 1]) ++k;
  return k;
}

// Two float16 values of x: its rounding and the rounding of what is left.
__device__ __forceinline__ void halves(float x, float &hi, float &lo) {
  hi = static_cast<float>(static_cast<_Float16>(x));
  lo = x - hi;
  // an infinity would leave a NaN, which the first value says already
  lo = lo == lo ? lo : 0.0f;
}

__device__ __forceinline__ void store_planes(uint16_t *hi_at, uint16_t *lo_at,
                                             const float (&x)[8]) {
  float hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) halves(x[e], hi[e], lo[e]);
  store<MTA_F16, 8, false>(hi_at, 0, hi);
  if (lo_at) store<MTA_F16, 8, false>(lo_at, 0, lo);
}

// Sum of a value of every lane of a workgroup of 256, in all of them.
__device__ __forceinline__ double sum256(double x, double *four) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d);
  __syncthreads();
  if (threadIdx.x % 64 == 0) four[threadIdx.x / 64] = x;
  __syncthreads();
  return (four[0] + four[1]) + (four[2] + four[3]);
}

// g' and, with a momentum, its new value and u.
struct Look {
  float s, c, mu;
  int nesterov;
  __device__ __forceinline__ float gradient(float g) const {
    return (g * s) * c;
  }
  __device__ __forceinline__ float next(float m, float g) const {
    return m * mu + g;
  }
  __device__ __forceinline__ float ahead(float m, float g) const {
    return nesterov ? g + mu * m : m;
  }
};
__device__ __forceinline__ Look look_of(const OrthoCall &c) {
  return Look{unscale_of(c), c.d_coef ? *c.d_coef : 1.0f, c.mu, c.nesterov};
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
  const OrthoSpace sp = ortho_space(it.rows, it.cols, it.planes);
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
  const OrthoSpace sp = ortho_space(it.rows, it.cols, it.planes);
  __shared__ double four[4];
  __shared__ float tile[kT][kT + 1];
  const int64_t parts = ortho_parts(it.rows, it.cols);
  const double mine =
      threadIdx.x < parts
          ? reinterpret_cast<const double *>(it.ws + sp.part)[threadIdx.x]
          : 0.0;
  const double norm = sqrt(sum256(mine, four)) + c.eps;
  const double factor = norm == 0.0 ? 0.0 : kScaleX / norm;
  const Look look = look_of(c);
  const bool skip = c.amp && c.amp->found_inf != 0.0f;
  const bool tall = it.rows > it.cols;
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
      store_planes(hi, hi + sp.plane_x, v);
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
    store_planes(hi, hi + sp.plane_x, v);
  }
}

// Eight results of a row: out, and the weights' step.
__device__ __forceinline__ void put_result(const OrthoItem &it,
                                           const OrthoCall &c, int64_t row,
                                           int64_t col, const float (&x)[8],
                                           bool skip) {
  if (row >= it.rows || col >= it.cols) return;
  const int n = static_cast<int>(min(int64_t{8}, it.cols - col));
  float y[8];
  if (it.out) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * it.scale;
    with_type(c.out_type, [&](auto type) {
      constexpr int T = decltype(type)::value;
      if (n == 8) {
        store8<T, false>(it.out, row * it.ldout + col, y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n) store_elem<T>(it.out, row * it.ldout + col + e, y[e]);
      }
    });
  }
  if (it.w && !skip) {
    const int64_t at = row * it.cols + col;
    const Raw8<MTA_F32> w = n == 8 ? load8<MTA_F32, false>(it.w, at)
                                   : load8_part<MTA_F32>(it.w, at, n, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = w[e] * c.decay + it.update * x[e];
    if (n == 8) {
      store8<MTA_F32, false>(it.w, at, y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) it.w[at + e] = y[e];
    }
    if (it.w16) {
      with_type(c.copy_type, [&](auto type) {
        constexpr int T = decltype(type)::value;
        if (n == 8) {
          store8<T, false>(it.w16, at, y);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < n) store_elem<T>(it.w16, at + e, y[e]);
        }
      });
    }
  }
}

// One tile of a step's product.
template <class C, int Step>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_ortho_product(const OrthoList l, const OrthoCall c) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  const uint32_t block = beside(blockIdx.x, gridDim.x);
  const int k = item_of(l, block);
  const OrthoItem &it = l.item[k];
  const OrthoSpace sp = ortho_space(it.rows, it.cols, it.planes);
  const uint32_t t = block - l.first[k];
  constexpr bool kSym = Step == kOrthoGram || Step == kOrthoSquare;
  const uint32_t side = static_cast<uint32_t>(sp.small + C::kBM - 1) / C::kBM;
  uint32_t tm, tn;
  if constexpr (kSym) {
    // tiles on and right of the diagonal, row by row
    uint32_t left = t;
    tm = 0;
    while (left >= side - tm) left -= side - tm++;
    tn = tm + left;
  } else {
    banded(t, side, static_cast<uint32_t>(sp.large + C::kBN - 1) / C::kBN, tm,
           tn);
  }
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  auto *x_old = reinterpret_cast<uint16_t *>(it.ws + sp.x + c.which * sp.next_x);
  auto *x_new = reinterpret_cast<uint16_t *>(it.ws + sp.x + (1 - c.which) * sp.next_x);
  auto *pa = reinterpret_cast<uint16_t *>(it.ws + sp.a);
  auto *pb = reinterpret_cast<uint16_t *>(it.ws + sp.a + sp.next_a);
  auto *da = reinterpret_cast<float *>(it.ws + sp.diag);
  auto *db = reinterpret_cast<float *>(it.ws + sp.diag + sp.next_diag);
  const Operand x{x_old, sp.plane_x, sp.pitch_x, sp.small, sp.small};
  const Operand a{pa, sp.plane_a, sp.pitch_a, sp.small, sp.small};
  const Operand b{pb, sp.plane_a, sp.pitch_a, sp.small, sp.small};
  const Pairs pairs = pairs_of(it.planes);
  const int64_t deep_x = (sp.large + 63) / 64 * 64;
  const int64_t deep_a = (sp.small + 63) / 64 * 64;
  f32x16 acc[C::kRM][C::kRN];

  if constexpr (kSym) {
    if constexpr (Step == kOrthoGram)
      tile_product<C, true, kAlong, kAlong>(x, x, pairs, m0, n0, 0, deep_x, lds,
                                            acc);
    else
      tile_product<C, true, kAlong, kAlong>(a, a, pairs, m0, n0, 0, deep_a, lds,
                                            acc);
    uint16_t *to = Step == kOrthoGram ? pa : pb;
    float *diag = Step == kOrthoGram ? da : db;
    const bool two = it.planes > 1;
    const auto put = [&](int64_t row, int64_t col, float (&v)[8]) {
      if (row >= sp.small || col >= sp.pitch_a) return;
      const int64_t at = row * sp.pitch_a + col;
      constexpr float kTo = Step == kOrthoGram ? kScaleA : kScaleB;
      if constexpr (Step == kOrthoGram) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= 1.0f / (kScaleX * kScaleX);
      } else {
        // with A = D + O, D its diagonal: A A = O O + D O + O D + D D
        const Raw8<MTA_F16> hi = load8<MTA_F16, false>(pa, at);
        Raw8<MTA_F16> lo = fill8<MTA_F16>(0);
        if (two) lo = load8<MTA_F16, false>(pa + sp.plane_a, at);
        const float dr = da[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = (hi[e] + lo[e]) * (1.0f / kScaleA);
          const float dc = col + e < sp.small ? da[col + e] : 0.0f;
          const float oo = v[e] * (1.0f / (kScaleA * kScaleA));
          v[e] = row == col + e ? c.b * dr + c.c * (oo + dr * dr)
                                : c.b * o + c.c * (oo + (dr + dc) * o);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (row == col + e) diag[row] = v[e];
        v[e] = row == col + e || col + e >= sp.small ? 0.0f : v[e] * kTo;
      }
      store_planes(to + at, two ? to + at + sp.plane_a : nullptr, v);
    };
    tile_out<C, false>(
        lds, acc, true, tm != tn,
        [&](int m, int n, float (&v)[8]) { put(m0 + m, n0 + n, v); },
        [&](int n, int m, float (&v)[8]) { put(n0 + n, m0 + m, v); });
  } else {
    tile_product<C, true, kAlong, kAcross>(
        b, Operand{x_old, sp.plane_x, sp.pitch_x, sp.pitch_x, sp.small}, pairs,
        m0, n0, 0, deep_a, lds, acc);
    const bool tall = it.rows > it.cols;
    const bool skip = c.amp && c.amp->found_inf != 0.0f;
    const bool whole = c.whole || it.planes > 1;
    const auto next = [&](int m, int n, float (&v)[8]) {
      const int64_t row = m0 + m, col = n0 + n;
      if (row >= sp.small || col >= sp.pitch_x) return;
      const int64_t at = row * sp.pitch_x + col;
      const Raw8<MTA_F16> hi = load8<MTA_F16, false>(x_old, at);
      const Raw8<MTA_F16> lo = load8<MTA_F16, false>(x_old + sp.plane_x, at);
      const float e_i = db[row];
      // kept: times kScaleX; handed out: as it is
      constexpr float kTo = Step == kOrthoLast ? 1.0f / kScaleX : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float all = hi[e] + lo[e];
        v[e] = (c.a * all + (e_i * (whole ? all : hi[e]) +
                             v[e] * (1.0f / kScaleB))) *
               kTo;
      }
      if constexpr (Step == kOrthoNext) {
        store_planes(x_new + at, x_new + at + sp.plane_x, v);
      } else if (!tall) {
        put_result(it, c, row, col, v, skip);
      }
    };
    tile_out<C, Step == kOrthoLast>(
        lds, acc, true, Step == kOrthoLast && tall, next,
        [&](int n, int m, float (&v)[8]) {
          if constexpr (Step == kOrthoLast)
            put_result(it, c, n0 + n, m0 + m, v, skip);
        });
  }
}

template <class C>
hipError_t start(int step, const OrthoList &l, const OrthoCall &c,
                 hipStream_t s) {
  const uint32_t grid = l.first[l.count];
  switch (step) {
    case kOrthoGram:
      k_ortho_product<C, kOrthoGram><<<grid, C::kThreads, 0, s>>>(l, c);
      break;
    case kOrthoSquare:
      k_ortho_product<C, kOrthoSquare><<<grid, C::kThreads, 0, s>>>(l, c);
      break;
    case kOrthoNext:
      k_ortho_product<C, kOrthoNext><<<grid, C::kThreads, 0, s>>>(l, c);
      break;
    default:
      k_ortho_product<C, kOrthoLast><<<grid, C::kThreads, 0, s>>>(l, c);
  }
  return hipGetLastError();
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

hipError_t launch_ortho_product(int step, int tile, const OrthoList &l,
                                const OrthoCall &c, hipStream_t s) {
  return tile == 256 ? start<Tile256>(step, l, c, s)
                     : start<Tile128>(step, l, c, s);
}

}  // namespace mta
