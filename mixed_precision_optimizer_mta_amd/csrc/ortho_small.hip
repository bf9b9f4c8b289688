// ortho_small.hip -- orthogonalised updates of matrices of up to 64 rows or
// columns (adapters, small heads), in float64 on the matrix cores.
//
// A step X <- (a + b A + c A A) X multiplies X from the left by a polynomial of
// A = X X^T, and all of them commute: the steps' polynomials are multiplied
// together on the Gram matrix alone,
//   R = u u^T / (|u| + eps)^2,   F = 1,
//   each step:  Q = a + b R + c R R,   F = Q F,   R = R Q Q
// and u is read once more for the result F u / (|u| + eps).  |u|^2 is the trace
// of u u^T.  In 16 or 22 bits this would not do: an eigenvalue of R that a
// rounding has made negative grows by a^2 = 12 a step; from float64's 2^-53 five
// steps reach 2^-35, and the ten that are allowed 2^-17, on directions that are
// then 2^-8 of the result.
//
// Three launches whatever the steps, bound by their latencies: a 16 x 768
// bfloat16 matrix takes 20 us (4.6, 12.6 and 4.5 in kernels) where the products'
// way took 121.
#include "ortho_device.h"

namespace mta {
namespace {

typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kSide = kOrthoSmall;  // rows of X, at most
constexpr int kCols = 64;           // columns of X at a time
// Doubles between LDS rows: 16 rows a step of k apart lie in distinct banks.
constexpr int kPitch = 66;

// acc + a b^T of 16 x 16 by 4: a lane brings a[lane % 16][lane / 16] and
// b[lane % 16][lane / 16], and has rows 4 r + lane / 16 of column lane % 16.
__device__ __forceinline__ f64x4 mfma64(double a, double b, f64x4 acc) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, acc, 0, 0, 0);
}

// u of 64 columns of X from column l0 into LDS; with Update the momentum takes
// the gradient in.
template <int D, bool Update>
__device__ __forceinline__ void load_columns(const OrthoItem &it,
                                             const OrthoCall &c,
                                             const OrthoSmallSpace &sp,
                                             int64_t l0,
                                             double (&x)[kSide][kPitch]) {
  const Look look = look_of(c);
  const bool skip = c.amp && c.amp->found_inf != 0.0f;
  const bool tall = it.rows > it.cols;
  // runs of eight along the rows of u
  const int runs = tall ? sp.side / 8 : kCols / 8;
  const int rows = tall ? kCols : sp.side;
  for (int q = threadIdx.x; q < runs * rows; q += 256) {
    const int y = q / runs, i = q % runs * 8;
    const int64_t r = tall ? l0 + y : y, col = tall ? i : l0 + i;
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
        float now[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float gr = look.gradient(g[e]);
          now[e] = Update || skip ? look.next(m[e], gr) : m[e];
          v[e] = look.ahead(now[e], gr);
        }
        if (Update && !skip) {
          if (n == 8) {
            store8<MTA_F32, false>(it.m, am, now);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (e < n) it.m[am + e] = now[e];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = look.gradient(g[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double u = e < n ? v[e] : 0.0;
      if (tall) x[i + e][y] = u;
      else x[y][i + e] = u;
    }
  }
}

// Block number b of the ones on and above the diagonal of n x n: row by row.
__device__ __forceinline__ void upper(int b, int n, int &row, int &col) {
  row = 0;
  while (b >= n - row) b -= n - row++;
  col = row + b;
}

// Part of u u^T: every parts-th run of 64 columns.
template <int D>
__global__ __launch_bounds__(256) void k_ortho_small_gram(const OrthoList l,
                                                          const OrthoCall c) {
  __shared__ double x[kSide][kPitch];
  const int k = item_of(l, blockIdx.x);
  const OrthoItem &it = l.item[k];
  const OrthoSmallSpace sp = ortho_small_space(it.rows, it.cols);
  const int part = static_cast<int>(blockIdx.x - l.first[k]);
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int n = sp.side / 16, blocks = n * (n + 1) / 2;
  constexpr int kEach = 3;  // blocks of a wave: ten among four
  int row[kEach], col[kEach];
  f64x4 acc[kEach];
#pragma unroll
  for (int t = 0; t < kEach; ++t) {
    upper(min(wave + 4 * t, blocks - 1), n, row[t], col[t]);
    acc[t] = f64x4{0, 0, 0, 0};
  }
  for (int64_t l0 = int64_t{part} * kCols; l0 < sp.large;
       l0 += int64_t{sp.parts} * kCols) {
    __syncthreads();
    load_columns<D, true>(it, c, sp, l0, x);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kEach; ++t) {
      if (wave + 4 * t >= blocks) break;
#pragma unroll
      for (int q = 0; q < kCols; q += 4)
        acc[t] = mfma64(x[row[t] * 16 + lane % 16][q + lane / 16],
                        x[col[t] * 16 + lane % 16][q + lane / 16], acc[t]);
    }
  }
  double *out = reinterpret_cast<double *>(it.ws) +
                int64_t{part} * sp.side * sp.side;
#pragma unroll
  for (int t = 0; t < kEach; ++t) {
    if (wave + 4 * t >= blocks) break;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      out[(row[t] * 16 + 4 * r + lane / 16) * sp.side + col[t] * 16 +
          lane % 16] = acc[t][r];
  }
}

// F / (|u| + eps), by one workgroup a matrix.  Bound by the float64 matrix rate
// of a CU (64 fused multiply-adds a clock): every product is symmetric, and only
// its blocks on and above the diagonal are computed, one or two a wave, and what is
// above the diagonal is copied below it in blocks on it too: rows are multiplied by
// rows, as p q^T, and what a rounding has made unlike on the two sides would grow
// by up to (a + |b|)^2 = 68 a step instead of staying as small as it is.
__global__ __launch_bounds__(1024) void k_ortho_small_factor(
    const OrthoList l, const OrthoCall c, const OrthoCoefficients co) {
  // R, Q, R Q and F
  __shared__ double at[4][kSide][kPitch];
  const OrthoItem &it = l.item[blockIdx.x];
  const OrthoSmallSpace sp = ortho_small_space(it.rows, it.cols);
  const int side = sp.side, n = side / 16, blocks = n * (n + 1) / 2;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  auto *parts = reinterpret_cast<double *>(it.ws);
  for (int b = wave; b < blocks * 4; b += 16) {
    int row, col;
    upper(b / 4, n, row, col);
    const int i = row * 16 + b % 4 * 4 + lane / 16, j = col * 16 + lane % 16;
    double sum = 0.0;
#pragma unroll 16
    for (int p = 0; p < sp.parts; ++p)
      sum += parts[(int64_t{p} * side + i) * side + j];
    if (i <= j) at[0][i][j] = at[0][j][i] = sum;
  }
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < side; ++i) trace += at[0][i][i];
  // (zeros stay zeros, however small eps is)
  const double f = trace == 0.0 ? 0.0 : 1.0 / (sqrt(trace) + c.eps);
  __syncthreads();
  for (int q = threadIdx.x; q < side * side; q += 1024)
    at[0][q / side][q % side] *= f * f;
  __syncthreads();

  // Block b of p times q.
  const auto product = [&](int b, const double (&p)[kSide][kPitch],
                           const double (&q)[kSide][kPitch]) {
    int row, col;
    upper(b, n, row, col);
    f64x4 acc{0, 0, 0, 0};
#pragma unroll 4
    for (int k = 0; k < side; k += 4)
      acc = mfma64(p[row * 16 + lane % 16][k + lane / 16],
                   q[col * 16 + lane % 16][k + lane / 16], acc);
    return acc;
  };
  // It and its mirror image into `to`, each value through `of(row, col, v)`.
  const auto put = [&](int b, double (&to)[kSide][kPitch], f64x4 acc,
                       auto &&of) {
    int row, col;
    upper(b, n, row, col);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = row * 16 + 4 * r + lane / 16, j = col * 16 + lane % 16;
      if (i > j) continue;
      const double v = of(i, j, acc[r]);
      to[i][j] = to[j][i] = v;
    }
  };
  const auto same = [](int, int, double v) { return v; };
  for (int s = 0; s < co.steps; ++s) {
    const double a = co.v[s][0], b2 = co.v[s][1], c2 = co.v[s][2];
    const bool last = s + 1 == co.steps;
    if (wave < blocks)
      put(wave, at[1], product(wave, at[0], at[0]),
          [&](int i, int j, double v) {
            return c2 * v + b2 * at[0][i][j] + (i == j ? a : 0.0);
          });
    __syncthreads();
    // F Q, kept until all have read F, and R Q: the waves that are left over
    // from one take the other
    f64x4 held{0, 0, 0, 0};
    if (s > 0 && wave < blocks) held = product(wave, at[3], at[1]);
    if (!last)
      for (int b = 15 - wave; b < blocks; b += 16)
        put(b, at[2], product(b, at[0], at[1]), same);
    __syncthreads();
    if (s > 0) {
      if (wave < blocks) put(wave, at[3], held, same);
    } else {
      for (int q = threadIdx.x; q < side * side; q += 1024)
        at[3][q / side][q % side] = at[1][q / side][q % side];
    }
    if (!last && wave < blocks)
      put(wave, at[0], product(wave, at[2], at[1]), same);
    __syncthreads();
  }
  double *out = parts + int64_t{sp.parts} * side * side;
  for (int q = threadIdx.x; q < side * side; q += 1024)
    out[q] = at[3][q / side][q % side] * f;
}

// 64 columns of the result: the factor times u.
template <int D>
__global__ __launch_bounds__(256) void k_ortho_small_apply(const OrthoList l,
                                                           const OrthoCall c) {
  __shared__ double f[kSide][kPitch], x[kSide][kPitch];
  const int k = item_of(l, blockIdx.x);
  const OrthoItem &it = l.item[k];
  const OrthoSmallSpace sp = ortho_small_space(it.rows, it.cols);
  const int side = sp.side, n = side / 16;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t l0 = int64_t{blockIdx.x - l.first[k]} * kCols;
  const double *factor = reinterpret_cast<const double *>(it.ws) +
                         int64_t{sp.parts} * side * side;
  for (int q = threadIdx.x * 2; q < side * side; q += 512) {
    typedef double f64x2 __attribute__((ext_vector_type(2)));
    *(f64x2 *)&f[q / side][q % side] = *(const f64x2 *)(factor + q);
  }
  load_columns<D, false>(it, c, sp, l0, x);
  __syncthreads();
  // a wave takes 16 columns
  f64x4 acc[kSide / 16];
#pragma unroll
  for (int b = 0; b < kSide / 16; ++b) acc[b] = f64x4{0, 0, 0, 0};
  for (int q = 0; q < side; q += 4) {
    const double v = x[q + lane / 16][wave * 16 + lane % 16];
#pragma unroll
    for (int b = 0; b < kSide / 16; ++b)
      if (b < n)
        acc[b] = mfma64(f[b * 16 + lane % 16][q + lane / 16], v, acc[b]);
  }
  __syncthreads();
  auto &y = reinterpret_cast<float (&)[kSide][kPitch]>(x);
#pragma unroll
  for (int b = 0; b < kSide / 16; ++b)
    if (b < n)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        y[b * 16 + 4 * r + lane / 16][wave * 16 + lane % 16] =
            static_cast<float>(acc[b][r]);
  __syncthreads();
  const bool skip = c.amp && c.amp->found_inf != 0.0f;
  const bool tall = it.rows > it.cols;
  const int runs = tall ? side / 8 : kCols / 8;
  const int rows = tall ? kCols : side;
  for (int q = threadIdx.x; q < runs * rows; q += 256) {
    const int r = q / runs, i = q % runs * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = tall ? y[i + e][r] : y[r][i + e];
    put_result(it, c, tall ? l0 + r : r, tall ? i : l0 + i, v, skip);
  }
}

}  // namespace

hipError_t launch_ortho_small_gram(const OrthoList &l, const OrthoCall &c,
                                   hipStream_t s) {
  with_type(c.type, [&](auto type) {
    k_ortho_small_gram<decltype(type)::value>
        <<<l.first[l.count], 256, 0, s>>>(l, c);
  });
  return hipGetLastError();
}

hipError_t launch_ortho_small_factor(const OrthoList &l, const OrthoCall &c,
                                     const OrthoCoefficients &k,
                                     hipStream_t s) {
  k_ortho_small_factor<<<l.count, 1024, 0, s>>>(l, c, k);
  return hipGetLastError();
}

hipError_t launch_ortho_small_apply(const OrthoList &l, const OrthoCall &c,
                                    hipStream_t s) {
  with_type(c.type, [&](auto type) {
    k_ortho_small_apply<decltype(type)::value>
        <<<l.first[l.count], 256, 0, s>>>(l, c);
  });
  return hipGetLastError();
}

}  // namespace mta
