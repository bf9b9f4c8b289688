// linear_kernels.hip -- the cross entropy of a linear output layer and its
// gradients on the matrix cores of gfx950, without keeping the logits.
//
//   z = h w^T,  p = softmax(z),  loss = sum weight (-log p[target])
//   dz = weight (p - [target]),  dh = dz w,  dw = dz^T h
//
// The forward is one product whose tiles leave two numbers a row, the largest
// logit and the sum of exponentials beside it (without the target's: 1 - p keeps
// its digits as p nears 1), and a kernel that joins a row's tiles.  The
// gradients take the vocabulary in pieces: the product again, its tiles written
// as dz in 16 bits, then dh += dz w and the piece of dw = dz^T h, which read dz,
// w and h as they lie, with k along or across.  Four products instead of the
// three that kept logits would need: logits in 32 bits for 8192 x 50257 are 1.6
// GB, whose writing and reading takes as long as the fourth.
//
// A float32 call has three bfloat16 planes for each operand and six products.
#include <algorithm>

#include "gemm_device.h"
#include "matrix_internal.h"

namespace mta {
namespace {

// dz of float16 is kept times 2^14: probabilities below 2^-14 of a largest
// weight keep their digits down to 2^-28.
template <int D>
constexpr float kRoom = D == MTA_F16 ? 16384.0f : 1.0f;

// Whether a row takes no part.
__device__ __forceinline__ bool left_out(const LinearArgs &l, int64_t r) {
  if (l.backward) return l.rows[r].weight == 0.0f;
  return l.a.targets[r] == l.a.ignore_index ||
         (l.a.weights && l.a.weights[r] == 0.0f);
}

// The weight of a row without weights, and the largest magnitude of any.
__global__ __launch_bounds__(1024) void k_linear_weights(const LinearArgs l) {
  const mta_linear_loss_args &a = l.a;
  int64_t count = 0;
  float most = 0.0f;
  for (int64_t r = threadIdx.x; r < a.rows; r += 1024) {
    if (l.backward) {
      most = fmaxf(most, fabsf(l.rows[r].weight));
    } else if (a.weights) {
      if (!left_out(l, r)) most = fmaxf(most, fabsf(a.weights[r]));
    } else {
      count += a.targets[r] != a.ignore_index;
    }
  }
  __shared__ int64_t counts[16];
  __shared__ float mosts[16];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) {
    count += __shfl_xor(count, d);
    most = fmaxf(most, __shfl_xor(most, d));
  }
  if (threadIdx.x % 64 == 0) {
    counts[threadIdx.x / 64] = count;
    mosts[threadIdx.x / 64] = most;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    count = 0;
    most = 0.0f;
    for (int k = 0; k < 16; ++k) {
      count += counts[k];
      most = fmaxf(most, mosts[k]);
    }
    const float each =
        count > 0 ? static_cast<float>(1.0 / static_cast<double>(count)) : 0.0f;
    l.scalars[0] = each;
    l.scalars[1] = l.backward || a.weights ? most : each;
  }
}

// The bfloat16 values that x is the sum of, largest first: each takes the next
// eight significant bits by cutting off the lower ones, so that differences are
// exact.  An infinity or NaN is carried by the first alone.
__device__ __forceinline__ void three(float x, uint16_t (&b)[3]) {
  const bool fine = __builtin_fabsf(x) < __builtin_inff();
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    uint32_t u = __float_as_uint(x) & 0xFFFF0000u;
    if (t == 0 && x != x) u = 0x7FC00000u;
    b[t] = static_cast<uint16_t>(u >> 16);
    x = fine ? x - __uint_as_float(u) : 0.0f;
  }
}

// Eight values into the planes of an operand.
template <int D>
__device__ __forceinline__ void put_planes(uint16_t *to, int64_t plane,
                                           const float (&v)[8]) {
  if constexpr (D == MTA_F32) {
    u32x4 w[3];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint16_t x[3], y[3];
      three(v[2 * k], x);
      three(v[2 * k + 1], y);
#pragma unroll
      for (int t = 0; t < 3; ++t)
        w[t][k] = x[t] | static_cast<uint32_t>(y[t]) << 16;
    }
#pragma unroll
    for (int t = 0; t < 3; ++t)
      *(MTA_GLOBAL u32x4 *)(to + t * plane) = w[t];
  } else {
    store8<D, false>(to, 0, v);
  }
}

// Rows of an operand into its planes, with zeros behind the last column and in
// the rows that are left out.
template <int D>
__global__ __launch_bounds__(256) void k_linear_pack(
    const LinearArgs l, const void *from, int64_t ld, int64_t rows,
    uint16_t *to, int64_t plane, bool mask) {
  const int64_t runs = l.pitch / 8;
  for (int64_t q = int64_t{blockIdx.x} * 256 + threadIdx.x; q < rows * runs;
       q += int64_t{gridDim.x} * 256) {
    const int64_t r = q / runs, i = (q - r * runs) * 8;
    const int64_t left = l.a.width - i;
    const int n = static_cast<int>(left >= 8 ? 8 : left > 0 ? left : 0);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0 && !(mask && left_out(l, r))) {
      const Raw8<D> x = n == 8 ? load8<D, false>(from, r * ld + i)
                               : load8_part<D>(from, r * ld + i, n, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = x[e];
    }
    put_planes<D>(to + r * l.pitch + i, plane, v);
  }
}

// e^x of x <= 0.  For float32 calls with all digits.
template <int D>
__device__ __forceinline__ float exponential(float x) {
  if constexpr (D == MTA_F32) return expf(x);
  else return __builtin_amdgcn_exp2f(x * 1.44269504f);
}

template <class C, int D>
__device__ __forceinline__ void logits_tile(const LinearArgs &l, int64_t m0,
                                            int64_t n0, MTA_LDS uint8_t *lds,
                                            f32x16 (&acc)[C::kRM][C::kRN]) {
  const Operand h{l.h, l.h_plane, l.pitch, l.a.rows, 0};
  const Operand w{l.w, l.w_plane, l.w_pitch, l.a.vocab, 0};
  tile_product<C, D == MTA_F16, kAlong, kAlong>(
      h, w, pairs_of(l.planes), m0, n0, 0, (l.a.width + 63) / 64 * 64, lds,
      acc);
}

// A tile of logits as each row's largest and its sum of exponentials.
template <class C, int D>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_linear_logits(const LinearArgs l) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  uint32_t tm, tn;
  banded(beside(blockIdx.x, gridDim.x),
         static_cast<uint32_t>((l.a.rows + C::kBM - 1) / C::kBM),
         static_cast<uint32_t>(l.tiles), tm, tn);
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  f32x16 acc[C::kRM][C::kRN];
  logits_tile<C, D>(l, m0, n0, lds, acc);

  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wr = wave / C::kWC, wc = wave % C::kWC;
  auto *side = (MTA_LDS f32x2 *)lds;  // [WC][BM]
  __syncthreads();
  // columns of this lane: n1 + 32 j + 8 q + e
  const int64_t n1 = n0 + wc * C::kTN + lane / 32 * 4;
  const int many =
      static_cast<int>(min(int64_t{C::kBN}, l.a.vocab - n1));
#pragma unroll
  for (int i = 0; i < C::kRM; ++i) {
    const int m = wr * C::kTM + i * 32 + lane % 32;
    const int64_t row = m0 + m;
    const int64_t target =
        row < l.a.rows ? ((const MTA_GLOBAL int64_t *)l.a.targets)[row] : -1;
    const int64_t far = target - n1;
    const int mine = far >= 0 && far < C::kBN ? static_cast<int>(far) : -1;
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < C::kRN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int at = j * 32 + r / 4 * 8 + r % 4;
        if (at >= many) acc[i][j][r] = -__builtin_inff();
        top = fmaxf(top, acc[i][j][r]);
      }
    top = fmaxf(top, __shfl_xor(top, 32));
    const float shift = top == -__builtin_inff() ? 0.0f : top;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < C::kRN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int at = j * 32 + r / 4 * 8 + r % 4;
        if (at == mine) {
          l.z_target[row] = acc[i][j][r];
        } else {
          sum += exponential<D>(acc[i][j][r] - shift);
        }
      }
    sum += __shfl_xor(sum, 32);
    if (lane < 32) side[wc * C::kBM + m] = f32x2{top, sum};
  }
  __syncthreads();
  for (int m = threadIdx.x; m < C::kBM; m += C::kThreads) {
    if (m0 + m >= l.a.rows) break;
    f32x2 v = side[m];
#pragma unroll
    for (int k = 1; k < C::kWC; ++k) {
      const f32x2 u = side[k * C::kBM + m];
      const float top = fmaxf(v[0], u[0]);
      const float shift = top == -__builtin_inff() ? 0.0f : top;
      v = f32x2{top, v[1] * exponential<D>(v[0] - shift) +
                         u[1] * exponential<D>(u[0] - shift)};
    }
    l.partial[tn * l.a.rows + m0 + m] = make_float2(v[0], v[1]);
  }
}

// Rows' tiles joined: 64 rows to a workgroup, 16 waves that take every 16th
// tile and are joined in order.
template <int D>
__global__ __launch_bounds__(1024) void k_linear_rows(const LinearArgs l) {
  const mta_linear_loss_args &a = l.a;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t row = int64_t{blockIdx.x} * 64 + lane;
  const auto join = [](float &top, float &sum, float t, float s) {
    const float most = fmaxf(top, t);
    const float shift = most == -__builtin_inff() ? 0.0f : most;
    sum = sum * exponential<D>(top - shift) + s * exponential<D>(t - shift);
    top = most;
  };
  float top = -__builtin_inff(), sum = 0.0f;
  if (row < a.rows) {
#pragma unroll 4
    for (int64_t t = wave; t < l.tiles; t += 16) {
      const float2 v = l.partial[t * a.rows + row];
      join(top, sum, v.x, v.y);
    }
  }
  __shared__ float2 side[16][64];
  side[wave][lane] = make_float2(top, sum);
  __syncthreads();
  if (wave != 0 || row >= a.rows) return;
#pragma unroll
  for (int k = 1; k < 16; ++k) join(top, sum, side[k][lane].x, side[k][lane].y);
  const int64_t target = a.targets[row];
  mta_linear_row r{0.0f, 0.0f, 0.0f, 0.0f};
  float logp = 0.0f;
  if (!left_out(l, row)) {
    r.weight = a.weights ? a.weights[row] : l.scalars[0];
    if (target < 0 || target >= a.vocab) {
      r.top = r.total = r.rest = logp = __builtin_nanf("");
    } else {
      const float zt = l.z_target[row];
      const float own = exponential<D>(zt - top);
      r.top = top;
      r.total = sum + own;
      r.rest = sum / r.total;
      logp = zt == top ? -log1pf(sum) : (zt - top) - logf(r.total);
      // (the largest may be infinite)
      if (!(own == own)) logp = own;
    }
  }
  l.rows[row] = r;
  if (a.logp) a.logp[row] = logp;
  l.terms[row] = r.weight == 0.0f ? 0.0 : -static_cast<double>(r.weight) * logp;
}

// The loss: each lane's terms in order, then the lanes'.
__global__ __launch_bounds__(1024) void k_linear_sum(const LinearArgs l) {
  double x = 0.0;
#pragma unroll 8
  for (int64_t r = threadIdx.x; r < l.a.rows; r += 1024) x += l.terms[r];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d);
  __shared__ double side[16];
  if (threadIdx.x % 64 == 0) side[threadIdx.x / 64] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
    x = 0.0;
    for (int k = 0; k < 16; ++k) x += side[k];
    *l.a.loss = static_cast<float>(x);
  }
}

// A tile of logits as dz, without the factor that all rows share.
template <class C, int D>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_linear_grad(const LinearArgs l) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  uint32_t tm, tn;
  banded(beside(blockIdx.x, gridDim.x),
         static_cast<uint32_t>((l.a.rows + C::kBM - 1) / C::kBM),
         static_cast<uint32_t>((l.count + C::kBN - 1) / C::kBN), tm, tn);
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  f32x16 acc[C::kRM][C::kRN];
  logits_tile<C, D>(l, m0, l.first + n0, lds, acc);
  const float most = l.scalars[1];
  const int64_t wide = (l.count + 63) / 64 * 64;
  tile_out<C, false>(
      lds, acc, true, false, [](int, int) { return 0; },
      [&](int m, int n, float (&v)[8], int) {
        const int64_t row = m0 + m, col = n0 + n;
        if (row >= l.deep_rows || col >= wide) return;
        mta_linear_row r{0.0f, 0.0f, 0.0f, 0.0f};
        int64_t target = -1;
        if (row < l.a.rows) {
          r = l.rows[row];
          target = l.a.targets[row] - l.first - col;
        }
        const float share =
            r.weight == 0.0f ? 0.0f : r.weight / most * kRoom<D>;
        const float each = share / r.total;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = e == target ? -r.rest * share
                                      : exponential<D>(v[e] - r.top) * each;
          v[e] = share == 0.0f || col + e >= l.count ? 0.0f : p;
        }
        put_planes<D>(l.z + row * l.pitch_z + col, l.z_plane, v);
      },
      [](int, int) { return 0; }, [](int, int, float (&)[8], int) {});
}

// The factor that all of dz shares.
template <int D>
__device__ __forceinline__ float shared_factor(const LinearArgs &l) {
  const float s = l.a.d_grad_scale ? *l.a.d_grad_scale : 1.0f;
  return s * (l.scalars[1] / kRoom<D>);
}

// Eight sums of a gradient's row, out.
template <int T>
__device__ __forceinline__ void put_out(void *to, int64_t at, int n,
                                        bool accumulate, float factor,
                                        float (&v)[8]) {
  if (accumulate) {
    const Raw8<T> old = n == 8 ? load8<T, false>(to, at)
                               : load8_part<T>(to, at, n, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * factor + old[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= factor;
  }
  if (n == 8) {
    store8<T, false>(to, at, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) store_elem<T>(to, at + e, v[e]);
  }
}

// Sums of a tile, rows x width, either out or to the workspace.
template <class C, int D>
__device__ __forceinline__ void gradient_out(
    const LinearArgs &l, MTA_LDS uint8_t *lds,
    const f32x16 (&acc)[C::kRM][C::kRN], int64_t m0, int64_t n0, int64_t rows,
    float *hold, bool add, void *to, int64_t ld, int64_t from, int type,
    bool accumulate) {
  const float factor = shared_factor<D>(l);
  tile_out<C, false>(
      lds, acc, true, false, [](int, int) { return 0; },
      [&](int m, int n, float (&v)[8], int) {
        const int64_t row = m0 + m, col = n0 + n;
        if (row >= rows || col >= l.a.width) return;
        if (hold) {  // (rows of whole runs)
          auto *at = (MTA_GLOBAL f32x4 *)(hold + row * l.pitch + col);
          f32x4 x{v[0], v[1], v[2], v[3]}, y{v[4], v[5], v[6], v[7]};
          if (add) {
            x += at[0];
            y += at[1];
          }
          at[0] = x;
          at[1] = y;
          return;
        }
        const int many =
            static_cast<int>(min(int64_t{8}, l.a.width - col));
        with_type(type, [&](auto t) {
          put_out<decltype(t)::value>(to, (from + row) * ld + col, many,
                                      accumulate, factor, v);
        });
      },
      [](int, int) { return 0; }, [](int, int, float (&)[8], int) {});
}

// dh (+)= dz w over a part of a piece.
template <class C, int D>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_linear_dh(const LinearArgs l, const int64_t part_k, const bool hold) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  const uint32_t rows = static_cast<uint32_t>((l.a.rows + C::kBM - 1) / C::kBM);
  const uint32_t cols =
      static_cast<uint32_t>((l.a.width + C::kBN - 1) / C::kBN);
  const uint32_t block = beside(blockIdx.x, gridDim.x);
  const uint32_t part = block / (rows * cols);
  uint32_t tm, tn;
  banded(block % (rows * cols), rows, cols, tm, tn);
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  const int64_t deep = (l.count + 63) / 64 * 64;
  const int64_t k0 = min(deep, part * part_k), k1 = min(deep, k0 + part_k);
  f32x16 acc[C::kRM][C::kRN];
  const Operand z{l.z, l.z_plane, l.pitch_z, l.a.rows, 0};
  const Operand w{l.w + l.first * l.w_pitch, l.w_plane, l.w_pitch,
                  (l.a.width + 7) / 8 * 8, l.count};
  tile_product<C, D == MTA_F16, kAlong, kAcross>(z, w, pairs_of(l.planes), m0,
                                                 n0, k0, k1, lds, acc);
  gradient_out<C, D>(
      l, lds, acc, m0, n0, l.a.rows,
      hold ? l.sum_h + part * l.a.rows * l.pitch : nullptr, l.first > 0, l.a.dh,
      l.a.lddh, 0, l.a.type, false);
}

// A piece of dw = dz^T h over a part of the rows.
template <class C, int D>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_linear_dw(const LinearArgs l, const int64_t part_k, const bool hold) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  const uint32_t rows = static_cast<uint32_t>((l.count + C::kBM - 1) / C::kBM);
  const uint32_t cols =
      static_cast<uint32_t>((l.a.width + C::kBN - 1) / C::kBN);
  const uint32_t block = beside(blockIdx.x, gridDim.x);
  const uint32_t part = block / (rows * cols);
  uint32_t tm, tn;
  banded(block % (rows * cols), rows, cols, tm, tn);
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  const int64_t k0 = min(l.deep_rows, part * part_k);
  const int64_t k1 = min(l.deep_rows, k0 + part_k);
  f32x16 acc[C::kRM][C::kRN];
  const Operand z{l.z, l.z_plane, l.pitch_z, (l.count + 63) / 64 * 64,
                  l.deep_rows};
  const Operand h{l.h, l.h_plane, l.pitch, l.pitch, l.a.rows};
  tile_product<C, D == MTA_F16, kAcross, kAcross>(z, h, pairs_of(l.planes), m0,
                                                  n0, k0, k1, lds, acc);
  gradient_out<C, D>(l, lds, acc, m0, n0, l.count,
                     hold ? l.sum_w + part * l.count * l.pitch : nullptr, false,
                     l.a.dw, l.a.lddw, l.first, l.a.dw_type, l.a.accumulate);
}

// Parts held in the workspace, joined in order and out.
template <int D>
__global__ __launch_bounds__(256) void k_linear_out(const LinearArgs l,
                                                    const bool dh,
                                                    const int parts) {
  const int64_t rows = dh ? l.a.rows : l.count;
  const float *from = dh ? l.sum_h : l.sum_w;
  const int64_t runs = (l.a.width + 7) / 8;
  const float factor = shared_factor<D>(l);
  for (int64_t q = int64_t{blockIdx.x} * 256 + threadIdx.x; q < rows * runs;
       q += int64_t{gridDim.x} * 256) {
    const int64_t r = q / runs, i = (q - r * runs) * 8;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const float *at = from + r * l.pitch + i;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const Raw8<MTA_F32> x =
          load8<MTA_F32, false>(at + k * rows * l.pitch, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += x[e];
    }
    const int many = static_cast<int>(min(int64_t{8}, l.a.width - i));
    with_type(dh ? l.a.type : l.a.dw_type, [&](auto t) {
      if (dh)
        put_out<decltype(t)::value>(l.a.dh, r * l.a.lddh + i, many, false,
                                    factor, v);
      else
        put_out<decltype(t)::value>(l.a.dw, (l.first + r) * l.a.lddw + i, many,
                                    l.a.accumulate, factor, v);
    });
  }
}

__global__ __launch_bounds__(256) void k_linear_none(const LinearArgs l) {
  const int64_t n = l.a.vocab * l.a.width;
  for (int64_t q = int64_t{blockIdx.x} * 256 + threadIdx.x; q < n;
       q += int64_t{gridDim.x} * 256) {
    const int64_t r = q / l.a.width, i = q - r * l.a.width;
    with_type(l.a.dw_type, [&](auto t) {
      store_elem<decltype(t)::value>(l.a.dw, r * l.a.lddw + i, 0.0f);
    });
  }
}

uint32_t up(int64_t n, int64_t d) {
  return static_cast<uint32_t>((n + d - 1) / d);
}

// f(tile, type) for the run-time ones.
template <typename F>
void with_tile(const LinearCut &c, int type, F &&f) {
  with_type(type, [&](auto t) {
    if (c.tile == 256) f(Tile256{}, t);
    else if (c.deep) f(TileDeep{}, t);
    else f(Tile128{}, t);
  });
}

}  // namespace

hipError_t launch_linear_weights(const LinearArgs &l, hipStream_t s) {
  k_linear_weights<<<1, 1024, 0, s>>>(l);
  return hipGetLastError();
}

hipError_t launch_linear_pack_h(const LinearArgs &l, hipStream_t s) {
  const int64_t runs = l.a.rows * (l.pitch / 8);
  const uint32_t grid = std::min<uint32_t>(up(runs, 256), 1u << 20);
  with_type(l.a.type, [&](auto t) {
    k_linear_pack<decltype(t)::value><<<grid, 256, 0, s>>>(
        l, l.a.h, l.a.ldh, l.a.rows, l.h, l.h_plane, true);
  });
  return hipGetLastError();
}

hipError_t launch_linear_pack_w(const LinearArgs &l, uint16_t *to,
                                hipStream_t s) {
  const int64_t runs = l.a.vocab * (l.pitch / 8);
  const uint32_t grid = std::min<uint32_t>(up(runs, 256), 1u << 20);
  with_type(l.a.type, [&](auto t) {
    k_linear_pack<decltype(t)::value><<<grid, 256, 0, s>>>(
        l, l.a.w, l.a.ldw, l.a.vocab, to, l.w_plane, false);
  });
  return hipGetLastError();
}

hipError_t launch_linear_logits(const LinearArgs &l, const LinearCut &c,
                                hipStream_t s) {
  with_tile(c, l.a.type, [&](auto tile, auto t) {
    using C = decltype(tile);
    k_linear_logits<C, decltype(t)::value>
        <<<up(l.a.rows, C::kBM) * static_cast<uint32_t>(l.tiles), C::kThreads,
           0, s>>>(l);
  });
  return hipGetLastError();
}

hipError_t launch_linear_rows(const LinearArgs &l, hipStream_t s) {
  if (l.a.rows > 0)
    with_type(l.a.type, [&](auto t) {
      k_linear_rows<decltype(t)::value><<<up(l.a.rows, 64), 1024, 0, s>>>(l);
    });
  k_linear_sum<<<1, 1024, 0, s>>>(l);
  return hipGetLastError();
}

hipError_t launch_linear_grad(const LinearArgs &l, const LinearCut &c,
                              hipStream_t s) {
  with_tile(c, l.a.type, [&](auto tile, auto t) {
    using C = decltype(tile);
    k_linear_grad<C, decltype(t)::value>
        <<<up(l.a.rows, C::kBM) * up(l.count, C::kBN), C::kThreads, 0, s>>>(l);
  });
  return hipGetLastError();
}

hipError_t launch_linear_dh(const LinearArgs &l, const LinearCut &c, bool hold,
                            hipStream_t s) {
  with_tile(c, l.a.type, [&](auto tile, auto t) {
    using C = decltype(tile);
    k_linear_dh<C, decltype(t)::value>
        <<<up(l.a.rows, C::kBM) * up(l.a.width, C::kBN) * c.parts, C::kThreads,
           0, s>>>(l, c.part_k, hold);
  });
  return hipGetLastError();
}

hipError_t launch_linear_dw(const LinearArgs &l, const LinearCut &c, bool hold,
                            hipStream_t s) {
  with_tile(c, l.a.type, [&](auto tile, auto t) {
    using C = decltype(tile);
    k_linear_dw<C, decltype(t)::value>
        <<<up(l.count, C::kBM) * up(l.a.width, C::kBN) * c.parts, C::kThreads,
           0, s>>>(l, c.part_k, hold);
  });
  return hipGetLastError();
}

hipError_t launch_linear_none(const LinearArgs &l, hipStream_t s) {
  if (!l.a.accumulate) k_linear_none<<<4096, 256, 0, s>>>(l);
  return hipGetLastError();
}

hipError_t launch_linear_out(const LinearArgs &l, bool dh, int parts,
                             hipStream_t s) {
  const int64_t runs =
      (dh ? l.a.rows : l.count) * ((l.a.width + 7) / 8);
  const uint32_t grid = std::min<uint32_t>(up(runs, 256), 1u << 20);
  with_type(l.a.type, [&](auto t) {
    k_linear_out<decltype(t)::value><<<grid, 256, 0, s>>>(l, dh, parts);
  });
  return hipGetLastError();
}

}  // namespace mta
