// linear_kernels.hip -- the cross entropy of a linear output layer and its
// gradients on the matrix cores of gfx950, without keeping the logits.
//
//   z = h w^T,  p = softmax(z),  loss = sum weight (-log p[target])
//   dz = weight (p - [target]),  dh = dz w,  dw = dz^T h
//
// Rows that are left out (padding, prompts) cost nothing: a first kernel lists
// the others, h is packed in that order, and every product ends at their number,
// which stays on the device.
//
// The forward is one product whose tiles leave two numbers a row, the largest
// logit and the sum of exponentials beside it (without the target's: 1 - p keeps
// its digits as p nears 1), and a kernel that joins a row's tiles.  The
// gradients take the vocabulary in pieces: the product again, its tiles written
// as dz in 16 bits, then dh += dz w and the piece of dw = dz^T h, which read dz,
// w and h as they lie, with k along or across.  Four products instead of the
// three that kept logits would need: memory is the reason.  Logits in 32 bits for
// 8192 x 50257 are 1.6 GB; writing and reading them would take 0.7 ms, the fourth
// product of 1600 columns 1.3.
//
// A float32 call has three bfloat16 planes for each operand and six products.
//
// Bound by the matrix pipes at the clock that this card's power allows: 14746
// rows of 768 against 50257 take 1.15 ms (990 TFLOP/s; the library's large
// product reaches 1228), 6554 rows of 1600 with gradients 4.3 ms (4.2 TFLOP of
// four products: 990).  8 rows take 24 us, 16.5 of them the product at 4.7 TB/s
// of w.
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

// A weight's part in the largest: an infinite one's would leave zeros of the
// other rows' dz, and NaN (a NaN's part is none, too).
__device__ __forceinline__ float finite_size(float weight) {
  const float x = fabsf(weight);
  return x < __builtin_inff() ? x : 0.0f;
}

// How many rows take part, the weight of a row without weights and the largest
// finite one.
__device__ __forceinline__ void put_counts(const LinearArgs &l, int all,
                                           float most) {
  if (!(most > 0.0f)) most = 1.0f;
  const float one =
      all > 0 ? static_cast<float>(1.0 / static_cast<double>(all)) : 0.0f;
  l.scalars[0] = one;
  l.scalars[1] = l.backward || l.a.weights ? most : one;
  *l.active = all;
}

// The rows that take part, in order, their number, the weight of a row without
// weights and the largest finite magnitude of any: one workgroup, a run of up to
// 64 rows a lane at a time, whose answers are bits of a word.
__global__ __launch_bounds__(1024) void k_linear_rows_in(const LinearArgs l) {
  const mta_linear_loss_args &a = l.a;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  __shared__ int counts[16];
  __shared__ float mosts[16];
  float most = 0.0f;
  int all = 0;
  constexpr int64_t kRun = 65536;
  for (int64_t base = 0; base < a.rows; base += kRun) {
    const int64_t n = min(a.rows - base, kRun);
    const int each = static_cast<int>((n + 1023) / 1024);
    const int64_t from = base + min(n, int64_t{each} * threadIdx.x);
    const int here = static_cast<int>(min(base + n - from, int64_t{each}));
    uint64_t in = 0;
    const auto mark = [&](auto &&takes_part) {
#pragma unroll 8
      for (int k = 0; k < here; ++k)
        if (takes_part(from + k)) in |= uint64_t{1} << k;
    };
    if (l.backward)
      mark([&](int64_t r) {
        const float w = l.rows[r].weight;
        most = fmaxf(most, finite_size(w));
        return w != 0.0f;
      });
    else if (a.weights)
      mark([&](int64_t r) {
        const float w = a.weights[r];
        const bool is = a.targets[r] != a.ignore_index && w != 0.0f;
        most = is ? fmaxf(most, finite_size(w)) : most;
        return is;
      });
    else
      mark([&](int64_t r) { return a.targets[r] != a.ignore_index; });
    // counts of the lanes before
    const int count = __popcll(in);
    int before = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int x = __shfl_up(before, d);
      if (lane >= d) before += x;
    }
    if (lane == 63) counts[wave] = before;
    __syncthreads();
    before += all - count;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (k < wave) before += counts[k];
      all += counts[k];
    }
    for (; in; in &= in - 1)
      l.index[before++] =
          static_cast<int>(from) + __ffsll(static_cast<long long>(in)) - 1;
    __syncthreads();
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) most = fmaxf(most, __shfl_xor(most, d));
  if (lane == 0) mosts[wave] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 1; k < 16; ++k) most = fmaxf(most, mosts[k]);
    put_counts(l, all, most);
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

// Rows of w into its planes, with zeros behind the last column.
template <int D>
__device__ __forceinline__ void pack_run(const LinearArgs &l, const void *from,
                                         int64_t row, int64_t i,
                                         uint16_t *to, int64_t plane) {
  const int64_t left = l.a.width - i;
  const int n = static_cast<int>(left >= 8 ? 8 : left > 0 ? left : 0);
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n > 0) {
    const Raw8<D> x = n == 8 ? load8<D, false>(from, row + i)
                             : load8_part<D>(from, row + i, n, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x[e];
  }
  put_planes<D>(to, plane, v);
}

template <int D>
__global__ __launch_bounds__(256) void k_linear_pack_w(const LinearArgs l,
                                                       uint16_t *to) {
  const int64_t runs = l.pitch / 8;
  for (int64_t q = int64_t{blockIdx.x} * 256 + threadIdx.x;
       q < l.a.vocab * runs; q += int64_t{gridDim.x} * 256) {
    const int64_t r = q / runs, i = (q - r * runs) * 8;
    pack_run<D>(l, l.a.w, r * l.a.ldw, i, to + r * l.pitch + i, l.w_plane);
  }
}

// The rows of h that take part, of which index[] has the numbers, into its planes,
// and zeros where the others' results are.
template <int D, typename Index>
__device__ __forceinline__ void pack_rows(const LinearArgs &l, int64_t active,
                                          Index index) {
  const int64_t runs = l.pitch / 8;
  for (int64_t q = int64_t{blockIdx.x} * blockDim.x + threadIdx.x;
       q < l.a.rows * runs; q += int64_t{gridDim.x} * blockDim.x) {
    const int64_t r = q / runs, i = (q - r * runs) * 8;
    if (r < active)
      pack_run<D>(l, l.a.h, index[r] * l.a.ldh, i, l.h + r * l.pitch + i,
                  l.h_plane);
    if (active == l.a.rows || !left_out(l, r)) continue;
    if (i == 0 && !l.backward) {
      l.rows[r] = mta_linear_row{0.0f, 0.0f, 0.0f, 0.0f};
      if (l.a.logp) l.a.logp[r] = 0.0f;
    }
    if (l.a.dh) {
      const int64_t left = l.a.width - i;
      const float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (left >= 8) {
        store8<D, false>(l.a.dh, r * l.a.lddh + i, v);
      } else {
        for (int e = 0; e < left; ++e)
          store_elem<D>(l.a.dh, r * l.a.lddh + i + e, 0.0f);
      }
    }
  }
}

template <int D>
__global__ __launch_bounds__(256) void k_linear_pack_h(const LinearArgs l) {
  pack_rows<D>(l, *l.active, l.index);
}

// Both for up to 1024 rows, whose workgroups find the rows each for itself: 3.5 us
// at 8 rows where the two launches take 3.3 and 3.1.
template <int D>
__global__ __launch_bounds__(1024) void k_linear_few_rows(const LinearArgs l) {
  const mta_linear_loss_args &a = l.a;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  __shared__ int counts[16], index[1024];
  __shared__ float mosts[16];
  const int64_t r = threadIdx.x;
  const bool in = r < a.rows && !left_out(l, r);
  const float w = !in          ? 0.0f
                  : l.backward ? l.rows[r].weight
                  : a.weights  ? a.weights[r]
                               : 0.0f;
  float most = finite_size(w);
  const uint64_t bits = __ballot(in);
#pragma unroll
  for (int d = 32; d > 0; d /= 2) most = fmaxf(most, __shfl_xor(most, d));
  if (lane == 0) {
    counts[wave] = __popcll(bits);
    mosts[wave] = most;
  }
  __syncthreads();
  int before = __popcll(bits & ((uint64_t{1} << lane) - 1)), all = 0;
  most = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    if (k < wave) before += counts[k];
    all += counts[k];
    most = fmaxf(most, mosts[k]);
  }
  if (in) {
    index[before] = threadIdx.x;
    if (blockIdx.x == 0) l.index[before] = threadIdx.x;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) put_counts(l, all, most);
  __syncthreads();
  pack_rows<D>(l, all, index);
}

// e^(z - top) with `shift` = shift_of(top): in one fused step, whose rounding of
// the shift is no larger than that of a logit of top's size; for float32 calls
// with all digits.
constexpr float kLog2e = 1.44269504f;
template <int D>
__device__ __forceinline__ float shift_of(float top) {
  // (nothing but -infinity, or what times log2(e) would be: exponentials of 0)
  constexpr float kLeast =
      D == MTA_F32 ? -3.40282347e38f : -3.40282347e38f / kLog2e;
  const float t = top < kLeast ? 0.0f : top;
  return D == MTA_F32 ? t : t * -kLog2e;
}
template <int D>
__device__ __forceinline__ float exponential(float z, float shift) {
  if constexpr (D == MTA_F32) return expf(z - shift);
  else return __builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, shift));
}

template <class C, int D>
__device__ __forceinline__ void logits_tile(const LinearArgs &l,
                                            int64_t active, int64_t m0,
                                            int64_t n0, MTA_LDS uint8_t *lds,
                                            f32x16 (&acc)[C::kRM][C::kRN]) {
  const Operand h{l.h, l.h_plane, l.pitch, active, 0};
  const Operand w{l.w, l.w_plane, l.w_pitch, l.a.vocab, 0};
  tile_product<C, D == MTA_F16, kAlong, kAlong>(
      h, w, pairs_of(l.planes), m0, n0, 0, (l.a.width + 63) / 64 * 64, lds,
      acc);
}

// The tile of workgroup number `block` where rows x cols of them are; false:
// there is none.
__device__ __forceinline__ bool my_tile(uint32_t block, uint32_t rows,
                                        uint32_t cols, uint32_t &tm,
                                        uint32_t &tn) {
  if (block >= rows * cols) return false;
  banded(beside(block, rows * cols), rows, cols, tm, tn);
  return true;
}

// A tile of logits as each row's largest and its sum of exponentials without
// the target's.
template <class C, int D>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_linear_logits(const LinearArgs l) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  const int64_t active = *l.active;
  uint32_t tm, tn;
  if (!my_tile(blockIdx.x,
               static_cast<uint32_t>((active + C::kBM - 1) / C::kBM),
               static_cast<uint32_t>(l.tiles), tm, tn))
    return;
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  f32x16 acc[C::kRM][C::kRN];
  logits_tile<C, D>(l, active, m0, n0, lds, acc);

  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int wr = wave % C::kWR, wc = wave / C::kWR;
  auto *side = (MTA_LDS f32x2 *)lds;  // [WC][BM]
  // columns of this lane: n1 + 32 j + 8 q + e
  const int64_t n1 = n0 + wc * C::kTN + lane / 32 * 4;
  const int many =
      static_cast<int>(min(int64_t{C::kBN}, l.a.vocab - n1));
  const auto column = [](int j, int r) { return j * 32 + r / 4 * 8 + r % 4; };
  if (n0 + C::kBN > l.a.vocab) {
#pragma unroll
    for (int i = 0; i < C::kRM; ++i)
#pragma unroll
      for (int j = 0; j < C::kRN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (column(j, r) >= many) acc[i][j][r] = -__builtin_inff();
  }
  int64_t target[C::kRM];
#pragma unroll
  for (int i = 0; i < C::kRM; ++i) {
    const int64_t row = min(m0 + wr * C::kTM + i * 32 + lane % 32, active - 1);
    target[i] = l.a.targets[l.index[row]] - n1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < C::kRM; ++i) {
    const int m = wr * C::kTM + i * 32 + lane % 32;
    float top = acc[i][0][0];
#pragma unroll
    for (int j = 0; j < C::kRN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, acc[i][j][r]);
    top = fmaxf(top, __shfl_xor(top, 32));
    const float shift = shift_of<D>(top);
    float sum = 0.0f;
    const bool mine = target[i] >= 0 && target[i] < C::kTN;
    if (__builtin_expect(__any(mine && m0 + m < active), 0)) {
      const int at = mine ? static_cast<int>(target[i]) : -1;
#pragma unroll
      for (int j = 0; j < C::kRN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float e = exponential<D>(acc[i][j][r], shift);
          if (column(j, r) == at) {
            if (m0 + m < active) l.z_target[m0 + m] = acc[i][j][r];
          } else {
            sum += e;
          }
        }
    } else {
      // (two sums: one would be a chain of additions as long as the row)
      float other = 0.0f;
#pragma unroll
      for (int j = 0; j < C::kRN; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
          sum += exponential<D>(acc[i][j][r], shift);
          other += exponential<D>(acc[i][j][r + 1], shift);
        }
      sum += other;
    }
    sum += __shfl_xor(sum, 32);
    if (lane < 32) side[wc * C::kBM + m] = f32x2{top, sum};
  }
  __syncthreads();
  for (int m = threadIdx.x; m < C::kBM; m += C::kThreads) {
    if (m0 + m >= active) break;
    f32x2 v = side[m];
#pragma unroll
    for (int k = 1; k < C::kWC; ++k) {
      const f32x2 u = side[k * C::kBM + m];
      const float top = fmaxf(v[0], u[0]), shift = shift_of<D>(top);
      v = f32x2{top, v[1] * exponential<D>(v[0], shift) +
                         u[1] * exponential<D>(u[0], shift)};
    }
    l.partial[tn * l.a.rows + m0 + m] = make_float2(v[0], v[1]);
  }
}

// Rows' tiles joined: `across` rows (up to 64) to a workgroup, one a lane, in 16
// waves and, with fewer rows, parts of waves that take every so many'th tile and
// are joined in order (8 rows, 393 tiles: 4.8 us, and 9.0 with a wave for 64 rows
// at all sizes).  A workgroup that has all rows sums the loss too.
template <int D>
__global__ __launch_bounds__(1024) void k_linear_rows(const LinearArgs l, int across) {
  const mta_linear_loss_args &a = l.a;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t at = int64_t{blockIdx.x} * 64 + lane % across;
  const int64_t active = *l.active;
  if (blockIdx.x * 64 >= active && gridDim.x > 1) return;
  const int parts = 1024 / across, part = threadIdx.x / across;
  const auto join = [](float &top, float &sum, float t, float s) {
    const float most = fmaxf(top, t), shift = shift_of<D>(most);
    sum = sum * exponential<D>(top, shift) + s * exponential<D>(t, shift);
    top = most;
  };
  float top = -__builtin_inff(), sum = 0.0f;
  if (at < active) {
    constexpr int kMany = 8;  // on their way at a time
    for (int64_t t = part; t < l.tiles; t += parts * kMany) {
      float2 v[kMany];
#pragma unroll
      for (int k = 0; k < kMany; ++k)
        v[k] = l.partial[min(t + parts * k, l.tiles - 1) * a.rows + at];
#pragma unroll
      for (int k = 0; k < kMany; ++k)
        if (t + parts * k < l.tiles) join(top, sum, v[k].x, v[k].y);
    }
  }
  for (int d = across; d < 64; d *= 2)
    join(top, sum, __shfl_xor(top, d), __shfl_xor(sum, d));
  __shared__ float2 side[16][64];
  side[wave][lane] = make_float2(top, sum);
  __syncthreads();
  if (wave != 0) return;
  double term = 0.0;
  if (at < active && lane < across) {
#pragma unroll
    for (int k = 1; k < 16; ++k)
      join(top, sum, side[k][lane].x, side[k][lane].y);
    const int64_t row = l.index[at], target = a.targets[row];
    mta_linear_row r;
    float logp;
    r.weight = a.weights ? a.weights[row] : l.scalars[0];
    if (target < 0 || target >= a.vocab) {
      r.top = r.total = r.rest = logp = __builtin_nanf("");
    } else {
      const float zt = l.z_target[at];
      const float own = exponential<D>(zt, shift_of<D>(top));
      r.top = top;
      r.total = sum + own;
      r.rest = sum / r.total;
      logp = zt == top ? -log1pf(sum) : (zt - top) - logf(r.total);
      // (no exponential of the row's is a number above 0: its largest logit is
      // infinite or, in 16 bits, beyond 2^128 / log2(e))
      if (!(r.total > 0.0f && r.total < __builtin_inff()))
        r.top = r.total = r.rest = logp = __builtin_nanf("");
    }
    l.rows[row] = r;
    if (a.logp) a.logp[row] = logp;
    term = -static_cast<double>(r.weight) * logp;
    l.terms[at] = term;
  }
  if (gridDim.x == 1) {
#pragma unroll
    for (int d = 32; d > 0; d /= 2) term += __shfl_xor(term, d);
    if (lane == 0) *a.loss = static_cast<float>(term);
  }
}

// The loss: each lane's terms in order, then the lanes'.
__global__ __launch_bounds__(1024) void k_linear_sum(const LinearArgs l) {
  double x = 0.0;
#pragma unroll 8
  for (int64_t r = threadIdx.x; r < *l.active; r += 1024) x += l.terms[r];
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

// What dz takes of a row, for the rows that take part and, up to a whole step of
// 64, rows of zeros.
template <int D>
__global__ __launch_bounds__(256) void k_linear_info(const LinearArgs l) {
  const int64_t active = *l.active, deep = (active + 63) / 64 * 64;
  const int64_t q = int64_t{blockIdx.x} * 256 + threadIdx.x;
  if (q >= deep) return;
  LinearInfo x{-__builtin_inff(), 0.0f, 0.0f, -1};
  if (D == MTA_F32) x.shift = __builtin_inff();
  if (q < active) {
    const int64_t row = l.index[q];
    const mta_linear_row r = l.rows[row];
    const float share = r.weight / l.scalars[1] * kRoom<D>;
    x.shift = shift_of<D>(r.top);
    x.each = share / r.total;
    x.own = -r.rest * share;
    const int64_t t = l.a.targets[row];
    x.target = t >= 0 && t < l.a.vocab ? static_cast<int>(t) : -1;
  }
  l.info[q] = x;
}

// The factor that all of dz shares (its own factors' product is exact in 64 bits,
// where small weights under a large scale do not leave the range of numbers).
template <int D>
__device__ __forceinline__ float shared_factor(const LinearArgs &l) {
  const double s = l.a.d_grad_scale ? *l.a.d_grad_scale : 1.0f;
  return static_cast<float>(s * l.scalars[1] * (1.0 / kRoom<D>));
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

// Sums of a tile, rows x width, either out, to row from + m or index[m], or to
// the workspace.
template <class C, int D>
__device__ __forceinline__ void gradient_out(
    const LinearArgs &l, MTA_LDS uint8_t *lds,
    const f32x16 (&acc)[C::kRM][C::kRN], int64_t m0, int64_t n0, int64_t rows,
    float *hold, bool add, void *to, int64_t ld, int64_t from,
    const int *index, int type, bool accumulate) {
  const float factor = shared_factor<D>(l);
  const int high = static_cast<int>(min(rows - m0, int64_t{C::kBM}));
  tile_out<C, false>(
      lds, acc, true, false,
      [&](int m, int) {
        return index ? int64_t{index[m0 + min(m, high - 1)]} : from + m0 + m;
      },
      [&](int m, int n, float (&v)[8], int64_t row) {
        const int64_t col = n0 + n;
        if (m >= high || col >= l.a.width) return;
        if (hold) {  // (rows of whole runs)
          auto *at = (MTA_GLOBAL f32x4 *)(hold + (m0 + m) * l.pitch + col);
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
          put_out<decltype(t)::value>(to, row * ld + col, many, accumulate,
                                      factor, v);
        });
      },
      [](int, int) { return 0; }, [](int, int, float (&)[8], int) {});
}

// A tile of logits as dz, without the factor that all rows share.
template <class C, int D>
__device__ __forceinline__ void make_dz(const LinearArgs &l,
                                        const LinearPiece &piece,
                                        int64_t active, uint32_t block,
                                        MTA_LDS uint8_t *lds) {
  uint32_t tm, tn;
  if (!my_tile(block, static_cast<uint32_t>((active + C::kBM - 1) / C::kBM),
               static_cast<uint32_t>((piece.count + C::kBN - 1) / C::kBN), tm,
               tn))
    return;
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  f32x16 acc[C::kRM][C::kRN];
  logits_tile<C, D>(l, active, m0, piece.first + n0, lds, acc);
  const int rows = static_cast<int>(
      min((active + 63) / 64 * 64 - m0, int64_t{C::kBM}));
  const int cols = static_cast<int>(
      min((piece.count + 63) / 64 * 64 - n0, int64_t{C::kBN}));
  const int there = static_cast<int>(min(piece.count - n0, int64_t{C::kBN}));
  const int from = static_cast<int>(piece.first + n0);
  uint16_t *to = piece.z + m0 * l.pitch_z + n0;
  const LinearInfo *info = l.info + m0;
  const uint32_t pitch = static_cast<uint32_t>(l.pitch_z);
  tile_out<C, false>(
      lds, acc, true, false,
      [&](int m, int) { return info[min(m, rows - 1)]; },
      [&](int m, int n, float (&v)[8], const LinearInfo &x) {
        if (m >= rows || n >= cols) return;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = exponential<D>(v[e], x.shift) * x.each;
        const int own = x.target - from - n;
        if (__any(own >= 0 && own < 8)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = e == own ? x.own : v[e];
        }
        if (there < C::kBN) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = n + e < there ? v[e] : 0.0f;
        }
        put_planes<D>(to + static_cast<uint32_t>(m) * pitch + n, l.z_plane, v);
      },
      [](int, int) { return 0; }, [](int, int, float (&)[8], int) {});
}

// dh (+)= dz w over a part of a piece.
template <class C, int D>
__device__ __forceinline__ void make_dh(const LinearArgs &l,
                                        const LinearPiece &piece,
                                        const LinearBack &back, int64_t active,
                                        uint32_t number,
                                        MTA_LDS uint8_t *lds) {
  const int parts = back.dh_parts;
  const uint32_t cols =
      static_cast<uint32_t>((l.a.width + C::kBN - 1) / C::kBN);
  const uint32_t tiles =
      static_cast<uint32_t>((active + C::kBM - 1) / C::kBM) * cols;
  if (number >= tiles * parts) return;
  const uint32_t block = beside(number, tiles * parts);
  const uint32_t part = block / tiles;
  uint32_t tm, tn;
  banded(block % tiles, tiles / cols, cols, tm, tn);
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  const int64_t deep = (piece.count + 63) / 64 * 64;
  const int64_t each = (deep / 64 + parts - 1) / parts * 64;
  const int64_t k0 = min(deep, part * each), k1 = min(deep, k0 + each);
  f32x16 acc[C::kRM][C::kRN];
  const Operand z{piece.z, l.z_plane, l.pitch_z, active, 0};
  const Operand w{l.w + piece.first * l.w_pitch, l.w_plane, l.w_pitch,
                  (l.a.width + 7) / 8 * 8, piece.count};
  tile_product<C, D == MTA_F16, kAlong, kAcross>(z, w, pairs_of(l.planes), m0,
                                                 n0, k0, k1, lds, acc);
  gradient_out<C, D>(
      l, lds, acc, m0, n0, active,
      back.hold_dh ? l.sum_h + part * l.a.rows * l.pitch : nullptr, piece.first > 0, l.a.dh,
      l.a.lddh, 0, l.index, l.a.type, false);
}

// A piece of dw = dz^T h over a part of the rows.
template <class C, int D>
__device__ __forceinline__ void make_dw(const LinearArgs &l,
                                        const LinearPiece &piece,
                                        const LinearBack &back, int64_t active,
                                        uint32_t number,
                                        MTA_LDS uint8_t *lds) {
  const int parts = back.dw_parts;
  const uint32_t rows = static_cast<uint32_t>((piece.count + C::kBM - 1) / C::kBM);
  const uint32_t cols =
      static_cast<uint32_t>((l.a.width + C::kBN - 1) / C::kBN);
  if (number >= rows * cols * parts) return;
  const uint32_t block = beside(number, rows * cols * parts);
  const uint32_t part = block / (rows * cols);
  uint32_t tm, tn;
  banded(block % (rows * cols), rows, cols, tm, tn);
  const int64_t m0 = int64_t{tm} * C::kBM, n0 = int64_t{tn} * C::kBN;
  const int64_t deep = (active + 63) / 64 * 64;
  const int64_t each = (deep / 64 + parts - 1) / parts * 64;
  const int64_t k0 = min(deep, part * each), k1 = min(deep, k0 + each);
  f32x16 acc[C::kRM][C::kRN];
  const Operand z{piece.z, l.z_plane, l.pitch_z, (piece.count + 63) / 64 * 64, deep};
  const Operand h{l.h, l.h_plane, l.pitch, l.pitch, active};
  tile_product<C, D == MTA_F16, kAcross, kAcross>(z, h, pairs_of(l.planes), m0,
                                                  n0, k0, k1, lds, acc);
  gradient_out<C, D>(l, lds, acc, m0, n0, piece.count,
                     back.hold_dw ? l.sum_w + part * piece.count * l.pitch : nullptr, false,
                     l.a.dw, l.a.lddw, piece.first, nullptr, l.a.dw_type,
                     l.a.accumulate);
}

// dh and dw of a piece and dz of the next one, or any of them: none needs
// another, and together they fill the compute units better than one after the
// other (8192 rows of 1600 are 224 tiles of dh).  Long sums come first.
template <class C, int D>
__global__ __launch_bounds__(C::kThreads)
    __attribute__((amdgpu_waves_per_eu(C::kPerSimd, C::kPerSimd))) void
    k_linear_back(const LinearArgs l, const LinearPiece piece,
                  const LinearPiece next, const LinearBack back) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds_[C::kLds];
  auto *lds = (MTA_LDS uint8_t *)lds_;
  const int64_t active = *l.active;
  const uint32_t block = blockIdx.x;
  if (block < back.first_dw)
    make_dh<C, D>(l, piece, back, active, block, lds);
  else if (block < back.first_dz)
    make_dw<C, D>(l, piece, back, active, block - back.first_dw, lds);
  else
    make_dz<C, D>(l, next, active, block - back.first_dz, lds);
}

// Parts held in the workspace, joined in order and out.
template <int D>
__global__ __launch_bounds__(256) void k_linear_out(
    const LinearArgs l, const LinearPiece piece, const bool dh,
    const int parts) {
  const int64_t rows = dh ? *l.active : piece.count;
  const int64_t step = (dh ? l.a.rows : piece.count) * l.pitch;
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
          load8<MTA_F32, false>(at + k * step, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += x[e];
    }
    const int many = static_cast<int>(min(int64_t{8}, l.a.width - i));
    with_type(dh ? l.a.type : l.a.dw_type, [&](auto t) {
      if (dh)
        put_out<decltype(t)::value>(l.a.dh, l.index[r] * l.a.lddh + i, many, false,
                                    factor, v);
      else
        put_out<decltype(t)::value>(l.a.dw, (piece.first + r) * l.a.lddw + i, many,
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

// f(tile, type) for the run-time ones; a small tile's workgroups that are too few
// for two on a CU get the deep one.
template <typename F>
void with_tile(int tile, uint32_t groups, int type, F &&f) {
  with_type(type, [&](auto t) {
    if (tile == 256) f(Tile256{}, t);
    else if (tile == 64) f(Tile64{}, t);
    else if (groups <= 256) f(TileDeep{}, t);
    else f(Tile128{}, t);
  });
}

}  // namespace

hipError_t launch_linear_rows_in(const LinearArgs &l, hipStream_t s) {
  const int64_t runs = l.a.rows * (l.pitch / 8);
  if (l.a.rows <= 1024) {
    with_type(l.a.type, [&](auto t) {
      k_linear_few_rows<decltype(t)::value>
          <<<std::clamp<uint32_t>(up(runs, 1024), 1, 1u << 20), 1024, 0, s>>>(l);
    });
    return hipGetLastError();
  }
  k_linear_rows_in<<<1, 1024, 0, s>>>(l);
  with_type(l.a.type, [&](auto t) {
    k_linear_pack_h<decltype(t)::value>
        <<<std::min<uint32_t>(up(runs, 256), 1u << 20), 256, 0, s>>>(l);
  });
  return hipGetLastError();
}

hipError_t launch_linear_pack_w(const LinearArgs &l, uint16_t *to,
                                hipStream_t s) {
  const uint32_t grid =
      std::min<uint32_t>(up(l.a.vocab * (l.pitch / 8), 256), 1u << 20);
  with_type(l.a.type, [&](auto t) {
    k_linear_pack_w<decltype(t)::value><<<grid, 256, 0, s>>>(l, to);
  });
  return hipGetLastError();
}

hipError_t launch_linear_info(const LinearArgs &l, hipStream_t s) {
  with_type(l.a.type, [&](auto t) {
    k_linear_info<decltype(t)::value>
        <<<up(l.a.rows + 63, 256), 256, 0, s>>>(l);
  });
  return hipGetLastError();
}

hipError_t launch_linear_logits(const LinearArgs &l, int tile, hipStream_t s) {
  const uint32_t grid = up(l.a.rows, tile) * static_cast<uint32_t>(l.tiles);
  with_tile(tile, grid, l.a.type, [&](auto which, auto t) {
    using C = decltype(which);
    k_linear_logits<C, decltype(t)::value><<<grid, C::kThreads, 0, s>>>(l);
  });
  return hipGetLastError();
}

hipError_t launch_linear_rows(const LinearArgs &l, hipStream_t s) {
  const uint32_t grid = std::max(1u, up(l.a.rows, 64));
  int across = 64;
  while (across > 1 && across / 2 >= l.a.rows) across /= 2;
  with_type(l.a.type, [&](auto t) {
    k_linear_rows<decltype(t)::value><<<grid, 1024, 0, s>>>(l, across);
  });
  if (grid > 1) k_linear_sum<<<1, 1024, 0, s>>>(l);
  return hipGetLastError();
}

hipError_t launch_linear_back(const LinearArgs &l, int tile,
                              const LinearPiece *piece,
                              const LinearPiece *next, LinearBack back,
                              hipStream_t s) {
  // (segments in wholes of eight, so that each begins on the first XCD)
  const auto eight = [](uint32_t n) { return (n + 7) / 8 * 8; };
  back.first_dw = back.first_dz = 0;
  if (piece && l.a.dh)
    back.first_dw = eight(up(l.a.rows, tile) * up(l.a.width, tile) *
                          back.dh_parts);
  back.first_dz = back.first_dw;
  if (piece && l.a.dw)
    back.first_dz += eight(up(piece->count, tile) * up(l.a.width, tile) *
                           back.dw_parts);
  uint32_t grid = back.first_dz;
  if (next) grid += up(l.a.rows, tile) * up(next->count, tile);
  const LinearPiece none{};
  with_tile(tile, grid, l.a.type, [&](auto which, auto t) {
    using C = decltype(which);
    k_linear_back<C, decltype(t)::value><<<grid, C::kThreads, 0, s>>>(
        l, piece ? *piece : none, next ? *next : none, back);
  });
  return hipGetLastError();
}

hipError_t launch_linear_none(const LinearArgs &l, hipStream_t s) {
  if (!l.a.accumulate) k_linear_none<<<4096, 256, 0, s>>>(l);
  return hipGetLastError();
}

hipError_t launch_linear_out(const LinearArgs &l, const LinearPiece &piece,
                             bool dh, int parts, hipStream_t s) {
  const int64_t runs =
      (dh ? l.a.rows : piece.count) * ((l.a.width + 7) / 8);
  const uint32_t grid = std::min<uint32_t>(up(runs, 256), 1u << 20);
  with_type(l.a.type, [&](auto t) {
    k_linear_out<decltype(t)::value>
        <<<grid, 256, 0, s>>>(l, piece, dh, parts);
  });
  return hipGetLastError();
}

}  // namespace mta
