// policy_kernels.hip -- the clipped policy loss with a KL term from the
// logits, forward and backward, on gfx950.
//
// A row's log-softmax needs its maximum and its sum of exponentials before
// the first gradient can be written, so the plain way reads the logits at
// least twice.  Here a row stays in the registers of the workgroup that reads
// it (65536 logits are 32 registers a lane of 1024 in 16 bits), so one call
// reads every logit once and writes every gradient once: bound by HBM.  Longer
// rows are read twice, the second time mostly from the memory-side cache.
//
// Numerics: exponentials are 2^((z - max) log2 e) in float32, a lane sums at
// most 64 (a streamed row: vocab / 1024) of them in float32, lanes are joined
// in float32 within a wave and in float64 across waves.  What follows for a
// row (its logp, ratio, clip, KL) is a handful of float64 operations of one
// wave: exp(d) - d - 1 and 1 - p lose every digit of a float32 near 0.
#include "ops_device.h"

namespace mta {
namespace {

constexpr float kInf = __builtin_inff();
constexpr float kLog2E = 1.44269504088896341f;

// The bits of -infinity, which pad a row: they add 0 to its sum.
template <int D>
constexpr uint32_t kMinusInf =
    D == MTA_F32 ? 0xFF800000u : D == MTA_BF16 ? 0xFF80u : 0xFC00u;

struct PolicyRow {
  float coef;  // d loss / d logp, weight included
  double lse, logp;
  double sums[kPolicySums];
};

// The row's scalars from its maximum and the sum of exp(z - max).
__device__ PolicyRow policy_row(const mta_policy_args &a, int64_t row, float w,
                                float za, float top, double total) {
  PolicyRow r;
  const double logtotal = log(total);
  r.lse = double{top} + logtotal;
  r.logp = (double{za} - double{top}) - logtotal;
  const double adv = a.advantages[row];
  const double ratio = exp(r.logp - double{a.old_logp[row]});
  const double lo = 1.0 - a.clip_low, hi = 1.0 + a.clip_high;
  // comparisons that keep a NaN ratio
  const double cut = ratio < lo ? lo : ratio > hi ? hi : ratio;
  const double plain = ratio * adv, clipped = cut * adv;
  const bool over = plain > clipped;
  double loss = over ? -clipped : -plain;
  double slope = over ? 0.0 : -plain;
  double kl = 0.0;
  if (a.ref_logp) {
    const double d = double{a.ref_logp[row]} - r.logp;
    const double e = expm1(d);
    kl = e - d;
    loss += a.kl_coef * kl;
    slope -= a.kl_coef * e;
  }
  r.coef = static_cast<float>(double{w} * slope);
  r.sums[0] = double{w} * loss;
  r.sums[1] = double{w} * kl;
  r.sums[2] = over ? double{w} : 0.0;
  return r;
}

// Maximum or sum over the 64 lanes of a wave, in every lane.
__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
  return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Threads to a row; a workgroup is at least four waves.
template <int Threads>
constexpr int kRows = Threads < 256 ? 256 / Threads : 1;

// A row's shared values, one set a row of the workgroup.
template <int Threads>
struct RowShared {
  float top[Threads / 64];
  float sum[Threads / 64];
  float gain, chosen;
};

// Units >= 0: that many runs of eight logits to a lane, kept in registers.
// Units == 0: the row is streamed, twice.
template <int D, int Threads, int Units>
__global__ __launch_bounds__(Threads * kRows<Threads>) void k_policy(
    const mta_policy_args a) {
  constexpr int kWaves = Threads / 64;
  constexpr bool kOneWave = Threads == 64;
  __shared__ RowShared<Threads> shared[kRows<Threads>];
  const int slot_in = threadIdx.x / Threads;
  RowShared<Threads> &sh = shared[slot_in];
  const int tid = threadIdx.x % Threads;
  const int wave = tid / 64;
  const int64_t slot =
      static_cast<int64_t>(blockIdx.x) * kRows<Threads> + slot_in;
  const int64_t slots = static_cast<int64_t>(gridDim.x) * kRows<Threads>;
  const int64_t vocab = a.vocab;
  const int64_t units = (vocab + 7) / 8;
  const float S = a.d_grad_scale ? *a.d_grad_scale : 1.0f;
  double sums[kPolicySums] = {0.0, 0.0, 0.0};

  const auto load = [&](int64_t base, int64_t u) {
    const int64_t left = vocab - u * 8;
    if (left >= 8) return load8<D, Units != 0>(a.logits, base + u * 8);
    return load8_part<D>(a.logits, base + u * 8,
                         static_cast<int>(left > 0 ? left : 0), kMinusInf<D>);
  };
  const auto store = [&](int64_t base, int64_t u, const float(&x)[8]) {
    const int64_t left = vocab - u * 8;
    if (left >= 8) {
      store8<D, true>(a.dlogits, base + u * 8, x);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) store_elem<D>(a.dlogits, base + u * 8 + k, x[k]);
    }
  };
  const auto sync = [&] {
    if constexpr (!kOneWave) __syncthreads();
  };

  for (int64_t row = slot; row < a.rows; row += slots) {
    const float w = a.weights
                        ? a.weights[row]
                        : static_cast<float>(1.0 / static_cast<double>(a.rows));
    const int64_t zbase = row * a.ld, gbase = row * a.ldd;
    if (w == 0.0f) {
      const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (a.dlogits)
        for (int64_t u = tid; u < units; u += Threads) store(gbase, u, zero);
      if (tid == 0) {
        if (a.logp) a.logp[row] = 0.0f;
        if (a.saved) a.saved[row] = mta_policy_row{0.0, 0.0f, 0};
      }
      continue;
    }
    const int64_t action = a.actions[row];
    const bool inside = action >= 0 && action < vocab;
    const float za = inside ? load_elem<D>(a.logits, zbase + action)
                            : __builtin_nanf("");

    // the row's maximum, and its sum of 2^((z - max) log2 e)
    Raw8<D> z[Units ? Units : 1];
    float top = -kInf, sum = 0.0f;
    if constexpr (Units != 0) {
#pragma unroll
      for (int j = 0; j < Units; ++j)
        z[j] = load(zbase, tid + j * Threads);
#pragma unroll
      for (int j = 0; j < Units; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) top = fmaxf(top, z[j][k]);
    } else {
      // running maximum and sum; a lane that has seen only -inf has 0
      for (int64_t u = tid; u < units; u += Threads) {
        const Raw8<D> x = load(zbase, u);
        float m = top;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, x[k]);
        if (m != top)
          sum *= __builtin_amdgcn_exp2f((top - m) * kLog2E);
        top = m;
        const float ref = m == -kInf ? 0.0f : m;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sum += __builtin_amdgcn_exp2f((x[k] - ref) * kLog2E);
      }
    }
    float all = wave_max(top);
    if constexpr (!kOneWave) {
      if (tid % 64 == 0) sh.top[wave] = all;
      sync();
#pragma unroll
      for (int i = 0; i < kWaves; ++i) all = fmaxf(all, sh.top[i]);
    }
    if constexpr (Units != 0) {
#pragma unroll
      for (int j = 0; j < Units; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sum += __builtin_amdgcn_exp2f((z[j][k] - all) * kLog2E);
    } else {
      sum *= __builtin_amdgcn_exp2f((top - all) * kLog2E);
    }
    top = all;
    sum = wave_sum(sum);
    double total = sum;
    if constexpr (!kOneWave) {
      if (tid % 64 == 0) sh.sum[wave] = sum;
      sync();
      total = 0.0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) total += sh.sum[i];
    }

    float gain = 0.0f, chosen = 0.0f;  // S * coef; the action's gradient
    if (wave == 0) {
      const PolicyRow r = policy_row(a, row, w, za, top, total);
      gain = S * r.coef;
      chosen = static_cast<float>(-expm1(r.logp)) * gain;
      if (tid == 0) {
        if (a.logp) a.logp[row] = static_cast<float>(r.logp);
        if (a.saved) a.saved[row] = mta_policy_row{r.lse, r.coef, 1};
        sh.gain = gain;
        sh.chosen = chosen;
#pragma unroll
        for (int i = 0; i < kPolicySums; ++i) sums[i] += r.sums[i];
      }
    }
    if (a.dlogits) {
      if constexpr (!kOneWave) {
        sync();
        gain = sh.gain;
        chosen = sh.chosen;
      }
      gain = -gain / static_cast<float>(total);
      const auto put = [&](int64_t u, const Raw8<D> &x) {
        float g[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          g[k] = __builtin_amdgcn_exp2f((x[k] - top) * kLog2E) * gain;
        store(gbase, u, g);
      };
      if constexpr (Units != 0) {
#pragma unroll
        for (int j = 0; j < Units; ++j)
          if (tid + j * Threads < units) put(tid + j * Threads, z[j]);
      } else {
        for (int64_t u = tid; u < units; u += Threads) put(u, load(zbase, u));
      }
      // the action's own gradient, by the lane that wrote its run
      if (inside && tid == (action / 8) % Threads)
        store_elem<D>(a.dlogits, gbase + action, chosen);
    }
    // the shared values are rewritten by the next row
    sync();
  }
  if (tid == 0) {
    double *out = static_cast<double *>(a.workspace) + slot * kPolicySums;
#pragma unroll
    for (int i = 0; i < kPolicySums; ++i) out[i] = sums[i];
  }
}

// The partial sums joined in one fixed order.
__global__ __launch_bounds__(1024) void k_policy_stats(const double *part,
                                                       int slots,
                                                       float *stats) {
  __shared__ double sh[1024];
  const int tid = threadIdx.x;
  for (int i = 0; i < kPolicySums; ++i) {
    double s = 0.0;
    for (int k = tid; k < slots; k += 1024) s += part[k * kPolicySums + i];
    sh[tid] = s;
    __syncthreads();
    for (int o = 512; o; o >>= 1) {
      if (tid < o) sh[tid] += sh[tid + o];
      __syncthreads();
    }
    if (tid == 0) stats[i] = static_cast<float>(sh[0]);
    __syncthreads();
  }
}

// dlogits from what the forward saved.  A workgroup takes a stretch of one
// row, so that a few long rows fill the card too.
constexpr int kBackThreads = 256;
constexpr int kBackUnroll = 4;
constexpr int kBackUnits = kBackThreads * kBackUnroll;

template <int D>
__global__ __launch_bounds__(kBackThreads) void k_policy_backward(
    const mta_policy_args a, int64_t parts) {
  const float S = a.d_grad_scale ? *a.d_grad_scale : 1.0f;
  const int64_t n = a.rows * parts;
  for (int64_t b = blockIdx.x; b < n; b += gridDim.x) {
    const int64_t row = b / parts;
    const int64_t u0 = (b - row * parts) * kBackUnits + threadIdx.x;
    const int64_t zbase = row * a.ld, gbase = row * a.ldd;
    const mta_policy_row r = a.saved[row];
    const int64_t action = a.actions[row];
    const bool on = r.on != 0;
    const float gain = S * r.coef;
    const float hi = static_cast<float>(r.lse);
    const float lo = hi - hi == 0.0f
                         ? static_cast<float>(r.lse - double{hi}) * kLog2E
                         : 0.0f;
    Raw8<D> z[kBackUnroll];
    int n_in[kBackUnroll];
#pragma unroll
    for (int j = 0; j < kBackUnroll; ++j) {
      const int64_t u = u0 + j * kBackThreads;
      const int64_t left = a.vocab - u * 8;
      n_in[j] = static_cast<int>(left >= 8 ? 8 : left > 0 ? left : 0);
      if (!on) continue;
      if (n_in[j] == 8) z[j] = load8<D, true>(a.logits, zbase + u * 8);
      else z[j] = load8_part<D>(a.logits, zbase + u * 8, n_in[j], 0);
    }
#pragma unroll
    for (int j = 0; j < kBackUnroll; ++j) {
      const int64_t u = u0 + j * kBackThreads;
      float g[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float p =
            __builtin_amdgcn_exp2f(__builtin_fmaf(z[j][k] - hi, kLog2E, -lo));
        const float d = u * 8 + k == action ? 1.0f - p : -p;
        g[k] = on ? gain * d : 0.0f;
      }
      if (n_in[j] == 8) {
        store8<D, true>(a.dlogits, gbase + u * 8, g);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < n_in[j]) store_elem<D>(a.dlogits, gbase + u * 8 + k, g[k]);
      }
    }
  }
}

template <int D, int Threads, int Units>
hipError_t start(const mta_policy_args &a, hipStream_t stream) {
  const int64_t groups =
      (a.rows + kRows<Threads> - 1) / kRows<Threads>;
  const int grid = static_cast<int>(groups < kPolicyGrid ? groups : kPolicyGrid);
  if (grid > 0)
    k_policy<D, Threads, Units>
        <<<grid, Threads * kRows<Threads>, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_policy_stats<<<1, 1024, 0, stream>>>(
      static_cast<const double *>(a.workspace), grid * kRows<Threads>,
      a.stats);
  return hipGetLastError();
}

// The smallest number of runs a lane that holds the row.
template <int D, int Threads, int Units>
hipError_t start_units(const mta_policy_args &a, hipStream_t stream) {
  if constexpr (Units < 8) {
    if (a.vocab > int64_t{Threads} * 8 * Units)
      return start_units<D, Threads, Units + 1>(a, stream);
  }
  return start<D, Threads, Units>(a, stream);
}

}  // namespace

hipError_t launch_policy(const mta_policy_args &a, hipStream_t stream) {
  return with_type(a.type, [&](auto d) {
    constexpr int D = decltype(d)::value;
    // a wave, four or sixteen to a row: as few as hold it, since a smaller
    // group waits less at its joins
    if (a.vocab <= 64 * 64) return start_units<D, 64, 1>(a, stream);
    if (a.vocab <= 256 * 64) return start_units<D, 256, 3>(a, stream);
    if (a.vocab <= 1024 * 64) return start_units<D, 1024, 3>(a, stream);
    return start<D, 1024, 0>(a, stream);
  });
}

hipError_t launch_policy_backward(const mta_policy_args &a,
                                  hipStream_t stream) {
  const int64_t units = (a.vocab + 7) / 8;
  const int64_t parts = (units + kBackUnits - 1) / kBackUnits;
  const int64_t n = a.rows * parts;
  if (n == 0) return hipSuccess;
  const int grid = static_cast<int>(n < (1 << 22) ? n : 1 << 22);
  return with_type(a.type, [&](auto d) {
    k_policy_backward<decltype(d)::value>
        <<<grid, kBackThreads, 0, stream>>>(a, parts);
    return hipGetLastError();
  });
}

}  // namespace mta
