// policy_kernels.hip -- the clipped policy loss with a KL term from the
// logits, forward and backward, on gfx950.
//
// A row's log-softmax needs its maximum and its sum of exponentials before
// the first gradient can be written, so the plain way reads the logits at
// least twice.  Here a row stays in the registers of the workgroup that reads
// it (65536 logits are 32 registers a lane of 1024 in 16 bits), so one call
// reads every logit once and writes every gradient once: bound by HBM (8192
// rows of 50257 bfloat16 logits, a fifth of them masked, at 5.5 TB/s).  Longer
// rows are read twice, the second time mostly from the memory-side cache.
//
// Numerics: exponentials are 2^((z - max) log2 e) in float32, a lane sums at
// most 64 (a streamed row: vocab / 1024) of them in float32, lanes are joined
// in float32 within a wave and in float64 across waves.  The action's own
// exponential stays out of that sum: where it is 1 and the others are small,
// 1 - p is their sum, of which a float32 1 + sum keeps little or nothing.
// What follows for a row (its logp, ratio, clip, KL) is a handful of float64
// operations of one wave: exp(d) - d - 1 and 1 - p lose every digit of a
// float32 near 0.
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
  double logp;
  double sums[kPolicySums];
};

// e^x in float64 is 2^k (1 + p): x = k ln 2 + r with |r| <= ln(2) / 2, p the
// Taylor series of e^r - 1 to r^12 (the next term is below 2^-50 of it).  A row
// needs two of these and a logarithm from one wave that the others wait for;
// the library's, which round to the last bit, take twice the time and (their
// tables of constants kept over the loop of rows) three times the registers.
struct Exp {
  double p, k;
};

__device__ __forceinline__ Exp exp_parts(double x) {
  const double k = __builtin_rint(x * 1.4426950408889634);
  double r = __builtin_fma(-k, 0x1.62e42fefa39efp-1, x);
  r = __builtin_fma(-k, 0x1.abc9e3b39803fp-56, r);
  double p = 1.0 / 479001600.0;
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p * r, r, r);
  return Exp{p, k};
}

// e^x - 1, which has the digits of x near 0 and none of e^x far below it.
__device__ __forceinline__ double exp_less_1(double x) {
  const Exp e = exp_parts(x);
  const double s = __builtin_ldexp(1.0, static_cast<int>(e.k));
  double y = __builtin_fma(s, e.p, s - 1.0);
  if (x > 709.0) y = __builtin_inf();
  if (x < -100.0) y = -1.0;
  return y;
}

// e^x, which has them.
__device__ __forceinline__ double exp_full(double x) {
  const Exp e = exp_parts(x);
  double y = __builtin_ldexp(1.0 + e.p, static_cast<int>(e.k));
  if (x > 709.0) y = __builtin_inf();
  if (x < -745.0) y = 0.0;
  return y;
}

// ln(1 + s) in float64 for s >= 0: 1 + s = m 2^e with m in [1/sqrt 2, sqrt 2),
// ln m = 2 atanh t, t = (m - 1) / (m + 1), |t| < 0.172, its series to t^17.
// Where e is 0, m - 1 is s itself, with the digits that 1 + s rounds away.
__device__ __forceinline__ double ln_plus_1(double s) {
  double m = __builtin_amdgcn_frexp_mant(1.0 + s);
  int e = __builtin_amdgcn_frexp_exp(1.0 + s);
  if (m < 0.70710678118654752) {
    m += m;
    --e;
  }
  const double d = e == 0 ? s : m - 1.0;
  const double t = d / (2.0 + d), u = t * t;
  double p = 2.0 / 17.0;
  p = __builtin_fma(p, u, 2.0 / 15.0);
  p = __builtin_fma(p, u, 2.0 / 13.0);
  p = __builtin_fma(p, u, 2.0 / 11.0);
  p = __builtin_fma(p, u, 2.0 / 9.0);
  p = __builtin_fma(p, u, 2.0 / 7.0);
  p = __builtin_fma(p, u, 2.0 / 5.0);
  p = __builtin_fma(p, u, 2.0 / 3.0);
  p = __builtin_fma(p, u, 2.0);
  return __builtin_fma(static_cast<double>(e), 0x1.62e42fefa39efp-1, p * t);
}

// What the caller gives for a row.
struct RowInputs {
  float w, old_logp, advantage, ref_logp, scale;
  int64_t action;
};

// The row's scalars from its maximum, the sum of exp(z - max) over all entries
// but the action's, and the action's own.  Where the action is the maximum its
// own is exactly 1, so logp = -ln(1 + others) has every digit of `others`.
__device__ __forceinline__ PolicyRow policy_row(const mta_policy_args &a,
                                                const RowInputs &in, float za,
                                                float top, double others,
                                                float own) {
  PolicyRow r;
  const double logtotal = ln_plus_1(others + (double{own} - 1.0));
  r.logp = (double{za} - double{top}) - logtotal;
  const double adv = in.advantage, w = in.w;
  const double ratio = exp_full(r.logp - double{in.old_logp});
  const double lo = 1.0 - a.clip_low, hi = 1.0 + a.clip_high;
  // comparisons that keep a NaN ratio
  const double cut = ratio < lo ? lo : ratio > hi ? hi : ratio;
  const double plain = ratio * adv, clipped = cut * adv;
  const bool over = plain > clipped;
  double loss = over ? -clipped : -plain;
  double slope = over ? 0.0 : -plain;
  double kl = 0.0;
  if (a.ref_logp) {
    const double d = double{in.ref_logp} - r.logp;
    const double e = exp_less_1(d);
    kl = e > 1e300 ? e : e - d;  // (not infinity - infinity)
    if (a.kl_coef != 0.0) {  // (0 * infinity)
      loss += a.kl_coef * kl;
      slope -= a.kl_coef * e;
    }
  }
  r.coef = static_cast<float>(w * slope);
  r.sums[0] = w * loss;
  r.sums[1] = w * kl;
  r.sums[2] = over ? w : 0.0;
  return r;
}

// A value that every lane has, in scalar registers: the row needs the others.
__device__ __forceinline__ float uniform(float x) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}
__device__ __forceinline__ double uniform(double x) {
  const uint64_t u = __double_as_longlong(x);
  const uint64_t lo = static_cast<uint32_t>(
      __builtin_amdgcn_readfirstlane(static_cast<int>(u)));
  const uint64_t hi = static_cast<uint32_t>(
      __builtin_amdgcn_readfirstlane(static_cast<int>(u >> 32)));
  return __longlong_as_double(static_cast<long long>(hi << 32 | lo));
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

// A row as whole runs of eight logits from its first address that is a
// multiple of Align, and up to Align / size + 7 single logits at its two ends,
// one to each of the first lanes.  Rows of an odd length start anywhere: with
// runs from each row's first element the same batch of 50257 columns took 352
// us (271 now).
struct Cut {
  uint32_t head, units, vocab;
  // The end of the row that lane i holds; `vocab` or more: none.
  __device__ __forceinline__ uint32_t edge(uint32_t i) const {
    return i < head ? i : i + units * 8;
  }
};

template <int D, int Align>
__device__ __forceinline__ Cut cut_row(const void *row, uint32_t vocab) {
  const uint32_t off =
      static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) % Align;
  Cut c;
  c.head = (Align - off) % Align / sizeof(elem<D>);
  if (c.head > vocab) c.head = vocab;
  c.units = (vocab - c.head) / 8;
  c.vocab = vocab;
  return c;
}

// Rows of a workgroup, which is at least four waves.
template <int Threads>
constexpr int kRows = Threads < 256 ? 256 / Threads : 1;

// What the waves of a row tell each other.
template <int Threads>
struct RowShared {
  float top[Threads / 64];
  float sum[Threads / 64];
  float gain, chosen;
};

// A run with element k (the same in every lane) made -infinity.
template <int D>
__device__ __forceinline__ Raw8<D> without(Raw8<D> x, uint32_t k) {
  constexpr int kWords = Raw8<D>::kWords, kEach = 8 / kWords;
  const uint32_t inf = kEach == 1 ? kMinusInf<D> : kMinusInf<D> * 0x10001u;
  const uint32_t bits = kEach == 1 ? ~0u : 0xFFFFu << (k % kEach * 16);
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const uint32_t m = k / kEach == static_cast<uint32_t>(w) ? bits : 0u;
    x.w[w] = (x.w[w] & ~m) | (inf & m);
  }
  return x;
}

// Runs of a streamed row that a lane has in flight.
constexpr int kBatch = 4;

// Units > 0: that many runs of eight logits to a lane, kept in registers.
// Units == 0: the row is streamed, twice.  A row is one workgroup's (or one
// wave's) and there is no loop over rows: over such a loop the compiler keeps
// the scalars' float64 constants in 60 registers.  A 16-bit row has 64 registers
// a lane, for two groups of sixteen waves on a CU: of seven runs six words are
// spilled around the scalars, of eight 13 (by one wave a row three from six runs
// on, and 15), 15 of the 840 MB that 8192 x 50304 bfloat16 write.
template <int D, int Threads, int Units>
__global__ __launch_bounds__(Threads * kRows<Threads>,
                             (D == MTA_F32 ? 4 : 8)) void k_policy(
    const mta_policy_args a, int64_t row0) {
  constexpr int kWaves = Threads / 64;
  constexpr bool kOneWave = Threads == 64;
  __shared__ RowShared<Threads> sh;
  const uint32_t tid = threadIdx.x % Threads;
  const uint32_t wave =
      __builtin_amdgcn_readfirstlane(threadIdx.x / 64) % kWaves;
  const int64_t row =
      row0 + int64_t{blockIdx.x} * kRows<Threads> +
      (kOneWave ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : 0);
  if (row >= a.rows) return;
  const uint32_t vocab = static_cast<uint32_t>(a.vocab);
  const elem<D> *zrow = static_cast<const elem<D> *>(a.logits) + row * a.ld;
  elem<D> *grow =
      a.dlogits ? static_cast<elem<D> *>(a.dlogits) + row * a.ldd : nullptr;
  double *out = static_cast<double *>(a.workspace) + row * kPolicySums;
  const Cut cut = cut_row<D, kOneWave ? 16 : 128>(zrow, vocab);
  const uint32_t units = cut.units, edge = cut.edge(tid);
  const bool has_edge = edge < vocab;
  const auto at = [&](uint32_t u) { return cut.head + u * 8; };
  const auto load = [&](uint32_t u) {
    return load8<D, Units != 0>(zrow, at(u));
  };

  // all at once: each is a trip to memory
  RowInputs in;
  in.w = a.weights ? a.weights[row]
                   : static_cast<float>(1.0 / static_cast<double>(a.rows));
  in.action = a.actions[row];
  in.old_logp = a.old_logp[row];
  in.advantage = a.advantages[row];
  in.ref_logp = a.ref_logp ? a.ref_logp[row] : 0.0f;
  in.scale = a.d_grad_scale ? *a.d_grad_scale : 1.0f;
  if (in.w == 0.0f) {
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (grow) {
      for (uint32_t u = tid; u < units; u += Threads)
        store8<D, true>(grow, at(u), zero);
      if (has_edge) store_elem<D>(grow, edge, 0.0f);
    }
    if (tid == 0) {
      if (a.logp) a.logp[row] = 0.0f;
      if (a.saved) a.saved[row] = mta_policy_row{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kPolicySums; ++i) out[i] = 0.0;
    }
    return;
  }

  // the row's maximum, and its sum of 2^((z - max) log2 e)
  Raw8<D> z[Units ? Units : 1];
  float top = -kInf, sum = 0.0f;
  if constexpr (Units != 0) {
#pragma unroll
    for (int j = 0; j < Units; ++j) {
      const uint32_t u = tid + j * Threads;
      if (u < units) z[j] = load(u);
      else z[j] = fill8<D>(kMinusInf<D>);
    }
  }
  const int64_t action = in.action;
  const bool inside = action >= 0 && action < a.vocab;
  float za = inside ? load_elem<D>(zrow, action) : __builtin_nanf("");
  // the action's place: element `chosen_k` of run `chosen_u` (no run: none of
  // them), or an end; the sum is over the others
  const uint32_t c = static_cast<uint32_t>(action) - cut.head;
  const uint32_t chosen_u = inside && c < units * 8 ? c / 8 : ~0u;
  const uint32_t chosen_k = c % 8;
  const bool chosen_edge =
      inside && has_edge && edge == static_cast<uint32_t>(action);
  float ze = has_edge ? load_elem<D>(zrow, edge) : -kInf;
  if constexpr (Units != 0) {
#pragma unroll
    for (int j = 0; j < Units; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, z[j][k]);
    // (the maximum before the change: the compiler would keep two rows, and
    // the loss alone of 7934 x 16384 bfloat16 take 73 us, not 58)
#pragma unroll
    for (int j = 0; j < Units; ++j)
#pragma unroll
      for (int k = 0; k < Raw8<D>::kWords; ++k)
        __asm__("" : "+v"(z[j].w[k]) : "v"(top));
#pragma unroll
    for (int j = 0; j < Units; ++j)
      if (tid + j * Threads == chosen_u) z[j] = without<D>(z[j], chosen_k);
  } else {
    // running maximum and sum; a lane that has seen only -inf has 0
    for (uint32_t u = tid; u < units; u += Threads * kBatch) {
      Raw8<D> x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (u + j * Threads < units) x[j] = load(u + j * Threads);
        else x[j] = fill8<D>(kMinusInf<D>);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (u + j * Threads == chosen_u) x[j] = without<D>(x[j], chosen_k);
      float m = top;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, x[j][k]);
      if (m != top) sum *= __builtin_amdgcn_exp2f((top - m) * kLog2E);
      top = m;
      const float ref = m == -kInf ? 0.0f : m;
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          sum += __builtin_amdgcn_exp2f((x[j][k] - ref) * kLog2E);
    }
  }
  const float seen = top;  // what `sum` is relative to (streamed)
  top = fmaxf(top, ze);
  if constexpr (Units == 0) top = fmaxf(top, za);
  if (chosen_edge) ze = -kInf;
  // the compiler would keep a 16-bit row widened from here on: pinned, its
  // registers stay half as many
  const auto pin = [&] {
    if constexpr (Units != 0 && D != MTA_F32) {
#pragma unroll
      for (int j = 0; j < Units; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) __asm__("" : "+v"(z[j].w[k]));
    }
  };
  pin();
  float all = wave_max(top);
  if constexpr (!kOneWave) {
    if (tid % 64 == 0) sh.top[wave] = all;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) all = fmaxf(all, sh.top[i]);
  }
  all = uniform(all);
  za = uniform(za);
  if constexpr (Units != 0) {
#pragma unroll
    for (int j = 0; j < Units; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        sum += __builtin_amdgcn_exp2f((z[j][k] - all) * kLog2E);
  } else {
    sum *= __builtin_amdgcn_exp2f((seen - all) * kLog2E);
  }
  top = all;
  sum += __builtin_amdgcn_exp2f((ze - all) * kLog2E);
  sum = wave_sum(sum);
  double others = sum;
  if constexpr (!kOneWave) {
    if (tid % 64 == 0) sh.sum[wave] = sum;
    __syncthreads();
    others = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) others += sh.sum[i];
  }
  others = uniform(others);
  const float own = uniform(__builtin_amdgcn_exp2f((za - all) * kLog2E));
  const float total = uniform(static_cast<float>(others + double{own}));

  float gain = 0.0f, chosen = 0.0f;  // S * coef; the action's gradient
  if (wave == 0) {
    const PolicyRow r = policy_row(a, in, za, top, others, own);
    gain = r.coef * in.scale;
    const float rest =  // 1 - p
        static_cast<float>(others) * __builtin_amdgcn_rcpf(total);
    chosen = rest * gain;
    if (tid == 0) {
      if (a.logp) a.logp[row] = static_cast<float>(r.logp);
      if (a.saved) a.saved[row] = mta_policy_row{top, total, r.coef, rest};
      if constexpr (!kOneWave) {
        sh.gain = gain;
        sh.chosen = chosen;
      }
#pragma unroll
      for (int i = 0; i < kPolicySums; ++i) out[i] = r.sums[i];
    }
  }
  if (!grow) return;
  if constexpr (!kOneWave) {
    __syncthreads();
    gain = uniform(sh.gain);
    chosen = uniform(sh.chosen);
  }
  gain = uniform(-gain / total);
  // the exponentials are formed again: the compiler would keep those of the
  // sum, twice the row's registers
  __asm__("" : "+s"(top));
  pin();
  const auto grad = [&](float x) {
    return __builtin_amdgcn_exp2f((x - top) * kLog2E) * gain;
  };
  const auto put = [&](uint32_t u, const Raw8<D> &x) {
    float g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = grad(x[k]);
    store8<D, true>(grow, at(u), g);
  };
  if constexpr (Units != 0) {
#pragma unroll
    for (int j = 0; j < Units; ++j)
      if (tid + j * Threads < units) put(tid + j * Threads, z[j]);
  } else {
    for (uint32_t u = tid; u < units; u += Threads * kBatch) {
      Raw8<D> x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (u + j * Threads < units) x[j] = load(u + j * Threads);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (u + j * Threads < units) put(u + j * Threads, x[j]);
    }
  }
  if (has_edge) store_elem<D>(grow, edge, grad(ze));
  // the action's own gradient, by the lane that wrote its place
  if (chosen_edge || (chosen_u != ~0u && tid == chosen_u % Threads))
    store_elem<D>(grow, action, chosen);
}

// The rows' sums joined in one fixed order: a workgroup takes a stretch of
// `per` rows; a second launch (of one, with `stats`) joins the stretches.
__global__ __launch_bounds__(1024) void k_policy_stats(const double *part,
                                                       int64_t n, int64_t per,
                                                       double *joined,
                                                       float *stats) {
  __shared__ double sh[kPolicySums][16];
  const int tid = threadIdx.x;
  const int64_t lo = blockIdx.x * per;
  const int64_t hi = n < lo + per ? n : lo + per;
  double s[kPolicySums] = {0.0, 0.0, 0.0};
  for (int64_t k = lo + tid; k < hi; k += 1024)
#pragma unroll
    for (int i = 0; i < kPolicySums; ++i) s[i] += part[k * kPolicySums + i];
#pragma unroll
  for (int i = 0; i < kPolicySums; ++i) {
#pragma unroll
    for (int o = 32; o; o >>= 1) s[i] += __shfl_xor(s[i], o);
    if (tid % 64 == 0) sh[i][tid / 64] = s[i];
  }
  __syncthreads();
  if (tid < kPolicySums) {
    double v = 0.0;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += sh[tid][k];
    if (stats) stats[tid] = static_cast<float>(v);
    else joined[blockIdx.x * kPolicySums + tid] = v;
  }
}

// dlogits from what the forward saved.  A workgroup takes a stretch of one
// row, so that a few long rows fill the card too.
constexpr int kBackThreads = 256;
constexpr int kBackUnroll = 4;
constexpr int kBackUnits = kBackThreads * kBackUnroll;

template <int D>
__global__ __launch_bounds__(kBackThreads) void k_policy_backward(
    const mta_policy_args a, int64_t row0, uint32_t parts) {
  const uint32_t tid = threadIdx.x;
  const uint32_t part = blockIdx.x % parts;
  const int64_t row = row0 + blockIdx.x / parts;
  const uint32_t vocab = static_cast<uint32_t>(a.vocab);
  const elem<D> *zrow = static_cast<const elem<D> *>(a.logits) + row * a.ld;
  elem<D> *grow = static_cast<elem<D> *>(a.dlogits) + row * a.ldd;
  const Cut cut = cut_row<D, 128>(zrow, vocab);
  const uint32_t u0 = part * kBackUnits + tid;
  const uint32_t edge = part == 0 ? cut.edge(tid) : vocab;
  const mta_policy_row r = a.saved[row];
  if (r.total == 0.0f) {  // a row of weight 0: others have 1 or more, or NaN
    const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kBackUnroll; ++j) {
      const uint32_t u = u0 + j * kBackThreads;
      if (u < cut.units) store8<D, true>(grow, cut.head + u * 8, zero);
    }
    if (edge < vocab) store_elem<D>(grow, edge, 0.0f);
    return;
  }
  Raw8<D> z[kBackUnroll];
#pragma unroll
  for (int j = 0; j < kBackUnroll; ++j) {
    const uint32_t u = u0 + j * kBackThreads;
    if (u < cut.units) z[j] = load8<D, true>(zrow, cut.head + u * 8);
  }
  const float ze = edge < vocab ? load_elem<D>(zrow, edge) : 0.0f;
  const int64_t action = a.actions[row];
  const float gain = r.coef * (a.d_grad_scale ? *a.d_grad_scale : 1.0f);
  // as in the forward, to the bit
  const float each = -gain / r.total, chosen = r.rest * gain;
  const auto grad = [&](float x, uint32_t at) {
    return at == action ? chosen
                        : __builtin_amdgcn_exp2f((x - r.top) * kLog2E) * each;
  };
#pragma unroll
  for (int j = 0; j < kBackUnroll; ++j) {
    const uint32_t u = u0 + j * kBackThreads;
    if (u >= cut.units) continue;
    const uint32_t at = cut.head + u * 8;
    float g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = grad(z[j][k], at + k);
    store8<D, true>(grow, at, g);
  }
  if (edge < vocab) store_elem<D>(grow, edge, grad(ze, edge));
}

template <int D, int Threads, int Units>
hipError_t start(const mta_policy_args &a, hipStream_t stream) {
  constexpr int64_t kMost = int64_t{1} << 21;  // below 2^32 threads a launch
  const int64_t groups = (a.rows + kRows<Threads> - 1) / kRows<Threads>;
  for (int64_t g = 0; g < groups; g += kMost) {
    const int64_t n = groups - g < kMost ? groups - g : kMost;
    k_policy<D, Threads, Units>
        <<<static_cast<int>(n), Threads * kRows<Threads>, 0, stream>>>(
            a, g * kRows<Threads>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const double *part = static_cast<const double *>(a.workspace);
  int64_t n = a.rows;
  if (n > kPolicyJoin) {
    // stretches of at least kPolicyJoin rows, at most kPolicyJoin of them
    int64_t per = (n + kPolicyJoin - 1) / kPolicyJoin;
    if (per < kPolicyJoin) per = kPolicyJoin;
    const int64_t m = (n + per - 1) / per;
    double *joined = static_cast<double *>(a.workspace) + n * kPolicySums;
    k_policy_stats<<<static_cast<int>(m), 1024, 0, stream>>>(part, n, per,
                                                             joined, nullptr);
    part = joined;
    n = m;
  }
  k_policy_stats<<<1, 1024, 0, stream>>>(part, n, n, nullptr, a.stats);
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
    // group waits less at its joins.  A float32 row of sixteen waves leaves
    // room for one group on a CU, whose loads, sums and stores then take
    // turns: streamed, two groups overlap theirs and the second reading comes
    // from the memory-side cache (2047 rows of 50257 with their gradient 205
    // us, 212 when kept; the loss alone 67 us, 98 when kept).
    if (a.vocab <= 64 * 64) return start_units<D, 64, 1>(a, stream);
    if (a.vocab <= 256 * 64) return start_units<D, 256, 3>(a, stream);
    if constexpr (D != MTA_F32)
      if (a.vocab <= 1024 * 64) return start_units<D, 1024, 3>(a, stream);
    return start<D, 1024, 0>(a, stream);
  });
}

hipError_t launch_policy_backward(const mta_policy_args &a,
                                  hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  // (the row's ends go with its first part)
  const int64_t units = a.vocab / 8;
  const int64_t parts = units > 0 ? (units + kBackUnits - 1) / kBackUnits : 1;
  const int64_t most = (int64_t{1} << 22) / parts;  // rows of a launch
  return with_type(a.type, [&](auto d) {
    for (int64_t row = 0; row < a.rows; row += most) {
      const int64_t n = a.rows - row < most ? a.rows - row : most;
      k_policy_backward<decltype(d)::value>
          <<<static_cast<int>(n * parts), kBackThreads, 0, stream>>>(
              a, row, static_cast<uint32_t>(parts));
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
}

}  // namespace mta
