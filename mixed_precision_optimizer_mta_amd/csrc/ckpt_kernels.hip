// ckpt_kernels.hip -- 8-bit activation checkpoints on gfx950: pack (with an
// activation function's value), unpack, and the activation's backward.
//
// One kernel walks all three.  A lane takes 16 bytes of a tensor, eight
// columns in 16 bits or four in 32; the four or eight neighbouring lanes of a
// block of 32 find its largest magnitude with two or three permutes.  The scale
// is a power of two, so its exponent comes from the bits of that magnitude and
// both the scaling and the kept value are exact; the only rounding is the
// hardware's nearest-even conversion to e4m3.
//
// Bound by HBM: 3.03 bytes move per element of a 16-bit pack or unpack, 5.03
// with an activation or its backward, against 10 to 40 vector instructions
// (but for gelu's erf in 16 bits: 8192 x 6400 takes 66 us where silu takes 47).
#include "ops_device.h"

namespace mta {
namespace {

constexpr float kInf = __builtin_inff();
constexpr float kLog2E = 1.44269504088896341f;

// e^x through the hardware's 2^x: relative error 2^-22 + |x| 2^-24, far inside
// a 16-bit result's rounding.
__device__ __forceinline__ float fast_exp(float x) {
  return __builtin_amdgcn_exp2f(x * kLog2E);
}

// e^x for x <= 0 to two steps of 2^-24, for float32 results: the argument's
// fraction f = x log2 e - n, |f| <= 1/2, from log2 e in two parts, and 2^f 2^n
// (a subnormal one too).
__device__ __forceinline__ float fine_exp(float x) {
  x = x < -110.0f ? -110.0f : x;  // (2^-158 is 0; a NaN stays)
  const float n = __builtin_rintf(x * kLog2E);
  float f = __builtin_fmaf(x, kLog2E, -n);
  f = __builtin_fmaf(x, 1.9259630e-8f, f);
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), static_cast<int>(n));
}

template <int D>
__device__ __forceinline__ float exp_of_negative(float x) {
  return D == MTA_F32 ? fine_exp(x) : fast_exp(x);
}

// s = 1 / (1 + e^-u) and t = s (1 - s).
struct Sigmoid {
  float s, t;
};

template <int D>
__device__ __forceinline__ Sigmoid sigmoid(float u) {
  if constexpr (D == MTA_F32) {
    // from e = e^-|u|, which neither overflows nor cancels: 1 / (1 + e) is the
    // hardware's with one Newton step.  8192 x 6400 silu and its backward take
    // 80 and 82 us, as with the 16-bit form's 2^x and reciprocal (79 and 81);
    // the library's exponential and quotients take 85 and 89.
    const float e = fine_exp(-__builtin_fabsf(u)), d = 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);
    const float small = e * r;
    return Sigmoid{u < 0.0f ? small : r, small * r};
  } else {
    const float s = __builtin_amdgcn_rcpf(1.0f + fast_exp(-u));
    return Sigmoid{s, s * (1.0f - s)};
  }
}

// sqrt(2/pi) (x + 0.044715 x^3), doubled: gelu_tanh(x) = x sigmoid(this).
__device__ __forceinline__ float tanh_arg2(float x) {
  const float c = 1.5957691216057308f;
  return x * __builtin_fmaf(c * 0.044715f * x, x, c);
}

// x * 0 where sigmoid underflows at x = -inf would be NaN; the limit is 0.
template <int D, int Act>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (Act == MTA_ACT_RELU) {
    return x > 0.0f ? x : (x != x ? x : 0.0f);
  } else if constexpr (Act == MTA_ACT_GELU) {
    const float h = 0.5f * x;
    const float r = __builtin_fmaf(h, erff(x * 0.70710678118654752f), h);
    return x == -kInf ? 0.0f : r;
  } else {
    const float r =
        x * sigmoid<D>(Act == MTA_ACT_SILU ? x : tanh_arg2(x)).s;
    return x == -kInf ? 0.0f : r;
  }
}

// The slope at a kept value, which is finite or NaN.
template <int D, int Act>
__device__ __forceinline__ float act_slope(float x) {
  if constexpr (Act == MTA_ACT_RELU) {
    return x > 0.0f ? 1.0f : (x != x ? x : 0.0f);
  } else if constexpr (Act == MTA_ACT_SILU) {
    const Sigmoid y = sigmoid<D>(x);
    // past |x| = 2^8, s (1 - s) is 0 and x s (1 - s) must not become inf * 0
    return y.t == 0.0f ? y.s : __builtin_fmaf(x, y.t, y.s);
  } else if constexpr (Act == MTA_ACT_GELU) {
    const float phi =
        __builtin_fmaf(0.5f, erff(x * 0.70710678118654752f), 0.5f);
    const float d = exp_of_negative<D>(-0.5f * x * x) * 0.3989422804014327f;
    return d == 0.0f ? phi : __builtin_fmaf(x, d, phi);
  } else {
    const Sigmoid y = sigmoid<D>(tanh_arg2(x));
    const float c = 1.5957691216057308f;
    const float du = __builtin_fmaf(3.0f * c * 0.044715f * x, x, c);
    return y.t == 0.0f ? y.s : __builtin_fmaf(x * y.t, du, y.s);
  }
}

// The largest of the four or eight lanes of a block.
template <int Lanes>
__device__ __forceinline__ float block_max(float x) {
  const int a = __builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xF, 0xF,
                                         false);  // lanes 1 0 3 2
  x = fmaxf(x, __int_as_float(a));
  const int b = __builtin_amdgcn_mov_dpp(__float_as_int(x), 0x4E, 0xF, 0xF,
                                         false);  // lanes 2 3 0 1
  x = fmaxf(x, __int_as_float(b));
  if constexpr (Lanes == 8) {
    const int c = __builtin_amdgcn_mov_dpp(__float_as_int(x), 0x141, 0xF, 0xF,
                                           false);  // lanes 7 6 5 4 3 2 1 0
    x = fmaxf(x, __int_as_float(c));
  }
  return x;
}

// The largest magnitude kept of a type: four significant bits below its
// overflow.
template <int D>
constexpr float kMost = D == MTA_F16 ? 61440.0f : 0x1.ep+127f;

// Biased exponent of the smallest 2^k, k >= -117, with top <= 448 * 2^k:
// 448 is 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_byte(float top) {
  const uint32_t u = __float_as_uint(top);
  const int b = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u);
  return static_cast<uint32_t>(max(b, 10));
}

// Where a lane's run of columns lies.
struct Place {
  int64_t row;
  uint32_t col;   // first column
  int valid;      // columns of it inside the tensor; -1: no run
};

// A run's codes: four to a word.
template <int N>
struct Codes {
  typedef uint32_t type __attribute__((ext_vector_type(N / 4)));
};

template <int D, int Mode, int Act>
__global__ __launch_bounds__(kCkptThreads) void k_ckpt(const CkptList list) {
  // the tensor of this workgroup
  uint32_t t = 0;
  while (t + 1 < list.count && blockIdx.x >= list.first[t + 1]) ++t;
  const CkptItem &it = list.item[t];
  constexpr int kN = ckpt_unit(D), kLanes = MTA_CKPT_BLOCK / kN;
  typedef typename Codes<kN>::type codes;
  const uint32_t lane = threadIdx.x;
  const uint64_t stride =
      uint64_t{list.first[t + 1] - list.first[t]} * it.chunk;

  for (uint64_t base = uint64_t{blockIdx.x - list.first[t]} * it.chunk;
       base < it.units; base += stride) {
    const bool flat = it.row_units == 0;
    const uint64_t row0 = flat ? 0 : base / it.row_units;
    const uint32_t off0 =
        flat ? 0 : static_cast<uint32_t>(base - row0 * it.row_units);

    Place at[kCkptUnroll];
    Raw<D, kN> in[kCkptUnroll];
    codes code[kCkptUnroll];
    uint32_t sb[kCkptUnroll];
    // every load of the chunk before any use
#pragma unroll
    for (int j = 0; j < kCkptUnroll; ++j) {
      const uint64_t u = base + j * kCkptThreads + lane;
      // (whole blocks at a time; as one comparison with the smaller end a
      // large bfloat16 list packs in 38.5 us instead of 33.7)
      if (u >= it.units || j * kCkptThreads >= it.chunk) {
        at[j].valid = -1;
        continue;
      }
      int64_t ex;
      if (flat) {
        at[j] = Place{0, 0, kN};
        ex = static_cast<int64_t>(u) * kN;
      } else {
        const uint32_t o = off0 + j * kCkptThreads + lane;
        const uint32_t dr = o / it.row_units;
        const uint32_t col = (o - dr * it.row_units) * kN;
        const int left = static_cast<int>(it.cols) - static_cast<int>(col);
        at[j].row = static_cast<int64_t>(row0 + dr);
        at[j].col = col;
        at[j].valid = max(0, min(kN, left));
        ex = at[j].row * it.ldx + col;
      }
      if constexpr (Mode != kCkptUnpack) {
        if (at[j].valid == kN) in[j] = load<D, kN, true>(it.x, ex);
        else in[j] = load_part<D, kN>(it.x, ex, at[j].valid, 0);
      }
      if constexpr (Mode != kCkptPack) {
        code[j] = __builtin_nontemporal_load(
            (const MTA_GLOBAL codes *)(it.q) + u);
        sb[j] = ((const MTA_GLOBAL uint8_t *)it.scale)[u / kLanes];
      }
    }
#pragma unroll
    for (int j = 0; j < kCkptUnroll; ++j) {
      if (at[j].valid < 0) continue;
      const uint64_t u = base + j * kCkptThreads + lane;
      const int64_t ey =
          flat ? static_cast<int64_t>(u) * kN
               : at[j].row * it.ldy + at[j].col;
      float out[kN];
      if constexpr (Mode == kCkptPack) {
        float v[kN], top = 0.0f;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const float x = in[j][k];
          const float a = __builtin_fabsf(x);
          const bool fine = a < kInf;
          top = fmaxf(top, fine ? a : 0.0f);
          v[k] = fine ? __builtin_amdgcn_fmed3f(x, -kMost<D>, kMost<D>)
                      : __builtin_nanf("");
          if constexpr (Act != MTA_ACT_NONE) out[k] = act_value<D, Act>(x);
        }
        const uint32_t b = scale_byte(block_max<kLanes>(fminf(top, kMost<D>)));
        const float inv = __uint_as_float((254u - b) << 23);
        codes w;
#pragma unroll
        for (int h = 0; h < kN / 4; ++h) {
          int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv,
                                                  v[4 * h + 1] * inv, 0,
                                                  false);
          c = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv,
                                              v[4 * h + 3] * inv, c, true);
          w[h] = static_cast<uint32_t>(c);
        }
        ((MTA_GLOBAL codes *)it.q)[u] = w;
        if (lane % kLanes == 0)
          ((MTA_GLOBAL uint8_t *)it.scale)[u / kLanes] =
              static_cast<uint8_t>(b);
      } else {
        const float s = __uint_as_float(sb[j] << 23);
#pragma unroll
        for (int h = 0; h < kN / 4; ++h) {
          const int c = static_cast<int>(code[j][h]);
          const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(c, false);
          const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
          out[4 * h] = lo[0] * s;
          out[4 * h + 1] = lo[1] * s;
          out[4 * h + 2] = hi[0] * s;
          out[4 * h + 3] = hi[1] * s;
        }
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          if constexpr (Mode == kCkptBackward)
            out[k] = in[j][k] * act_slope<D, Act>(out[k]);
          else if constexpr (D == MTA_F16)  // a NaN passes the comparisons
            out[k] = out[k] > 65504.0f    ? 65504.0f
                     : out[k] < -65504.0f ? -65504.0f
                                          : out[k];
        }
      }
      if constexpr (Mode != kCkptPack || Act != MTA_ACT_NONE) {
        if (at[j].valid == kN) {
          store<D, kN, true>(it.y, ey, out);
        } else {
#pragma unroll
          for (int k = 0; k < kN; ++k)
            if (k < at[j].valid) store_elem<D>(it.y, ey + k, out[k]);
        }
      }
    }
  }
}

template <int D, int Mode, int Act>
hipError_t start(const CkptList &list, hipStream_t stream) {
  k_ckpt<D, Mode, Act>
      <<<list.first[list.count], kCkptThreads, 0, stream>>>(list);
  return hipGetLastError();
}

template <int D, int Mode>
hipError_t start_act(int act, const CkptList &list, hipStream_t stream) {
  switch (act) {
    case MTA_ACT_RELU: return start<D, Mode, MTA_ACT_RELU>(list, stream);
    case MTA_ACT_SILU: return start<D, Mode, MTA_ACT_SILU>(list, stream);
    case MTA_ACT_GELU: return start<D, Mode, MTA_ACT_GELU>(list, stream);
    default: return start<D, Mode, MTA_ACT_GELU_TANH>(list, stream);
  }
}

}  // namespace

hipError_t launch_ckpt(int mode, int type, int act, const CkptList &list,
                       hipStream_t stream) {
  return with_type(type, [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (mode == kCkptUnpack)
      return start<D, kCkptUnpack, MTA_ACT_NONE>(list, stream);
    if (mode == kCkptBackward)
      return start_act<D, kCkptBackward>(act, list, stream);
    if (act == MTA_ACT_NONE)
      return start<D, kCkptPack, MTA_ACT_NONE>(list, stream);
    return start_act<D, kCkptPack>(act, list, stream);
  });
}

}  // namespace mta
