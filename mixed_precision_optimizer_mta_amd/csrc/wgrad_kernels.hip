// wgrad_kernels.hip -- weight and bias gradient of a linear layer from the
// 8-bit checkpoint of its input, on the matrix cores of gfx950.
//
//   dW[o][i] = sum_t dY[t][o] * kept[t][i],   db[o] = sum_t dY[t][o]
//
// A kept value is an e4m3 code times a power of two: exact in bfloat16, so
// the product runs on the bfloat16 matrix instructions without any rounding
// but that of its float32 sums, and the checkpoint is read at one byte a
// value.  A float16 (float32) dY is split into two (three) bfloat16 values
// whose sum it is, one matrix product each.
//
// Both operands lie with the contracted index t as their rows, while a matrix
// instruction wants eight consecutive t of one column in a lane.  They are
// staged in LDS as they lie, and read back with the transposing LDS load
// (16 lanes read four rows of 16 columns and get four rows of one column
// each).
#include "ops_device.h"

namespace mta {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// 64 bytes behind each LDS row: the four rows of a transposing load, and the
// two column halves that are read together, then lie in distinct banks.
constexpr int kPad = 32;

template <int D>
constexpr int kTerms = D == MTA_BF16 ? 1 : D == MTA_F16 ? 2 : 3;

// The bfloat16 values that a dy is the sum of, largest first.  Each takes the
// next eight significant bits of what is left by cutting the lower ones off,
// so a difference is exact and no value grows past its source.  An infinity
// or NaN is carried by the first alone.
template <int D>
__device__ __forceinline__ void split8(const Raw8<D> &x,
                                       uint32_t (&w)[kTerms<D>][4]) {
  if constexpr (D == MTA_BF16) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[0][k] = x.w[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t u[2][kTerms<D>];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = x[2 * k + h];
        const bool fine = __builtin_fabsf(v) < __builtin_inff();
#pragma unroll
        for (int t = 0; t < kTerms<D>; ++t) {
          uint32_t b = __float_as_uint(v) & 0xFFFF0000u;
          // a NaN of low bits only would be cut to an infinity
          if (t == 0 && v != v) b = 0x7FC00000u;
          u[h][t] = b;
          v = fine ? v - __uint_as_float(b) : 0.0f;
        }
      }
#pragma unroll
      for (int t = 0; t < kTerms<D>; ++t)
        w[t][k] = (u[0][t] >> 16) | u[1][t];
    }
  }
}

// Sixteen codes of one block to bfloat16.
__device__ __forceinline__ void kept16(const u32x4 &code, uint32_t sb,
                                       u32x4 (&out)[2]) {
  const float s = __uint_as_float(sb << 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    out[k / 2][2 * (k % 2)] = __builtin_bit_cast(
        uint32_t,
        __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code[k], s, false));
    out[k / 2][2 * (k % 2) + 1] = __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code[k], s, true));
  }
}

__device__ __forceinline__ bf16x8 transposed(const uint16_t *lds, int stride) {
  typedef __attribute__((address_space(3))) s16x4 lds4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)lds);
  const s16x4 b =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(lds + 4 * stride));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return __builtin_bit_cast(bf16x8, v);
}

// A sum into dw or db, in the gradient's type.
__device__ __forceinline__ void put(void *p, int64_t i, float x, int gtype,
                                    int accumulate) {
  if (gtype == MTA_F32) {
    if (accumulate) x += load_elem<MTA_F32>(p, i);
    store_elem<MTA_F32>(p, i, x);
  } else if (gtype == MTA_BF16) {
    if (accumulate) x += load_elem<MTA_BF16>(p, i);
    store_elem<MTA_BF16>(p, i, x);
  } else {
    if (accumulate) x += load_elem<MTA_F16>(p, i);
    store_elem<MTA_F16>(p, i, x);
  }
}

// A workgroup's tile of BO x BI outputs over its part of the tokens; WO x WI
// waves of 32 x 32 matrix tiles; Step tokens at a time through two LDS
// buffers.
template <int D, int BO, int BI, int WO, int WI, int Step>
struct Wgrad {
  static constexpr int kThreads = 64 * WO * WI;
  static constexpr int kT = kTerms<D>;
  static constexpr int kStrideO = BO + kPad, kStrideI = BI + kPad;
  static constexpr int kUnitsO = Step * (BO / 8);   // 8 values each
  static constexpr int kUnitsI = Step * (BI / 16);  // 16 codes each
  static constexpr int kPerO = kUnitsO / kThreads, kPerI = kUnitsI / kThreads;
  static constexpr int kMo = BO / WO / 32, kMi = BI / WI / 32;
  static_assert(kUnitsO % kThreads == 0 && kUnitsI % kThreads == 0, "");
  static_assert(kThreads % (BO / 8) == 0 && kThreads % (BI / 16) == 0, "");
  struct Buffer {
    uint16_t o[kT][Step * kStrideO];
    uint16_t i[Step * kStrideI];
  };
};

template <int D, int BO, int BI, int WO, int WI, int Step>
__global__ __launch_bounds__(64 * WO *WI) void k_wgrad(const WgradArgs a,
                                                       int tiles_i, int tiles,
                                                       int64_t per_split) {
  using K = Wgrad<D, BO, BI, WO, WI, Step>;
  __shared__ __attribute__((aligned(16))) typename K::Buffer buf[2];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int split = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int64_t o0 = int64_t{tile / tiles_i} * BO;
  const int64_t i0 = int64_t{tile % tiles_i} * BI;
  const int64_t t0 = split * per_split;
  const int64_t t1 = min(a.tokens, t0 + per_split);
  const int steps = static_cast<int>((t1 - t0 + Step - 1) / Step);
  const bool bias = a.db && i0 == 0;

  // what this lane stages: fixed columns, kPerO (kPerI) of the step's rows
  const int co = tid % (BO / 8), ro = tid / (BO / 8);
  const int ci = tid % (BI / 16), ri = tid / (BI / 16);
  constexpr int kRowsO = K::kThreads / (BO / 8);
  constexpr int kRowsI = K::kThreads / (BI / 16);
  const int64_t left_o = a.fout - (o0 + co * 8);
  const int n_o = static_cast<int>(left_o >= 8 ? 8 : left_o > 0 ? left_o : 0);
  const bool in_i = i0 + ci * 16 < a.ldq;

  Raw8<D> y[K::kPerO];
  u32x4 code[K::kPerI];
  uint32_t sb[K::kPerI];
  float db[8] = {0, 0, 0, 0, 0, 0, 0, 0};

  const auto fetch = [&](int step) {
    const int64_t t = t0 + int64_t{step} * Step;
#pragma unroll
    for (int j = 0; j < K::kPerO; ++j) {
      const int64_t r = t + ro + j * kRowsO;
      const int64_t at = r * a.lddy + o0 + co * 8;
      if (r < t1 && n_o == 8) y[j] = load8<D, false>(a.dy, at);
      else y[j] = load8_part<D>(a.dy, at, r < t1 ? n_o : 0, 0);
    }
#pragma unroll
    for (int j = 0; j < K::kPerI; ++j) {
      const int64_t r = t + ri + j * kRowsI;
      code[j] = u32x4{0, 0, 0, 0};
      sb[j] = 0;
      if (r < t1 && in_i) {
        const int64_t at = r * a.ldq + i0 + ci * 16;
        code[j] = *(const MTA_GLOBAL u32x4 *)(a.q + at);
        sb[j] = ((const MTA_GLOBAL uint8_t *)a.scale)[at / MTA_CKPT_BLOCK];
      }
    }
  };
  const auto stage = [&](typename K::Buffer &b) {
#pragma unroll
    for (int j = 0; j < K::kPerO; ++j) {
      uint32_t w[K::kT][4];
      split8<D>(y[j], w);
#pragma unroll
      for (int t = 0; t < K::kT; ++t)
        *(u32x4 *)&b.o[t][(ro + j * kRowsO) * K::kStrideO + co * 8] =
            u32x4{w[t][0], w[t][1], w[t][2], w[t][3]};
      if (bias) {
#pragma unroll
        for (int k = 0; k < 8; ++k) db[k] += y[j][k];
      }
    }
#pragma unroll
    for (int j = 0; j < K::kPerI; ++j) {
      u32x4 v[2];
      kept16(code[j], sb[j], v);
      u32x4 *at = (u32x4 *)&b.i[(ri + j * kRowsI) * K::kStrideI + ci * 16];
      at[0] = v[0];
      at[1] = v[1];
    }
  };

  f32x16 acc[K::kMo][K::kMi];
#pragma unroll
  for (int x = 0; x < K::kMo; ++x)
#pragma unroll
    for (int v = 0; v < K::kMi; ++v)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[x][v][r] = 0.0f;

  const int wo = (wave / WI) * (BO / WO), wi = (wave % WI) * (BI / WI);
  // this lane's place in a transposing load of 32 columns x 16 tokens
  const int tr = (lane / 32) * 8 + (lane % 16) / 4;
  const int tc = ((lane / 16) % 2) * 16 + (lane % 4) * 4;

  if (steps > 0) {
    fetch(0);
    stage(buf[0]);
    fetch(1);
  }
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const typename K::Buffer &b = buf[s & 1];
#pragma unroll
    for (int k = 0; k < Step / 16; ++k) {
      bf16x8 fi[K::kMi];
#pragma unroll
      for (int v = 0; v < K::kMi; ++v)
        fi[v] = transposed(
            &b.i[(k * 16 + tr) * K::kStrideI + wi + v * 32 + tc], K::kStrideI);
#pragma unroll
      for (int t = K::kT - 1; t >= 0; --t) {
#pragma unroll
        for (int x = 0; x < K::kMo; ++x) {
          const bf16x8 fo = transposed(
              &b.o[t][(k * 16 + tr) * K::kStrideO + wo + x * 32 + tc],
              K::kStrideO);
#pragma unroll
          for (int v = 0; v < K::kMi; ++v)
            acc[x][v] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                fo, fi[v], acc[x][v], 0, 0, 0);
        }
      }
    }
    if (s + 1 < steps) {
      stage(buf[(s + 1) & 1]);
      fetch(s + 2);
    }
    __syncthreads();
  }

  // D[o][i]: lane % 32 is the column i, the rows o are 4 (lane / 32) +
  // r % 4 + 8 (r / 4)
#pragma unroll
  for (int x = 0; x < K::kMo; ++x)
#pragma unroll
    for (int v = 0; v < K::kMi; ++v) {
      const int64_t i = i0 + wi + v * 32 + lane % 32;
      if (i >= a.fin) continue;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t o =
            o0 + wo + x * 32 + (lane / 32) * 4 + r % 4 + 8 * (r / 4);
        if (o >= a.fout) continue;
        if (a.part)
          a.part[(split * a.fout + o) * a.fin + i] = acc[x][v][r];
        else
          put(a.dw, o * a.lddw + i, acc[x][v][r], a.gtype, a.accumulate);
      }
    }
  if (bias) {
    // the rows of a column are joined in order
    float *sum = (float *)&buf[0];
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[ro * BO + co * 8 + k] = db[k];
    __syncthreads();
    for (int c = tid; c < BO; c += K::kThreads) {
      if (o0 + c >= a.fout) continue;
      float s = 0.0f;
      for (int r = 0; r < kRowsO; ++r) s += sum[r * BO + c];
      if (a.part_db) a.part_db[split * a.fout + o0 + c] = s;
      else put(a.db, o0 + c, s, a.gtype, a.accumulate);
    }
  }
}

// The parts' sums joined in order.
__global__ __launch_bounds__(256) void k_wgrad_join(const WgradArgs a,
                                                    int splits) {
  const int64_t n = a.fout * a.fin;
  const int64_t all = n + (a.db ? a.fout : 0);
  for (int64_t e = int64_t{blockIdx.x} * 256 + threadIdx.x; e < all;
       e += int64_t{gridDim.x} * 256) {
    const bool w = e < n;
    const float *p = w ? a.part + e : a.part_db + (e - n);
    const int64_t pitch = w ? n : a.fout;
    float s = 0.0f;
    for (int k = 0; k < splits; ++k) s += p[k * pitch];
    if (w) put(a.dw, e / a.fin * a.lddw + e % a.fin, s, a.gtype, a.accumulate);
    else put(a.db, e - n, s, a.gtype, a.accumulate);
  }
}

constexpr int kTileO = 128, kTileI = 128, kStep = 32;

}  // namespace

WgradShape wgrad_shape(int64_t tokens, int64_t fin, int64_t fout, int type,
                       int cus) {
  WgradShape s{};
  s.tile_o = kTileO;
  s.tile_i = kTileI;
  s.step = kStep;
  s.terms = type == MTA_BF16 ? 1 : type == MTA_F16 ? 2 : 3;
  // no input features: the bias gradient alone still takes a column of tiles
  s.tiles = ((fout + kTileO - 1) / kTileO) *
            (((fin > 0 ? fin : 1) + kTileI - 1) / kTileI);
  const int64_t steps = (tokens + kStep - 1) / kStep;
  int64_t splits = s.tiles > 0 ? (2 * cus + s.tiles - 1) / s.tiles : 1;
  if (splits > steps / 8) splits = steps / 8;
  if (splits < 1) splits = 1;
  s.per_split = (steps + splits - 1) / splits * kStep;
  s.splits = s.per_split > 0
                 ? static_cast<int>((tokens + s.per_split - 1) / s.per_split)
                 : 1;
  if (s.splits < 1) s.splits = 1;
  return s;
}

hipError_t launch_wgrad(const WgradArgs &a, const WgradShape &s,
                        hipStream_t stream) {
  const int tiles_i =
      static_cast<int>(((a.fin > 0 ? a.fin : 1) + s.tile_i - 1) / s.tile_i);
  const int grid = static_cast<int>(s.tiles * s.splits);
  if (grid == 0) return hipSuccess;
  const hipError_t e = with_type(a.type, [&](auto d) {
    k_wgrad<decltype(d)::value, kTileO, kTileI, 2, 2, kStep>
        <<<grid, 256, 0, stream>>>(a, tiles_i, static_cast<int>(s.tiles),
                                   s.per_split);
    return hipGetLastError();
  });
  if (e != hipSuccess || s.splits == 1) return e;
  const int64_t n = a.fout * a.fin + (a.db ? a.fout : 0);
  const int64_t blocks = (n + 255) / 256;
  k_wgrad_join<<<static_cast<int>(blocks < 65536 ? blocks : 65536), 256, 0,
                 stream>>>(a, s.splits);
  return hipGetLastError();
}

}  // namespace mta
