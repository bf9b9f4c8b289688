// wgrad_kernels.hip -- weight and bias gradient of a linear layer from the
// 8-bit checkpoint of its input, on the matrix cores of gfx950.
//
//   dW[o][i] = sum_t dY[t][o] * kept[t][i],   db[o] = sum_t dY[t][o]
//
// A kept value is an e4m3 code times a power of two: exact in bfloat16, so the
// product runs on the bfloat16 matrix instructions without any rounding but
// that of its float32 sums, and the checkpoint is read at one byte a value.
// A float16 dY is multiplied on the float16 instructions where every kept
// value is exact in float16 too, as those of float16 activations are; a
// kernel looks at the checkpoint first.  Otherwise a float16 (float32) dY is
// split into the two (three) bfloat16 values whose sum it is, one product each.
//
// Both operands lie with the contracted index t as their rows, while a matrix
// instruction wants eight consecutive t of one column in a lane.  They are
// staged in LDS as they lie (the codes converted on the way) and read back
// with the transposing LDS load: 16 lanes read four rows of 16 columns and
// each gets four rows of one column.
//
// Bound by the LDS and the matrix pipes, which take turns: a step of a
// workgroup, 32 tokens, is 32 KiB of transposing reads (which reach 128 bytes a
// clock here), 16 KiB of writes (64 to 77), 16 loads of a wave and 32 matrix
// instructions, and the counters have the LDS busy for 51% of the time and the
// matrix pipes for 41%.  A workgroup of four waves takes a tile of 128 x 128,
// and three share a CU, so that one's reads run under another's products: 8192
// tokens of 4096 x 4096 in bfloat16 in 294 to 310 us (890 to 935 TFLOP/s),
// 308 without the order that sched_group_barrier asks for where it is 294 with
// it; one workgroup of 256^2 with the same inner loop, whose eight waves keep
// step, was 1 to 3% slower.  A tile's sums are written with all tests of types
// outside and, when added to the gradient, with 32 old values on their way at
// once: one after the other they cost 8 us a workgroup (4 steps of tokens 16.3
// us, now 8.6; 1024 tokens, 768 -> 2304, 27.0, now 16 to 18).
#include "ops_device.h"

namespace mta {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTile = kWgradTile;  // outputs of a workgroup, each way
constexpr int kStep = kWgradStep;  // tokens at a time
constexpr int kThreads = 256;
// 64 bytes behind each LDS row: the four rows of a transposing load, and the
// two column halves that are read together, then lie in distinct banks.
constexpr int kPitch = kTile + 32;

// How dY is multiplied.
enum Mode { kBf16, kF16, kF16Split, kF32Split };

template <int M>
struct Stage {
  static constexpr int kType =
      M == kBf16 ? MTA_BF16 : M == kF32Split ? MTA_F32 : MTA_F16;
  static constexpr int kTerms = M == kF32Split ? 3 : M == kF16Split ? 2 : 1;
  // Two buffers of 10 KiB and 10 for each term; three, two and two workgroups
  // of 168, 256 and 256 registers a lane.
  static constexpr int kWavesPerSimd = kTerms == 1 ? 3 : 2;
  struct Operand {
    uint16_t at[kStep][kPitch];
  };
  struct Buffer {
    Operand o[kTerms], i;
  };
};

// The bfloat16 values that v is the sum of, largest first, each in the upper
// half of a word.  Each takes the next eight significant bits of what is left
// by cutting the lower ones off, so a difference is exact and no value grows
// past its source.  An infinity or NaN is carried by the first alone.
template <int Terms>
__device__ __forceinline__ void split(float v, uint32_t (&b)[Terms]) {
  const bool fine = __builtin_fabsf(v) < __builtin_inff();
#pragma unroll
  for (int t = 0; t < Terms; ++t) {
    b[t] = __float_as_uint(v) & 0xFFFF0000u;
    // a NaN of low bits only would be cut to an infinity
    if (t == 0 && v != v) b[t] = 0x7FC00000u;
    v = fine ? v - __uint_as_float(b[t]) : 0.0f;
  }
}

// Four codes of one block times their scale, as two words of 16-bit values.
template <int M>
__device__ __forceinline__ void kept4(uint32_t code, float scale,
                                      uint32_t &lo, uint32_t &hi) {
  if constexpr (M == kF16) {
    lo = __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(code, scale, false));
    hi = __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(code, scale, true));
  } else {
    lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                          code, scale, false));
    hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(
                                          code, scale, true));
  }
}

// The magnitude of a whole number below 2^32; 0 of a NaN.
__device__ __forceinline__ uint32_t whole(float x) {
  return x == x ? static_cast<uint32_t>(__builtin_fabsf(x)) : 0u;
}

// The run `n` elements (0 to 7) further on; its last n are anything.
template <int D>
__device__ __forceinline__ Raw8<D> slide(Raw8<D> x, int n) {
  constexpr int kWords = Raw8<D>::kWords, kEach = 8 / kWords;
#pragma unroll
  for (int h = 4; h >= kEach; h /= 2) {
    const int d = h / kEach;
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      x.w[k] = n & h ? x.w[k + d < kWords ? k + d : k] : x.w[k];
  }
  if constexpr (kEach == 2) {
    const uint32_t bits = (n & 1) * 16;
#pragma unroll
    for (int k = 0; k < kWords; ++k)
      x.w[k] = __builtin_amdgcn_alignbit(
          x.w[k + 1 < kWords ? k + 1 : k], x.w[k], bits);
  }
  return x;
}

// Eight tokens of one column, from `p` in this lane's place.
__device__ __forceinline__ s16x8 transposed(const uint16_t *p) {
  typedef __attribute__((address_space(3))) s16x4 lds4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
  const s16x4 b =
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + 4 * kPitch));
  return s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

template <int M>
__device__ __forceinline__ f32x16 multiply(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (M == kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(
        __builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        __builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
        0);
}

// An address kept in scalar registers: the compiler would fold a lane's offset
// into it and add the two in every lane.
__device__ __forceinline__ const MTA_GLOBAL uint8_t *scalar(
    const MTA_GLOBAL uint8_t *p) {
  __asm__("" : "+s"(p));
  return p;
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

// The output tile number t: down bands of eight rows of tiles, so that tiles
// that run together share their operands' columns.
__device__ __forceinline__ void tile_at(const WgradGrid &g, int64_t t,
                                        int64_t &o, int64_t &i) {
  constexpr int64_t kBand = 8;
  const int64_t band = t / (kBand * g.tiles_i), first = band * kBand;
  const int64_t height = min(kBand, g.tiles_o - first);
  const int64_t u = t - first * g.tiles_i;
  o = (first + u % height) * kTile;
  i = u / height * kTile;
}

// Work item `w` of n, such that workgroups that run on one of the eight XCDs
// (blocks are dealt out in turn) take neighbouring ones.
__device__ __forceinline__ int64_t neighbours(int64_t w, int64_t n) {
  const int64_t x = w % 8, each = n / 8, more = n % 8;
  return x * each + min(x, more) + w / 8;
}

// Whether every kept value is exact in float16, as those of a float16 tensor
// are.  Most blocks' scales say so; the others' codes are looked at (a block of
// small values, such as the single column behind whole blocks often is, or of
// zeros).  A workgroup answers for a stretch of blocks.
__global__ __launch_bounds__(256) void k_wgrad_range(const WgradArgs a,
                                                     int64_t blocks) {
  constexpr int kEach = 4;  // blocks a lane has in flight
  const int64_t stride = int64_t{gridDim.x} * 256;
  int fine = 1;
  for (int64_t e = int64_t{blockIdx.x} * 256 + threadIdx.x; e < blocks;
       e += stride * kEach) {
    uint32_t s[kEach];
    u32x4 q[kEach][2];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      s[j] = e + j * stride < blocks
                 ? ((const MTA_GLOBAL uint8_t *)a.scale)[e + j * stride]
                 : kFloat16Scales[0];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (s[j] < kFloat16Scales[0] || s[j] > kFloat16Scales[1]) {
        const auto *at = (const MTA_GLOBAL u32x4 *)a.q + (e + j * stride) * 2;
        q[j][0] = at[0];
        q[j][1] = at[1];
      }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (s[j] < kFloat16Scales[0] || s[j] > kFloat16Scales[1]) {
        // a code times 2^9 is its number of steps; a NaN becomes 0
        uint32_t steps = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = static_cast<int>(q[j][k / 4][k % 4]);
            const f32x2 v =
                h ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, 512.0f, true)
                  : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, 512.0f, false);
            steps |= whole(v[0]) | whole(v[1]);
          }
        if (!float16_holds(s[j], steps)) fine = 0;
      }
  }
  fine = __syncthreads_and(fine);
  if (threadIdx.x == 0) a.range[blockIdx.x] = fine;
}

// Groups > 1: so many times the waves work on a tile, each group of four on
// its own share of the tokens with its own LDS buffers, and are joined in LDS
// at the end.
template <int M, int Groups>
__global__ __launch_bounds__(kThreads * Groups)
    __attribute__((amdgpu_waves_per_eu(Stage<M>::kWavesPerSimd))) void
    k_wgrad(const WgradArgs a, const WgradGrid g) {
  using K = Stage<M>;
  constexpr int D = K::kType, kTerms = K::kTerms;
  constexpr int kRounds = kStep / 16;
  const int group =
      Groups == 1 ? 0
                  : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
  const int tid = threadIdx.x % kThreads, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);

  if constexpr (M == kF16 || M == kF16Split) {
    const int fine =
        __syncthreads_and(tid < g.ranges ? a.range[tid] : 1);
    if (fine != (M == kF16)) return;
  }

  // Whole tiles first, then the parts of the cut ones.
  const int64_t block = blockIdx.x;
  const bool cut = block >= g.whole;
  int64_t tile, part = 0;
  if (!cut) {
    tile = neighbours(block, g.whole);
  } else {
    const int64_t w = neighbours(block - g.whole, g.cut * g.parts);
    part = w / g.cut;
    tile = g.whole + w % g.cut;
  }
  int64_t o0, i0;
  tile_at(g, tile, o0, i0);
  const int64_t t0 = cut ? part * g.part_tokens : 0;
  const int64_t t1 = cut ? min(a.tokens, t0 + g.part_tokens) : a.tokens;

  __shared__ typename K::Buffer bufs[Groups][2];
  auto &buf = bufs[group];

  // A lane stages eight columns of dY in tokens row_o and row_o + 16, and
  // sixteen of the checkpoint in token row_i.
  constexpr int kRowsO = kThreads / (kTile / 8), kRowsI = kThreads / (kTile / 16);
  constexpr int kNO = kStep / kRowsO;
  static_assert(kNO == 2 && kRowsI == kStep, "a step is staged in one go");
  const int co = tid % (kTile / 8) * 8, row_o = tid / (kTile / 8);
  const int ci = tid % (kTile / 16) * 16, row_i = tid / (kTile / 16);
  const int64_t pitch_s = a.ldq / MTA_CKPT_BLOCK;
  // Columns past the last whole run are the last one's again: what comes of
  // them is not written.  A run that the last column ends inside is moved to
  // its place when it is staged (loaded by elements instead, the last tiles
  // of 1601 outputs made 8192 tokens of 1600 features take 120 us, not 76).
  const int64_t col_o = min(o0 + co, max(int64_t{0}, a.fout - 8));
  const int64_t col_i = min(i0 + ci, max(int64_t{0}, a.ldq - 16));
  const int64_t lane_o = (col_o - o0 + row_o * a.lddy) * int64_t{sizeof(elem<D>)};
  const int behind = static_cast<int>(min(int64_t{7}, o0 + co - col_o));
  const uint32_t lane_i = static_cast<uint32_t>(col_i - i0 + row_i * a.ldq);
  const uint32_t lane_s = static_cast<uint32_t>(
      col_i / MTA_CKPT_BLOCK - i0 / MTA_CKPT_BLOCK + row_i * pitch_s);

  struct Fetched {
    Raw8<D> o[kNO];
    u32x4 code;
    uint32_t scale;
  } raw[2];
  float db[8] = {0, 0, 0, 0, 0, 0, 0, 0};

  // A step that lies inside the tensors, loaded without a test.
  const auto fetch = [&](int step, Fetched &x) {
    const int64_t t = t0 + int64_t{step} * kStep;
#pragma unroll
    for (int j = 0; j < kNO; ++j) {
      const auto *p = scalar(
          (const MTA_GLOBAL uint8_t *)a.dy +
          ((t + j * kRowsO) * a.lddy + o0) * int64_t{sizeof(elem<D>)});
#pragma unroll
      for (int h = 0; h < Raw8<D>::kWords / 4; ++h) {
        const u32x4 v =
            *(const MTA_GLOBAL typename Wide<D>::type *)(p + lane_o + h * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) x.o[j].w[4 * h + k] = v[k];
      }
    }
    x.code = *(const MTA_GLOBAL u32x4 *)(
        scalar((const MTA_GLOBAL uint8_t *)a.q + t * a.ldq + i0) + lane_i);
    x.scale = *(scalar((const MTA_GLOBAL uint8_t *)a.scale + t * pitch_s +
                       i0 / MTA_CKPT_BLOCK) +
                lane_s);
  };
  // Any step: what lies outside is zero.
  const auto fetch_edge = [&](int step, Fetched &x) {
    const int64_t t = t0 + int64_t{step} * kStep;
    const int64_t left = a.fout - (o0 + co);
    const int n = static_cast<int>(left >= 8 ? 8 : left > 0 ? left : 0);
#pragma unroll
    for (int j = 0; j < kNO; ++j) {
      const int64_t r = t + row_o + j * kRowsO;
      const int64_t at = r * a.lddy + o0 + co;
      if (r < t1 && n == 8) x.o[j] = load8<D, false>(a.dy, at);
      else x.o[j] = load8_part<D>(a.dy, at, r < t1 ? n : 0, 0);
    }
    x.code = u32x4{0, 0, 0, 0};
    x.scale = 0;
    const int64_t r = t + row_i;
    if (r < t1 && i0 + ci < a.ldq) {
      const int64_t at = r * a.ldq + i0 + ci;
      x.code = *(const MTA_GLOBAL u32x4 *)(a.q + at);
      x.scale = ((const MTA_GLOBAL uint8_t *)a.scale)[at / MTA_CKPT_BLOCK];
    }
  };
  const auto stage = [&](typename K::Buffer &b, const Fetched &x, auto with_bias,
                         auto ragged) {
#pragma unroll
    for (int j = 0; j < kNO; ++j) {
      Raw8<D> dy = x.o[j];
      if constexpr (decltype(ragged)::value) dy = slide<D>(dy, behind);
      uint32_t w[kTerms][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (kTerms == 1) {
          w[0][k] = dy.w[k];
        } else {
          uint32_t u[kTerms], v[kTerms];
          split<kTerms>(dy[2 * k], u);
          split<kTerms>(dy[2 * k + 1], v);
#pragma unroll
          for (int t = 0; t < kTerms; ++t) w[t][k] = (u[t] >> 16) | v[t];
        }
      }
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
        *(u32x4 *)&b.o[t].at[row_o + j * kRowsO][co] =
            u32x4{w[t][0], w[t][1], w[t][2], w[t][3]};
      if constexpr (decltype(with_bias)::value) {
#pragma unroll
        for (int k = 0; k < 8; ++k) db[k] += dy[k];
      }
    }
    const float s = __uint_as_float(x.scale << 23);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4];
      kept4<M>(x.code[2 * h], s, w[0], w[1]);
      kept4<M>(x.code[2 * h + 1], s, w[2], w[3]);
      *(u32x4 *)&b.i.at[row_i][ci + h * 8] = u32x4{w[0], w[1], w[2], w[3]};
    }
  };

  // Waves lie two by two, each with 2 x 2 matrix tiles of 32 x 32.
  // The second and third terms of a float32 dY have their own sums: three
  // roundings to the first one's size for every sixteen tokens would be 1.3e-6
  // of the result after 16384, where one is 5e-7.
  constexpr int kSums = kTerms == 3 ? 2 : 1;
  f32x16 acc[kSums][2][2];
#pragma unroll
  for (int u = 0; u < kSums; ++u)
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[u][x][v][r] = 0.0f;
  const int wo = wave / 2 * 64, wi = wave % 2 * 64;
  // this lane's place in a transposing load of 32 columns x 16 tokens
  const int tr = (lane / 32) * 8 + (lane % 16) / 4;
  const int tc = ((lane / 16) % 2) * 16 + (lane % 4) * 4;
  // the next round's operands beside this one's, but for three terms, whose
  // second sums have the registers
  constexpr int kSets = kTerms == 3 ? 1 : 2;
  s16x8 fo[kSets][kTerms][2], fi[kSets][2];
  const auto read = [&](const typename K::Buffer &b, int k, int set) {
#pragma unroll
    for (int v = 0; v < 2; ++v)
      fi[set][v] = transposed(&b.i.at[k * 16 + tr][wi + v * 32 + tc]);
#pragma unroll
    for (int t = 0; t < kTerms; ++t)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        fo[set][t][x] = transposed(&b.o[t].at[k * 16 + tr][wo + x * 32 + tc]);
  };

  // Steps [from, to), each fetched by `get`.  While step s is multiplied, step
  // s + 1 goes to LDS and steps s + 2 and s + 3 are on their way.
  const auto run = [&](int from, int to, auto &&get, auto with_bias,
                       auto ragged) {
    const int n = to - from;
    if (n <= 0) return;
    get(from, raw[0]);
    stage(buf[0], raw[0], with_bias, ragged);
    // (past the end: the last step again)
    get(min(from + 1, to - 1), raw[0]);
    get(min(from + 2, to - 1), raw[1]);
    __syncthreads();
    const auto step = [&](int s, typename K::Buffer &b, typename K::Buffer &next,
                          Fetched &x, auto steady) {
      if constexpr (kSets == 2) read(b, 0, 0);
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        const int set = k % kSets;
        if constexpr (kSets == 1) read(b, k, 0);
        else if (k + 1 < kRounds) read(b, k + 1, (k + 1) % kSets);
#pragma unroll
        for (int t = kTerms - 1; t >= 0; --t)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              f32x16 &sum = acc[t == 0 ? 0 : kSums - 1][m][v];
              sum = multiply<M>(fo[set][t][m], fi[set][v], sum);
            }
        if (k == 0) {
          if (decltype(steady)::value || s + 1 < n) stage(next, x, with_bias, ragged);
          if (decltype(steady)::value || s + 3 < n) get(from + s + 3, x);
        }
        if constexpr (kTerms == 1) {
          // a product, two reads of the next round's operands, a few others'
          // instructions, and so on
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            if (k == 0) __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
    };
    int s = 0;
    for (; s + 4 < n; s += 2) {
      step(s, buf[0], buf[1], raw[0], std::true_type{});
      step(s + 1, buf[1], buf[0], raw[1], std::true_type{});
    }
    for (; s < n; s += 2) {
      step(s, buf[0], buf[1], raw[0], std::false_type{});
      if (s + 1 < n) step(s + 1, buf[1], buf[0], raw[1], std::false_type{});
    }
    __syncthreads();
  };
  const bool bias = a.db && i0 == 0;
  const bool inside = a.fout >= 8 && a.ldq > 0;
  // Every group takes the same number of steps that lie inside, then the same
  // number of others, some of them past the end.
  const int steps = static_cast<int>((t1 - t0 + kStep - 1) / kStep);
  const int inner = inside ? static_cast<int>((t1 - t0) / kStep / Groups) : 0;
  const int outer = (steps - inner * Groups + Groups - 1) / Groups;
  const int from = group * inner, edge = inner * Groups + group * outer;
  if (o0 + kTile > a.fout && a.fout % 8 != 0)
    run(from, from + inner, fetch, std::true_type{}, std::true_type{});
  else if (bias)
    run(from, from + inner, fetch, std::true_type{}, std::false_type{});
  else
    run(from, from + inner, fetch, std::false_type{}, std::false_type{});
  run(edge, edge + outer, fetch_edge, std::true_type{}, std::false_type{});
  if constexpr (kSums == 2) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int v = 0; v < 2; ++v) acc[0][x][v] += acc[1][x][v];
  }
  // the groups' sums joined in order
  if constexpr (Groups > 1) {
    f32x4 *at = (f32x4 *)&bufs[0][0];
    static_assert(sizeof bufs >= kTile * kTile * 4, "a tile fits");
#pragma unroll
    for (int u = 1; u < Groups; ++u) {
      if (group == u) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const f32x16 &c = acc[0][q / 8][q / 4 % 2];
          const int r = q % 4 * 4;
          at[q * kThreads + tid] = f32x4{c[r], c[r + 1], c[r + 2], c[r + 3]};
        }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const f32x4 y = at[q * kThreads + tid];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[0][q / 8][q / 4 % 2][q % 4 * 4 + k] += y[k];
        }
      }
      __syncthreads();
    }
  }

  // D[o][i]: lane % 32 is the column i, the rows o are 4 (lane / 32) +
  // r % 4 + 8 (r / 4).  A part's tile goes to the workspace whole.
  if (group == 0) {
    const auto row = [](int x, int r) { return x * 32 + r % 4 + 8 * (r / 4); };
    const int64_t o1 = o0 + wo + (lane / 32) * 4, i1 = i0 + wi + lane % 32;
    if (cut) {
      float *out = a.part + ((tile - g.whole) * g.parts + part) *
                                int64_t{kTile * kTile};
      const int first = (wo + (lane / 32) * 4) * kTile + wi + lane % 32;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            out[first + row(x, r) * kTile + v * 32] = acc[0][x][v][r];
    } else {
      const auto write = [&](auto type, auto whole) {
        constexpr int T = decltype(type)::value;
        const int64_t place = (lane / 32 * 4 * a.lddw + lane % 32) *
                              int64_t{sizeof(elem<T>)};
        const auto at = [&](int x, int v, int r) {
          return (void *)(scalar((const MTA_GLOBAL uint8_t *)a.dw +
                                 ((o0 + wo + row(x, r)) * a.lddw + i0 + wi +
                                  v * 32) *
                                     int64_t{sizeof(elem<T>)}) +
                          place);
        };
        const auto is = [&](int x, int v, int r) {
          return decltype(whole)::value ||
                 (o1 + row(x, r) < a.fout && i1 + v * 32 < a.fin);
        };
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // the old values of 32 sums before the first is stored: otherwise
          // each load waits for the one before it
          if (a.accumulate) {
            float old[2][16];
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
              for (int r = 0; r < 16; ++r)
                old[v][r] = is(x, v, r) ? load_elem<T>(at(x, v, r), 0) : 0.0f;
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
              for (int r = 0; r < 16; ++r) acc[0][x][v][r] += old[v][r];
          }
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (is(x, v, r)) store_elem<T>(at(x, v, r), 0, acc[0][x][v][r]);
        }
      };
      with_type(a.gtype, [&](auto type) {
        if (o0 + kTile <= a.fout && i0 + kTile <= a.fin)
          write(type, std::true_type{});
        else
          write(type, std::false_type{});
      });
    }
  }
  if (bias) {
    // a column's rows are joined in order
    float *sum = (float *)&bufs[0][0];
    const int row = group * kRowsO + row_o;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[row * kTile + co + k] = db[k];
    __syncthreads();
    if (threadIdx.x < kTile && o0 + tid < a.fout) {
      float s = 0.0f;
      for (int r = 0; r < kRowsO * Groups; ++r) s += sum[r * kTile + tid];
      if (cut) a.part_db[part * a.fout + o0 + tid] = s;
      else put(a.db, o0 + tid, s, a.gtype, a.accumulate);
    }
  }
}

// The cut tiles' parts joined in order: a workgroup takes 16 rows of a tile.
__global__ __launch_bounds__(256) void k_wgrad_join(const WgradArgs a,
                                                    const WgradGrid g) {
  constexpr int kStrips = kTile / 16;
  const int64_t which = blockIdx.x / kStrips;
  const int strip = blockIdx.x % kStrips;
  int64_t o0, i0;
  tile_at(g, g.whole + which, o0, i0);
  const float *p = a.part + which * g.parts * int64_t{kTile * kTile} +
                   strip * 16 * kTile;
  f32x4 s[2] = {};
  const int at = threadIdx.x * 4;
  const auto part = [&](int k, int j) {
    return *(const MTA_GLOBAL f32x4 *)(p + k * int64_t{kTile * kTile} + at +
                                       j * 1024);
  };
  int k = 0;
  for (; k + 4 <= g.parts; k += 4) {  // four on their way at a time
    f32x4 y[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j) y[u][j] = part(k + u, j);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j] += y[u][j];
  }
  for (; k < g.parts; ++k)
#pragma unroll
    for (int j = 0; j < 2; ++j) s[j] += part(k, j);
  with_type(a.gtype, [&](auto type) {
    constexpr int T = decltype(type)::value;
    const int64_t o = o0 + strip * 16 + at / kTile, i = i0 + at % kTile;
    const auto is = [&](int j, int u) {
      return o + j * 8 < a.fout && i + u < a.fin;
    };
    if (a.accumulate) {
      f32x4 old[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          old[j][u] = is(j, u)
                          ? load_elem<T>(a.dw, (o + j * 8) * a.lddw + i + u)
                          : 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j] += old[j];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (is(j, u))
          store_elem<T>(a.dw, (o + j * 8) * a.lddw + i + u, s[j][u]);
  });
  if (a.db && i0 == 0 && strip == 0 && threadIdx.x < kTile) {
    const int64_t o = o0 + threadIdx.x;
    if (o < a.fout) {
      float b = 0.0f;
      for (k = 0; k < g.parts; ++k) b += a.part_db[k * a.fout + o];
      put(a.db, o, b, a.gtype, a.accumulate);
    }
  }
}

template <int M>
hipError_t start(const WgradArgs &a, const WgradGrid &g, hipStream_t stream) {
  const int n = static_cast<int>(g.whole + g.cut * g.parts);
  if (g.grouped) {
    constexpr int kGroups = Stage<M>::kWavesPerSimd;
    k_wgrad<M, kGroups><<<n, kThreads * kGroups, 0, stream>>>(a, g);
  } else {
    k_wgrad<M, 1><<<n, kThreads, 0, stream>>>(a, g);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_wgrad(const WgradArgs &a, const WgradGrid &g,
                        hipStream_t stream) {
  hipError_t e;
  if (a.type == MTA_BF16) {
    e = start<kBf16>(a, g, stream);
  } else if (a.type == MTA_F32) {
    e = start<kF32Split>(a, g, stream);
  } else {
    // one of the two finds that it is not wanted and ends
    if (g.ranges > 0)
      k_wgrad_range<<<g.ranges, 256, 0, stream>>>(
          a, a.tokens * (a.ldq / MTA_CKPT_BLOCK));
    e = start<kF16>(a, g, stream);
    if (e == hipSuccess) e = start<kF16Split>(a, g, stream);
  }
  if (e != hipSuccess || g.cut == 0) return e;
  k_wgrad_join<<<static_cast<int>(g.cut * (kTile / 16)), 256, 0, stream>>>(a,
                                                                           g);
  return hipGetLastError();
}

}  // namespace mta
