// gemm_device.h -- the tiled matrix product that the operators of
// include/mta_matrix.h are built on, for the matrix cores of gfx950.
//
//   acc[m][n] = sum over pairs p, sum over k of A_p[m][k] * B_p[n][k]
//
// with 16-bit elements and float32 sums.  A and B are read either as they lie
// with k contiguous (kAlong) or with k as their rows (kAcross); a product of
// more than 16 bits an element is a list of pairs of 16-bit planes, so that
// each pair is one more run over k with the same sums.
//
// A workgroup takes a tile of BM x BN.  Its operands come to LDS without
// passing registers (16 bytes a lane), ST buffers of BK values of k deep, so
// that ST - 1 of them are on their way while one is multiplied.  A wave has
// the fragments of the next 16 k on their way from LDS while it multiplies
// these, one read or one load behind each matrix instruction; the barrier of a
// buffer stands before the last 16 k of the one before, whose fragments are
// out of LDS by then.
//
// In LDS the 16-byte chunks of a row lie rotated: a plain layout would put the
// rows that a fragment's lanes read together into the same banks.
//
// Bound by power on this card: tiles of 256 x 256 in eight waves with BK 32,
// 4 buffers and with 64, 2 buffers, and in four waves of 128 x 128 each, all
// take 8192 x 8192 x 4160 at 1075 to 1130 TFLOP/s with the matrix pipes busy
// for 60 to 70% of a clock that falls to 1.6 GHz.  The library's product is at
// 1228 there.  Tiles of 128 x 128, two workgroups a CU, are at 1000.
#pragma once

#include "matrix_internal.h"
#include "ops_device.h"

namespace mta {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

#define MTA_LDS __attribute__((address_space(3)))

enum Lay { kAlong, kAcross };

template <int BM, int BN, int WR, int WC, int BK, int ST, int PerSimd>
struct Tile {
  static constexpr int kBM = BM, kBN = BN, kBK = BK, kST = ST;
  static constexpr int kWR = WR, kWC = WC;
  static constexpr int kPerSimd = PerSimd;         // waves on a SIMD
  static constexpr int kThreads = 64 * WR * WC;
  static constexpr int kTM = BM / WR, kTN = BN / WC;  // outputs of a wave
  static constexpr int kRM = kTM / 32, kRN = kTN / 32;
  static constexpr int kNA = BM * BK / 8 / kThreads;  // loads of a lane
  static constexpr int kNB = BN * BK / 8 / kThreads;
  static constexpr int kStage = (BM + BN) * BK * 2;   // bytes
  static constexpr int kLds = kStage * ST;
  static_assert(kNA * kThreads * 8 == BM * BK, "whole loads");
  static_assert(kNB * kThreads * 8 == BN * BK, "whole loads");
  static_assert(BM >= 64 && BN >= 64, "a turn stays in a row of LDS");
};

// One operand: planes of 16-bit elements, `plane` elements apart, rows of ld.
struct Operand {
  const uint16_t *p;
  int64_t plane;
  int64_t ld;
  int64_t extent;  // rows (kAlong) or columns (kAcross) that are there: more
                   // are read again from the last ones
  int64_t depth;   // kAcross: rows that are there, as above
};

// Which planes are multiplied, two bits each, the smallest products first, so
// that few roundings have the size of the whole sum.
struct Pairs {
  int count;
  uint32_t a, b;
};
__host__ __device__ constexpr Pairs pairs_of(int planes) {
  // 1: hi hi.  2: lo hi, hi lo, hi hi.  3: 2 0, 0 2, 1 1, 1 0, 0 1, 0 0.
  return planes == 1   ? Pairs{pair_count(1), 0, 0}
         : planes == 2 ? Pairs{pair_count(2), 0x01, 0x04}
                       : Pairs{pair_count(3), 0x052, 0x118};
}

// A value that is the same in all lanes, for the scalar registers.
__device__ __forceinline__ uint32_t scalar(uint32_t x) {
  return __builtin_amdgcn_readfirstlane(x);
}
__device__ __forceinline__ float scalar(float x) {
  return __uint_as_float(scalar(__float_as_uint(x)));
}
__device__ __forceinline__ const MTA_GLOBAL uint8_t *scalar(
    const MTA_GLOBAL uint8_t *p) {
  const uint64_t x = (uint64_t)p;
  return (const MTA_GLOBAL uint8_t *)(
      uint64_t{scalar(static_cast<uint32_t>(x))} |
      uint64_t{scalar(static_cast<uint32_t>(x >> 32))} << 32);
}

// Sixteen bytes a lane from base + off to lds + 16 * lane (base and lds the
// same in a wave).  m0 is a register that the compiler keeps for itself, of which
// it warns; it is told all the same that this writes it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void to_lds(const MTA_GLOBAL uint8_t *base,
                                       uint32_t off, uint32_t lds) {
  __asm__ volatile(
      "s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
      :
      : "v"(off), "s"(base), "s"(lds)
      : "m0", "memory");
}
#pragma clang diagnostic pop

template <bool F16>
__device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(
        __builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        __builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
        0);
}

// How an operand of R rows (or columns) by BK lies in LDS, how a lane loads its
// share of it, and where it reads a fragment.
template <int L, int R, int BK, int Threads>
struct Slab {
  static constexpr int kRow = L == kAlong ? BK : R;  // elements of an LDS row
  static constexpr int kChunks = kRow / 8;
  static constexpr int kLoads = R * BK / 8 / Threads;
  // 256 bytes of LDS are all its banks: the rows that lie as far apart as that
  // and the lanes of a read want at once get different chunks.
  static __device__ __forceinline__ int turn(int row) {
    if constexpr (L == kAlong)
      return kChunks == 8 ? (row >> 1) & 7 : (row >> 2) & 3;
    else  // (rows of 64 are half the banks)
      return kChunks == 8 ? (row & 2) << 1 : (row & 3) << 2;
  }
  // Row and first element of chunk number q of the slab.
  static __device__ __forceinline__ int row_of(int q) { return q / kChunks; }
  static __device__ __forceinline__ int first_of(int q) {
    const int row = q / kChunks;
    return ((q % kChunks) ^ turn(row)) * 8;
  }
  // Bytes from the slab to this lane's part of the fragment of 16 values of k
  // from kk * 16 and 32 rows from 0.
  static __device__ __forceinline__ uint32_t place(int lane, int kk) {
    if constexpr (L == kAlong) {
      const int row = lane % 32, c = kk * 2 + lane / 32;
      return (row * kRow + ((c ^ turn(row)) * 8)) * 2;
    } else {
      const int k = kk * 16 + (lane / 32) * 8 + (lane % 16) / 4;
      const int x = ((lane / 16) % 2) * 16 + (lane % 4) * 4;
      return (k * kRow + (((x / 8) ^ turn(k)) * 8) + x % 8) * 2;
    }
  }
  // Fragment number i (32 rows on each) at `at`, a place() in the slab.
  static __device__ __forceinline__ s16x8 read(MTA_LDS uint8_t *slab,
                                               uint32_t at, int i) {
    if constexpr (L == kAlong) {
      return *(MTA_LDS s16x8 *)(slab + at + i * 32 * kRow * 2);
    } else {
      // 32 columns on: four chunks, and a turn is a multiple of four
      typedef MTA_LDS s16x4 lds4;
      MTA_LDS uint8_t *p = slab + (at ^ (i * 64));
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds4 *)(p + 4 * kRow * 2));
      return s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
  }
};

// The sums of the tile at (m0, n0) over k in [k0, k1), both multiples of 64:
// lane l of a wave has, of its 32 x 32 blocks acc[i][j], the row m = l % 32 and
// the columns n = 8 (r / 4) + 4 (l / 32) + r % 4.  Where an operand with k
// across ends before k1, its last row is taken again, and the other one has
// zeros there.
// `lds` has C::kLds bytes; on return no load is on its way, but other waves may
// still read it.
template <class C, bool F16, int LA, int LB>
__device__ __forceinline__ void tile_product(
    const Operand &a, const Operand &b, const Pairs pairs, int64_t m0,
    int64_t n0, int64_t k0, int64_t k1, MTA_LDS uint8_t *lds,
    f32x16 (&acc)[C::kRM][C::kRN]) {
  using SA = Slab<LA, C::kBM, C::kBK, C::kThreads>;
  using SB = Slab<LB, C::kBN, C::kBK, C::kThreads>;
  constexpr int kPer = C::kNA + C::kNB, kR = C::kBK / 16;
  constexpr int kReads = C::kRM + C::kRN, kM = C::kRM * C::kRN;
  constexpr int kSlots = kM > kReads ? kM : kReads;
  const int tid = threadIdx.x, lane = tid % 64;
  const int wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int wr = wave % C::kWR, wc = wave / C::kWR;

#pragma unroll
  for (int i = 0; i < C::kRM; ++i)
#pragma unroll
    for (int j = 0; j < C::kRN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int each = static_cast<int>((k1 - k0) / C::kBK);
  const int steps = each * pairs.count;
  if (steps == 0) return;

  // A lane's loads: rows and chunks are fixed, and for operands with k along
  // the row so are the offsets.
  uint32_t off_a[C::kNA], off_b[C::kNB];
  const auto offsets = [&](auto slab, const Operand &x, int64_t at,
                           uint32_t (&off)[decltype(slab)::kLoads], int lay,
                           int64_t left) {
    using S = decltype(slab);
#pragma unroll
    for (int j = 0; j < S::kLoads; ++j) {
      const int q = j * C::kThreads + tid;
      const int row = S::row_of(q), first = S::first_of(q);
      if (lay == kAlong) {
        const int most = static_cast<int>(
            x.extent - 1 - at < C::kBM + C::kBN ? x.extent - 1 - at
                                                : C::kBM + C::kBN);
        off[j] = static_cast<uint32_t>(min(row, most)) *
                     static_cast<uint32_t>(x.ld * 2) +
                 first * 2;
      } else {
        const int64_t last = x.extent - 8 - at;  // multiples of 8
        const int most = static_cast<int>(last < 1024 ? last : 1024);
        const int deep =
            static_cast<int>(left - 1 < C::kBK ? left - 1 : C::kBK);
        off[j] = static_cast<uint32_t>(min(row, deep)) *
                     static_cast<uint32_t>(x.ld * 2) +
                 min(first, most) * 2;
      }
    }
  };
  if constexpr (LA == kAlong) offsets(SA{}, a, m0, off_a, LA, 0);
  if constexpr (LB == kAlong) offsets(SB{}, b, n0, off_b, LB, 0);
  const auto *pa = (const MTA_GLOBAL uint8_t *)a.p +
                   (LA == kAlong ? m0 * a.ld + k0 : k0 * a.ld + m0) * 2;
  const auto *pb = (const MTA_GLOBAL uint8_t *)b.p +
                   (LB == kAlong ? n0 * b.ld + k0 : k0 * b.ld + n0) * 2;

  // The next step to load: its pair and its place in k.
  int load_pair = 0, load_k = 0, loads = 0;
  const MTA_GLOBAL uint8_t *la, *lb;
  const auto aim = [&] {
    // (past the end: the last step again, which nobody reads)
    const int x = (pairs.a >> (2 * load_pair)) & 3;
    const int y = (pairs.b >> (2 * load_pair)) & 3;
    const int64_t from = k0 + int64_t{load_k} * C::kBK;
    if constexpr (LA == kAlong) {
      la = pa + x * a.plane * 2 + int64_t{load_k} * (C::kBK * 2);
    } else {
      const int64_t row = min(from, a.depth - 1);
      la = pa + (x * a.plane + (row - k0) * a.ld) * 2;
      offsets(SA{}, a, m0, off_a, LA, a.depth - row);
    }
    if constexpr (LB == kAlong) {
      lb = pb + y * b.plane * 2 + int64_t{load_k} * (C::kBK * 2);
    } else {
      const int64_t row = min(from, b.depth - 1);
      lb = pb + (y * b.plane + (row - k0) * b.ld) * 2;
      offsets(SB{}, b, n0, off_b, LB, b.depth - row);
    }
    la = scalar(la);
    lb = scalar(lb);
    if (++loads < steps && ++load_k == each) {
      load_k = 0;
      ++load_pair;
    }
  };
  const uint32_t lds0 = scalar((uint32_t)(uintptr_t)lds) + wave * 1024;
  const auto load1 = [&](uint32_t stage, int j) {
    if (j < C::kNA)
      to_lds(la, off_a[j < C::kNA ? j : 0], stage + j * C::kThreads * 16);
    else
      to_lds(lb, off_b[j < C::kNA ? 0 : j - C::kNA],
             stage + C::kBM * C::kBK * 2 + (j - C::kNA) * C::kThreads * 16);
  };

  // A wave whose outputs lie behind the last row or column only brings its share
  // of the operands.  (Waves that share a SIMD lie far apart in n, so that a
  // tile with few columns left uses all SIMDs: 1600 columns are 6.25 tiles.)
  const int64_t high = a.extent - m0, wide = b.extent - n0;
  if (wr * C::kTM >= high || wc * C::kTN >= wide) {
#pragma unroll
    for (int s = 0; s < C::kST - 1; ++s) {
      aim();
#pragma unroll
      for (int j = 0; j < kPer; ++j) load1(lds0 + s * C::kStage, j);
    }
    __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kPer * (C::kST - 2))
                     : "memory");
    __builtin_amdgcn_s_barrier();
    int cur = 0;
    for (int s = 0; s < steps; ++s) {
      const int far = cur == 0 ? C::kST - 1 : cur - 1;
      aim();
#pragma unroll
      for (int j = 0; j < kPer; ++j) load1(lds0 + far * C::kStage, j);
      __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kPer * (C::kST - 2))
                       : "memory");
      __builtin_amdgcn_s_barrier();
      cur = cur + 1 == C::kST ? 0 : cur + 1;
    }
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return;
  }

  uint32_t at_a[kR], at_b[kR];
#pragma unroll
  for (int kk = 0; kk < kR; ++kk) {
    at_a[kk] = SA::place(lane, kk);
    at_b[kk] = SB::place(lane, kk);
  }
  s16x8 fa[2][C::kRM], fb[2][C::kRN];
  const auto read1 = [&](MTA_LDS uint8_t *s, int kk, int set, int q) {
    if (q < C::kRN) {
      MTA_LDS uint8_t *slab = s + C::kBM * C::kBK * 2;
      fb[set][q] = LB == kAlong
                       ? SB::read(slab + wc * C::kTN * C::kBK * 2, at_b[kk], q)
                       : SB::read(slab, at_b[kk] ^ (wc * C::kTN * 2), q);
    } else if (q < kReads) {
      fa[set][q - C::kRN] =
          LA == kAlong
              ? SA::read(s + wr * C::kTM * C::kBK * 2, at_a[kk], q - C::kRN)
              : SA::read(s, at_a[kk] ^ (wr * C::kTM * 2), q - C::kRN);
    }
  };

#pragma unroll
  for (int s = 0; s < C::kST - 1; ++s) {
    aim();
#pragma unroll
    for (int j = 0; j < kPer; ++j) load1(lds0 + s * C::kStage, j);
  }
  __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(kPer * (C::kST - 2)) : "memory");
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
#pragma unroll
  for (int q = 0; q < kReads; ++q) read1(lds, 0, 0, q);

  // One load behind so many matrix instructions; all of them before the wait
  // when there are only two buffers.
  constexpr int kSpace =
      C::kST == 2 ? kM * (kR - 1) / kPer : kR * kM / kPer;
  static_assert(kSpace >= 1 && kSpace * kPer <= kR * kM, "loads fit a step");
  int cur = 0;
  for (int s = 0; s < steps; ++s) {
    const int far = cur == 0 ? C::kST - 1 : cur - 1;
    const uint32_t to = lds0 + far * C::kStage;
    MTA_LDS uint8_t *here = lds + cur * C::kStage;
    const int after = cur + 1 == C::kST ? 0 : cur + 1;
    MTA_LDS uint8_t *next = lds + after * C::kStage;
    aim();
#pragma unroll
    for (int kk = 0; kk < kR; ++kk) {
      const int set = kk & 1;
      if (kk == kR - 1) {
        // what the next step reads is in LDS, and this one's fragments are out
        constexpr int kSent =
            kM * (kR - 1) / kSpace < kPer ? kM * (kR - 1) / kSpace : kPer;
        constexpr int kLeft = kPer * (C::kST - 3) + kSent;
        static_assert(kLeft >= 0 && kLeft < 64, "a count of loads");
        __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLeft)
                         : "memory");
        __builtin_amdgcn_s_barrier();
        __asm__ volatile("" ::: "memory");
      }
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        if (q < kM) {
          // neighbours share a fragment
          const int i = q / C::kRN;
          const int j = i & 1 ? C::kRN - 1 - q % C::kRN : q % C::kRN;
          acc[i][j] = mfma<F16>(fb[set][j], fa[set][i], acc[i][j]);
        }
        if (kk + 1 < kR) read1(here, kk + 1, set ^ 1, q);
        else read1(next, 0, set ^ 1, q);
        const int g = kk * kM + q;
        if (q < kM && g % kSpace == kSpace - 1 && g / kSpace < kPer)
          load1(to, g / kSpace);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    cur = after;
  }
  __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

// The sums through LDS, up to 64 rows of a wave's columns at a time, to
//   emit(m, n, v, x)    eight columns n .. n + 7 of a row, where `direct`
//   turned(n, m, v, x)  eight rows m .. m + 7 of a column, where `mirror`: with
//                       Fold what emit has made of them
// with m and n counted from the tile's corner and x what look(m, n) or
// ahead(n, m) gave some turns earlier (they are also asked for what lies behind
// the tile): global memory is on its way meanwhile.
// Loops are rolled: a workgroup runs this code once, and straight through it
// was 20 to 60 KB to fetch.
template <class C, bool Fold, class Look, class Emit, class Ahead, class Turned>
__device__ __forceinline__ void tile_out(
    MTA_LDS uint8_t *lds, const f32x16 (&acc)[C::kRM][C::kRN], bool direct,
    bool mirror, Look &&look, Emit &&emit, Ahead &&ahead, Turned &&turned) {
  constexpr int kH = C::kTM < 64 ? C::kTM : 64, kW = C::kTN;  // at a time
  constexpr int kBlocks = C::kTM / kH, kChunks = kW / 4;
  // lanes beside each other in a row (a column), rows (columns) of a turn, turns
  constexpr int kAlongRow = kW / 8, kRows = 64 / kAlongRow, kTurns = kH / kRows;
  constexpr int kAlongCol = kH / 8, kCols = 64 / kAlongCol,
                kTurnsCol = kW / kCols;
  constexpr int kWave = kH * kW * 4;
  static_assert(C::kTM % kH == 0 && kTurns % 2 == 0 && kTurnsCol % 2 == 0,
                "whole turns");
  static_assert(C::kWR * C::kWC * kWave <= C::kLds, "the staging fits");
  const int lane = threadIdx.x % 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int m_at = wave % C::kWR * C::kTM, n_at = wave / C::kWR * C::kTN;
  // rows of chunks of four, turned by the row so that lanes of a write or a
  // read meet in few banks
  auto *mine = (MTA_LDS float *)(lds + wave * kWave);
  const auto chunk = [&](int m, int c) {
    return (MTA_LDS f32x4 *)(mine + m * kW + ((c ^ (m & (kChunks - 1))) * 4));
  };
  // so many turns' memory is on its way (sums that wait for the second 64 rows
  // leave fewer registers)
  constexpr int kAhead =
      kTurns < 4 || (kBlocks > 1 && sizeof(decltype(look(0, 0))) > 48) ? 2 : 4;
  constexpr int kAheadCol = kTurnsCol < 4 ? 2 : 4;
  decltype(look(0, 0)) seen[kAhead];
  const int m = lane / kAlongRow, n = lane % kAlongRow * 8;
  if (direct) {
#pragma unroll
    for (int p = 0; p < kAhead; ++p)
      seen[p] = look(m_at + p * kRows + m, n_at + n);
  }
  __syncthreads();
#pragma unroll 1
  for (int b = 0; b < kBlocks; ++b) {
    const int m_b = m_at + b * kH;
#pragma unroll
    for (int i = 0; i < C::kRM; ++i) {
      if (i / (kH / 32) != b) continue;
#pragma unroll
      for (int j = 0; j < C::kRN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *chunk(i % (kH / 32) * 32 + lane % 32, j * 8 + q * 2 + lane / 32) =
              f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                    acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
    __builtin_amdgcn_wave_barrier();
    if (direct) {
#pragma unroll 1
      for (int h = 0; h < kTurns; h += kAhead) {
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
          const int row = (h + p) * kRows + m;
          const f32x4 f = *chunk(row, n / 4);
          const f32x4 g = *chunk(row, n / 4 + 1);
          float v[8] = {f[0], f[1], f[2], f[3], g[0], g[1], g[2], g[3]};
          emit(m_b + row, n_at + n, v, seen[p]);
          if constexpr (Fold) {
            *chunk(row, n / 4) = f32x4{v[0], v[1], v[2], v[3]};
            *chunk(row, n / 4 + 1) = f32x4{v[4], v[5], v[6], v[7]};
          }
          // (past the end: the next rows)
          seen[p] = look(m_b + row + kAhead * kRows, n_at + n);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
    if (mirror) {
      const int across = lane / kAlongCol, down = lane % kAlongCol * 8;
      decltype(ahead(0, 0)) next[kAheadCol];
#pragma unroll
      for (int p = 0; p < kAheadCol; ++p)
        next[p] = ahead(n_at + p * kCols + across, m_b + down);
#pragma unroll 1
      for (int h = 0; h < kTurnsCol; h += kAheadCol) {
#pragma unroll
        for (int p = 0; p < kAheadCol; ++p) {
          const int at = (h + p) * kCols + across;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            v[e] = ((MTA_LDS float *)chunk(down + e, at / 4))[at % 4];
          turned(n_at + at, m_b + down, v, next[p]);
          next[p] = ahead(n_at + at + kAheadCol * kCols, m_b + down);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Work item `w` of n, such that workgroups that run on one of the eight XCDs
// (blocks are dealt out in turn) take neighbouring ones.
__device__ __forceinline__ uint32_t beside(uint32_t w, uint32_t n) {
  const uint32_t x = w % 8, each = n / 8, more = n % 8;
  return x * each + min(x, more) + w / 8;
}

// Tile number t of rows x cols of them, down bands of eight rows.
__device__ __forceinline__ void banded(uint32_t t, uint32_t rows, uint32_t cols,
                                       uint32_t &row, uint32_t &col) {
  const uint32_t first = t / (8 * cols) * 8;
  const uint32_t height = min(8u, rows - first);
  const uint32_t u = t - first * cols;
  row = first + u % height;
  col = u / height;
}

// The tiles: the large one, whose workgroup fills a CU, the small one, of which
// a CU holds two, and the small one for launches that bring a CU no second one:
// four buffers, since there is nobody else to hide a load's way (768 x 768 over
// 768: 0.8 us a step of 64 with two).
using Tile256 = Tile<256, 256, 2, 4, 32, 4, 2>;
using Tile128 = Tile<128, 128, 2, 2, 64, 2, 2>;
using TileDeep = Tile<128, 128, 2, 2, 64, 4, 1>;
// For products that would leave CUs without a tile.
using Tile64 = Tile<64, 64, 2, 2, 64, 4, 2>;

}  // namespace mta
