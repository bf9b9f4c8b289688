// ops_internal.h -- types shared by the host side and the gfx950 kernels of
// the operators of include/mta_ops.h.  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/mta_ops.h"
#include "mta_internal.h"

namespace mta {

// ---- 8-bit checkpoints --------------------------------------------------

constexpr int kCkptThreads = 256;
// Elements a lane handles at a time, 16 bytes: a wave's accesses are then one
// run of memory.
constexpr int ckpt_unit(int type) { return type == MTA_F32 ? 4 : 8; }
constexpr int kCkptUnroll = 4;  // units a lane has in flight, at most
constexpr int kCkptTensors = 32;  // tensors in one launch (they travel in the
                                  // kernel's arguments, 4 KiB at most)

// One tensor of a launch.  Its work is `units` runs of ckpt_unit columns, row
// by row and `row_units` to a row (whole blocks of them, so that the four or
// eight lanes of a scale's block never part).  A tensor whose rows follow each
// other without gaps and are whole blocks long is one row (flat).
struct CkptItem {
  const void *x;
  void *y;
  uint8_t *q;
  uint8_t *scale;
  int64_t ldx, ldy;
  uint64_t units;
  uint32_t cols;
  uint32_t row_units;  // 0: flat
  uint32_t chunk;      // units a workgroup handles at a time
};

struct CkptList {
  CkptItem item[kCkptTensors];
  uint32_t first[kCkptTensors + 1];  // first workgroup of each tensor; the
                                     // last entry is the grid
  uint32_t count;
};
static_assert(sizeof(CkptList) <= 4000, "kernel argument space");

enum CkptMode { kCkptPack = 0, kCkptUnpack = 1, kCkptBackward = 2 };

hipError_t launch_ckpt(int mode, int type, int act, const CkptList &list,
                       hipStream_t stream);

// ---- weight gradient from a checkpoint ----------------------------------

constexpr int kWgradTile = 128;  // outputs of a workgroup, each way
constexpr int kWgradStep = 32;   // tokens it takes at a time
constexpr int kWgradRanges = 256;  // answers about the values' range, at most

// Whether kept values of one scale are the same in float16: multiples of 2^-24
// of at most 65504 (their four significant bits always fit).  `steps` are their
// magnitudes in units of the scale's smallest code, 2^(scale - 127 - 9), or'ed:
// the lowest bit is the lowest of any, the highest the highest.
__host__ __device__ inline bool float16_holds(uint32_t scale, uint32_t steps) {
  if (steps == 0) return true;
  const int unit = static_cast<int>(scale) - 127 - 9;
  return unit + __builtin_ctz(steps) >= -24 &&
         unit + 31 - __builtin_clz(steps) <= 15;
}
// Scales with which it holds for every code: the smallest code is then 2^-24
// or more, the largest 57344 or less.
constexpr uint32_t kFloat16Scales[2] = {112, 134};

// The workgroups of a launch: `whole` tiles of the output over all tokens,
// then `cut` tiles in `parts` parts of `part_tokens` each.
struct WgradGrid {
  int64_t tiles_o, tiles_i;
  int64_t whole, cut;
  int64_t part_tokens;
  int parts;
  int ranges;  // workgroups that look at the kept values (float16 dy)
  int grouped;  // workgroups of as many waves as a CU holds
};

WgradGrid wgrad_grid(int64_t tokens, int64_t fin, int64_t fout, int type,
                     int cus);

struct WgradArgs {
  const uint8_t *q, *scale;
  const void *dy;
  void *dw, *db;
  float *part;     // [cut][parts][tile][tile]
  float *part_db;  // [parts][fout]
  int *range;      // [ranges]
  int64_t tokens, fin, fout, lddy, lddw;
  int64_t ldq;
  int type, gtype, accumulate;
};

hipError_t launch_wgrad(const WgradArgs &args, const WgradGrid &grid,
                        hipStream_t stream);

// ---- policy loss --------------------------------------------------------

static_assert(sizeof(mta_policy_row) == 16, "saved row layout");

// A row leaves its terms of the three sums in the workspace; more than
// kPolicyJoin rows are joined in stretches first.
constexpr int kPolicySums = 3;
constexpr int64_t kPolicyJoin = 4096;

hipError_t launch_policy(const mta_policy_args &args, hipStream_t stream);
hipError_t launch_policy_backward(const mta_policy_args &args,
                                  hipStream_t stream);

}  // namespace mta
