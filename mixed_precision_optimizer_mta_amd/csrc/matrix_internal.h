// matrix_internal.h -- types shared by the host side and the gfx950 kernels of
// the operators of include/mta_matrix.h.  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/mta_matrix.h"
#include "mta_internal.h"

namespace mta {

// Elements between the rows of a plane of n columns: whole steps of 64, and
// not a multiple of 1024, whose rows would lie in few of the memory's channels.
__host__ __device__ constexpr int64_t plane_pitch(int64_t n) {
  const int64_t p = (n + 63) / 64 * 64;
  return p % 1024 == 0 ? p + 64 : p;
}

// Products of planes that make one product: all but those of the smallest.
__host__ __device__ constexpr int pair_count(int planes) {
  return planes == 1 ? 1 : planes == 2 ? 3 : 6;
}

// ---- orthogonalised updates ---------------------------------------------

constexpr int kOrthoItems = 40;  // matrices of a launch (they travel in the
                                 // kernel's arguments, 4 KiB at most)
constexpr int kOrthoParts = 256;  // workgroups that sum a matrix's squares

// One matrix of a launch.  Its iterate X is [small, large].
struct OrthoItem {
  const void *g;
  float *m;
  void *out;
  float *w;
  void *w16;
  uint8_t *ws;
  int64_t ldg, ldout;
  uint32_t rows, cols;
  float scale;   // of out
  float update;  // -lr scale, of w
};

struct OrthoList {
  OrthoItem item[kOrthoItems];
  uint32_t first[kOrthoItems + 1];  // first workgroup of each matrix; the
                                    // entry behind the last one is the grid
  uint32_t count;
};

// What all launches of a call share.
struct OrthoCall {
  const float *d_coef;
  const mta_amp_state *amp;
  double eps;
  float mu;
  float decay;  // of w
  // a product of two symmetric matrices: e0 P Q + e1 P + e2, of the buffers
  // number p, q and out
  float e0, e1, e2;
  int p, q, out;
  // X from buffer `out`; what is left of X behind its first plane is multiplied
  // by its diagonal too (whole), or by `rest`
  float rest;
  int type, out_type, copy_type, nesterov;
  int planes;   // of a product's operands: 2 with `precise`
  int cuts;     // parts of k that A is summed in
  int whole;
  int which;    // the X that is read; the other one is written
  int steps_of;  // e0 and e1 are those of a polynomial of A
  // What singular values grow by, at most, to the end of this product's steps
  // and to the end of the next ones' (0: X is handed out)
  float grown, grows;
};
static_assert(sizeof(OrthoList) + sizeof(OrthoCall) +
                      sizeof(double) * 3 * MTA_ORTHO_STEPS + 8 <=
                  4096,
              "kernel argument space");

// Up to so many rows or columns a matrix takes the way of the small: its Gram
// matrix and the polynomial of it in float64.
constexpr int kOrthoSmall = 64;
__host__ __device__ inline bool ortho_is_small(int64_t rows, int64_t cols) {
  return rows <= kOrthoSmall || cols <= kOrthoSmall;
}

// A small matrix's part of the workspace: partial Gram matrices of `side` rows,
// whole blocks of 16, and the polynomial's factor.
struct OrthoSmallSpace {
  int64_t small, large;
  int side, parts;
  int64_t bytes;
};
__host__ __device__ inline OrthoSmallSpace ortho_small_space(int64_t rows,
                                                             int64_t cols) {
  OrthoSmallSpace s;
  s.small = rows < cols ? rows : cols;
  s.large = rows < cols ? cols : rows;
  s.side = static_cast<int>((s.small + 15) / 16 * 16);
  // 64 columns at a time; few enough parts for one workgroup to read
  const int64_t tiles = (s.large + 63) / 64;
  const int64_t most = s.side > 32 ? 32 : 64;
  s.parts = static_cast<int>(tiles < most ? tiles : most);
  s.bytes = (s.parts + 1) * static_cast<int64_t>(s.side) * s.side * 8;
  return s;
}

// A matrix's part of the workspace: two X of two planes each, three symmetric
// matrices of `planes` planes, their diagonals, the partial sums of squares and
// the first X's norm, a float.
constexpr int kOrthoSquares = 3;
struct OrthoSpace {
  int64_t small, large, pitch_x, pitch_a;
  int64_t plane_x, plane_a;          // elements
  // offsets in bytes, and from the first to the next
  int64_t x, next_x, a, next_a, diag, next_diag, part, norm, bytes;
  int64_t cut;  // partial sums of A: [cuts][small][pitch_a] floats
};
__host__ __device__ inline OrthoSpace ortho_space(int64_t rows, int64_t cols,
                                                  int planes, int cuts) {
  OrthoSpace s;
  s.small = rows < cols ? rows : cols;
  s.large = rows < cols ? cols : rows;
  s.pitch_x = plane_pitch(s.large);
  s.pitch_a = plane_pitch(s.small);
  s.plane_x = s.small * s.pitch_x;
  s.plane_a = s.small * s.pitch_a;
  const auto round = [](int64_t x) { return (x + 255) / 256 * 256; };
  s.x = 0;
  s.next_x = round(s.plane_x * 2 * 2);
  s.a = s.x + 2 * s.next_x;
  s.next_a = round(s.plane_a * planes * 2);
  s.diag = s.a + kOrthoSquares * s.next_a;
  s.next_diag = round(s.pitch_a * 4);  // zeros behind the last
  s.part = s.diag + kOrthoSquares * s.next_diag;
  s.norm = s.part + kOrthoParts * 8;
  s.cut = s.norm + 256;
  s.bytes = s.cut + (cuts > 1 ? round(cuts * s.plane_a * 4) : 0);
  return s;
}

// The tiles of a product's workgroups, and those of the kernels before it.
// After a Gram product in parts: 64 x 64 of A, and what mirrors it.
hipError_t launch_ortho_join(const OrthoList &l, const OrthoCall &c,
                             hipStream_t s);
enum OrthoStep { kOrthoGram, kOrthoTimes, kOrthoNext, kOrthoLast };
constexpr int kOrthoLoadTile = 64;
// Workgroups that sum a matrix's squares: 64 elements a lane, as long as they
// are few enough for one read of their sums by every workgroup that follows.
__host__ __device__ inline int64_t ortho_parts(int64_t rows, int64_t cols) {
  const int64_t n = (rows * cols + 16383) / 16384;
  return n < 1 ? 1 : n < kOrthoParts ? n : kOrthoParts;
}
hipError_t launch_ortho_norm(const OrthoList &l, const OrthoCall &c,
                             hipStream_t s);
hipError_t launch_ortho_load(const OrthoList &l, const OrthoCall &c,
                             hipStream_t s);
hipError_t launch_ortho_small_gram(const OrthoList &l, const OrthoCall &c,
                                   hipStream_t s);
// coefficients: a, b, c of each step
struct OrthoCoefficients {
  double v[MTA_ORTHO_STEPS][3];
  int steps;
};
hipError_t launch_ortho_small_factor(const OrthoList &l, const OrthoCall &c,
                                     const OrthoCoefficients &k, hipStream_t s);
hipError_t launch_ortho_small_apply(const OrthoList &l, const OrthoCall &c,
                                    hipStream_t s);
// tile: 256, 128 or 64; deep: no CU gets a second workgroup
hipError_t launch_ortho_product(int step, int tile, bool deep,
                                const OrthoList &l,
                                const OrthoCall &c, hipStream_t s);

// ---- cross entropy of a linear output layer -----------------------------

static_assert(sizeof(mta_linear_row) == 16, "saved row layout");

// The course of a call.
struct LinearPlan {
  int planes;
  bool copy_w;          // w does not lie as the products want it
  int64_t pitch;        // of h's and w's planes
  int64_t piece;        // columns of the vocabulary at a time, all but the last
  int64_t pieces;
  int64_t pitch_z;      // of dz
  int64_t deep_rows;    // rows of dz, at most: whole steps of 64
  int tile;             // of the forward's product
  int back_tile;        // of the others
  int dh_parts, dw_parts;  // of k, whose sums are joined
  bool hold_dh, hold_dw;  // sums held in the workspace before they go out
  // offsets in the workspace
  int64_t active, scalars, terms, rows, index, info, z_target, partial, h, w,
      z[2], sum_h, sum_w, bytes;
};

// What dz takes of a row, besides the factor that all rows share.
struct LinearInfo {
  float shift;  // of its exponentials
  float each;   // weight / total
  float own;    // the target's value
  int target;   // -1: none
};

// Rows that take part come first, in order, in h, z_target, partial, terms, info
// and dz: index[] says which they are, *active how many.
struct LinearArgs {
  mta_linear_loss_args a;
  mta_linear_row *rows;   // of the workspace or the caller's
  int *active;
  int *index;             // [rows]
  LinearInfo *info;       // [deep_rows]
  float *scalars;         // [0] weight of a row without weights, [1] largest
                          // finite one
  double *terms;          // [rows] of the loss
  float *z_target;        // [rows]
  float2 *partial;        // [tiles][rows]: largest, sum without the target
  uint16_t *h;            // planes
  const uint16_t *w;
  float *sum_h, *sum_w;   // [parts][rows or piece][pitch]
  int64_t h_plane, w_plane, w_pitch, z_plane;
  int64_t pitch, pitch_z;
  int64_t tiles;          // of the vocabulary
  int planes;
  int backward;           // rows are the caller's, and say what is left out
};

// A piece of the vocabulary, and its dz.
struct LinearPiece {
  int64_t first, count;
  uint16_t *z;  // planes
};

// The parts of dh's and dw's sums, whether they are held in the workspace, and
// the first workgroups of dw and of dz.
struct LinearBack {
  int dh_parts, dw_parts, hold_dh, hold_dw;
  uint32_t first_dw, first_dz;
};

// the rows that take part, and h's planes
hipError_t launch_linear_rows_in(const LinearArgs &l, hipStream_t s);
hipError_t launch_linear_info(const LinearArgs &l, hipStream_t s);
hipError_t launch_linear_pack_w(const LinearArgs &l, uint16_t *to,
                                hipStream_t s);
hipError_t launch_linear_logits(const LinearArgs &l, int tile, hipStream_t s);
hipError_t launch_linear_rows(const LinearArgs &l, hipStream_t s);
// dh and dw of `piece` and dz of `next`, either of which may be null.  Held dh is
// added to what is there after the first piece.
hipError_t launch_linear_back(const LinearArgs &l, int tile,
                              const LinearPiece *piece,
                              const LinearPiece *next, LinearBack back,
                              hipStream_t s);
// dw of no rows
hipError_t launch_linear_none(const LinearArgs &l, hipStream_t s);
// what is held, out
hipError_t launch_linear_out(const LinearArgs &l, const LinearPiece &piece,
                             bool dh, int parts, hipStream_t s);

}  // namespace mta
