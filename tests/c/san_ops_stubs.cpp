// san_ops_stubs.cpp -- the kernel launchers behind include/mta_ops.h, replaced
// for the host-only sanitizer build of ops_host.cpp
// (tests/test_ops_sanitizers.py).  The driver (san_ops.c) makes only calls
// that are refused or have no work; reaching a launcher is a failure.
#include <cstdio>
#include <cstdlib>

#include "../../mixed_precision_optimizer_mta_amd/csrc/ops_internal.h"

namespace mta {

[[noreturn]] static void reached(const char *what) {
  std::fprintf(stderr, "san_ops_stubs: %s reached in a host-only test\n",
               what);
  std::exit(3);
}

hipError_t launch_ckpt(int, int, int, const CkptList &, hipStream_t) {
  reached("launch_ckpt");
}
hipError_t launch_wgrad(const WgradArgs &, const WgradGrid &, hipStream_t) {
  reached("launch_wgrad");
}
hipError_t launch_policy(const mta_policy_args &, hipStream_t) {
  reached("launch_policy");
}
hipError_t launch_policy_backward(const mta_policy_args &, hipStream_t) {
  reached("launch_policy_backward");
}

}  // namespace mta

// Whether the weight gradient's grid covers its outputs and tokens once: all
// tiles, and for the cut ones parts of which none is empty and the last ends
// past the tokens.
extern "C" int san_wgrad_grid(int64_t tokens, int64_t fin, int64_t fout,
                              int type, int cus) {
  const mta::WgradGrid g = mta::wgrad_grid(tokens, fin, fout, type, cus);
  const int64_t t = mta::kWgradTile;
  if (g.tiles_o != (fout + t - 1) / t) return 1;
  if (g.tiles_i != (fin > 0 ? (fin + t - 1) / t : 1)) return 2;
  if (g.whole < 0 || g.cut < 0 || g.whole + g.cut != g.tiles_o * g.tiles_i)
    return 3;
  if (g.cut == 0 ? g.parts != 1 : g.parts < 2) return 4;
  if (g.part_tokens % mta::kWgradStep) return 5;
  if (g.cut && (g.parts * g.part_tokens < tokens ||
                (g.parts - 1) * g.part_tokens >= tokens))
    return 6;
  if (g.grouped && g.whole + g.cut * g.parts > cus) return 7;
  if (g.ranges < 0 || g.ranges > mta::kWgradRanges ||
      (g.ranges > 0) != (type == MTA_F16 && tokens > 0 && fin > 0))
    return 8;
  return 0;
}
