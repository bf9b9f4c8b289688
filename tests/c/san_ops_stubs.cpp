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
