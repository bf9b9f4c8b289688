// san_matrix_stubs.cpp -- the kernel launchers behind include/mta_matrix.h,
// replaced for the host-only sanitizer build of matrix_host.cpp
// (tests/test_matrix_sanitizers.py).  The driver (san_matrix.c) makes only
// calls that are refused or have no work; reaching a launcher is a failure.
#include <cstdio>
#include <cstdlib>

#include "../../mixed_precision_optimizer_mta_amd/csrc/matrix_internal.h"

namespace mta {

[[noreturn]] static void reached(const char *what) {
  std::fprintf(stderr, "san_matrix_stubs: %s reached in a host-only test\n",
               what);
  std::exit(3);
}

hipError_t launch_ortho_join(const OrthoList &, const OrthoCall &,
                             hipStream_t) {
  reached("launch_ortho_join");
}
hipError_t launch_ortho_norm(const OrthoList &, const OrthoCall &,
                             hipStream_t) {
  reached("launch_ortho_norm");
}
hipError_t launch_ortho_load(const OrthoList &, const OrthoCall &,
                             hipStream_t) {
  reached("launch_ortho_load");
}
hipError_t launch_ortho_small_gram(const OrthoList &, const OrthoCall &,
                                   hipStream_t) {
  reached("launch_ortho_small_gram");
}
hipError_t launch_ortho_small_factor(const OrthoList &, const OrthoCall &,
                                     const OrthoCoefficients &, hipStream_t) {
  reached("launch_ortho_small_factor");
}
hipError_t launch_ortho_small_apply(const OrthoList &, const OrthoCall &,
                                    hipStream_t) {
  reached("launch_ortho_small_apply");
}
hipError_t launch_ortho_product(int, int, bool, const OrthoList &,
                                const OrthoCall &, hipStream_t) {
  reached("launch_ortho_product");
}
hipError_t launch_linear_rows_in(const LinearArgs &, hipStream_t) {
  reached("launch_linear_rows_in");
}
hipError_t launch_linear_info(const LinearArgs &, hipStream_t) {
  reached("launch_linear_info");
}
hipError_t launch_linear_pack_w(const LinearArgs &, uint16_t *, hipStream_t) {
  reached("launch_linear_pack_w");
}
hipError_t launch_linear_logits(const LinearArgs &, int, hipStream_t) {
  reached("launch_linear_logits");
}
hipError_t launch_linear_rows(const LinearArgs &, hipStream_t) {
  reached("launch_linear_rows");
}
hipError_t launch_linear_back(const LinearArgs &, int, const LinearPiece *,
                              const LinearPiece *, LinearBack, hipStream_t) {
  reached("launch_linear_back");
}
hipError_t launch_linear_none(const LinearArgs &, hipStream_t) {
  reached("launch_linear_none");
}
hipError_t launch_linear_out(const LinearArgs &, const LinearPiece &, bool,
                             int, hipStream_t) {
  reached("launch_linear_out");
}

}  // namespace mta
