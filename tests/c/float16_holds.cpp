// float16_holds.cpp -- float16_holds of ops_internal.h for every scale and code,
// and every pair of codes, against its definition: the values survive a rounding
// to float16.  Exits 0 and prints "same" when all agree.
#include <cmath>
#include <cstdio>

#include "../../mixed_precision_optimizer_mta_amd/csrc/ops_internal.h"

// x rounded to float16's grid: eleven significant bits, steps of 2^-24 at
// least, infinity past 65504.
static double to_float16(double x) {
  if (x == 0.0) return x;
  int e;
  std::frexp(x, &e);  // x = f 2^e, 1/2 <= |f| < 1
  const double step = std::ldexp(1.0, e - 11 < -24 ? -24 : e - 11);
  const double y = std::nearbyint(x / step) * step;
  return std::fabs(y) > 65504.0 ? std::copysign(INFINITY, x) : y;
}

int main() {
  int held = 0;
  for (unsigned scale = 0; scale < 256; ++scale) {
    bool want[127];
    uint32_t steps[127];
    for (int m = 0; m < 127; ++m) {
      const double v =
          m < 8 ? std::ldexp(m, -9) : std::ldexp(8 + m % 8, m / 8 - 10);
      const double x = std::ldexp(v, static_cast<int>(scale) - 127);
      want[m] = to_float16(x) == x;
      steps[m] = static_cast<uint32_t>(v * 512.0);
      held += want[m];
      if (scale >= mta::kFloat16Scales[0] && scale <= mta::kFloat16Scales[1] &&
          !want[m])
        return 2;
    }
    for (int a = 0; a < 127; ++a)
      for (int b = 0; b < 127; ++b)
        if (mta::float16_holds(scale, steps[a] | steps[b]) !=
            (want[a] && want[b])) {
          std::fprintf(stderr, "scale %u codes %d and %d\n", scale, a, b);
          return 1;
        }
  }
  std::printf("same %d\n", held);
  return 0;
}
