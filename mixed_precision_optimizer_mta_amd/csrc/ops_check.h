// ops_check.h -- what the operators' host sides check their arguments with.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "mta_internal.h"

namespace mta {
namespace check {

inline int fail(int code, const char *fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  return mta::report(code, msg);
}

inline int ok() { return mta::report(MTA_OK, ""); }

inline bool known_type(int t) {
  return t == MTA_F32 || t == MTA_BF16 || t == MTA_F16;
}

inline int64_t size_of(int type) { return type == MTA_F32 ? 4 : 2; }

inline bool aligned(const void *p, int64_t a) {
  return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(a - 1)) == 0;
}

// Sizes beyond this would overflow 64-bit byte offsets.
constexpr int64_t kMostBytes = int64_t{1} << 60;

// rows * pitch * size fits.
inline bool fits(int64_t rows, int64_t pitch, int64_t size) {
  return rows == 0 || pitch == 0 || rows <= kMostBytes / size / pitch;
}

// A buffer of `rows` runs of `width` bytes, `pitch` bytes apart.
struct Region {
  uintptr_t lo, hi;  // first byte, one past the last
  uintptr_t pitch, width;
  const char *name;
  int64_t tensor;  // of a list, or -1
  bool written;
  const void *pair;  // a buffer that this one may be, element for element
};

inline Region region(const void *p, int64_t rows, int64_t pitch, int64_t width,
              const char *name, int64_t tensor, bool written,
              const void *pair = nullptr) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  const uintptr_t bytes =
      rows > 0 && width > 0
          ? static_cast<uintptr_t>((rows - 1) * pitch + width)
          : 0;
  return Region{lo,     lo + bytes, static_cast<uintptr_t>(pitch),
                static_cast<uintptr_t>(width), name, tensor, written, pair};
}

// Whether two buffers share a byte.  Column slices of one wide buffer lie
// between each other's rows without doing so.
inline bool shares(const Region &a, const Region &b) {  // a.lo <= b.lo
  if (a.lo == a.hi || b.lo == b.hi || b.lo >= a.hi) return false;
  if (a.pitch != b.pitch || a.pitch == 0) return true;
  const uintptr_t d = (b.lo - a.lo) % a.pitch;
  return !(d >= a.width && d + b.width <= a.pitch);
}

inline int check_regions(std::vector<Region> *r) {
  std::sort(r->begin(), r->end(),
            [](const Region &a, const Region &b) { return a.lo < b.lo; });
  for (size_t i = 0; i < r->size(); ++i)
    for (size_t j = i + 1; j < r->size() && (*r)[j].lo < (*r)[i].hi; ++j) {
      const Region &a = (*r)[i], &b = (*r)[j];
      if (!a.written && !b.written) continue;
      // in place: the same elements of the same tensor
      if (a.lo == b.lo && a.hi == b.hi && a.pitch == b.pitch &&
          a.tensor == b.tensor &&
          (a.pair == reinterpret_cast<const void *>(b.lo) ||
           b.pair == reinterpret_cast<const void *>(a.lo)))
        continue;
      if (!shares(a, b)) continue;
      if (a.tensor < 0)
        return fail(MTA_EINVAL, "buffers overlap: %s and %s", a.name, b.name);
      return fail(MTA_EINVAL,
                  "buffers overlap: tensor %lld %s and tensor %lld %s",
                  static_cast<long long>(a.tensor), a.name,
                  static_cast<long long>(b.tensor), b.name);
    }
  return MTA_OK;
}

// Compute units of the current device.
inline int current_cus(int *cus) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e == hipSuccess)
    e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
  if (e != hipSuccess || *cus <= 0)
    return fail(MTA_EHIP, "cannot read the compute-unit count: %s",
                hipGetErrorString(e));
  return MTA_OK;
}

}  // namespace check
}  // namespace mta
