// ops_device.h -- device helpers of the operators of include/mta_ops.h:
// element types, wide loads and stores at any element's address, and the
// 8-bit checkpoint's codes.
#pragma once

#include <type_traits>

#include "ops_internal.h"

namespace mta {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

#define MTA_GLOBAL __attribute__((address_space(1)))

template <int D>
using elem = typename std::conditional<D == MTA_F32, float, uint16_t>::type;

// float32 of a 16-bit element in the low half of h, exact.
template <int D>
__device__ __forceinline__ float widen(uint32_t h) {
  if constexpr (D == MTA_BF16) return __uint_as_float(h << 16);
  else
    return static_cast<float>(
        __builtin_bit_cast(_Float16, static_cast<uint16_t>(h)));
}

// Two float32 to two 16-bit elements in one word, each rounded to
// nearest-even (a NaN stays a NaN).
template <int D>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if constexpr (D == MTA_BF16) {
    const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    const f16x2 v = {static_cast<_Float16>(lo), static_cast<_Float16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
  }
}

template <int D>
__device__ __forceinline__ elem<D> narrow(float x) {
  if constexpr (D == MTA_F32) return x;
  else return static_cast<uint16_t>(narrow2<D>(x, x));
}

template <int D>
__device__ __forceinline__ float load_elem(const void *p, int64_t i) {
  const auto v = ((const MTA_GLOBAL elem<D> *)p)[i];
  if constexpr (D == MTA_F32) return v;
  else return widen<D>(v);
}

template <int D>
__device__ __forceinline__ void store_elem(void *p, int64_t i, float x) {
  ((MTA_GLOBAL elem<D> *)p)[i] = narrow<D>(x);
}

// N consecutive elements as they lie in memory, in words of 16 bytes.
template <int D, int N>
struct Raw {
  static constexpr int kWords = D == MTA_F32 ? N : N / 2;
  static_assert(kWords % 4 == 0, "whole 16-byte accesses");
  uint32_t w[kWords];

  __device__ __forceinline__ float operator[](int k) const {
    if constexpr (D == MTA_F32) return __uint_as_float(w[k]);
    else if constexpr (D == MTA_BF16)
      return __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
    else return widen<D>((k & 1 ? w[k / 2] >> 16 : w[k / 2]) & 0xFFFFu);
  }
};

template <int D>
using Raw8 = Raw<D, 8>;

// A 16-byte access at an element's address.  gfx950 serves it at any
// alignment in one instruction, so rows of odd lengths need no element path.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
template <int D>
struct Wide {
  typedef u32x4_at2 type;
};
template <>
struct Wide<MTA_F32> {
  typedef u32x4_at4 type;
};

template <int D, int N, bool Stream>
__device__ __forceinline__ Raw<D, N> load(const void *p, int64_t i) {
  const auto *a =
      (const MTA_GLOBAL typename Wide<D>::type *)((const MTA_GLOBAL elem<D> *)p +
                                                  i);
  Raw<D, N> r;
#pragma unroll
  for (int h = 0; h < Raw<D, N>::kWords / 4; ++h) {
    const u32x4 v = Stream ? __builtin_nontemporal_load(a + h) : a[h];
#pragma unroll
    for (int k = 0; k < 4; ++k) r.w[4 * h + k] = v[k];
  }
  return r;
}

// The first n (below N) of N elements; the rest are `fill`.
template <int D, int N>
__device__ __forceinline__ Raw<D, N> load_part(const void *p, int64_t i, int n,
                                               uint32_t fill) {
  Raw<D, N> r;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t v = fill;
    if (k < n) {
      const auto e = ((const MTA_GLOBAL elem<D> *)p)[i + k];
      if constexpr (D == MTA_F32) v = __float_as_uint(e);
      else v = e;
    }
    if constexpr (D == MTA_F32) r.w[k] = v;
    else if (k & 1) r.w[k / 2] |= v << 16;
    else r.w[k / 2] = v;
  }
  return r;
}

// Eight times the element with bits `v`.
template <int D>
__device__ __forceinline__ Raw8<D> fill8(uint32_t v) {
  Raw8<D> r;
#pragma unroll
  for (int k = 0; k < Raw8<D>::kWords; ++k)
    r.w[k] = D == MTA_F32 ? v : v | v << 16;
  return r;
}

template <int D, int N, bool Stream>
__device__ __forceinline__ void store(void *p, int64_t i, const float (&x)[N]) {
  auto *a = (MTA_GLOBAL typename Wide<D>::type *)((MTA_GLOBAL elem<D> *)p + i);
#pragma unroll
  for (int h = 0; h < Raw<D, N>::kWords / 4; ++h) {
    u32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (D == MTA_F32) v[k] = __float_as_uint(x[4 * h + k]);
      else v[k] = narrow2<D>(x[2 * k], x[2 * k + 1]);
    }
    if constexpr (Stream) __builtin_nontemporal_store(v, a + h);
    else a[h] = v;
  }
}

// The same of eight elements.
template <int D, bool Stream>
__device__ __forceinline__ Raw8<D> load8(const void *p, int64_t i) {
  return load<D, 8, Stream>(p, i);
}
template <int D>
__device__ __forceinline__ Raw8<D> load8_part(const void *p, int64_t i, int n,
                                              uint32_t fill) {
  return load_part<D, 8>(p, i, n, fill);
}
template <int D, bool Stream>
__device__ __forceinline__ void store8(void *p, int64_t i,
                                       const float (&x)[8]) {
  store<D, 8, Stream>(p, i, x);
}

// Calls f(std::integral_constant<int, T>) for the run-time element type.
template <typename F>
__host__ __device__ __forceinline__ auto with_type(int type, F &&f) {
  switch (type) {
    case MTA_BF16: return f(std::integral_constant<int, MTA_BF16>{});
    case MTA_F16: return f(std::integral_constant<int, MTA_F16>{});
    default: return f(std::integral_constant<int, MTA_F32>{});
  }
}

}  // namespace mta
