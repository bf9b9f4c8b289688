// ortho_device.h -- what the kernels of orthogonalised updates share: a launch's
// matrices, u from a gradient and its momentum, and where results go.
#pragma once

#include "matrix_internal.h"
#include "ops_device.h"

namespace mta {
namespace {

__device__ __forceinline__ float unscale_of(const OrthoCall &c) {
  return c.amp ? static_cast<float>(1.0 / static_cast<double>(c.amp->scale))
               : 1.0f;
}

__device__ __forceinline__ int item_of(const OrthoList &l, uint32_t block) {
  int k = 0;
  while (k + 1 < static_cast<int>(l.count) && block >= l.first[k + 1]) ++k;
  return k;
}

// Sum of a value of every lane of a workgroup of 256, in all of them.
__device__ __forceinline__ double sum256(double x, double *four) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d);
  __syncthreads();
  if (threadIdx.x % 64 == 0) four[threadIdx.x / 64] = x;
  __syncthreads();
  return (four[0] + four[1]) + (four[2] + four[3]);
}

// g' and, with a momentum, its new value and u.
struct Look {
  float s, c, mu;
  int nesterov;
  __device__ __forceinline__ float gradient(float g) const {
    return (g * s) * c;
  }
  __device__ __forceinline__ float next(float m, float g) const {
    return m * mu + g;
  }
  __device__ __forceinline__ float ahead(float m, float g) const {
    return nesterov ? g + mu * m : m;
  }
};
__device__ __forceinline__ Look look_of(const OrthoCall &c) {
  return Look{unscale_of(c), c.d_coef ? *c.d_coef : 1.0f, c.mu, c.nesterov};
}

// X of a matrix whose norm is far below eps begins far below 1, where float16
// values have few digits: it is kept times 2^n, with n the most that leaves
// singular values below 1 until they have grown by `grown`.  0 for any other
// matrix (and for NaN).
__device__ __forceinline__ int lift_of(float norm, float grown) {
  const float x = norm * grown;
  if (!(x > 0.0f && x < 1.0f)) return 0;
  int e;
  frexpf(x, &e);
  return min(-e, 100);
}

// Eight results of a row: out, and the weights' step.
__device__ __forceinline__ void put_result(const OrthoItem &it,
                                           const OrthoCall &c, int64_t row,
                                           int64_t col, const float (&x)[8],
                                           bool skip) {
  if (row >= it.rows || col >= it.cols) return;
  const int n = static_cast<int>(min(int64_t{8}, it.cols - col));
  float y[8];
  if (it.out) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e] * it.scale;
    with_type(c.out_type, [&](auto type) {
      constexpr int T = decltype(type)::value;
      if (n == 8) {
        store8<T, false>(it.out, row * it.ldout + col, y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < n) store_elem<T>(it.out, row * it.ldout + col + e, y[e]);
      }
    });
  }
  if (it.w && !skip) {
    const int64_t at = row * it.cols + col;
    const Raw8<MTA_F32> w = n == 8 ? load8<MTA_F32, false>(it.w, at)
                                   : load8_part<MTA_F32>(it.w, at, n, 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = w[e] * c.decay + it.update * x[e];
    if (n == 8) {
      store8<MTA_F32, false>(it.w, at, y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) it.w[at + e] = y[e];
    }
    if (it.w16) {
      with_type(c.copy_type, [&](auto type) {
        constexpr int T = decltype(type)::value;
        if (n == 8) {
          store8<T, false>(it.w16, at, y);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < n) store_elem<T>(it.w16, at + e, y[e]);
        }
      });
    }
  }
}

}  // namespace
}  // namespace mta
