// Sums of squares at the scale of their largest entries.
#pragma once

#include "orth_kernel.cuh"

namespace specv {

__device__ __forceinline__ void squares_join(ScaledSquares& a, const ScaledSquares& b) {
  const float m = fmaxf(a.m, b.m), x = a.m / m, y = b.m / m;  // (powers of two)
  a.s = a.s * (x * x) + b.s * (y * y);
  a.m = m;
}
__device__ __forceinline__ ScaledSquares squares_shfl(const ScaledSquares& a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)};
}
__device__ __forceinline__ void squares_warp(ScaledSquares& a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) squares_join(a, squares_shfl(a, o));
}

// The sum over a CTA of 256 threads, in a fixed order, for all of them.
__device__ __forceinline__ void squares_cta(ScaledSquares& a, ScaledSquares (&warps)[8], ScaledSquares& sum) {
  squares_warp(a);
  if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = a;
  __syncthreads();
  if (threadIdx.x < 32) {
    ScaledSquares w = warps[threadIdx.x % 8];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) squares_join(w, squares_shfl(w, o));
    if (threadIdx.x == 0) sum = w;
  }
  __syncthreads();
}

constexpr float kSquaresLeast = 1.17549435e-38f;  // 2^-126

template <int VW>
__device__ __forceinline__ void squares_add(ScaledSquares& a, float& inv, const float (&x)[VW]) {
  float most = 0.f;
#pragma unroll
  for (int k = 0; k < VW; ++k) most = fmaxf(most, fabsf(x[k]));
  if (most >= 2.f * a.m) {
    // the power of two at or below it (infinity: its own, and the sum becomes NaN)
    const float m = __uint_as_float(__float_as_uint(most) & 0x7f800000u);
    const float f = a.m / m;  // (rarely: the first vector, and where entries double)
    a.s *= f * f;
    a.m = m;
    inv = 1.f / m;
  }
#pragma unroll
  for (int k = 0; k < VW; ++k) {
    const float y = x[k] * inv;
    a.s = fmaf(y, y, a.s);
  }
}

}  // namespace specv
