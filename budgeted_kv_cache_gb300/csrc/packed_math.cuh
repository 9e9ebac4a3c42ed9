// Packed fp32 arithmetic and small functions shared by the 4-bit cache and the
// prompt attention.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ void unpair(uint64_t v, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(z) / z for |z| <= 1 as a polynomial of degree 6 in z^2, fitted at
// Chebyshev points: tanh within 1.8e-7 of its value.
__device__ constexpr float kTanh[7] = {0.9999999403953552f,  -0.33332857489585876f, 0.13325397670269012f, -0.05346517637372017f,
                                       0.020305519923567772f, -0.006217069923877716f, 0.0010455535957589746f};

// Two values from u = z^2.
__device__ __forceinline__ uint64_t tanh_over_z(uint64_t u) {
  uint64_t r = pair(kTanh[6], kTanh[6]);
#pragma unroll
  for (int k = 5; k >= 0; --k) r = fma2(r, u, pair(kTanh[k], kTanh[k]));
  return r;
}

// One value from z.
__device__ __forceinline__ float poly_tanh_over_z(float z) {
  const float u = z * z;
  float r = kTanh[6];
#pragma unroll
  for (int k = 5; k >= 0; --k) r = fmaf(r, u, kTanh[k]);
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace kvc
