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

// tanh(z) / z for |z| <= kTanhRange as a polynomial of degree 4 in z^2, fitted
// at Chebyshev points: tanh within 1.2e-7 (and 2.2e-7 of its value).
constexpr float kTanhRange = 0.625f;
__device__ constexpr float kTanh[5] = {0.9999998807907104f, -0.3333197236061096f, 0.13304771482944489f, -0.05183185636997223f,
                                       0.015063672326505184f};

__device__ __forceinline__ float tanh_over_z(float z) {
  const float u = z * z;
  float r = kTanh[4];
#pragma unroll
  for (int k = 3; k >= 0; --k) r = fmaf(r, u, kTanh[k]);
  return r;
}

// Base-2 cap tanh(x / cap) of one score x, z = x / cap: the polynomial where z
// is small, else cap (1 - 2 / (1 + e^2z)), which is off by about 2^-21 cap.
// That is coarse beside scores far below a cap of more than kFineCap, so tiles
// under such caps choose score by score and not as a whole.
constexpr float kFineCap = 1024.f;

__device__ __forceinline__ float capped_base2(float x, float z, float cap) {
  constexpr float kLog2e = 1.4426950408889634f;
  const float far = fmaf(-2.f * cap, rcp_approx(1.f + ex2_approx(z * (2.f * kLog2e))), cap);
  return (fabsf(z) <= kTanhRange ? x * tanh_over_z(z) : far) * kLog2e;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace kvc
