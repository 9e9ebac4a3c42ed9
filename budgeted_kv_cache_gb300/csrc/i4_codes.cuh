// Rows of a 4-bit cache: quantised, dequantised, and as operands of matrix
// instructions.
#pragma once

#include "kvc_internal.cuh"
#include "packed_math.cuh"

namespace kvc {

constexpr unsigned kFull = 0xffffffffu;

// Quantises the 8 elements of this lane (`LANES` adjacent lanes share a
// scale): packed codes, and the scale's bits.
//   scale = max / 7 rounded to the scale's format, code = rint(x / scale).
// Both quotients are q0 = x y, q = q0 + (x - q0 b) y (Markstein) with y within
// one ulp of 1 / b.  The codes equal those of IEEE division: checked for every
// bf16 mantissa against every bf16 and fp16 scale mantissa with y one ulp off
// either way; and so does the rounded scale, because a / 7 for a bf16 a is
// never within an ulp of a tie of either format (checked for every a).  rint
// is an addition of 1.5 x 2^23 (a conversion to integer runs at a quarter of
// the rate); the eight sums, 8 larger than their codes, are packed by shifted
// additions and the offset is taken out at the end.  Everything but the
// packing works on two elements per instruction.
// Scales that are subnormal or clipped (where the quotient may exceed 7.5)
// take the slow way.
template <bool ROW, int LANES>
__device__ __forceinline__ uint32_t quantise8(const uint4& w, uint16_t* bits) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
  __nv_bfloat162 mx = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&r[0]));
#pragma unroll
  for (int i = 1; i < 4; ++i) mx = __hmax2(mx, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&r[i])));
  float amax = fmaxf(__low2float(mx), __high2float(mx));
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  float sc = div_by_recip(amax, 7.f, 0x1.24924ap-3f);       // the reciprocal of 7, rounded
  uint16_t sb;
  if (ROW) {
    sb = __half_as_ushort(__float2half_rn(sc));
    sc = __half2float(__ushort_as_half(sb));
  } else {
    sb = float_to_bf16_bits(sc);
    sc = bf16_bits_to_float(sb);
  }
  if (!(amax > 0.f)) {                           // a group of zeros: codes 0, scale 1
    sc = 1.f;
    sb = ROW ? 0x3c00 : 0x3f80;
  }
  const bool fast = ROW ? sc >= 0x1p-14f && sc < 65504.f : recip_div_ok(sc);
  if (__all_sync(kFull, fast)) {
    const float y = rcp_approx(sc);
    const uint64_t y2 = pair(y, y), nb2 = pair(-sc, -sc), round2 = pair(12582920.f, 12582920.f);
    uint32_t pk = 0u - 0x3f400000u;                          // the exponents' part of the sum below
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x2 = pair(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
      const uint64_t q0 = mul2(x2, y2);
      float lo, hi;
      unpair(add2(fma2(fma2(q0, nb2, x2), y2, q0), round2), &lo, &hi);
      pk += (__float_as_uint(lo) << (8 * i)) + (__float_as_uint(hi) << (8 * i + 4));
    }
    *bits = sb;
    return pk ^ 0x88888888u;
  }
  sc = 1.f;
  if (amax > 0.f) {
    const float s = __fdiv_rn(amax, 7.f);
    if (ROW) sc = fmaxf(fminf(__half2float(__float2half_rn(s)), 65504.f), 0x1p-24f);
    else sc = fmaxf(bf16_bits_to_float(float_to_bf16_bits(s)), __uint_as_float(0x00010000u));   // 2^-133
  }
  *bits = ROW ? __half_as_ushort(__float2half_rn(sc)) : float_to_bf16_bits(sc);
  uint32_t pk = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(i & 1 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
    const int q = max(-7, min(7, amax > 0.f ? __float2int_rn(__fdiv_rn(x, sc)) : 0));
    pk |= static_cast<uint32_t>(q & 0xf) << (4 * i);
  }
  return pk;
}

// The 8 codes of a word times their scale, as bf16 in element order, each
// rounded once: codes are exact in bf16 (136 + code - 136), a bf16 scale
// multiplies them in bf16, an fp16 scale in fp32.
__device__ __forceinline__ uint4 dequantise8(uint32_t w, uint16_t scale, bool row_mode) {
  uint32_t c[4];                                 // elements (0,4), (1,5), (2,6), (3,7)
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = ((w >> (4 * k)) & 0x000f000fu) ^ 0x43084308u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(c[k]) : "r"(x), "r"(0x43084308u));
  }
  if (row_mode) {
    const float s = __half2float(__ushort_as_half(scale));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(c[k] << 16) * s, __uint_as_float(c[k] & 0xffff0000u) * s);
      c[k] = *reinterpret_cast<const uint32_t*>(&p);
    }
  } else {
    const uint32_t s2 = scale * 0x10001u;
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(c[k]) : "r"(s2));
  }
  return make_uint4(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410), __byte_perm(c[0], c[1], 0x7632),
                    __byte_perm(c[2], c[3], 0x7632));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D (16 x 8) += A (16 x 16) B (16 x 8), bf16 in, fp32 out.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The codes in bits 0..3 and 16..19 of w as a bf16 pair.
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43084308, 0x6a;" : "=r"(r) : "r"(w));      // (w & mask) ^ magic
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0x43084308u));
  return r;
}

// Scales of one key times `by`, as fp32.
__device__ __forceinline__ void put_scales(float* to, uint2 s, float by) {
  *reinterpret_cast<float4*>(to) =
      make_float4(__uint_as_float(s.x << 16) * by, __uint_as_float(s.x & 0xffff0000u) * by, __uint_as_float(s.y << 16) * by,
                  __uint_as_float(s.y & 0xffff0000u) * by);
}
__device__ __forceinline__ void put_scales(float* to, uint32_t s, float by) {
  *reinterpret_cast<float2*>(to) = make_float2(__uint_as_float(s << 16) * by, __uint_as_float(s & 0xffff0000u) * by);
}
__device__ __forceinline__ void put_scales(float* to, uint16_t s, float by) { *to = __half2float(__ushort_as_half(s)) * by; }

}  // namespace kvc
