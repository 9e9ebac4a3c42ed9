// Rotary positions: the tables of cosines and sines, and the rotation of fresh
// queries and keys by them.
//
// Tables: cos and sin of p theta_i for every position p.  Angles are counted in
// turns as 64-bit fractions (theta_i / 2 pi 2^64, see rope_turns.h), so p theta_i is
// one integer product whose overflow drops the whole turns: off by 2^-30 of angle
// at position 2^31 - 1, where a product in fp32 is off by whole radians at a million
// positions and fp64 runs at a sixtieth of the fp32 rate here.  What is left of the nearest quarter turn (at
// most an eighth of a turn) goes through two polynomials in its square, fitted
// at Chebyshev points (within 1e-7 of sin and cos after their fp32 roundings).
// Written once, 8 bytes a (position, pair).
//
// Rotation: x' = x C - y S, y' = y C + x S for the pairs (x, y), in fp32 with
// the order of kvc_compact_rerotate_quant and no fused multiply-add, rounded
// once to bf16.  Bound by the rows, read and written once.  A lane takes sixteen
// elements of a row in two 16-byte pieces (both halves of eight pairs, or eight
// interleaved pairs), reads their eight cosines and sines once and applies them
// to one head after another: the tables cost 1 / heads of a read per row.
//
// Measured: tables of 1,048,576 positions x 64 pairs 84 us = 6.4 TB/s, 95 % of
// the measured bandwidth; 32,768 tokens of 32 and 8 heads, d = 128, 107 us = 6.5
// TB/s, 95 %.
#include <algorithm>

#include "kvc_internal.cuh"
#include "packed_math.cuh"

namespace kvc {

namespace {

constexpr int kThreads = kRopeThreads;
constexpr int kBatch = 4;                        // heads of a thread whose loads are in flight together

// sin(2 pi t) = t S(t^2) and cos(2 pi t) = 1 + t^2 C(t^2) for |t| <= 1/8.
__device__ constexpr float kSin[4] = {6.2831854820251465f, -41.3416633605957f, 81.59254455566406f, -75.401611328125f};
__device__ constexpr float kCos[4] = {-19.739208221435547f, 64.93936920166016f, -85.44882202148438f, 59.42410659790039f};

// cos and sin of `turns` 2^-32 turns.
__device__ __forceinline__ float2 cos_sin(uint32_t turns) {
  const uint32_t quarter = (turns + 0x20000000u) >> 30;
  const float t = static_cast<float>(static_cast<int32_t>(turns - (quarter << 30))) * 0x1p-32f;
  const float u = t * t;
  const float s = t * fmaf(fmaf(fmaf(kSin[3], u, kSin[2]), u, kSin[1]), u, kSin[0]);
  const float c = fmaf(u, fmaf(fmaf(fmaf(kCos[3], u, kCos[2]), u, kCos[1]), u, kCos[0]), 1.f);
  const bool odd = quarter & 1;
  const float x = odd ? s : c, y = odd ? c : s;
  // quarter 1: (-sin, cos); 2: (-cos, -sin); 3: (sin, -cos)
  return make_float2(__uint_as_float(__float_as_uint(x) ^ (((quarter + 1) & 2) << 30)),
                     __uint_as_float(__float_as_uint(y) ^ ((quarter & 2) << 30)));
}

// One thread: four pairs of every position from its first on, `step` apart.
__global__ void __launch_bounds__(kThreads) rope_tables_kernel(const RopeTableArgs a) {
  wait_for_previous_kernel();
  let_next_kernel_start();
  const int groups = a.half / 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads / groups;
  const int g = static_cast<int>(id % groups);
  int64_t p = id / groups;
  if (p >= step) return;                           // threads behind the last whole position
  uint64_t f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = a.turns[4 * g + k];
  for (; p < a.max_pos; p += step) {
    float2 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // to the nearest 2^-32
      v[k] = cos_sin(static_cast<uint32_t>((f[k] * static_cast<uint64_t>(p) + 0x80000000ull) >> 32));
      v[k].x *= a.magnitude;
      v[k].y *= a.magnitude;
    }
    const int64_t at = p * a.half + 4 * g;
    *reinterpret_cast<float4*>(a.cos + at) = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
    *reinterpret_cast<float4*>(a.sin + at) = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
  }
}

__device__ __forceinline__ float bf16_at(const uint4& w, int i) {
  const uint32_t x = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
  return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
}

// The pair (x, y) turned by (c, s), each result rounded to bf16.
__device__ __forceinline__ void turn(float x, float y, float c, float s, float* x1, float* y1) {
  *x1 = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  *y1 = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// D: head dimension.  Block: a.tokens tokens (a power of two) times the heads
// that then fit, D / 16 lanes a row; blockIdx.y takes the heads in strides.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 16;
  const int lane = threadIdx.x % LPR, row = threadIdx.x / LPR;
  const int per_block = kThreads / LPR >> a.token_bits;            // heads side by side
  uint32_t block;
  const int bl = static_cast<int>(a.by_blocks.divmod(blockIdx.x, &block)), b = bl / a.L, l = bl - b * a.L;
  const int64_t token = (static_cast<int64_t>(block) << a.token_bits) + (row & ((1 << a.token_bits) - 1));
  wait_for_previous_kernel();
  let_next_kernel_start();
  if (token >= (a.n_rows ? clamp_count(a.n_rows[b], a.n) : a.n)) return;
  const int p = a.pos[static_cast<int64_t>(b) * a.n + token];
  const int h0 = blockIdx.y * per_block + (row >> a.token_bits), stride = gridDim.y * per_block;
  if (p < 0 || p >= a.max_pos) {
    if (a.unit_status && lane == 0)
      for (int h = h0; h < a.units; h += stride) a.unit_status[bl * a.units + h] = KVC_UNIT_BAD_INDEX;
    return;
  }
  const bool turned = lane * 16 < a.rotary_dim;
  if (!turned && a.in_place) return;
  float c[8], s[8];
  if (turned) {
    const int64_t at = static_cast<int64_t>(p) * (a.rotary_dim / 2) + lane * 8;
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const float4 x = *reinterpret_cast<const float4*>(a.cos + at + k), y = *reinterpret_cast<const float4*>(a.sin + at + k);
      c[k] = x.x, c[k + 1] = x.y, c[k + 2] = x.z, c[k + 3] = x.w;
      s[k] = y.x, s[k + 1] = y.y, s[k + 2] = y.z, s[k + 3] = y.w;
    }
    if (a.inverse) {
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] = -s[k];
    }
  }
  // this lane's two pieces of a row: the pairs' halves, or sixteen elements side by side
  const int first = turned && !PAIRS ? lane * 8 : lane * 16;
  const int second = turned && !PAIRS ? a.rotary_dim / 2 + lane * 8 : lane * 16 + 8;
  auto place = [&](const kvc_strides& st, int h) {
    return b * st.batch + l * st.layer + h * st.head + token * st.token;
  };
  // heads of the queries, then those of the keys
  const int heads = a.Hq + a.Hkv;
  for (int h = h0; h < heads; h += kBatch * stride) {
    uint4 w[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int hh = h + k * stride;
      if (hh < heads) {
        const __nv_bfloat16* x = hh < a.Hq ? a.q + place(a.qs, hh) : a.k + place(a.ks, hh - a.Hq);
        w[k][0] = *reinterpret_cast<const uint4*>(x + first);
        w[k][1] = *reinterpret_cast<const uint4*>(x + second);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int hh = h + k * stride;
      if (hh >= heads) break;
      if (turned) {
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = PAIRS ? bf16_at(w[k][i >> 2], 2 * i & 7) : bf16_at(w[k][0], i);
          const float v = PAIRS ? bf16_at(w[k][i >> 2], (2 * i & 7) + 1) : bf16_at(w[k][1], i);
          turn(u, v, c[i], s[i], &x[i], &y[i]);
        }
        if (PAIRS) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            w[k][e] = make_uint4(pack_bf16x2(x[4 * e], y[4 * e]), pack_bf16x2(x[4 * e + 1], y[4 * e + 1]),
                                 pack_bf16x2(x[4 * e + 2], y[4 * e + 2]), pack_bf16x2(x[4 * e + 3], y[4 * e + 3]));
        } else {
          w[k][0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
          w[k][1] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
      }
      __nv_bfloat16* o = hh < a.Hq ? a.q_out + place(a.qos, hh) : a.k_out + place(a.kos, hh - a.Hq);
      *reinterpret_cast<uint4*>(o + first) = w[k][0];
      *reinterpret_cast<uint4*>(o + second) = w[k][1];
    }
  }
}

}  // namespace

cudaError_t launch_rope_tables(const RopeTableArgs& a, int sms, cudaStream_t stream) {
  const int64_t threads = (a.max_pos * (a.half / 4) + kThreads - 1) / kThreads;
  const int64_t blocks = std::min<int64_t>(threads, 8LL * sms);
  return launch_after(rope_tables_kernel, dim3(static_cast<unsigned>(std::max<int64_t>(1, blocks))), kThreads, 0, stream, a);
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.by_blocks.d) * a.B * a.L, a.split);
  const bool pairs = a.layout == KVC_ROPE_INTERLEAVED;
  if (a.d == 128) return launch_after(pairs ? rope_kernel<128, true> : rope_kernel<128, false>, grid, kThreads, 0, stream, a);
  return launch_after(pairs ? rope_kernel<64, true> : rope_kernel<64, false>, grid, kThreads, 0, stream, a);
}

}  // namespace kvc
