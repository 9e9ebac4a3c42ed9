// Score modifiers and visibility of the prompt attention and the 4-bit
// attention, and a plain tiled attention over any key source.
#pragma once

#include <math.h>

#include "kvc_internal.cuh"

namespace kvc {

// x = (q . k) * scale -> capped and biased logit.
__device__ __forceinline__ float mod_score(float x, float softcap, float slope, float dist) {
  if (softcap > 0.f) x = softcap * tanhf(x / softcap);
  return x - slope * fabsf(dist);
}

__device__ __forceinline__ bool sees(int64_t p_q, int64_t p_k, int window, int64_t prefix) {
  return p_k < prefix || (p_k <= p_q && (window == 0 || p_q - p_k < window));
}

constexpr int kPlainRows = 16, kPlainKeys = 64, kPlainThreads = 128;

// One block: kPlainRows packed rows (row = query * G + head of the group) of
// one unit over all its keys, fp32 throughout.  Src supplies, for a unit and
// a block of rows: rows(), keys(), query(r), key / value elements, positions
// and visibility.  With `mass` set the block makes a second pass over the
// keys for one tile of keys and every row (see i4_attn.cu).
template <int D, class Src>
__device__ void plain_attention(const Src& src, int row0) {
  __shared__ float qs[kPlainRows][D], ks[kPlainKeys][D + 1], s[kPlainRows][kPlainKeys];
  __shared__ float sm[kPlainRows], sl[kPlainRows], sc[kPlainRows];
  const int tid = threadIdx.x;
  const int rows = min(kPlainRows, src.rows() - row0);
  if (rows <= 0) return;
  for (int i = tid; i < kPlainRows * D; i += kPlainThreads)
    qs[i / D][i % D] = i / D < rows ? src.query(row0 + i / D, i % D) : 0.f;
  if (tid < kPlainRows) sm[tid] = -INFINITY, sl[tid] = 0.f;
  constexpr int NO = kPlainRows * D / kPlainThreads;     // outputs of a thread: one column, NO rows
  float acc[NO] = {};
  const int col = tid % D, r0 = tid / D * NO;
  const int64_t n = src.keys();
  for (int64_t j0 = 0; j0 < n; j0 += kPlainKeys) {
    __syncthreads();
    for (int i = tid; i < kPlainKeys * D; i += kPlainThreads)
      ks[i / D][i % D] = j0 + i / D < n ? src.key(j0 + i / D, i % D) : 0.f;
    __syncthreads();
    for (int e = tid; e < kPlainRows * kPlainKeys; e += kPlainThreads) {
      const int r = e / kPlainKeys, j = e % kPlainKeys;
      float x = 0.f;
      for (int c = 0; c < D; ++c) x += qs[r][c] * ks[j][c];
      s[r][j] = r < rows && j0 + j < n ? src.score(row0 + r, j0 + j, x) : -INFINITY;
    }
    __syncthreads();
    for (int i = tid; i < kPlainKeys * D; i += kPlainThreads)
      ks[i / D][i % D] = j0 + i / D < n ? src.value(j0 + i / D, i % D) : 0.f;
    if (tid < kPlainRows) {
      float m = sm[tid], l = 0.f;
      for (int j = 0; j < kPlainKeys; ++j) m = fmaxf(m, s[tid][j]);
      const float m0 = m == -INFINITY ? 0.f : m;
      for (int j = 0; j < kPlainKeys; ++j) l += s[tid][j] = expf(s[tid][j] - m0);
      sc[tid] = expf(sm[tid] - m0);
      sl[tid] = sl[tid] * sc[tid] + l;
      sm[tid] = m;
    }
    __syncthreads();
    for (int o = 0; o < NO; ++o) {
      const int r = r0 + o;
      float x = acc[o] * sc[r];
      for (int j = 0; j < kPlainKeys; ++j) {
        const float p = s[r][j];
        if (p > 0.f) x += p * ks[j][col];
      }
      acc[o] = x;
    }
  }
  __syncthreads();
  for (int o = 0; o < NO; ++o) {
    const int r = r0 + o;
    if (r < rows) src.store(row0 + r, col, sl[r] > 0.f ? acc[o] / sl[r] : 0.f);
  }
  if (tid < rows) src.store_lse(row0 + tid, sl[tid] > 0.f ? sm[tid] + logf(sl[tid]) : -INFINITY);
}

}  // namespace kvc
