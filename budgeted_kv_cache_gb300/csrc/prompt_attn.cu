// Attention of a prompt, a chunk of one or single tokens over a bf16 cache
// (PASK Eq. 1) with score modifiers, documents and a prefix.
#include "attn_rows.cuh"

namespace kvc {

namespace {

struct PromptSrc {
  const PromptArgs& a;
  int b, l, g;
  int nq, first;              // queries, position of query 0
  int64_t nk, prefix;
  __device__ PromptSrc(const PromptArgs& a_, int u) : a(a_) {
    b = u / (a.L * a.Hkv), l = u / a.Hkv % a.L, g = u % a.Hkv;
    nk = a.kv_len ? max(0, min(static_cast<int>(a.T), a.kv_len[b])) : a.T;
    nq = a.q_len ? clamp_count(a.q_len[b], a.n_q) : a.n_q;
    first = static_cast<int>(nk) - nq;
    prefix = a.mods.prefix_len ? a.mods.prefix_len[b] : 0;
  }
  __device__ int rows() const { return nq * a.G; }
  __device__ int64_t keys() const { return nk; }
  __device__ float query(int r, int c) const {
    return __bfloat162float(a.q[b * a.qs.batch + l * a.qs.layer + (g * a.G + r % a.G) * a.qs.head +
                                (r / a.G) * a.qs.token + c]);
  }
  __device__ int64_t at(int64_t j) const { return b * a.kvs.batch + l * a.kvs.layer + g * a.kvs.head + j * a.kvs.token; }
  __device__ bool dead(int64_t j) const { return a.docs && a.docs[b * a.T + j] < 0; }
  __device__ float key(int64_t j, int c) const { return dead(j) ? 0.f : __bfloat162float(a.k[at(j) + c]); }
  __device__ float value(int64_t j, int c) const { return dead(j) ? 0.f : __bfloat162float(a.v[at(j) + c]); }
  __device__ float score(int r, int64_t j, float x) const {
    const int64_t p = first + r / a.G;
    if (p < 0 || !sees(p, j, a.mods.window, prefix)) return -INFINITY;
    if (a.docs) {
      const int32_t doc = a.docs[b * a.T + j];
      if (doc < 0 || doc != a.docs[b * a.T + p]) return -INFINITY;
    }
    return mod_score(x * a.scale, a.mods.softcap, a.mods.slopes ? a.mods.slopes[g * a.G + r % a.G] : 0.f,
                     static_cast<float>(p - j));
  }
  __device__ void store(int r, int c, float x) const {
    a.out[b * a.os.batch + l * a.os.layer + (g * a.G + r % a.G) * a.os.head + (r / a.G) * a.os.token + c] =
        __float2bfloat16_rn(x);
  }
  __device__ void store_lse(int r, float x) const {
    if (a.lse) a.lse[((static_cast<int64_t>(b) * a.L + l) * (a.Hkv * a.G) + g * a.G + r % a.G) * a.n_q + r / a.G] = x;
  }
};

template <int D>
__global__ void __launch_bounds__(kPlainThreads) prompt_plain_kernel(const PromptArgs a) {
  for (int u = blockIdx.y; u < a.U; u += gridDim.y) {
    plain_attention<D>(PromptSrc(a, u), blockIdx.x * kPlainRows);
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.n_q) * a.G;
  const dim3 grid(static_cast<unsigned>((rows + kPlainRows - 1) / kPlainRows), a.U < 65535 ? a.U : 65535);
  if (a.d == 128) prompt_plain_kernel<128><<<grid, kPlainThreads, 0, stream>>>(a);
  else prompt_plain_kernel<64><<<grid, kPlainThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
