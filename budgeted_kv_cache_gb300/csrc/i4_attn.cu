// Attention over the rows of a 4-bit cache, with score modifiers; optionally
// adds the softmax weights to the rows' mass.
#include "attn_rows.cuh"

namespace kvc {

namespace {

struct I4Src {
  const I4AttnArgs& a;
  int u, b, l, g;
  int n, next;
  int64_t prefix, base;
  bool row_mode;
  __device__ I4Src(const I4AttnArgs& a_, int u_) : a(a_), u(u_) {
    b = u / (a.L * a.Hkv), l = u / a.Hkv % a.L, g = u % a.Hkv;
    n = clamp_count(a.rows.count[u], a.rows.capacity);
    next = a.rows.next_pos[u];
    prefix = a.mods.prefix_len ? a.mods.prefix_len[b] : INT64_MIN;
    base = static_cast<int64_t>(u) * a.rows.capacity;
    row_mode = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  }
  __device__ int rows() const { return a.n_q * a.G; }
  __device__ int64_t keys() const { return n; }
  __device__ float query(int r, int c) const {
    return __bfloat162float(a.q[b * a.qs.batch + l * a.qs.layer + (g * a.G + r % a.G) * a.qs.head +
                                (r / a.G) * a.qs.token + c]);
  }
  __device__ float element(const void* codes, const void* scales, int64_t j, int c) const {
    const int d = a.d;
    const uint8_t byte = static_cast<const uint8_t*>(codes)[(base + j) * (d / 2) + c / 2];
    const int code = static_cast<int>((c & 1 ? byte >> 4 : byte & 15) ^ 8) - 8;
    const uint16_t s = static_cast<const uint16_t*>(scales)[row_mode ? base + j : (base + j) * (d / 32) + c / 32];
    return code * (row_mode ? __half2float(__ushort_as_half(s)) : bf16_bits_to_float(s));
  }
  __device__ float key(int64_t j, int c) const { return element(a.rows.k, a.rows.k_scale, j, c); }
  __device__ float value(int64_t j, int c) const { return element(a.rows.v, a.rows.v_scale, j, c); }
  __device__ float score(int r, int64_t j, float x) const {
    const int i = r / a.G;
    const int64_t p = a.q_pos ? a.q_pos[b * a.n_q + i] : static_cast<int64_t>(next) - a.n_q + i;
    const int64_t pk = a.rows.pos[base + j];
    if (!sees(p, pk, a.mods.window, prefix)) return -INFINITY;
    return mod_score(x * a.scale, a.mods.softcap, a.mods.slopes ? a.mods.slopes[g * a.G + r % a.G] : 0.f,
                     static_cast<float>(p - pk));
  }
  __device__ void store(int r, int c, float x) const {
    a.out[b * a.os.batch + l * a.os.layer + (g * a.G + r % a.G) * a.os.head + (r / a.G) * a.os.token + c] =
        __float2bfloat16_rn(x);
  }
  __device__ int64_t lse_at(int r) const {
    return ((static_cast<int64_t>(b) * a.L + l) * (a.Hkv * a.G) + g * a.G + r % a.G) * a.n_q + r / a.G;
  }
  __device__ void store_lse(int r, float x) const {
    if (a.lse) a.lse[lse_at(r)] = x;
  }
};

template <int D>
__global__ void __launch_bounds__(kPlainThreads) i4_plain_kernel(const I4AttnArgs a) {
  for (int u = blockIdx.y; u < a.U; u += gridDim.y) {
    plain_attention<D>(I4Src(a, u), blockIdx.x * kPlainRows);
    __syncthreads();
  }
}

// mass[j] += sum over the rows of exp(x_rj - lse_r), one warp per key.
template <int D>
__global__ void __launch_bounds__(kPlainThreads) i4_mass_kernel(const I4AttnArgs a) {
  for (int u = blockIdx.y; u < a.U; u += gridDim.y) {
    const I4Src src(a, u);
    const int lane = threadIdx.x & 31;
    for (int64_t j = blockIdx.x * (kPlainThreads / 32) + (threadIdx.x >> 5); j < src.n;
         j += gridDim.x * (kPlainThreads / 32)) {
      float k[D / 32], sum = 0.f;
      for (int c = 0; c < D / 32; ++c) k[c] = src.key(j, c * 32 + lane);
      for (int r = 0; r < src.rows(); ++r) {
        float x = 0.f;
        for (int c = 0; c < D / 32; ++c) x += src.query(r, c * 32 + lane) * k[c];
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        x = src.score(r, j, x);
        if (x > -INFINITY) sum += expf(x - a.lse[src.lse_at(r)]);
      }
      if (lane == 0) a.rows.mass[src.base + j] += sum;
    }
  }
}

}  // namespace

cudaError_t launch_i4_attn(const I4AttnArgs& a, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(a.n_q) * a.G;
  const unsigned y = a.U < 65535 ? a.U : 65535;
  const dim3 grid(static_cast<unsigned>((rows + kPlainRows - 1) / kPlainRows), y);
  const dim3 mgrid(static_cast<unsigned>((a.rows.capacity + 31) / 32), y);
  if (a.d == 128) i4_plain_kernel<128><<<grid, kPlainThreads, 0, stream>>>(a);
  else i4_plain_kernel<64><<<grid, kPlainThreads, 0, stream>>>(a);
  if (a.add_mass) {
    if (a.d == 128) i4_mass_kernel<128><<<mgrid, kPlainThreads, 0, stream>>>(a);
    else i4_mass_kernel<64><<<mgrid, kPlainThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace kvc
