// Attention of a tree of drafted tokens over the rows of a 4-bit cache and over
// the tree's own bf16 rows, with score modifiers.
//
// Node i of a tree stands at position next_pos + depth(i) and sees the cached
// rows, its ancestors and itself.  Parents come before their children, so a
// node's ancestors are met by walking up once while the tree's keys are taken
// from the last to the first.
#include <algorithm>

#include "kvc_internal.cuh"
#include "packed_math.cuh"

namespace kvc {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Element i (0..7) of a word of codes.
__device__ __forceinline__ float code_at(uint32_t w, int i) {
  return static_cast<float>(static_cast<int32_t>(w << (28 - 4 * i)) >> 28);
}

__device__ __forceinline__ float scale_at(const void* scales, int64_t row, int group, int groups) {
  if (groups == 1) return __half2float(static_cast<const __half*>(scales)[row]);
  return bf16_bits_to_float(static_cast<const uint16_t*>(scales)[row * groups + group]);
}

// One warp per query row; a lane takes a key of 32 for the scores and D / 32 columns for the values.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) tree_rows_kernel(const TreeArgs a) {
  __shared__ float sq[kWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = a.n * a.G, u = blockIdx.y + blockIdx.z * 65535, r = blockIdx.x * kWarps + warp;
  wait_for_previous_kernel();
  let_next_kernel_start();
  if (u >= a.U || r >= R) return;
  const int b = u / (a.L * a.Hkv), l = u / a.Hkv % a.L, g = u % a.Hkv;
  const int node = r / a.G, head = g * a.G + r % a.G;
  if (a.n_nodes && node >= a.n_nodes[b]) return;
  const int32_t* parent = a.parent + static_cast<int64_t>(b) * a.n;
  int depth = 0;
  bool bad = false;
  auto above = [&](int i) {
    const int p = parent[i];
    if (p >= -1 && p < i) return p;
    bad = true;
    return -1;
  };
  for (int i = above(node); i >= 0; i = above(i)) ++depth;
  if (bad && lane == 0 && a.unit_status) a.unit_status[u] = KVC_UNIT_BAD_INDEX;
  const int count = clamp_count(a.rows.count[u], a.rows.capacity);
  const int p_q = a.rows.next_pos[u] + depth;
  const int prefix = a.mods.prefix_len ? a.mods.prefix_len[b] : INT32_MIN;
  const float slope = a.mods.slopes ? a.mods.slopes[head] : 0.f;
  const int64_t q_at = b * a.qs.batch + l * a.qs.layer + head * a.qs.head + node * a.qs.token;
  for (int c = lane; c < D; c += 32) sq[warp][c] = __bfloat162float(a.q[q_at + c]) * a.scale;
  __syncwarp();
  float m = -INFINITY, sum = 0.f, o[D / 32] = {};
  // 32 keys: this lane's score x of the natural base and whether it is seen; value(j, c) of key j
  auto step = [&](float x, int p_k, bool seen, auto value) {
    const int far = p_q - p_k;
    if (a.mods.softcap > 0.f) x = capped_base2(x, x / a.mods.softcap, a.mods.softcap);
    else x *= kLog2e;
    x -= slope * kLog2e * fabsf(static_cast<float>(far));
    if (!seen || (a.mods.window && far >= a.mods.window && p_k >= prefix)) x = -INFINITY;
    float top = x;
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, k));
    if (top == -INFINITY) return;
    const float to = fmaxf(m, top), f = m == -INFINITY ? 0.f : ex2_approx(m - to);
    m = to;
    const float w = ex2_approx(x - m);
    float all = w;
    for (int k = 16; k; k >>= 1) all += __shfl_xor_sync(kFull, all, k);
    sum = fmaf(sum, f, all);
    for (int c = 0; c < D / 32; ++c) o[c] *= f;
    for (int j = 0; j < 32; ++j) {
      const float wj = __shfl_sync(kFull, w, j);
      if (wj > 0.f)
        for (int c = 0; c < D / 32; ++c) o[c] = fmaf(wj, value(j, c), o[c]);
    }
  };
  const int64_t base = static_cast<int64_t>(u) * a.rows.capacity;
  const int groups = a.rows.quant_mode == KVC_QUANT_ROW_FP16 ? 1 : D / 32;
  for (int j0 = 0; j0 < count; j0 += 32) {
    const int j = j0 + lane;
    const int64_t row = base + min(j, count - 1);
    float x = 0.f;
    for (int w = 0; w < D / 8; ++w) {
      const uint32_t codes = static_cast<const uint32_t*>(a.rows.k)[row * (D / 8) + w];
      const float s = scale_at(a.rows.k_scale, row, w / 4, groups);
      for (int e = 0; e < 8; ++e) x = fmaf(code_at(codes, e) * s, sq[warp][8 * w + e], x);
    }
    step(x, a.rows.pos[row], j < count, [&](int jj, int c) {
      const int64_t row = base + j0 + jj;
      const int d = lane * (D / 32) + c;
      return code_at(static_cast<const uint32_t*>(a.rows.v)[row * (D / 8) + d / 8], d % 8) *
             scale_at(a.rows.v_scale, row, d / 32, groups);
    });
  }
  const int64_t new_at = b * a.news.batch + l * a.news.layer + g * a.news.head;
  int cur = node, left = depth;                    // the lowest ancestor not met yet, and its depth
  for (int j0 = node / 32 * 32; j0 >= 0; j0 -= 32) {
    bool seen = false;
    int p_k = p_q;
    while (cur >= j0) {
      if (cur == j0 + lane) seen = true, p_k = p_q - (depth - left);
      cur = above(cur);
      --left;
    }
    const int64_t row = new_at + static_cast<int64_t>(min(j0 + lane, node)) * a.news.token;
    float x = 0.f;
    for (int c = 0; c < D; ++c) x = fmaf(__bfloat162float(a.k_new[row + c]), sq[warp][c], x);
    step(x, p_k, seen, [&](int jj, int c) {
      return __bfloat162float(a.v_new[new_at + static_cast<int64_t>(j0 + jj) * a.news.token + lane * (D / 32) + c]);
    });
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  __nv_bfloat16* out = a.out + b * a.os.batch + l * a.os.layer + head * a.os.head + node * a.os.token + lane * (D / 32);
  for (int c = 0; c < D / 32; ++c) out[c] = __float2bfloat16_rn(o[c] * inv);
  if (lane == 0 && a.lse)
    a.lse[((static_cast<int64_t>(b) * a.L + l) * (a.Hkv * a.G) + head) * a.n + node] = (m + log2f(sum)) * kLn2;
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const dim3 grid((a.n * a.G + kWarps - 1) / kWarps, std::min(a.U, 65535), (a.U + 65534) / 65535);
  return launch_after(a.d == 128 ? tree_rows_kernel<128> : tree_rows_kernel<64>, grid, kWarps * 32, 0, stream, a);
}

}  // namespace kvc
