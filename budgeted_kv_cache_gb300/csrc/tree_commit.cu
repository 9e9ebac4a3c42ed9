// The accepted path of a drafted tree: its softmax weights added to the mass of
// the cached rows, its own rows quantised behind them.
//
// Mass.  mass[j] += sum over the path's queries r of 2^(y_rj - lse_r), with the
// row statistics that the tree's attention left, so one pass over the key codes
// and scales is enough and nothing is joined.  Bound by those bytes (72 and 8 of
// mass a row at d = 128) for up to about 16 query rows, by the products behind
// them.  As in the attention over the 4-bit cache: a warp works alone on tiles
// of 32 keys, its copies three tiles ahead; S = K Q^T with the codes, exact in
// bf16, in the 16-row operand, the key scales applied to the groups' partial
// sums in fp32.  More than 32 query rows take another pass over the codes each.
//
// Measured, replayed (d = 128, the path of 4 to 7 nodes of 4 heads): 8 units of
// 2,304 rows 6.3 us, 576 of them 50 us = 2.2 TB/s, 64 units of 20K to 32K rows, 5
// nodes of 3 heads, capped, a scale per row, 54 us = 2.5 TB/s.  What is left is
// latency: three warps a scheduler, which issues in 47 to 56 % of its cycles.
//
// Rows.  One block per unit, launched with the mass (only the counters, which
// the other kernel reads, wait for it): d / 8 lanes a row, as kvc_i4_append.  A row's own mass is
// the weight that it got from the path behind it: few products, a lane each.
#include <algorithm>
#include <type_traits>

#include "i4_codes.cuh"
#include "kvc_internal.cuh"
#include "packed_math.cuh"

namespace kvc {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 32;                        // keys per warp tile
constexpr int kStages = 4;
constexpr int kRowThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// Distance back to a position that lies before p (up to 2^32 - 1: positions are any 32-bit integers).
__device__ __forceinline__ uint32_t behind(int p, int before) { return static_cast<uint32_t>(p) - static_cast<uint32_t>(before); }

// A unit's path: its nodes, and whether they and their rows are fit to be committed (else n = 0).
struct Path {
  int u, b, l, g, n, count, status;
  int64_t base;
  const int32_t* node;
  // called by whole warps
  __device__ __forceinline__ Path(const TreeCommitArgs& a, int u_) : u(u_) {
    b = u / (a.L * a.Hkv), l = u / a.Hkv % a.L, g = u % a.Hkv;
    node = a.path + static_cast<int64_t>(b) * a.max_path;
    // every load at once: nodes behind the path are not looked at
    static_assert(KVC_TREE_MAX_PATH <= 64, "two nodes a lane");
    const int lane = threadIdx.x & 31;
    const int first = lane < a.max_path ? node[lane] : 0, second = lane + 32 < a.max_path ? node[lane + 32] : 0;
    n = clamp_count(a.path_len[b], a.max_path);
    count = a.rows.count[u];
    base = static_cast<int64_t>(u) * a.rows.capacity;
    status = KVC_UNIT_OK;
    const bool bad = count < 0 || count > a.rows.capacity || (lane < n && (first < 0 || first >= a.n)) ||
                     (lane + 32 < n && (second < 0 || second >= a.n));
    if (__any_sync(kFull, bad)) status = KVC_UNIT_BAD_INDEX;
    else if (n > a.rows.capacity - count) status = KVC_UNIT_FULL;
    if (status != KVC_UNIT_OK) n = 0;
  }
  __device__ __forceinline__ int64_t q_at(const TreeCommitArgs& a, int i, int h) const {
    return b * a.qs.batch + l * a.qs.layer + static_cast<int64_t>(g * a.G + h) * a.qs.head + node[i] * a.qs.token;
  }
  // base 2; infinity, which makes every weight 0, for a row that saw nothing
  __device__ __forceinline__ float lse2(const TreeCommitArgs& a, int i, int h) const {
    const float x = a.row_lse[((static_cast<int64_t>(b) * a.L + l) * (a.Hkv * a.G) + g * a.G + h) * a.n + node[i]];
    return x == -INFINITY ? INFINITY : x * kLog2e;
  }
  __device__ __forceinline__ int64_t new_at(const TreeCommitArgs& a, const kvc_strides& s, int row) const {
    return b * s.batch + l * s.layer + g * s.head + row * s.token;
  }
};

template <int D, bool ROW>
struct Smem {
  alignas(128) uint8_t codes[kWarps][kStages][kTile][D / 2];
  alignas(16) float scale[kWarps][kTile][ROW ? 1 : D / 32];
  int32_t pos[kWarps][kTile];
};

// NT: query rows of a pass / 8.  MODS: some change of the scores is asked for.
template <int D, int NT, bool ROW, bool MODS>
__global__ void __launch_bounds__(kThreads, NT == 4 ? 3 : 4) tree_mass_kernel(const TreeCommitArgs a) {
  constexpr int NG = D / 32, CH = D / 32;          // scale groups; 16-byte chunks per row
  __shared__ Smem<D, ROW> s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u = blockIdx.y + blockIdx.z * 65535;
  if (u >= a.U) return;
  wait_for_previous_kernel();
  let_next_kernel_start();
  const Path un(a, u);
  if (un.n == 0) return;
  const int next = a.rows.next_pos[u], prefix = MODS && a.mods.prefix_len ? a.mods.prefix_len[un.b] : INT32_MIN;
  const int R = un.n * a.G, tiles = (un.count + kTile - 1) / kTile;
  // with a window every split takes tiles in turn, so that all of them have a part of what is seen
  const bool windowed = MODS && a.mods.window;
  const int split = blockIdx.x, splits = gridDim.x;
  int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / splits),
      t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / splits);
  if (windowed) t0 = split * kWarps, t1 = tiles;
  const int stride = windowed ? kWarps * splits : kWarps;

  auto swz = [](int row, int chunk) { return D == 128 ? chunk ^ ((row >> 1) & 3) : chunk ^ ((row >> 2) & 1); };
  constexpr int RPC = 32 / CH;                     // rows per copy instruction of a warp
  const int c_row = lane / CH, c_chunk = lane % CH;
  const uint32_t c_dst = smem_u32(&s.codes[warp][0][c_row][swz(c_row, c_chunk) * 16]);
  const uint8_t* const c_src = static_cast<const uint8_t*>(a.rows.k) + (un.base + c_row) * (D / 2) + c_chunk * 16;
  auto copy_tile = [&](int i, int st, bool wanted) {
    if (i < t1 && wanted) {
      const uint8_t* src = c_src + static_cast<int64_t>(i) * (kTile * D / 2);
      const int left = un.count - i * kTile - c_row;
#pragma unroll
      for (int r = 0; r < kTile; r += RPC)
        cp_async16(c_dst + st * (kTile * D / 2) + r * (D / 2), r < left ? src + r * (D / 2) : c_src - c_row * (D / 2), r < left);
    }
    cp_async_commit();
  };
  using Scales = typename std::conditional<ROW, uint16_t, typename std::conditional<D == 128, uint2, uint32_t>::type>::type;
  Scales ks_next = {};
  int32_t pos_next = 0;
  float old_next = 0.f;
  auto fetch = [&](int i) {
    const int j = i * kTile + lane;
    ks_next = Scales{};
    if (i < t1 && j < un.count) {
      ks_next = static_cast<const Scales*>(a.rows.k_scale)[un.base + j];
      if (MODS) pos_next = a.rows.pos[un.base + j];
      old_next = a.rows.mass[un.base + j];
    }
  };
  auto position = [&](int i) {
    const int j = i * kTile + lane;
    return i < t1 && j < un.count ? a.rows.pos[un.base + j] : 0;
  };
  // seen by the path's first node (and so by any), or in the prefix
  auto seen_by_any = [&](int i, int32_t p) {
    return __any_sync(kFull, i < t1 && i * kTile + lane < un.count && (behind(next, p) < static_cast<uint32_t>(a.mods.window) || p < prefix)) != 0;
  };
  const bool capped = MODS && a.mods.softcap > 0.f, biased = MODS && a.mods.slopes;
  const float pre = capped ? a.scale : a.scale * kLog2e;
  const float inv_cap = capped ? fminf(1.f / a.mods.softcap, 1e30f) : 0.f;

#pragma unroll 1
  for (int r0 = 0; r0 < R; r0 += NT * 8) {
    if (r0) cp_async_wait<0>(), __syncwarp();
    bool ahead[kStages - 1];                       // of the tiles on their way
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int at = t0 + warp + i * stride;
      ahead[i] = !windowed || seen_by_any(at, position(at));
      copy_tile(at, i, ahead[i]);
    }
    fetch(t0 + warp);
    int32_t pos_far = windowed ? position(t0 + warp + (kStages - 1) * stride) : 0;
    uint32_t qf[NT][NG][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + g, rc = min(r, R - 1);
      const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + un.q_at(a, rc / a.G, rc % a.G) + 8 * t;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const uint4 w = r < R ? *reinterpret_cast<const uint4*>(q + 32 * gr) : make_uint4(0, 0, 0, 0);
        qf[nt][gr][0] = __byte_perm(w.x, w.z, 0x5410);       // elements (0,4), (1,5), (2,6), (3,7) of the lane's eight
        qf[nt][gr][1] = __byte_perm(w.x, w.z, 0x7632);
        qf[nt][gr][2] = __byte_perm(w.y, w.w, 0x5410);
        qf[nt][gr][3] = __byte_perm(w.y, w.w, 0x7632);
      }
    }
    // query rows 2t, 2t + 1 of each column block
    float lse[NT][2], slope[NT][2];
    int p_q[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + nt * 8 + 2 * t + e, rc = min(r, R - 1), i = rc / a.G;
        lse[nt][e] = r < R ? un.lse2(a, i, rc % a.G) : INFINITY;       // 2^(y - inf) = 0
        p_q[nt][e] = next + i;
        slope[nt][e] = biased ? a.mods.slopes[un.g * a.G + rc % a.G] * kLog2e : 0.f;
      }
    int st = 0;
#pragma unroll 1
    for (int i = t0 + warp; i < t1; i += stride) {
      const int far = i + (kStages - 1) * stride;
      const bool wanted = !windowed || seen_by_any(far, pos_far);
      copy_tile(far, (st + kStages - 1) % kStages, wanted);
      if (windowed) pos_far = position(far + stride);
      put_scales(&s.scale[warp][lane][0], ks_next, pre);
      if (MODS) s.pos[warp][lane] = pos_next;
      const float old = old_next;
      const bool now = ahead[0];
#pragma unroll
      for (int k = 0; k + 1 < kStages - 1; ++k) ahead[k] = ahead[k + 1];
      ahead[kStages - 2] = wanted;
      fetch(i + stride);
      cp_async_wait<kStages - 1>();
      __syncwarp();
      if (now) {
        const uint8_t* kc = &s.codes[warp][st][0][0];
        float sum[4];                              // of keys g, g + 8, g + 16, g + 24
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          // without modifiers the sums begin at -lse: y is the weight's exponent
          float y[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) y[nt][c] = ROW || MODS ? 0.f : -lse[nt][c & 1];
          const int k0 = sub * 16 + g, k1 = k0 + 8;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(kc + k0 * (D / 2) + swz(k0, gr) * 16 + t * 4);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(kc + k1 * (D / 2) + swz(k1, gr) * 16 + t * 4);
            const uint32_t lo[4] = {code_pair(w0), code_pair(w1), code_pair(w0 >> 4), code_pair(w1 >> 4)};
            const uint32_t hi[4] = {code_pair(w0 >> 8), code_pair(w1 >> 8), code_pair(w0 >> 12), code_pair(w1 >> 12)};
            const float f0 = s.scale[warp][k0][ROW ? 0 : gr], f1 = s.scale[warp][k1][ROW ? 0 : gr];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (ROW) {
                mma16816(y[nt], lo, qf[nt][gr][0], qf[nt][gr][1]);
                mma16816(y[nt], hi, qf[nt][gr][2], qf[nt][gr][3]);
                if (gr == NG - 1) {
                  const uint64_t begin = MODS ? 0 : pair(-lse[nt][0], -lse[nt][1]);
                  unpair(fma2(pair(y[nt][0], y[nt][1]), pair(f0, f0), begin), &y[nt][0], &y[nt][1]);
                  unpair(fma2(pair(y[nt][2], y[nt][3]), pair(f1, f1), begin), &y[nt][2], &y[nt][3]);
                }
              } else {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816(acc, lo, qf[nt][gr][0], qf[nt][gr][1]);
                mma16816(acc, hi, qf[nt][gr][2], qf[nt][gr][3]);
                unpair(fma2(pair(acc[0], acc[1]), pair(f0, f0), pair(y[nt][0], y[nt][1])), &y[nt][0], &y[nt][1]);
                unpair(fma2(pair(acc[2], acc[3]), pair(f1, f1), pair(y[nt][2], y[nt][3])), &y[nt][2], &y[nt][3]);
              }
            }
          }
          if (MODS) {
            const int pk[2] = {s.pos[warp][k0], s.pos[warp][k1]};
            if (capped) {
              float big = 0.f;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; c += 2) big = fmax3(big, fabsf(y[nt][c]), fabsf(y[nt][c + 1]));
              if (__all_sync(kFull, big * inv_cap <= kTanhRange)) {
                const uint64_t z2 = pair(inv_cap, inv_cap);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 4; c += 2) {
                    const uint64_t x = pair(y[nt][c], y[nt][c + 1]), z = mul2(x, z2), w = mul2(z, z);
                    uint64_t p = pair(kTanh[4] * kLog2e, kTanh[4] * kLog2e);
#pragma unroll
                    for (int k = 3; k >= 0; --k) p = fma2(p, w, pair(kTanh[k] * kLog2e, kTanh[k] * kLog2e));
                    unpair(mul2(x, p), &y[nt][c], &y[nt][c + 1]);
                  }
              } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 4; ++c) y[nt][c] = capped_base2(y[nt][c], y[nt][c] * inv_cap, a.mods.softcap);
              }
            }
            if (biased) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  y[nt][c] = fmaf(-slope[nt][c & 1], static_cast<float>(behind(p_q[nt][c & 1], pk[c >> 1])), y[nt][c]);
            }
            if (windowed) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (behind(p_q[nt][c & 1], pk[c >> 1]) >= static_cast<uint32_t>(a.mods.window) && pk[c >> 1] >= prefix) y[nt][c] = -INFINITY;
            }
          }
          uint64_t all[2] = {0, 0};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float w0 = y[nt][2 * k], w1 = y[nt][2 * k + 1];
              if (MODS) unpair(add2(pair(w0, w1), pair(-lse[nt][0], -lse[nt][1])), &w0, &w1);
              all[k] = add2(all[k], pair(ex2_approx(w0), ex2_approx(w1)));
            }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float w0, w1;
            unpair(all[k], &w0, &w1);
            sum[2 * sub + k] = w0 + w1;
          }
        }
        // over the query rows of the four lanes; lane (g, t) then keeps that of key 8 t + g
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sum[k] += __shfl_xor_sync(kFull, sum[k], 1);
          sum[k] += __shfl_xor_sync(kFull, sum[k], 2);
        }
        const float mine = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
        const float add = __shfl_sync(kFull, mine, (lane & 7) * 4 + (lane >> 3));
        const int j = i * kTile + lane;
        if (j < un.count) a.rows.mass[un.base + j] = old + add;
      }
      __syncwarp();
      st = (st + 1) % kStages;
    }
  }
  cp_async_wait<0>();
}

template <int D, bool ROW>
__global__ void __launch_bounds__(kRowThreads) tree_rows_commit_kernel(const TreeCommitArgs a) {
  constexpr int LPR = D / 8, RPB = kRowThreads / LPR, NS = ROW ? 1 : D / 32;
  __shared__ float sk[kRowThreads / 32][D];
  // With q the kernel in front is the one that adds the mass: it touches rows in use alone, and nothing began before
  // everything in front of it was done.  Only the counters, which it reads, wait for it.
  if (!a.q) wait_for_previous_kernel();
  const Path un(a, blockIdx.x);
  if (un.status != KVC_UNIT_OK && threadIdx.x == 0 && a.unit_status) a.unit_status[un.u] = un.status;
  if (un.n == 0) {
    if (a.q) wait_for_previous_kernel();           // whoever comes behind this kernel comes behind that one too
    return;
  }
  const int next = a.rows.next_pos[un.u];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int64_t row0 = un.base + un.count;
  for (int j0 = 0; j0 < un.n; j0 += RPB) {         // whole warps: a group's lanes share their maximum
    const int j = j0 + sub, jc = min(j, un.n - 1);
    const int64_t src = un.new_at(a, a.news, un.node[jc]) + piece * 8;
    const uint4 w[2] = {*reinterpret_cast<const uint4*>(a.k_new + src), *reinterpret_cast<const uint4*>(a.v_new + src)};
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint16_t bits;
      const uint32_t pk = quantise8<ROW, ROW ? LPR : 4>(w[v], &bits);
      if (j >= un.n) continue;
      static_cast<uint32_t*>(v ? a.rows.v : a.rows.k)[(row0 + j) * LPR + piece] = pk;
      if (ROW ? piece == 0 : (piece & 3) == 0)
        static_cast<uint16_t*>(v ? a.rows.v_scale : a.rows.k_scale)[(row0 + j) * NS + (ROW ? 0 : piece / 4)] = bits;
      if (a.k_out)
        *reinterpret_cast<uint4*>((v ? a.v_out : a.k_out) + un.new_at(a, a.outs, j) + piece * 8) = dequantise8(pk, bits, ROW);
    }
    if (j < un.n && piece == 0) a.rows.pos[row0 + j] = next + j;
  }
  if (a.rows.mass) {
    const int prefix = a.mods.prefix_len ? a.mods.prefix_len[un.b] : INT32_MIN;
    for (int j = warp; j < un.n; j += kRowThreads / 32) {
      float sum = 0.f;
      if (a.q) {
        const __nv_bfloat16* k = a.k_new + un.new_at(a, a.news, un.node[j]);
        __syncwarp();
        for (int c = lane; c < D; c += 32) sk[warp][c] = __bfloat162float(k[c]);
        __syncwarp();
        for (int r = j * a.G + lane; r < un.n * a.G; r += 32) {        // the queries of node j and those behind it
          const int i = r / a.G, h = r % a.G;
          const __nv_bfloat16* q = a.q + un.q_at(a, i, h);
          float x = 0.f;
#pragma unroll 4
          for (int c = 0; c < D; c += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(q + c);
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x = fmaf(__uint_as_float(v[e] << 16), sk[warp][c + 2 * e], x);
              x = fmaf(__uint_as_float(v[e] & 0xffff0000u), sk[warp][c + 2 * e + 1], x);
            }
          }
          x *= a.scale;
          if (a.mods.softcap > 0.f) x = capped_base2(x, x * fminf(1.f / a.mods.softcap, 1e30f), a.mods.softcap);
          else x *= kLog2e;
          if (a.mods.slopes) x -= a.mods.slopes[un.g * a.G + h] * kLog2e * static_cast<float>(i - j);
          if (!a.mods.window || i - j < a.mods.window || next + j < prefix) sum += ex2_approx(x - un.lse2(a, i, h));
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      }
      if (lane == 0) a.rows.mass[row0 + j] = sum;
    }
  }
  if (a.q) wait_for_previous_kernel();
  __syncthreads();
  if (threadIdx.x == 0) {
    a.rows.count[un.u] = un.count + un.n;
    a.rows.next_pos[un.u] = next + un.n;
  }
}

template <int D, bool ROW>
cudaError_t launch_one(const TreeCommitArgs& a, cudaStream_t stream) {
  if (a.q) {
    const bool mods = a.mods.softcap > 0.f || a.mods.slopes || a.mods.window;
    const int rows = a.max_path * a.G;
    const dim3 grid(a.splits, std::min(a.U, 65535), (a.U + 65534) / 65535);
    auto go = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      return launch_after(mods ? tree_mass_kernel<D, NT, ROW, true> : tree_mass_kernel<D, NT, ROW, false>, grid, kThreads, 0,
                          stream, a);
    };
    const cudaError_t e = rows <= 8    ? go(std::integral_constant<int, 1>{})
                          : rows <= 16 ? go(std::integral_constant<int, 2>{})
                                       : go(std::integral_constant<int, 4>{});
    if (e != cudaSuccess) return e;
  }
  return launch_after(tree_rows_commit_kernel<D, ROW>, dim3(a.U), kRowThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_tree_commit(const TreeCommitArgs& a, cudaStream_t stream) {
  const bool row = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  if (a.d == 128) return row ? launch_one<128, true>(a, stream) : launch_one<128, false>(a, stream);
  return row ? launch_one<64, true>(a, stream) : launch_one<64, false>(a, stream);
}

}  // namespace kvc
