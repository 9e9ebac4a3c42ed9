// Attention over the rows of a 4-bit cache, with score modifiers; optionally
// adds the softmax weights to the rows' mass.
//
// HBM-bound by the codes and scales (144 bytes a row at d = 128) as long as a
// row's 256 codes are turned into operands in about six SM cycles, so the
// design counts instructions per code.
//   * One warp works alone on tiles of 32 rows (keys): its own asynchronous
//     copies, two tiles ahead (three with more than eight query rows), its
//     own running maximum and sum, no barrier in the loop; the warps of a
//     block and the blocks of a unit are joined at the end (PASK Eq. 15).
//   * Plain causal scores have a kernel of their own; caps, slopes, windows
//     and prefixes share the other.  With a window, the codes of tiles that
//     no query row sees are not read, and a unit's splits take its tiles in
//     turn, so that all of them have a part of what is seen (32 units of 100K
//     to 131K rows, window 8,192: 47 us without mass, 107 when every split
//     read a run of tiles).
//   * Both products put the codes in the 16-row operand and the packed query
//     rows (row r = query r / G, head r % G of the unit) in the 8-column one:
//     S^T = K Q^T and O^T = V^T P^T, so eight query rows cost one instruction.
//     A pair of codes becomes a bf16 pair by one logical operation
//     ((w & 0x000f000f) ^ 0x43084308 = 136 + code) and one subtraction, both
//     exact; the scales never touch the codes:
//   * the key scale of a group multiplies that group's partial sum in fp32;
//     the value scale multiplies the weight, which is rounded to bf16 once
//     after it, per group of 32 columns (mma.sync takes operands of one type,
//     and the codes are exact in bf16: half a step, 2^-8 of a weight, as much
//     as the output's own rounding; the row's sum and the mass take the
//     unrounded weight).
//   * The order of d inside a product is free: a lane takes the eight codes of
//     one 32-bit word as they lie, and the queries are laid out to match.  For
//     the values a byte permutation pairs the words of two rows.
//   * Shared rows are swizzled in 16-byte chunks so that both access patterns
//     (8 rows x 4 words, and 4 row pairs x 4 words) meet every bank once.
// With mass, the loop leaves each row's logits (base 2) in the workspace and a
// second kernel, which also joins the blocks' outputs, adds 2^(y - lse) over
// the query rows, in order.  It is launched ahead of its data, so it costs a
// few latencies and no gap.  (One kernel, a cluster per unit joined through
// distributed shared memory with the logits kept there, was measured: 8.5 us
// against 7.2 for 8 units of 2,304 rows, 28 against 20 for 144 units.)
//
// Measured, replayed from a graph (d = 128, four heads a unit, g32 scales, one
// query): 32 units of 100K to 131K rows 120 us without mass = 4.7 TB/s (the
// copies alone take 104 us; 62 % of the ALU cycles turn codes into operands),
// 142 us with it (the logits' round trip), 172 with a cap, whatever the scores; 8 units of 2,304 rows 7.1 us with
// mass, two launches' latencies.  64 units of 300 to 9,000 rows, d = 64, 15
// query rows, capped, slopes and a window of 4,096: 16.6 us.
#include <algorithm>
#include <type_traits>

#include "i4_codes.cuh"
#include "kvc_internal.cuh"
#include "packed_math.cuh"

namespace kvc {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 32;                        // keys per warp tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;                     // log2 growth of the maximum that forces a rescale

struct Unit {
  int u, b, l, g, n, R;
  int64_t base;
  __device__ __forceinline__ Unit(const I4AttnArgs& a, int u_) : u(u_) {
    b = u / (a.L * a.Hkv), l = u / a.Hkv % a.L, g = u % a.Hkv;
    n = clamp_count(a.rows.count[u], a.rows.capacity);
    R = a.n_q * a.G;
    base = static_cast<int64_t>(u) * a.rows.capacity;
  }
  __device__ __forceinline__ int64_t q_at(const I4AttnArgs& a, const kvc_strides& s, int r) const {
    return b * s.batch + l * s.layer + static_cast<int64_t>(g * a.G + r % a.G) * s.head +
           static_cast<int64_t>(r / a.G) * s.token;
  }
  __device__ __forceinline__ int64_t lse_at(const I4AttnArgs& a, int r) const {
    return ((static_cast<int64_t>(b) * a.L + l) * (a.Hkv * a.G) + g * a.G + r % a.G) * a.n_q + r / a.G;
  }
};

// Keys [t0, t1) tiles of split `split` of a unit with n rows in use.
__device__ __forceinline__ void split_range(const I4AttnArgs& a, int n, int split, int* t0, int* t1) {
  const int tiles = (n + kTile - 1) / kTile;
  *t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / a.splits);
  *t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / a.splits);
}

// NT: query rows of a block / 8.  ROW: one scale per row.
template <int D, int NT, bool ROW>
struct Smem {
  // one column block: four blocks (of 128 registers a thread) per SM with three stages; else fewer and larger
  static constexpr int kStages = NT == 1 ? 3 : 4, kBlocks = NT == 1 ? 4 : NT == 2 ? 3 : 2;
  union {
    alignas(128) uint8_t codes[kWarps][kStages][2][kTile][D / 2];
    // after the loop: the block's outputs, and those of half its warps at a time
    struct {
      alignas(16) float o[NT * 8][D + 4];
      float part[kWarps / 2][NT * 8][D + 4];
    };
  };
  alignas(16) float scale[kWarps][2][kTile][ROW ? 1 : D / 32];
  int32_t pos[kWarps][kTile];
  float m[kWarps][NT * 8], l[kWarps][NT * 8];
  float2 ml[NT * 8];                               // of the block
};

// Two weights of adjacent query rows as bf16 operands; with FINE also what the rounding left of them (then off by 2^-18).
template <bool FINE>
__device__ __forceinline__ void weights(float x, float y, uint32_t* w, uint32_t* rest) {
  const uint32_t hi = pack_bf16x2(x, y);
  *w = transpose8x8(hi);
  if constexpr (FINE) *rest = transpose8x8(pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u)));
}

// MODS: some change of the scores (cap, slopes, window, prefix) is asked for.
// TREE: the queries are the nodes of a drafted tree (a.tree, at most 32 query
// rows): at next_pos + depth, over the cached rows and over the tree's own bf16
// rows, which the last warp of the last split takes behind its tiles.  Weights
// go in as two bf16 operands, so that they are no coarser than where more query
// rows take fp16 ones (8 units of 131,072 rows, 4 query rows: 42 us with one
// operand, 48 with two; fp16 would need the values' sizes tile by tile).
template <int D, int NT, bool ROW, bool MODS, bool TREE>
__global__ void __launch_bounds__(kThreads, (Smem<D, NT, ROW>::kBlocks)) i4_attn_kernel(const I4AttnArgs a) {
  constexpr int NG = D / 32;                       // scale groups
  constexpr int CH = D / 32;                       // 16-byte chunks per row
  extern __shared__ __align__(128) uint8_t raw[];
  using S = Smem<D, NT, ROW>;
  constexpr int kStages = S::kStages;
  S& s = *reinterpret_cast<S*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (static_cast<int>(blockIdx.y + blockIdx.z * 65535) >= a.U) return;
  wait_for_previous_kernel();
  let_next_kernel_start();                         // not before: it reads the counts while this kernel runs
  const Unit un(a, blockIdx.y + blockIdx.z * 65535);
  // what does not depend on the rows in use is on its way before anything waits for them
  const int32_t next = a.rows.next_pos[un.u];
  const int prefix = MODS && a.mods.prefix_len ? a.mods.prefix_len[un.b] : INT32_MIN;
  const int split = blockIdx.x % a.splits, r0 = blockIdx.x / a.splits * (NT * 8);
  // a tree's nodes, one a lane: ancestors (and the node itself) as bits, depth
  uint32_t above = 0;
  int depth = 0, nodes = 0;
  if constexpr (TREE) {
    nodes = a.tree.n_nodes ? clamp_count(a.tree.n_nodes[un.b], a.n_q) : a.n_q;
    const int32_t* parent = a.tree.parent + static_cast<int64_t>(un.b) * a.n_q;
    const int up = lane < nodes ? parent[lane] : -1;
    const bool fine = up >= -1 && up < lane;       // parents come before their children
    if (lane < nodes && !fine && a.tree.unit_status) a.tree.unit_status[un.u] = KVC_UNIT_BAD_INDEX;
    above = 1u << lane;
    int at = fine ? up : -1;
    for (int i = 1; i < a.n_q; ++i) {              // all lanes together: every step up is another lane's parent
      if (at >= 0) above |= 1u << at, ++depth;
      const int p = __shfl_sync(kFull, fine ? up : -1, max(at, 0));
      at = at >= 0 ? p : -1;
    }
  }
  uint32_t qf[NT][NG][4];                          // operand of both products' k-steps of a group
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + nt * 8 + g;
    const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + un.q_at(a, a.qs, min(r, un.R - 1)) + 8 * t;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      const uint4 w = r < un.R ? *reinterpret_cast<const uint4*>(q + 32 * gr) : make_uint4(0, 0, 0, 0);
      // elements (0,4), (1,5), (2,6), (3,7) of the lane's eight
      qf[nt][gr][0] = __byte_perm(w.x, w.z, 0x5410);
      qf[nt][gr][1] = __byte_perm(w.x, w.z, 0x7632);
      qf[nt][gr][2] = __byte_perm(w.y, w.w, 0x5410);
      qf[nt][gr][3] = __byte_perm(w.y, w.w, 0x7632);
    }
  }

  // this block's tiles: t0, t0 + 1, .. below t1, one warp after another; with a window every split takes each splits-th
  // four, so that all of them have a part of what is seen
  const bool windowed = MODS && a.mods.window;
  int t0, t1;
  split_range(a, un.n, split, &t0, &t1);
  if (windowed) t0 = split * kWarps, t1 = (un.n + kTile - 1) / kTile;
  const int stride = windowed ? kWarps * a.splits : kWarps;

  // one warp's copies of tile i: this lane's 16-byte chunk of every 32 / CH rows; rows past n filled with zeros
  auto swz = [](int row, int chunk) { return D == 128 ? chunk ^ ((row >> 1) & 3) : chunk ^ ((row >> 2) & 1); };
  constexpr int RPC = 32 / CH;                     // rows per copy instruction of a warp
  const int c_row = lane / CH, c_chunk = lane % CH;
  const uint32_t c_dst = smem_u32(&s.codes[warp][0][0][c_row][swz(c_row, c_chunk) * 16]);
  const int64_t c_src = (un.base + c_row) * (D / 2) + c_chunk * 16;
  const uint8_t* const c_k = static_cast<const uint8_t*>(a.rows.k) + c_src;
  const uint8_t* const c_v = static_cast<const uint8_t*>(a.rows.v) + c_src;
  auto copy_tile = [&](int i, int st, bool wanted) {
    if (i < t1 && wanted) {
      const int64_t at = static_cast<int64_t>(i) * (kTile * D / 2);
      const uint32_t dst = c_dst + st * (2 * kTile * D / 2);
      const int left = un.n - i * kTile - c_row;   // rows from this lane's first on
      if (i * kTile + kTile <= un.n) {
#pragma unroll
        for (int r = 0; r < kTile; r += RPC) {
          cp_async16(dst + r * (D / 2), c_k + at + r * (D / 2), true);
          cp_async16(dst + (kTile + r) * (D / 2), c_v + at + r * (D / 2), true);
        }
      } else {
#pragma unroll
        for (int r = 0; r < kTile; r += RPC) {
          const bool ok = r < left;
          cp_async16(dst + r * (D / 2), ok ? c_k + at + r * (D / 2) : c_k, ok);
          cp_async16(dst + (kTile + r) * (D / 2), ok ? c_v + at + r * (D / 2) : c_v, ok);
        }
      }
    }
    cp_async_commit();
  };
  // scales and position of this lane's key of tile i
  using Scales = typename std::conditional<ROW, uint16_t, typename std::conditional<D == 128, uint2, uint32_t>::type>::type;
  Scales ks_next = {}, vs_next = {};
  int32_t pos_next = 0;
  auto fetch = [&](int i) {
    const int j = i * kTile + lane;
    ks_next = vs_next = Scales{};                  // rows behind those in use: no garbage meets a zero weight
    if (i < t1 && j < un.n) {
      ks_next = static_cast<const Scales*>(a.rows.k_scale)[un.base + j];
      vs_next = static_cast<const Scales*>(a.rows.v_scale)[un.base + j];
      pos_next = a.rows.pos[un.base + j];
    }
  };
  // query rows 2t, 2t + 1 of each column block: limits, slopes; and the query operand
  int q_hi[NT][2], q_lo[NT][2];
  float slope[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = min(r0 + nt * 8 + 2 * t + e, un.R - 1), i = r / a.G;
      const int64_t p = TREE      ? static_cast<int64_t>(next) + __shfl_sync(kFull, depth, i)
                        : a.q_pos ? a.q_pos[un.b * a.n_q + i]
                                  : static_cast<int64_t>(next) - a.n_q + i;
      q_hi[nt][e] = static_cast<int>(max(p, static_cast<int64_t>(INT32_MIN)));
      q_lo[nt][e] = MODS && a.mods.window ? static_cast<int>(max(p - a.mods.window + 1, static_cast<int64_t>(INT32_MIN))) : INT32_MIN;
      slope[nt][e] = MODS && a.mods.slopes ? a.mods.slopes[un.g * a.G + r % a.G] * kLog2e : 0.f;
    }
  if (!MODS) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy_tile(t0 + warp + i * stride, i, true);
    fetch(t0 + warp);
  }

  const bool capped = MODS && a.mods.softcap > 0.f, biased = MODS && a.mods.slopes;
  const bool modified = capped || biased;
  const float pre = capped ? a.scale : a.scale * kLog2e;      // goes into the key scales
  const float inv_cap = capped ? fminf(1.f / a.mods.softcap, 1e30f) : 0.f;    // a smaller cap leaves no score either
  // limits over the block's query rows
  int hi_min = INT32_MAX, lo_max = INT32_MIN, hi_max = INT32_MIN, lo_min = INT32_MAX;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      hi_min = min(hi_min, q_hi[nt][e]);
      hi_max = max(hi_max, q_hi[nt][e]);
      lo_min = min(lo_min, q_lo[nt][e]);
      lo_max = max(lo_max, q_lo[nt][e]);
    }
  hi_min = __reduce_min_sync(kFull, hi_min);
  hi_max = __reduce_max_sync(kFull, hi_max);
  lo_min = __reduce_min_sync(kFull, lo_min);
  lo_max = __reduce_max_sync(kFull, lo_max);
  // With a window the positions of a tile are looked at before its copies are sent for: what no query row sees is not read.
  auto position = [&](int i) {
    const int j = i * kTile + lane;
    return i < t1 && j < un.n ? a.rows.pos[un.base + j] : 0;
  };
  auto seen_by_any = [&](int i, int32_t p) {
    return __any_sync(kFull, i < t1 && i * kTile + lane < un.n && ((p <= hi_max && p >= lo_min) || p < prefix)) != 0;
  };
  int32_t pos_far = 0;                             // of the tile that is copied next
  if (MODS) {
    int32_t p[kStages - 1];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) p[i] = windowed ? position(t0 + warp + i * stride) : 0;
    if (windowed) pos_far = position(t0 + warp + (kStages - 1) * stride);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
      copy_tile(t0 + warp + i * stride, i, !windowed || seen_by_any(t0 + warp + i * stride, p[i]));
    fetch(t0 + warp);
  }
  float* const log_row = a.logits + (un.base + g) * a.logit_stride + r0 + 2 * t;      // [key][R rounded up to even]
  const uint32_t half_sel = (g >> 2) ? 0x7632u : 0x5410u;
  float m[NT][2], l[NT][2], o[NG][2][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
      for (int k = 0; k < 8; ++k) o[gr][k >> 2][nt][k & 3] = 0.f;
  }

  // ---- running maximum per query row over the warp's keys; logits y become weights
  auto take = [&](float (&y)[2][NT][4]) {
    bool grow = false;
    float top[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(y[0][nt][e], y[0][nt][e + 2]), fmaxf(y[1][nt][e], y[1][nt][e + 2]));
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, k));
        top[nt][e] = x;
        grow |= x - m[nt][e] > kGrow;
      }
    if (__any_sync(kFull, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (!(top[nt][e] > m[nt][e])) continue;
          const float f = m[nt][e] == -INFINITY ? 0.f : ex2_approx(m[nt][e] - top[nt][e]);
          m[nt][e] = top[nt][e];
          l[nt][e] *= f;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              o[gr][mt][nt][e] *= f;
              o[gr][mt][nt][e + 2] *= f;
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float& x = y[k >> 1][nt][(k & 1) * 2 + e];
          x = ex2_approx(x - ref);
          l[nt][e] += x;
        }
      }
  };

  int st = 0;
#pragma unroll 1
  for (int i = t0 + warp; i < t1; i += stride) {
    const int far = i + (kStages - 1) * stride;
    copy_tile(far, (st + kStages - 1) % kStages, !windowed || seen_by_any(far, pos_far));
    if (windowed) pos_far = position(far + stride);
    // scales and positions of this tile: one lane per key, then to all
    put_scales(&s.scale[warp][0][lane][0], ks_next, pre);
    put_scales(&s.scale[warp][1][lane][0], vs_next, 1.f);
    s.pos[warp][lane] = pos_next;
    // does every query row see every key of the tile?
    const bool mine = i * kTile + lane < un.n;
    const bool clear = __all_sync(kFull, mine && pos_next <= hi_min && (!MODS || pos_next >= lo_max));
    const bool none = !clear && windowed && !seen_by_any(i, pos_next);
    fetch(i + stride);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    if (none) {
      if (a.logits && mine) {
        float* dst = a.logits + (un.base + i * kTile + lane) * a.logit_stride + r0;
        for (int c = 0; c < min(NT * 8, a.logit_stride - r0); c += 2)
          *reinterpret_cast<float2*>(dst + c) = make_float2(-INFINITY, -INFINITY);
      }
      __syncwarp();
      st = (st + 1) % kStages;
      continue;
    }
    const uint8_t* kc = &s.codes[warp][st][0][0][0];
    const uint8_t* vc = &s.codes[warp][st][1][0][0];
    auto scale_f = [&](int which, int key, float (&f)[NG]) {
      const float* w = &s.scale[warp][which][key][0];
      if constexpr (ROW) {
        f[0] = w[0];
      } else if constexpr (NG == 4) {
        const float4 v = *reinterpret_cast<const float4*>(w);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(w);
        f[0] = v.x, f[1] = v.y;
      }
    };

    // ---- y = logits in base 2: y[sub][nt][c], key 16 sub + g (+ 8 for c >= 2), query row 2t + (c & 1)
    float y[2][NT][4];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) y[sub][nt][c] = 0.f;
      const int k0 = sub * 16 + g, k1 = k0 + 8;
      float f0[NG], f1[NG];
      scale_f(0, k0, f0);
      scale_f(0, k1, f1);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(kc + k0 * (D / 2) + swz(k0, gr) * 16 + t * 4);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(kc + k1 * (D / 2) + swz(k1, gr) * 16 + t * 4);
        const uint32_t lo[4] = {code_pair(w0), code_pair(w1), code_pair(w0 >> 4), code_pair(w1 >> 4)};
        const uint32_t hi[4] = {code_pair(w0 >> 8), code_pair(w1 >> 8), code_pair(w0 >> 12), code_pair(w1 >> 12)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (ROW) {
            mma16816(y[sub][nt], lo, qf[nt][gr][0], qf[nt][gr][1]);
            mma16816(y[sub][nt], hi, qf[nt][gr][2], qf[nt][gr][3]);
          } else {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816(acc, lo, qf[nt][gr][0], qf[nt][gr][1]);
            mma16816(acc, hi, qf[nt][gr][2], qf[nt][gr][3]);
            y[sub][nt][0] = fmaf(acc[0], f0[gr], y[sub][nt][0]);
            y[sub][nt][1] = fmaf(acc[1], f0[gr], y[sub][nt][1]);
            y[sub][nt][2] = fmaf(acc[2], f1[gr], y[sub][nt][2]);
            y[sub][nt][3] = fmaf(acc[3], f1[gr], y[sub][nt][3]);
          }
        }
      }
      if constexpr (ROW) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) y[sub][nt][c] *= c < 2 ? f0[0] : f1[0];
      }
      if (modified || !clear) {
        const int pk[2] = {s.pos[warp][k0], s.pos[warp][k1]};
        if (capped) {
          // cap tanh(x / cap): a polynomial while the warp's |x / cap| is small, else cap (1 - 2 / (1 + e^(2 x / cap)))
          float big = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) big = fmaxf(big, fabsf(y[sub][nt][c]));
          if (__all_sync(kFull, big * inv_cap <= kTanhRange)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) y[sub][nt][c] *= tanh_over_z(y[sub][nt][c] * inv_cap) * kLog2e;
          } else if (a.mods.softcap > kFineCap) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) y[sub][nt][c] = capped_base2(y[sub][nt][c], y[sub][nt][c] * inv_cap, a.mods.softcap);
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                y[sub][nt][c] = fmaf(-2.f * a.mods.softcap, rcp_approx(1.f + ex2_approx(y[sub][nt][c] * (inv_cap * (2.f * kLog2e)))),
                                     a.mods.softcap) * kLog2e;
          }
        }
        if (biased) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              y[sub][nt][c] = fmaf(-slope[nt][c & 1], static_cast<float>(__sad(q_hi[nt][c & 1], pk[c >> 1], 0u)), y[sub][nt][c]);
        }
        if (!clear) {
          const bool in_use[2] = {i * kTile + k0 < un.n, i * kTile + k1 < un.n};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int e = c & 1, k = c >> 1;
              const bool seen = in_use[k] && ((pk[k] <= q_hi[nt][e] && (!MODS || pk[k] >= q_lo[nt][e])) || (MODS && pk[k] < prefix));
              if (!seen) y[sub][nt][c] = -INFINITY;
            }
        }
      }
      if (a.logits) {
        float* dst = log_row + (static_cast<int64_t>(i) * kTile + sub * 16) * a.logit_stride;
        if (clear || i * kTile + k0 < un.n) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (r0 + nt * 8 + 2 * t < a.logit_stride)
              *reinterpret_cast<float2*>(dst + nt * 8) = make_float2(y[sub][nt][0], y[sub][nt][1]);
        }
        if (clear || i * kTile + k1 < un.n) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (r0 + nt * 8 + 2 * t < a.logit_stride)
              *reinterpret_cast<float2*>(dst + 8 * a.logit_stride + nt * 8) = make_float2(y[sub][nt][2], y[sub][nt][3]);
        }
      }
    }

    take(y);

    // ---- O^T += V^T P^T
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int k0 = sub * 16 + g, k1 = k0 + 8;
      float f0[NG], f1[NG];
      scale_f(1, k0, f0);
      scale_f(1, k1, f1);
      uint32_t pb[NT][2], rest[NT][2];
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        if (!ROW || gr == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            weights<TREE>(y[sub][nt][0] * f0[gr], y[sub][nt][1] * f0[gr], &pb[nt][0], &rest[nt][0]);
            weights<TREE>(y[sub][nt][2] * f1[gr], y[sub][nt][3] * f1[gr], &pb[nt][1], &rest[nt][1]);
          }
        }
        uint32_t w[4];                             // rows 2t, 2t + 1, 2t + 8, 2t + 9; word g & 3 of the chunk
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = sub * 16 + 2 * t + (k & 1) + (k >> 1) * 8;
          w[k] = *reinterpret_cast<const uint32_t*>(vc + key * (D / 2) + swz(key, gr) * 16 + (g & 3) * 4);
        }
        const uint32_t x0 = __byte_perm(w[0], w[1], half_sel), x1 = __byte_perm(w[2], w[3], half_sel);
        const uint32_t a0[4] = {code_pair(x0), code_pair(x0 >> 4), code_pair(x1), code_pair(x1 >> 4)};
        const uint32_t a1[4] = {code_pair(x0 >> 8), code_pair(x0 >> 12), code_pair(x1 >> 8), code_pair(x1 >> 12)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(o[gr][0][nt], a0, pb[nt][0], pb[nt][1]);
          mma16816(o[gr][1][nt], a1, pb[nt][0], pb[nt][1]);
          if constexpr (TREE) {
            mma16816(o[gr][0][nt], a0, rest[nt][0], rest[nt][1]);
            mma16816(o[gr][1][nt], a1, rest[nt][0], rest[nt][1]);
          }
        }
      }
    }
    __syncwarp();
    st = (st + 1) % kStages;
  }
  cp_async_wait<0>();

  if constexpr (TREE) {
    if (split == a.splits - 1 && warp == kWarps - 1 && nodes > 0) {
      const int64_t base = un.b * a.tree.news.batch + un.l * a.tree.news.layer + un.g * a.tree.news.head;
      float y[2][NT][4] = {};
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int k0 = sub * 16 + g, k1 = k0 + 8;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          auto piece = [&](int k) {
            return k < nodes ? *reinterpret_cast<const uint4*>(a.tree.k_new + base + k * a.tree.news.token + 32 * gr + 8 * t)
                             : make_uint4(0, 0, 0, 0);
          };
          const uint4 w0 = piece(k0), w1 = piece(k1);
          const uint32_t lo[4] = {__byte_perm(w0.x, w0.z, 0x5410), __byte_perm(w1.x, w1.z, 0x5410),
                                  __byte_perm(w0.x, w0.z, 0x7632), __byte_perm(w1.x, w1.z, 0x7632)};
          const uint32_t hi[4] = {__byte_perm(w0.y, w0.w, 0x5410), __byte_perm(w1.y, w1.w, 0x5410),
                                  __byte_perm(w0.y, w0.w, 0x7632), __byte_perm(w1.y, w1.w, 0x7632)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(y[sub][nt], lo, qf[nt][gr][0], qf[nt][gr][1]);
            mma16816(y[sub][nt], hi, qf[nt][gr][2], qf[nt][gr][3]);
          }
        }
        const int pk[2] = {next + __shfl_sync(kFull, depth, k0), next + __shfl_sync(kFull, depth, k1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t mine = __shfl_sync(kFull, above, min(r0 + nt * 8 + 2 * t + e, un.R - 1) / a.G);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float& x = y[sub][nt][2 * k + e];
              x *= pre;
              if (capped) x = capped_base2(x, x * inv_cap, a.mods.softcap);
              if (biased) x = fmaf(-slope[nt][e], static_cast<float>(__sad(q_hi[nt][e], pk[k], 0u)), x);
              const int j = k ? k1 : k0;
              if (j >= nodes || !((mine >> j) & 1) || (MODS && pk[k] < q_lo[nt][e] && pk[k] >= prefix)) x = -INFINITY;
            }
          }
      }
      take(y);
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        uint32_t pb[NT][2], rest[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          weights<TREE>(y[sub][nt][0], y[sub][nt][1], &pb[nt][0], &rest[nt][0]);
          weights<TREE>(y[sub][nt][2], y[sub][nt][3], &pb[nt][1], &rest[nt][1]);
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          uint2 w[4];                              // four columns of rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = sub * 16 + 2 * t + (k & 1) + (k >> 1) * 8;
            w[k] = key < nodes ? *reinterpret_cast<const uint2*>(a.tree.v_new + base + key * a.tree.news.token + 32 * gr +
                                                                 8 * (g & 3) + 4 * (g >> 2))
                               : make_uint2(0, 0);
          }
          const uint32_t a0[4] = {__byte_perm(w[0].x, w[1].x, 0x5410), __byte_perm(w[0].x, w[1].x, 0x7632),
                                  __byte_perm(w[2].x, w[3].x, 0x5410), __byte_perm(w[2].x, w[3].x, 0x7632)};
          const uint32_t a1[4] = {__byte_perm(w[0].y, w[1].y, 0x5410), __byte_perm(w[0].y, w[1].y, 0x7632),
                                  __byte_perm(w[2].y, w[3].y, 0x5410), __byte_perm(w[2].y, w[3].y, 0x7632)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816(o[gr][0][nt], a0, pb[nt][0], pb[nt][1]);
            mma16816(o[gr][1][nt], a1, pb[nt][0], pb[nt][1]);
            mma16816(o[gr][0][nt], a0, rest[nt][0], rest[nt][1]);
            mma16816(o[gr][1][nt], a1, rest[nt][0], rest[nt][1]);
          }
        }
      }
    }
  }

  // ---- join the warps: sums over the lanes' keys, one reference maximum, outputs added in warp order
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) l[nt][e] += __shfl_xor_sync(kFull, l[nt][e], k);
      if (g == 0) {
        s.m[warp][nt * 8 + 2 * t + e] = m[nt][e];
        s.l[warp][nt * 8 + 2 * t + e] = l[nt][e];
      }
    }
  __syncthreads();
  auto block_max = [&](int c) {
    float x = s.m[0][c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) x = fmaxf(x, s.m[w][c]);
    return x;
  };
  float f[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) f[nt][e] = m[nt][e] == -INFINITY ? 0.f : ex2_approx(m[nt][e] - block_max(nt * 8 + 2 * t + e));
  const int rows_here = min(NT * 8, un.R - r0);
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    if (warp / (kWarps / 2) == half) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = nt * 8 + 2 * t + e;
          if (c >= rows_here) continue;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr)
            *reinterpret_cast<float4*>(&s.part[warp % (kWarps / 2)][c][32 * gr + 8 * (g & 3) + 4 * (g >> 2)]) =
                make_float4(o[gr][0][nt][e] * f[nt][e], o[gr][0][nt][e + 2] * f[nt][e], o[gr][1][nt][e] * f[nt][e],
                            o[gr][1][nt][e + 2] * f[nt][e]);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows_here * (D / 4); i += kThreads) {
      const int c = i / (D / 4), d0 = i % (D / 4) * 4;
      float4 x = half ? *reinterpret_cast<const float4*>(&s.o[c][d0]) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps / 2; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(&s.part[w][c][d0]);
        x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
      }
      *reinterpret_cast<float4*>(&s.o[c][d0]) = x;
    }
    __syncthreads();
  }
  if (threadIdx.x < NT * 8) {
    const int c = threadIdx.x;
    const float mm = block_max(c);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      // (a sum of NaN has no maximum)
      if (s.m[w][c] != -INFINITY || (TREE && isnan(s.l[w][c]))) sum = fmaf(s.l[w][c], ex2_approx(s.m[w][c] - mm), sum);
    s.ml[c] = make_float2(mm, sum);
  }
  __syncthreads();
  constexpr int LPR = D / 8;                       // lanes per output row
  for (int c = threadIdx.x / LPR; c < rows_here; c += kThreads / LPR) {
    const int r = r0 + c, d0 = threadIdx.x % LPR * 8;
    const float2 ml = s.ml[c];
    const float* x = &s.o[c][d0];
    if (a.splits > 1) {
      const int64_t part = (static_cast<int64_t>(un.u) * un.R + r) * a.splits + split;
#pragma unroll
      for (int k = 0; k < 8; k += 4)
        *reinterpret_cast<float4*>(a.part_o + part * D + d0 + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
      if (d0 == 0) a.part_ml[part] = ml;
    } else if (!TREE || r < nodes * a.G) {         // (rows behind a tree's nodes are left as they were)
      const float inv = ml.y > 0.f ? 1.f / ml.y : 0.f;
      *reinterpret_cast<uint4*>(a.out + un.q_at(a, a.os, r) + d0) =
          make_uint4(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv),
                     pack_bf16x2(x[4] * inv, x[5] * inv), pack_bf16x2(x[6] * inv, x[7] * inv));
      if (d0 == 0) {
        // (of a tree's row of NaN: NaN)
        const bool none = TREE ? ml.y == 0.f : !(ml.y > 0.f);
        if (a.lse) a.lse[un.lse_at(a, r)] = none ? -INFINITY : (ml.x + log2f(ml.y)) * kLn2;
        if (a.part_ml) a.part_ml[static_cast<int64_t>(un.u) * un.R + r] = ml;
      }
    }
  }
}

// Second kernel: blocks [0, a.merge_blocks) of a unit join the splits of its
// rows, the others add the weights of their keys to the mass.
constexpr int kFinThreads = 256;
// Query rows up to which a thread adds a key's weights alone.  Measured: 4 rows of 32 units of 100K to 131K keys 142 us
// alone, 172 by groups of lanes; 128 rows of 8 units of 8,192 keys 176 us alone (each lane's logits lie 512 bytes from
// the next one's), 63 by groups.
constexpr int kFewRows = 8;

template <int D>
__global__ void __launch_bounds__(kFinThreads, 4) i4_finish_kernel(const I4AttnArgs a) {
  extern __shared__ float lse2[];                  // base-2 log-sum-exp of each row (mass blocks)
  if (static_cast<int>(blockIdx.y + blockIdx.z * 65535) >= a.U) return;
  const Unit un(a, blockIdx.y + blockIdx.z * 65535);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_previous_kernel();
  // Every load that does not depend on another is issued first: this kernel is a few latencies long.
  if (static_cast<int>(blockIdx.x) < a.merge_blocks) {
    const int r = blockIdx.x * (kFinThreads / 32) + warp;
    if (r >= un.R) return;
    const int64_t part = (static_cast<int64_t>(un.u) * un.R + r) * a.splits;
    const float* src = a.part_o + part * D + lane * (D / 32);
    float2 v[kMaxSplits / 32];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMaxSplits / 32; ++k)
      v[k] = k * 32 + lane < a.splits ? a.part_ml[part + k * 32 + lane] : make_float2(-INFINITY, 0.f);
    float x[D / 32] = {}, sum = 0.f;
    constexpr int kAhead = 8;
    using Vec = typename std::conditional<D == 128, float4, float2>::type;
    Vec o[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) o[i] = *reinterpret_cast<const Vec*>(src + min(i, a.splits - 1) * D);
#pragma unroll
    for (int k = 0; k < kMaxSplits / 32; ++k) top = fmaxf(top, v[k].x);
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, k));
    float w[kMaxSplits / 32];
#pragma unroll
    for (int k = 0; k < kMaxSplits / 32; ++k) {
      w[k] = v[k].x == -INFINITY ? 0.f : ex2_approx(v[k].x - top);
      sum = fmaf(v[k].y, w[k], sum);
    }
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(kFull, sum, k);
#pragma unroll
    for (int k = 0; k < kMaxSplits / 32; ++k) {
#pragma unroll 1
      for (int i0 = 0; i0 < 32 && k * 32 + i0 < a.splits; i0 += kAhead) {
        if (k + i0 > 0) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i)
            o[i] = *reinterpret_cast<const Vec*>(src + static_cast<int64_t>(min(k * 32 + i0 + i, a.splits - 1)) * D);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float wi = __shfl_sync(kFull, w[k], i0 + i);       // 0 past the last split
          const float* e = reinterpret_cast<const float*>(&o[i]);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) x[c] = fmaf(e[c], wi, x[c]);
        }
      }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    __nv_bfloat16* out = a.out + un.q_at(a, a.os, r) + lane * (D / 32);
#pragma unroll
    for (int c = 0; c < D / 32; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(x[c] * inv, x[c + 1] * inv);
    if (lane == 0 && a.lse) a.lse[un.lse_at(a, r)] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
    return;
  }
  // Mass.  Few query rows: four keys of a thread at once, two query rows per load.  More: a group of lanes per key, each
  // with two query rows, so that a warp reads keys that follow each other as one piece.  Loads of keys past the rows in
  // use stay inside the unit's logits (their values are not used).
  const bool few = un.R <= kFewRows;
  const int j0 = (blockIdx.x - a.merge_blocks) * a.mass_keys, cap = a.rows.capacity;
  auto key_at = [&](int j, int k) { return un.base + min(j + k * kFinThreads, cap - 1); };
  float old[4];
  float2 y[2][4];                                // of rows 0..3
  auto load = [&](int j, int r, float2 (&to)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) to[k] = *reinterpret_cast<const float2*>(a.logits + key_at(j, k) * a.logit_stride + r);
  };
  auto load_first = [&](int j) {
#pragma unroll
    for (int k = 0; k < 4; ++k) old[k] = a.rows.mass[key_at(j, k)];
    load(j, 0, y[0]);
    load(j, min(2, a.logit_stride - 2), y[1]);
  };
  if (few) load_first(j0 + threadIdx.x);
  // base-2 log-sum-exps; splits <= kMaxSplits: four per lane, read once, of `rows` rows together
  auto statistics = [&](int r, auto rows_c) {
    constexpr int rows = decltype(rows_c)::value, stride = kFinThreads / 32;
    float2 v[rows][kMaxSplits / 32];
#pragma unroll
    for (int i = 0; i < rows; ++i) {
      const float2* ml = a.part_ml + (static_cast<int64_t>(un.u) * un.R + min(r + i * stride, un.R - 1)) * a.splits;
#pragma unroll
      for (int k = 0; k < kMaxSplits / 32; ++k)
        v[i][k] = k * 32 + lane < a.splits ? ml[k * 32 + lane] : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int i = 0; i < rows; ++i) {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < kMaxSplits / 32; ++k) top = fmaxf(top, v[i][k].x);
      for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, k));
#pragma unroll
      for (int k = 0; k < kMaxSplits / 32; ++k)
        if (v[i][k].x != -INFINITY) sum = fmaf(v[i][k].y, ex2_approx(v[i][k].x - top), sum);
      for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(kFull, sum, k);
      // nothing seen: every logit is -inf
      if (lane == 0 && r + i * stride < un.R) lse2[r + i * stride] = sum > 0.f ? top + log2f(sum) : 0.f;
    }
  };
  if (few) {
    if (warp < un.R) statistics(warp, std::integral_constant<int, 1>{});
  } else {
#pragma unroll 1
    for (int r = warp; r < un.R; r += kFinThreads / 32 * 4) statistics(r, std::integral_constant<int, 4>{});
  }
  const int j1 = min(un.n, j0 + a.mass_keys);
  __syncthreads();
  if (!few) {
    const int pairs = a.logit_stride / 2;
    int group = 4;                                 // lanes of a key
    while (group < pairs && group < 32) group *= 2;
    const int keys = 32 / group, own = lane & (group - 1), step = kFinThreads / 32 * keys;
    for (int jb = j0 + warp * keys; jb < j1; jb += 4 * step) {
      const int j = jb + lane / group;
      float was[4], sum[4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) was[k] = own == 0 ? a.rows.mass[un.base + min(j + k * step, cap - 1)] : 0.f;
      for (int q = own; q < pairs; q += group) {
        float2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          v[k] = *reinterpret_cast<const float2*>(a.logits + (un.base + min(j + k * step, cap - 1)) * a.logit_stride + 2 * q);
        const bool two = 2 * q + 1 < un.R;         // a padding column adds nothing
        const float l0 = lse2[2 * q], l1 = two ? lse2[2 * q + 1] : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] += ex2_approx(v[k].x - l0) + (two ? ex2_approx(v[k].y - l1) : 0.f);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        for (int o = 1; o < group; o <<= 1) sum[k] += __shfl_xor_sync(kFull, sum[k], o);
        if (own == 0 && j + k * step < j1) a.rows.mass[un.base + j + k * step] = was[k] + sum[k];
      }
    }
    return;
  }
  for (int j = j0 + threadIdx.x; j < j1; j += kFinThreads * 4) {
    if (j >= j0 + kFinThreads) load_first(j);
    float sum[4] = {};
    for (int r = 0; r < un.R; r += 2) {
      if (r >= 4) {
        if ((r >> 1) & 1) load(j, r, y[1]);
        else load(j, r, y[0]);
      }
      const bool two = r + 1 < un.R;             // a padding column adds nothing
      const float l0 = lse2[r], l1 = two ? lse2[r + 1] : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = (r >> 1) & 1 ? y[1][k] : y[0][k];
        sum[k] += ex2_approx(v.x - l0) + (two ? ex2_approx(v.y - l1) : 0.f);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (j + k * kFinThreads < j1) a.rows.mass[un.base + j + k * kFinThreads] = old[k] + sum[k];
  }
}

template <int D, int NT, bool ROW, bool TREE = false>
cudaError_t launch_one(const I4AttnArgs& a, cudaStream_t stream) {
  // the plain scores' kernel is one of its own: with the branches of the others in its loop it takes 3-4 % longer
  const bool mods = a.mods.softcap > 0.f || a.mods.slopes || a.mods.window || a.mods.prefix_len;
  auto kernel = mods ? i4_attn_kernel<D, NT, ROW, true, TREE> : i4_attn_kernel<D, NT, ROW, false, TREE>;
  const int bytes = static_cast<int>(sizeof(Smem<D, NT, ROW>));
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int R = a.n_q * a.G;
  const dim3 grid((R + NT * 8 - 1) / (NT * 8) * a.splits, std::min(a.U, 65535), (a.U + 65534) / 65535);
  return launch_after(kernel, grid, kThreads, bytes, stream, a);
}

template <int D, bool ROW>
cudaError_t launch_rows(const I4AttnArgs& a, cudaStream_t stream) {
  const int R = a.n_q * a.G;
  if (R <= 8) return launch_one<D, 1, ROW>(a, stream);
  if (R <= 16) return launch_one<D, 2, ROW>(a, stream);
  return launch_one<D, 4, ROW>(a, stream);
}

}  // namespace

cudaError_t launch_i4_attn(const I4AttnArgs& a, cudaStream_t stream) {
  const bool row = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  cudaError_t e = a.d == 128 ? (row ? launch_rows<128, true>(a, stream) : launch_rows<128, false>(a, stream))
                             : (row ? launch_rows<64, true>(a, stream) : launch_rows<64, false>(a, stream));
  const int mass_blocks = a.add_mass ? (a.rows.capacity + a.mass_keys - 1) / a.mass_keys : 0;
  if (e != cudaSuccess || a.merge_blocks + mass_blocks == 0) return e;
  const dim3 grid(a.merge_blocks + mass_blocks, std::min(a.U, 65535), (a.U + 65534) / 65535);
  const size_t bytes = a.add_mass ? static_cast<size_t>(a.n_q) * a.G * sizeof(float) : 0;
  return launch_after(a.d == 128 ? i4_finish_kernel<128> : i4_finish_kernel<64>, grid, kFinThreads, bytes, stream, a);
}

cudaError_t launch_i4_tree(const I4AttnArgs& a, cudaStream_t stream) {
  const bool row = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  const int R = a.n_q * a.G;
  auto go = [&](auto d, auto r) -> cudaError_t {
    constexpr int D = decltype(d)::value;
    constexpr bool ROW = decltype(r)::value;
    if (R <= 8) return launch_one<D, 1, ROW, true>(a, stream);
    if constexpr (D == 64)
      if (R > 16) return launch_one<D, 4, ROW, true>(a, stream);
    return launch_one<D, 2, ROW, true>(a, stream);
  };
  using D128 = std::integral_constant<int, 128>;
  using D64 = std::integral_constant<int, 64>;
  if (a.d == 128) return row ? go(D128{}, std::true_type{}) : go(D128{}, std::false_type{});
  return row ? go(D64{}, std::true_type{}) : go(D64{}, std::false_type{});
}

}  // namespace kvc
