// Attention of a prompt, a chunk of one or single tokens over a bf16 cache
// (PASK Eq. 1) with score modifiers, documents and a prefix.
//
// Rows.  The G heads that share a KV head are packed: row r of a unit is
// query r / G of head r % G, so one read of a key tile serves all of them and
// a single token fills G rows of a tile instead of one.
//
// One CTA per SM works on one item: a block of 256 rows of a unit (two tiles
// of 128 that share every key and value tile) or, where that leaves SMs idle
// or the unit has no more, of 128 rows, whose two streams take the key tiles
// in turn.  Either way two streams run against each other on the tensor core:
// while the warps of one turn scores into weights, the other's products run.
// Per step of a stream
//   S = Q K^T      tcgen05, operands in shared memory, S in tensor memory
//   softmax        128 threads, one row each: S to registers, running maximum
//                  and sum (base 2), P = 2^(y - m) rounded to bf16 and stored
//                  over S in tensor memory; the accumulator is rescaled only
//                  when the maximum grew by more than 2^8 (P then stays below
//                  2^8 and every sum in fp32), which a row does a few times
//   O += P V       tcgen05, P from tensor memory, V read as an MN-major
//                  operand straight from its TMA tile.  P is rounded to bf16
//                  because the product wants the values' own type: half a step,
//                  2^-8 of a weight, as much as the output's own rounding; the
//                  row's sum is that of the unrounded weights
// Few rows: the keys of an item are split over CTAs and the partial (m, l, O)
// joined by PASK Eq. 15 in a second kernel.
//
// A capped score is s times a polynomial in s^2 while |s scale / cap| stays
// within 0.625 over a warp's tile (else cap (1 - 2 / (1 + e^2z))); slopes add
// two packed operations an element pair.  Where the polynomial's coefficients
// for s leave fp32's range (caps far above or below the scale), and where caps
// above 1,024 would make the second form coarse, another instance of the kernel
// works in z = s scale / cap and chooses the form score by score (as a branch
// of the first one it cost every capped call 2 to 6 %: spills).
//
// Masks.  An item walks only key tiles that some of its rows see; a tile that
// every row of a warp sees whole takes no mask.  Values of keys that no row of
// the item sees are zeroed in shared memory (0 x NaN is NaN in a product).
//
// Outputs are staged in shared memory; a warp whose 32 rows are whole queries
// sends them by tensor copies (documents 84.8 us, 86.6 by its own stores),
// others store whole rows.
//
// Warp roles (12 warps): 0-3 and 4-7 softmax of stream 0 and 1 (a row of 128
// scores per thread in registers: their warpgroups take 200 registers a
// thread, the third gives them up and keeps 104; 2 x 200 + 104 = 3 x 168, what
// the block was launched with), 8 barriers, the item and every TMA copy (the
// first queries and keys are sent for before the block has met), 9 TMEM owner
// and MMA issuer.  Every wait is bounded; one that gives up raises a shared
// abort flag, the unit is marked KVC_UNIT_TIMEOUT and the CTA drains its
// copies and MMAs before it frees tensor memory.
//
// Bounds.  A step of 128 x 128 scores at d = 128 takes the tensor core 1,024
// cycles and its softmax 640 warp instructions a warp, 1,150 with a cap, which
// two warps per scheduler cannot hide behind each other's latencies: about
// 1,400 and 2,300 cycles a step.  Measured, replayed from a graph (32 query
// heads over 8, d = 128): 8,192 causal tokens 350 us = 1,570 TFLOP/s, 84 % of
// the measured bf16 peak, tensor pipe 67 % active; capped 523 us = 1,050
// TFLOP/s, 751 us with scores past 0.625 of the cap in every tile.  One token over
// 16 sequences of up to 32,768: 180 us = 6.5 TB/s, 96 % of the measured
// bandwidth; 208 us capped, 268 past 0.625.  300 tokens: 9.3 us.  Beside its
// steps an item costs about 11,000 cycles: 1,400 to set up, 2,300 until the
// first scores are there, 2,200 to read and stage its outputs, 1,200 until the
// next block of the SM begins.
// Tried and slower: one persistent CTA per SM with its outputs under the next
// item's loads (407 us against 389: a value stage less, spills), scores read
// from tensor memory in parts (422 against 365: spills).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvc_internal.cuh"
#include "packed_math.cuh"
#include "tc_attn.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 384;                    // three warpgroups of 168 registers a thread at launch
constexpr int kTileRows = 128;
constexpr int kKeys = 128;                       // keys per tile
constexpr uint32_t kTmemCols = 512;              // S0, S1, O0, O1 of 128 columns each
constexpr uint32_t kOCol = 256;
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;                     // log2 growth of the maximum that forces a rescale

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTile = kChunks * kChunkBytes;          // a Q, K or V tile
  static constexpr int kNk = D == 128 ? 2 : 4, kNv = D == 128 ? 3 : 4;
  static constexpr int kSmem = (2 + kNk + kNv) * kTile + 1024 /* alignment */ + 512 /* Bars */;
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_store_5d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// Until the stores of this thread have read their sources.
__device__ __forceinline__ void tma_store_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}

// What an item covers.
struct Item {
  int u, b, l, g, split;
  int row0, rows;              // first packed row, packed rows of the item (<= 256)
  int nk, first, pre;          // keys, position of query 0, visible prefix
  int lo, hi;                  // keys [lo, hi) are seen through the causal window by some row
  int n, skip_at, skip;        // tiles to walk: index i is tile i, or i + skip from skip_at on
  int i0, i1;                  // indices of this split
};

__device__ __forceinline__ Item make_item(const PromptArgs& a, int id) {
  Item t;
  uint32_t split, u, g, l;
  const uint32_t qb_rev = a.by_units.divmod(a.by_splits.divmod(id, &split), &u);
  t.split = static_cast<int>(split);
  t.u = static_cast<int>(u);
  const int qb = a.n_blocks - 1 - static_cast<int>(qb_rev);      // long rows first: the causal tail fills the gaps
  t.b = static_cast<int>(a.by_layers.divmod(a.by_heads.divmod(u, &g), &l));
  t.l = static_cast<int>(l);
  t.g = static_cast<int>(g);
  t.nk = a.kv_len ? max(0, min(static_cast<int>(a.T), a.kv_len[t.b])) : static_cast<int>(a.T);
  const int nq = a.q_len ? clamp_count(a.q_len[t.b], a.n_q) : a.n_q;
  t.first = t.nk - nq;
  t.row0 = qb * a.block_rows;
  t.rows = min(a.block_rows, nq * a.G - t.row0);
  t.pre = a.mods.prefix_len ? max(0, min(t.nk, a.mods.prefix_len[t.b])) : 0;
  if (t.rows <= 0) {
    t.rows = t.lo = t.hi = t.n = t.skip = t.skip_at = t.i0 = t.i1 = 0;
    return t;
  }
  const int p_min = t.first + static_cast<int>(a.by_group.div(t.row0)),
            p_max = t.first + static_cast<int>(a.by_group.div(t.row0 + t.rows - 1));
  t.hi = max(0, p_max + 1);
  t.lo = a.mods.window && p_min >= a.mods.window ? p_min - a.mods.window + 1 : 0;
  t.lo = min(t.lo, t.hi);
  if (p_max < 0) t.pre = 0;
  const int pre_tiles = (t.pre + kKeys - 1) / kKeys;
  const int lo_tile = t.lo / kKeys, hi_tile = (t.hi + kKeys - 1) / kKeys;
  t.skip_at = pre_tiles;
  t.skip = max(0, lo_tile - pre_tiles);
  t.n = max(pre_tiles, hi_tile) - t.skip;
  if (hi_tile <= lo_tile) t.n = pre_tiles, t.skip = 0;
  t.i0 = static_cast<int>(a.by_splits.div(static_cast<uint32_t>(t.n) * split));      // tiles < 2^24, splits <= 256
  t.i1 = t.split + 1 == a.splits ? t.n : static_cast<int>(a.by_splits.div(static_cast<uint32_t>(t.n) * (split + 1)));
  return t;
}

__device__ __forceinline__ Item uniform_item(const Item& from) {
  static_assert(sizeof(Item) % 4 == 0, "an Item is ints");
  Item t;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(Item) / 4); ++i)
    reinterpret_cast<int*>(&t)[i] = uniform(reinterpret_cast<const int*>(&from)[i]);
  return t;
}

// The tiles of an item that may be seen, in order; every lane of the warp
// calls next() together.
struct TileWalk {
  int skip_at, skip, end;
  const int2* table;           // [tiles] (min, max) document of each key tile, or null
  int q_min, q_max;            // documents of the item's queries
  int at, base;
  uint32_t mask;
  __device__ TileWalk(const Item& t, const int2* table_, int q_min_, int q_max_)
      : skip_at(t.skip_at), skip(t.skip), end(t.i1), table(table_), q_min(q_min_), q_max(q_max_), at(t.i0), base(0), mask(0) {}
  __device__ __forceinline__ int tile(int i) const { return i + (i >= skip_at ? skip : 0); }
  __device__ __forceinline__ int next() {
    if (!table) return at < end ? tile(at++) : -1;
#pragma unroll 1
    while (mask == 0) {
      if (at >= end) return -1;
      const int i = at + (threadIdx.x & 31);
      bool ok = false;
      if (i < end) {
        const int2 d = table[tile(i)];
        ok = d.y >= q_min && d.x <= q_max;
      }
      mask = __ballot_sync(0xffffffffu, ok);
      base = at;
      at += 32;
    }
    const int i = base + __ffs(mask) - 1;          // uniform: a ballot's bits
    mask &= mask - 1;
    return tile(i);
  }
};

struct Bars {
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t sfull[2], phalf[2], pfull[2], odone[2], qfull[2], done;
  uint32_t tmem;
  int abort_flag;
  int q_min, q_max;
  int tiles[2];                // of each stream
  Item item;
};
static_assert(sizeof(Bars) <= 512, "Cfg::kSmem");

// One tile of keys or values; one tile of queries (one thread).
template <int D>
__device__ __forceinline__ void load_tile(uint8_t* to, uint64_t* full, const CUtensorMap& map, const Item& t, int tile) {
  mbar_arrive_expect_tx(smem_u32(full), Cfg<D>::kTile);
  for (int c = 0; c < Cfg<D>::kChunks; ++c)
    tma_load_5d(smem_u32(to + c * kChunkBytes), &map, smem_u32(full), c * 64, tile * kKeys, t.g, t.l, t.b);
}

template <int D>
__device__ __forceinline__ void load_queries(Bars& s, uint8_t* sq, const CUtensorMap& map, const PromptArgs& a, const Item& t,
                                             int i) {
  mbar_arrive_expect_tx(smem_u32(&s.qfull[i]), Cfg<D>::kTile);
  for (int c = 0; c < Cfg<D>::kChunks; ++c)
    tma_load_5d(smem_u32(sq + i * Cfg<D>::kTile + c * kChunkBytes), &map, smem_u32(&s.qfull[i]), c * 64, t.g * a.G,
                static_cast<int>(a.by_group.div(t.row0 + i * kTileRows)), t.l, t.b);
}

// The polynomial in x^2 with coefficients c, lowest first: of the odd function x p(x^2).
__device__ __forceinline__ uint64_t odd_factor(uint64_t x, const float (&c)[5]) {
  const uint64_t w = mul2(x, x);
  return fma2(fma2(fma2(fma2(pair(c[4], c[4]), w, pair(c[3], c[3])), w, pair(c[2], c[2])), w, pair(c[1], c[1])), w,
              pair(c[0], c[0]));
}

// D: head dimension.  CAP: the logits are capped; WIDE: by a cap that the
// polynomial in s does not serve (cap_is_wide).  BIAS: they get slopes.
template <int D, bool CAP, bool BIAS, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
              const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const PromptArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sq = base;                                  // two Q tiles
  uint8_t* sk = sq + 2 * C::kTile;
  uint8_t* sv = sk + C::kNk * C::kTile;
  Bars& s = *reinterpret_cast<Bars*>(sv + C::kNv * C::kTile);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s.abort_flag;
  // One thread of the load warp sets up the barriers, works out the item and sends for the first queries and keys
  // (the first tile of an item with documents depends on them), while another warp allocates tensor memory.
  if (warp == kLoadWarp && lane == 0) {
    if (a.q_tma) tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s.kfull[i]), 1);
      mbar_init(smem_u32(&s.kempty[i]), 1);
      mbar_init(smem_u32(&s.vfull[i]), 1);
      mbar_init(smem_u32(&s.vempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.sfull[i]), 1);
      mbar_init(smem_u32(&s.phalf[i]), 4);
      mbar_init(smem_u32(&s.pfull[i]), 4);
      mbar_init(smem_u32(&s.odone[i]), 1);
      mbar_init(smem_u32(&s.qfull[i]), a.q_tma ? 1 : 4);
    }
    mbar_init(smem_u32(&s.done), 1);
    s.abort_flag = 0;
    s.q_min = INT32_MAX;
    s.q_max = -1;
    fence_barrier_init();
    wait_for_previous_kernel();
    const Item t = make_item(a, blockIdx.x);
    s.item = t;
    if (t.rows > 0) {
      // (a.stall_unit: a test makes the first key tile's wait expect 16 bytes more than its copies bring)
      if (t.u == a.stall_unit) mbar_expect_tx(smem_u32(&s.kfull[0]), 16);
      if (a.q_tma) load_queries<D>(s, sq, map_q, a, t, 0);
      if (!a.docs && t.i0 < t.i1)
        load_tile<D>(sk, &s.kfull[0], map_k, t, t.i0 + (t.i0 >= t.skip_at ? t.skip : 0));
      if (a.q_tma && t.rows > kTileRows) load_queries<D>(s, sq, map_q, a, t, 1);
      if (a.o_tma) tma_prefetch_desc(&map_o);
    }
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s.tmem), kTmemCols);
    tmem_relinquish();
  }
  wait_for_previous_kernel();                            // its results, or the documents of the key tiles
  let_next_kernel_start();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s.tmem);
  const Item t = uniform_item(s.item);
  const bool share = t.rows > kTileRows;               // two Q tiles, or two streams over one
  if (t.rows == 0) {                                   // rows past the sequence's queries
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  const int32_t* docs = a.docs ? a.docs + static_cast<int64_t>(t.b) * a.T : nullptr;
  const int2* table = a.docs ? a.doc_tiles + static_cast<int64_t>(t.b) * a.n_tiles : nullptr;

  // Q tiles: one copy per 64 columns and tile where whole queries fill a tile's rows (the producer issues it), else
  // the softmax warps load their 32 rows, two at a time (16 lanes a row; four at d = 64), and store them in the
  // operand's swizzled chunks.  And the documents of the queries' positions.
  if (warp < 8) {
    const int tile = warp >> 2, row = tile * kTileRows + (threadIdx.x & 127);
    if (tile == 0 || share) {
      const bool ok = row < t.rows;
      const int pr = t.row0 + (ok ? row : 0);
      if (!a.q_tma) {
        const __nv_bfloat16* q = a.q + t.b * a.qs.batch + t.l * a.qs.layer;
        const int64_t own = static_cast<int64_t>(t.g * a.G + pr % a.G) * a.qs.head + static_cast<int64_t>(pr / a.G) * a.qs.token;
        constexpr int LPR = D / 8;
        const int chunk = lane % LPR;
        uint8_t* dst = sq + tile * C::kTile + (chunk >> 3) * kChunkBytes;
#pragma unroll 1
        for (int i0 = 0; i0 < LPR; i0 += 8) {
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (i0 + i) * (32 / LPR) + lane / LPR;
            const int64_t at = __shfl_sync(0xffffffffu, own, r);
            w[i] = row - lane + r < t.rows ? reinterpret_cast<const uint4*>(q + at)[chunk] : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rt = (warp & 3) * 32 + (i0 + i) * (32 / LPR) + lane / LPR;
            *reinterpret_cast<uint4*>(dst + rt * 128 + (((chunk & 7) ^ (rt & 7)) << 4)) = w[i];
          }
        }
      }
      if (docs) {
        const int p = t.first + pr / a.G;
        const int doc = ok && p >= 0 ? docs[p] : -1;
        const int lo = __reduce_min_sync(0xffffffffu, doc >= 0 ? doc : INT32_MAX), hi = __reduce_max_sync(0xffffffffu, doc);
        if (lane == 0) {
          atomicMin(&s.q_min, lo);
          atomicMax(&s.q_max, hi);
        }
      }
    }
    if (!a.q_tma) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.qfull[tile]));
    }
  }
  if (docs) __syncthreads();
  const int q_min = docs ? uniform(s.q_min) : 0, q_max = docs ? uniform(s.q_max) : 0;

  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (warp == kLoadWarp) {
    // -------------------------------------------------------------- TMA producer: K(i + 1) before V(i)
    TileWalk walk(t, table, q_min, q_max);
    auto load = [&](const CUtensorMap& map, uint8_t* ring, uint64_t* full, uint64_t* empty, uint32_t n, int i,
                    int tile) -> bool {
      const uint32_t st = i % n, ph = (i / n) & 1;
      if (!warp_wait(smem_u32(&empty[st]), ph ^ 1, abort_flag)) return false;
      if (lane == 0) load_tile<D>(ring + st * C::kTile, &full[st], map, t, tile);
      __syncwarp();
      return true;
    };
    int nk = 0, nv = 0;
    int cur = walk.next();
    bool ok = true;
    if (cur >= 0) {
      if (docs) ok = load(map_k, sk, s.kfull, s.kempty, C::kNk, 0, cur);      // else it is on its way
      if (ok) nk = 1;
    }
    while (cur >= 0 && ok) {
      const int nxt = walk.next();
      if (nxt >= 0) {
        if (!(ok = load(map_k, sk, s.kfull, s.kempty, C::kNk, nk, nxt))) break;
        ++nk;
      }
      if (!(ok = load(map_v, sv, s.vfull, s.vempty, C::kNv, nv, cur))) break;
      ++nv;
      cur = nxt;
    }
    // every copy issued above lands before the CTA exits
    if (a.q_tma) drain(smem_u32(&s.qfull[0]), 0);
    if (a.q_tma && share) drain(smem_u32(&s.qfull[1]), 0);
    for (int i = max(0, nk - C::kNk); i < nk; ++i)
      drain(smem_u32(&s.kfull[i % C::kNk]), (i / C::kNk) & 1);
    for (int i = max(0, nv - C::kNv); i < nv; ++i)
      drain(smem_u32(&s.vfull[i % C::kNv]), (i / C::kNv) & 1);
  } else if (warp == kMmaWarp) {
    // -------------------------------------------------------------- MMA issuer
    const uint32_t idesc_s = mma_idesc_bf16(128, kKeys);
    const uint32_t idesc_o = mma_idesc_bf16(128, D) | (1u << 16);     // B (values) MN-major
    TileWalk walk(t, table, q_min, q_max), walk_v(t, table, q_min, q_max);
    bool ok = warp_wait(smem_u32(&s.qfull[0]), 0, abort_flag);
    const uint32_t elected = elect_one();
    const uint64_t q_desc = sw128_desc(smem_u32(sq)), k_desc = sw128_desc(smem_u32(sk)), val_desc = v_desc(smem_u32(sv));
    int n_k = 0, n_v = 0;                // K and V tiles taken up
    bool k_more = true;
    // the scores of step x (stream x & 1); false when there is no such step
    auto scores = [&](int x) -> bool {
      const int h = x & 1;
      const bool fresh = !share || h == 0;
      if (fresh) {
        if (!k_more || walk.next() < 0) return k_more = false;
        const uint32_t st = n_k % C::kNk;
        if (!warp_wait(smem_u32(&s.kfull[st]), (n_k / C::kNk) & 1, abort_flag)) return ok = false;
        ++n_k;
      } else if (!k_more) {
        return false;
      }
      if (share && x == 1 && !warp_wait(smem_u32(&s.qfull[1]), 0, abort_flag)) return ok = false;
      tc_fence_after();
      const uint32_t st = (n_k - 1) % C::kNk;
      const uint64_t qd = q_desc + (share ? h : 0) * (C::kTile >> 4), kd = k_desc + st * (C::kTile >> 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = (ks >> 2) * (kChunkBytes >> 4) + (ks & 3) * 2;
        mma_ss(tmem + h * 128, qd + off, kd + off, idesc_s, ks > 0 ? 1u : 0u, elected);
      }
      commit(smem_u32(&s.sfull[h]), elected);
      if (!share || h == 1) commit(smem_u32(&s.kempty[st]), elected);
      return true;
    };
    auto values = [&](int x) -> bool {
      const int h = x & 1;
      if (!share || h == 0) {
        const int j0 = walk_v.next() * kKeys;
        const uint32_t st = n_v % C::kNv;
        if (!warp_wait(smem_u32(&s.vfull[st]), (n_v / C::kNv) & 1, abort_flag)) return false;
        ++n_v;
        // values of keys that no row of the item sees become zeros
        bool live = j0 + kKeys <= t.nk && (j0 + kKeys <= t.pre || (j0 >= t.lo && j0 + kKeys <= t.hi));
        if (docs) {
          const int2 d = table[j0 / kKeys];
          live = live && d.x >= q_min && d.y <= q_max;
        }
        if (!live) {
#pragma unroll 1
          for (int c = lane; c < kKeys; c += 32) {
            const int j = j0 + c;
            bool keep = j < t.nk && (j < t.pre || (j >= t.lo && j < t.hi));
            if (docs && keep) {
              const int doc = docs[j];
              keep = doc >= q_min && doc <= q_max;         // 0 <= q_min
            }
            if (!keep) {
              uint4* row = reinterpret_cast<uint4*>(sv + st * C::kTile + c * 128);
              for (int k = 0; k < C::kChunks; ++k)
                for (int i = 0; i < 8; ++i) row[k * (kChunkBytes / 16) + i] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      if (!warp_wait(smem_u32(&s.phalf[h]), (x >> 1) & 1, abort_flag)) return false;
      tc_fence_after();
      const uint32_t st = (n_v - 1) % C::kNv;
      const uint64_t vd = val_desc + st * (C::kTile >> 4);
      const uint32_t more = x > 1 ? 1u : 0u;
#pragma unroll
      for (int ks = 0; ks < kKeys / 32; ++ks)
        mma_ts(tmem + kOCol + h * 128, tmem + h * 128 + ks * 8, vd + ((ks * 16 * 128) >> 4), idesc_o, ks > 0 ? 1u : more,
               elected);
      if (!warp_wait(smem_u32(&s.pfull[h]), (x >> 1) & 1, abort_flag)) return false;
      tc_fence_after();
#pragma unroll
      for (int ks = kKeys / 32; ks < kKeys / 16; ++ks)
        mma_ts(tmem + kOCol + h * 128, tmem + h * 128 + ks * 8, vd + ((ks * 16 * 128) >> 4), idesc_o, 1u, elected);
      commit(smem_u32(&s.odone[h]), elected);
      if (!share || h == 1) commit(smem_u32(&s.vempty[st]), elected);
      return true;
    };
    if (ok) {
      int issued = 0;
      while (issued < 2 && scores(issued)) ++issued;
      for (int x = 0; ok && x < issued; ++x) {
        if (!(ok = values(x))) break;
        if (issued == x + 2 && scores(issued)) ++issued;
      }
    }
    // all MMAs issued above complete before tensor memory is freed
    commit(smem_u32(&s.done), elected);
    drain(smem_u32(&s.done), 0);
  }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int h = warp >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int row = (share ? h * kTileRows : 0) + r;
    const bool valid = row < t.rows;
    uint32_t in_group;                         // head of the group
    const int p = t.first + static_cast<int>(a.by_group.divmod(t.row0 + (valid ? row : 0), &in_group));
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_col = tmem + lanes + h * 128, o_col = tmem + lanes + kOCol + h * 128;
    const bool warp_valid = __any_sync(0xffffffffu, valid);
    // keys of this row: [row_lo, row_hi) and [0, row_pre)
    int row_hi = min(p + 1, t.nk), row_lo = a.mods.window && p >= a.mods.window ? p - a.mods.window + 1 : 0;
    int row_pre = t.pre;
    int my_doc = 0;
    if (docs) my_doc = p >= 0 && p < t.nk ? docs[p] : -1;
    if (p < 0 || my_doc < 0) row_hi = row_lo = row_pre = 0;
    // tiles that every row of the warp sees whole: keys [all_lo, all_hi) and [0, all_pre)
    const int all_lo = __reduce_max_sync(0xffffffffu, valid ? row_lo : 0);
    const int all_hi = __reduce_min_sync(0xffffffffu, valid ? row_hi : INT32_MAX);
    const int all_pre = __reduce_min_sync(0xffffffffu, valid ? row_pre : INT32_MAX);
    const float cs = CAP ? 1.f : a.scale * kLog2e;
    const float cap = a.mods.softcap;
    const float zs = !CAP ? 0.f : WIDE ? fminf(fmaxf(a.scale / cap, 0x1p-126f), 1e30f) : a.scale / cap;
    float tc[5];                               // the polynomial's coefficients for s
    if constexpr (CAP) {
      float f = a.scale * kLog2e;
#pragma unroll
      for (int k = 0; k < 5; ++k, f *= zs * zs) tc[k] = kTanh[k] * f;
    }
    // slope in units of y: base 2 behind a cap, raw scores otherwise
    const float bias = BIAS ? a.mods.slopes[t.g * a.G + static_cast<int>(in_group)] * (CAP ? kLog2e : 1.f / a.scale) : 0.f;
    const int all_pre_max = BIAS ? __reduce_max_sync(0xffffffffu, row_pre) : 0;
    float m = -INFINITY, l = 0.f;              // reference maximum (of y / cs) and sum of 2^(y - m cs)
    TileWalk walk(t, table, q_min, q_max);
    int n = 0;                                 // tiles of this stream
    bool fail = false;
    for (int i = 0;; ++i) {
      const int tile = walk.next();
      if (tile < 0) break;
      if (!share && (i & 1) != h) continue;
      if (!warp_wait(smem_u32(&s.sfull[h]), n & 1, abort_flag)) {
        fail = true;
        break;
      }
      ++n;
      tc_fence_after();
      if (!warp_valid) {                       // nothing of this warp is a row: the product's result is not read
        tc_fence_before();
        if (lane == 0) {
          mbar_arrive(smem_u32(&s.phalf[h]));
          mbar_arrive(smem_u32(&s.pfull[h]));
        }
        continue;
      }
      uint32_t sr[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32_issue(s_col + c * 32, sr[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
      float (&y)[4][32] = reinterpret_cast<float (&)[4][32]>(sr);
      const int j0 = tile * kKeys;
      // z = s scale / cap; cap tanh(z) log2 e = s times a polynomial in s^2 as long as the warp's |z| are small.  It
      // grows with s, so without slopes the maximum is that of s, and the polynomial is evaluated between the
      // exponentials (it fills the fp32 pipe while they wait for theirs).
      bool late = false;
      if constexpr (CAP && WIDE) {
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) big = fmaxf(big, fmaxf(fabsf(y[c][e]), fabsf(y[c][e + 1])));
        if (__all_sync(0xffffffffu, big * zs <= kTanhRange || !valid)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) y[c][e] *= tanh_over_z(y[c][e] * zs) * (a.scale * kLog2e);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) y[c][e] = capped_base2(y[c][e] * a.scale, y[c][e] * zs, cap);
        }
      } else if constexpr (CAP) {
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; e += 2) big = fmaxf(big, fmaxf(fabsf(y[c][e]), fabsf(y[c][e + 1])));
        if (__all_sync(0xffffffffu, big * zs <= kTanhRange || !valid)) {
          if constexpr (BIAS) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const uint64_t x = pair(y[c][e], y[c][e + 1]);
                unpair(mul2(x, odd_factor(x, tc)), &y[c][e], &y[c][e + 1]);
              }
          } else {
            late = true;
          }
        } else {
          // cap tanh(z) = cap (1 - 2 / (1 + e^2z)): right at both infinities
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              y[c][e] = fmaf(-2.f * cap, rcp_approx(1.f + ex2_approx(y[c][e] * (zs * (2.f * kLog2e)))), cap) * kLog2e;
        }
      }
      if constexpr (BIAS) {
        if (all_pre_max == 0) {
          // keys that are seen lie at or before the row: -slope |p - j| = slope (j - j0) - slope (p - j0)
          const float b0 = -bias * static_cast<float>(p - j0);
          const uint64_t s2 = pair(bias, bias), b2 = pair(b0, b0);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              unpair(add2(fma2(s2, pair(static_cast<float>(c * 32 + e), static_cast<float>(c * 32 + e + 1)), b2),
                          pair(y[c][e], y[c][e + 1])), &y[c][e], &y[c][e + 1]);
        } else {
          const float far = static_cast<float>(p - j0);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) y[c][e] = fmaf(-bias, fabsf(far - static_cast<float>(c * 32 + e)), y[c][e]);
        }
      }
      // masks, unless every row of the warp sees the whole tile
      const bool whole = j0 + kKeys <= all_pre || (j0 >= all_lo && j0 + kKeys <= all_hi);
      bool same = true;
      if (docs) {
        const int2 d = table[tile];
        same = __all_sync(0xffffffffu, (d.x == d.y && d.x == my_doc) || !valid);
      }
      if (!whole || !same) {
        uint32_t eq[4] = {~0u, ~0u, ~0u, ~0u};
        if (!same) {
          // the keys of each document that the warp's rows have, one document after another
          int kd[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) kd[c] = j0 + c * 32 + lane < t.nk ? docs[j0 + c * 32 + lane] : -1;
          uint32_t left = 0xffffffffu;
#pragma unroll 1
          while (left) {
            const int doc = __shfl_sync(0xffffffffu, my_doc, __ffs(left) - 1);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t hit = __ballot_sync(0xffffffffu, kd[c] == doc);
              if (my_doc == doc) eq[c] = hit;
            }
            left &= ~__ballot_sync(0xffffffffu, my_doc == doc);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int jc = j0 + c * 32;
          const uint32_t bits = (bit_range(row_lo - jc, row_hi - jc) | bit_range(0, row_pre - jc)) & eq[c];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(bits & (1u << e))) y[c][e] = -INFINITY;
        }
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = fmaxf(y[c][0], y[c][1]);
#pragma unroll
        for (int e = 2; e < 32; e += 2) mx[c] = fmaxf(mx[c], fmaxf(y[c][e], y[c][e + 1]));
      }
      float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (late) {                              // -inf stays: the leading coefficient is positive, see cap_is_wide
        const float w = top * top;
        top *= fmaf(fmaf(fmaf(fmaf(tc[4], w, tc[3]), w, tc[2]), w, tc[1]), w, tc[0]);
      }
      const bool grow = (top - m) * cs > kGrow;          // also from -inf
      if (__any_sync(0xffffffffu, grow)) {
        float f = 1.f;
        if (grow) {
          f = m == -INFINITY ? 0.f : ex2_approx((m - top) * cs);
          m = top;
          l *= f;
        }
        if (n > 1) {
          if (!warp_wait(smem_u32(&s.odone[h]), n & 1, abort_flag)) {     // the product of tile n - 2
            fail = true;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(o_col + c * 16, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(o_col + c * 16, o);
          }
        }
      }
      const float sub = m == -INFINITY ? 0.f : m * cs;
      const uint64_t cs2 = pair(cs, cs), sub2 = pair(-sub, -sub);
      uint64_t sum[2] = {0, 0};
      auto weights = [&](auto exponent) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float p0, p1;
            unpair(exponent(pair(y[c][e], y[c][e + 1])), &p0, &p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(p0, p1));
            pk[e / 2] = pack_bf16x2(p0, p1);
          }
          tmem_st16(s_col + c * 16, pk);
          if (c == 1) {                        // the product may start on the first half of the keys
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.phalf[h]));
          }
        }
      };
      if (CAP && !WIDE && !BIAS && late) weights([&](uint64_t x) { return fma2(x, odd_factor(x, tc), sub2); });
      else weights([&](uint64_t x) { return fma2(x, cs2, sub2); });
      float s0, s1;
      unpair(add2(sum[0], sum[1]), &s0, &s1);
      l += s0 + s1;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.pfull[h]));
    }
    // statistics of the row, once they are those of all its keys in this item
    const bool part = a.splits > 1;
    const int query = p - t.first, head = t.g * a.G + static_cast<int>(in_group);
    const int64_t prow = static_cast<int64_t>(t.u) * a.n_q * a.G + t.row0 + (valid ? row : 0);
    auto write_stats = [&](float top, float sum) {
      if (part)
        a.part_ml[prow * a.splits + t.split] = make_float2(top, sum);
      else if (a.lse)
        a.lse[((static_cast<int64_t>(t.b) * a.L + t.l) * (a.Hkv * a.G) + head) * a.n_q + query] =
            sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
    };
    float m2 = m == -INFINITY ? -INFINITY : m * cs;
    if (share && valid) write_stats(m2, l);      // while the last product of this stream runs
    // Without a tile there is no product to wait for, but the queries are on their way all the same, into the shared
    // memory that stages the outputs.
    if (!fail && !warp_wait(smem_u32(n > 0 ? &s.odone[h] : &s.qfull[share ? h : 0]), n > 0 ? (n - 1) & 1 : 0, abort_flag))
      fail = true;
    tc_fence_after();
    // One row tile: both streams hold an output for the same rows, in the same lanes of tensor memory.  They exchange
    // (m, l) through the unused second Q tile, and each joins and writes one half of the columns.
    int n_other = 0;
    float f0 = 1.f, f1 = 0.f;
    if (!share) {
      float2* ml = reinterpret_cast<float2*>(sq + C::kTile);
      ml[h * kTileRows + r] = make_float2(m2, l);
      if (r == 0) s.tiles[h] = n;
      tc_fence_before();
      fail = named_bar_or(1, 256, fail);                     // both streams' products are done
      tc_fence_after();
      n_other = uniform(s.tiles[h ^ 1]);
      const float2 o = ml[(h ^ 1) * kTileRows + r];
      const float mm = fmaxf(m2, o.x);
      f0 = m2 == -INFINITY ? 0.f : ex2_approx(m2 - mm);
      f1 = o.x == -INFINITY ? 0.f : ex2_approx(o.x - mm);
      // the same order of the sum on both sides
      l = h == 0 ? fmaf(l, f0, o.y * f1) : fmaf(o.y, f1, l * f0);
      m2 = mm;
      if (valid && h == 0) write_stats(m2, l);
    }
    if (!fail && warp_valid) {
      if (!part) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        f0 *= inv;
        f1 *= inv;
      }
      const int64_t own = static_cast<int64_t>(head) * a.os.head + static_cast<int64_t>(query) * a.os.token;
      // this stream's columns, staged in shared memory in 16-byte chunks (Q is not read any more)
      const int cols = share ? D : D / 2, col0 = share ? 0 : h * (D / 2);
      const int chunks = cols / 8, flip = min(chunks - 1, 7);
      // a warp's rows: 64 columns (or fewer) of all of them, then the next 64; chunks swizzled as a tensor copy takes them
      uint8_t* stage = sq + h * C::kTile + (share ? 0 : h * 4096) + quarter * (32 * chunks * 16);
      const int pitch = min(chunks, 8) * 16;
      float* part_o = a.part_o + (prow * a.splits + t.split) * D + col0;
      const uint32_t mine = o_col + col0, other = tmem + lanes + kOCol + (h ^ 1) * 128 + col0;
      auto put = [&](int c, const float (&x)[32]) {
        if (!valid) return;
        if (part) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part_o + c * 32 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4*>(stage + (c >> 1) * 4096 + lane * pitch + ((((c & 1) * 4 + e / 8) ^ (lane & flip)) << 4)) =
                make_uint4(pack_bf16x2(x[e], x[e + 1]), pack_bf16x2(x[e + 2], x[e + 3]),
                           pack_bf16x2(x[e + 4], x[e + 5]), pack_bf16x2(x[e + 6], x[e + 7]));
        }
      };
      // every column of this warp is on its way before the first is used; a stream without tiles holds nothing
      constexpr int kOwn = D / 32, kHalf = D / 64;
      uint32_t o[kOwn][32] = {};
      float x[32];
      if (share) {
        if (n > 0) {
#pragma unroll
          for (int c = 0; c < kOwn; ++c) tmem_ld32_issue(mine + c * 32, o[c]);
#pragma unroll
          for (int c = 0; c < kOwn; ++c) tmem_ld_wait(o[c]);
        }
#pragma unroll
        for (int c = 0; c < kOwn; ++c) {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(o[c][e]) * f0;
          put(c, x);
        }
      } else {
        if (n > 0) {
#pragma unroll
          for (int c = 0; c < kHalf; ++c) tmem_ld32_issue(mine + c * 32, o[c]);
        }
        if (n_other > 0) {
#pragma unroll
          for (int c = 0; c < kHalf; ++c) tmem_ld32_issue(other + c * 32, o[kHalf + c]);
        }
#pragma unroll
        for (int c = 0; c < kOwn; ++c) tmem_ld_wait(o[c]);
#pragma unroll
        for (int c = 0; c < kHalf; ++c) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[e] = fmaf(__uint_as_float(o[kHalf + c][e]), f1, __uint_as_float(o[c][e]) * f0);
          put(c, x);
        }
      }
      if (!part) {
        const int row0 = (share ? h * kTileRows : 0) + quarter * 32;
        if (a.o_tma && cols >= 64 && row0 + 32 <= t.rows) {
          // whole queries, all of them rows: one copy per 64 columns
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int q0 = static_cast<int>(a.by_group.div(t.row0 + row0));
            for (int c = 0; c < cols / 64; ++c)
              tma_store_5d(&map_o, smem_u32(stage + c * 4096), col0 + c * 64, t.g * a.G, q0, t.l, t.b);
            tma_store_wait();
          }
        } else {
          // from shared memory, whole rows (or halves) per store
          __syncwarp();
          const int chunk = lane & (chunks - 1), per = 32 / chunks;     // rows per instruction
          __nv_bfloat16* out = a.out + t.b * a.os.batch + t.l * a.os.layer + col0;
#pragma unroll 4
          for (int i = 0; i < chunks; ++i) {
            const int rr = i * per + lane / chunks;
            const int64_t at = __shfl_sync(0xffffffffu, own, rr);
            if (row0 + rr < t.rows)
              *(reinterpret_cast<uint4*>(out + at) + chunk) =
                  *reinterpret_cast<const uint4*>(stage + (chunk >> 3) * 4096 + rr * pitch + (((chunk & 7) ^ (rr & flip)) << 4));
          }
        }
      }
    }
    if (fail && lane == 0 && a.unit_status) a.unit_status[s.item.u] = KVC_UNIT_TIMEOUT;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the splits of a row (PASK Eq. 15): one warp per row.
template <int D>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const PromptArgs a) {
  const int64_t rows = static_cast<int64_t>(a.U) * a.n_q * a.G;
  const int64_t prow = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (prow >= rows) return;
  const int lane = threadIdx.x & 31;
  wait_for_previous_kernel();
  const int u = static_cast<int>(prow / (static_cast<int64_t>(a.n_q) * a.G));
  const int pr = static_cast<int>(prow % (static_cast<int64_t>(a.n_q) * a.G));
  const int b = u / (a.L * a.Hkv), l = u / a.Hkv % a.L, g = u % a.Hkv;
  if (a.q_len && pr / a.G >= clamp_count(a.q_len[b], a.n_q)) return;
  const float2* ml = a.part_ml + prow * a.splits;
  float top = -INFINITY;
  for (int i = lane; i < a.splits; i += 32) top = fmaxf(top, ml[i].x);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float x[D / 32] = {}, sum = 0.f;
  for (int i0 = 0; i0 < a.splits; i0 += 32) {
    // lane i holds split i's weight; the outputs of eight splits are on their way together
    const float2 v = i0 + lane < a.splits ? ml[i0 + lane] : make_float2(-INFINITY, 0.f);
    const float w = v.x == -INFINITY ? 0.f : ex2_approx(v.x - top);
    sum = fmaf(v.y, w, sum);
    const int n = min(32, a.splits - i0);
    const float* src = a.part_o + (prow * a.splits + i0) * D + lane * (D / 32);
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) x[c] = fmaf(src[i * D + c], wi, x[c]);
    }
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int head = g * a.G + pr % a.G;
  __nv_bfloat16* out = a.out + b * a.os.batch + l * a.os.layer + static_cast<int64_t>(head) * a.os.head +
                       static_cast<int64_t>(pr / a.G) * a.os.token + lane * (D / 32);
#pragma unroll
  for (int c = 0; c < D / 32; c += 2)
    *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(x[c] * inv, x[c + 1] * inv);
  if (lane == 0 && a.lse)
    a.lse[((static_cast<int64_t>(b) * a.L + l) * (a.Hkv * a.G) + head) * a.n_q + pr / a.G] =
        sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
}

// Smallest and largest document of each key tile: one warp per tile.
__global__ void __launch_bounds__(256) doc_tiles_kernel(const PromptArgs a) {
  wait_for_previous_kernel();
  let_next_kernel_start();
  const int tile = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (tile >= a.n_tiles) return;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    int lo = INT32_MAX, hi = INT32_MIN;
    for (int c = lane; c < kKeys; c += 32) {
      const int64_t j = static_cast<int64_t>(tile) * kKeys + c;
      if (j >= a.T) continue;
      const int d = a.docs[b * a.T + j];
      lo = min(lo, d);
      hi = max(hi, d);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) a.doc_tiles[static_cast<int64_t>(b) * a.n_tiles + tile] = make_int2(lo, hi);
  }
}

// Caps beyond kFineCap, and those whose last coefficient kTanh[4] scale log2(e)
// (scale / cap)^8 is no normal number: masked scores of -inf rely on its sign.
bool cap_is_wide(const PromptArgs& a) {
  const double z = static_cast<double>(a.scale) / a.mods.softcap, last = 0.015 * 1.44 * a.scale * std::pow(z, 8);
  return a.mods.softcap > kFineCap || last < 0x1p-124 || last > 0x1p118;
}

}  // namespace

size_t prompt_smem_bytes(int d) { return d == 128 ? Cfg<128>::kSmem : Cfg<64>::kSmem; }

cudaError_t launch_prompt(const PromptArgs& a, const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v,
                          const CUtensorMap& map_o, cudaStream_t stream) {
  if (a.docs) {
    const cudaError_t e = launch_after(doc_tiles_kernel, dim3((a.n_tiles + 7) / 8, std::min(a.B, 65535)), 256, 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.n_blocks) * a.U * a.splits);
  auto go = [&](auto kernel) -> cudaError_t {
    const int bytes = static_cast<int>(prompt_smem_bytes(a.d));
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(grid), kThreads, bytes, stream, map_q, map_k, map_v, map_o, a);
  };
  const bool bias = a.mods.slopes != nullptr;
  auto go_capped = [&](auto d) -> cudaError_t {
    constexpr int D = decltype(d)::value;
    if (!(a.mods.softcap > 0.f)) return bias ? go(prompt_kernel<D, false, true, false>) : go(prompt_kernel<D, false, false, false>);
    if (cap_is_wide(a)) return bias ? go(prompt_kernel<D, true, true, true>) : go(prompt_kernel<D, true, false, true>);
    return bias ? go(prompt_kernel<D, true, true, false>) : go(prompt_kernel<D, true, false, false>);
  };
  const cudaError_t e = a.d == 128 ? go_capped(std::integral_constant<int, 128>{}) : go_capped(std::integral_constant<int, 64>{});
  if (e != cudaSuccess || a.splits == 1) return e;
  const int64_t rows = static_cast<int64_t>(a.U) * a.n_q * a.G;
  const unsigned blocks = static_cast<unsigned>((rows + 7) / 8);
  return launch_after(a.d == 128 ? prompt_merge_kernel<128> : prompt_merge_kernel<64>, blocks, 256, 0, stream, a);
}

}  // namespace kvc
