// Attention of a tree of drafted tokens over the rows of a 4-bit cache and over
// the tree's own bf16 rows, with score modifiers.
//
// Rows.  The G heads that share a KV head are packed: row r of a unit is node
// r / G of head r % G.  A block works on one item: 256 rows of a unit (two tiles
// of 128 that share every key and value tile) or 128 rows, whose two streams
// take the key tiles in turn, over a part of the unit's keys: the cached rows in
// tiles of 128, then the tree's.  Partial outputs are joined by PASK Eq. 15 in a
// second kernel.
//
// Both products run on the tensor cores from operands that are exact: code *
// scale has 3 + 8 bits and an fp16 number 11, so the rows are turned into fp16,
// scaled by a power of two per tile that keeps them within its range (2^-ek for
// keys, 2^-ev for values; it is taken back in fp32: 2^ek goes into the softmax
// scale, 2^ev into the running maximum).  Elements more than 2^24 below the
// tile's largest lose bits to the format's end.  A scale per row in fp16 has 11
// bits itself: there the operands are the plain codes, and the scales multiply
// the scores and the weights in fp32.  Queries are scaled to fp16 per row alike;
// they, and the tree's rows, come in 8 bits.
//   S = Q K^T      tcgen05, both operands in shared memory, S in tensor memory
//   softmax        128 threads, one row each, in base 2; the weights are rounded
//                  to fp16 (2^-11 of a weight, and 2^-25 of the largest product
//                  of weight and value) and stored over S in tensor memory; the
//                  row's sum is that of the unrounded weights.  The accumulator
//                  is rescaled only when the maximum grew by more than 2^8
//   O += P V       tcgen05, P from tensor memory, V as an MN-major operand
// The order of d inside a product is free: the eight codes of a word lie as
// pairs (0,4), (1,5), (2,6), (3,7), and the queries, the tree's rows and the
// outputs are laid out to match, so that a pair costs a shift, a logical
// operation ((w & 0x03c003c0) ^ 0x4e004e00 = 24 + code) and a multiply-add.
//
// Masks.  Node i sees the cached rows (with a window those near enough), its
// ancestors and itself.  Parents come before their children, so the tree's tiles
// are taken from the last to the first and each row's ancestors are met by one
// walk up.  With a window, tiles that no row sees are not read: the warps that
// turn rows into operands decide, and say so to the others tile by tile.
//
// Warp roles (16 warps): 0-3 and 4-7 softmax of stream 0 and 1 (176 registers),
// 8-11 operands (104; a tile's codes on their way in registers while the one
// before is turned, tiles behind them prefetched to L2), 12 tensor memory and
// MMA issuer (56): 176 + 176 + 104 + 56 = 4 x 128, what the block was launched
// with.  Every wait is bounded; one that gives up raises a shared abort flag, the
// unit is marked KVC_UNIT_TIMEOUT and the block ends.
#include <algorithm>
#include <type_traits>

#include "kvc_internal.cuh"
#include "packed_math.cuh"
#include "tc_attn.cuh"

namespace kvc {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 512;
constexpr int kTileRows = 128;
constexpr int kKeys = 128;                       // keys per tile
constexpr uint32_t kTmemCols = 512;              // S0, S1, O0, O1 of 128 columns each
constexpr uint32_t kOCol = 256;
constexpr int kOperandWarp = 8, kMmaWarp = 12;   // the first of four; the only one
constexpr int kStages = 2;                       // key tiles, and value tiles, in shared memory
constexpr int kSlots = 4;                        // tiles whose description is held
constexpr int kAhead = 4;                        // tiles prefetched to L2 in front of the registers' own
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;                     // log2 growth of the maximum that forces a rescale

// What the operand warps say about a tile.
struct Tile {
  int j0;                      // its first key: a cached row's slot, or a node
  int tree;                    // the tree's own rows
  int ek, ev;                  // operands are rows times 2^-ek, 2^-ev
  int p_min;                   // smallest position
};

struct Bars {
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t sfull[2], phalf[2], pfull[2], odone[2], qfull[2], done;
  uint32_t tmem;
  int abort_flag;
  int total;                   // tiles of this item, once that is known
  int e_ref;                   // ev of the first of them
  int tiles[2];                // of each stream
  uint32_t top[kSlots][4][2];  // largest key and value scale that each operand warp met
  Tile tile[kSlots];
  int8_t q_exp[256];           // queries are rows times 2^-q_exp
  alignas(16) int32_t pos[kSlots][kKeys];
  alignas(16) float ks[kSlots][kKeys], vs[kSlots][kKeys];    // scale per row: of keys; of values times 2^-ev
};

template <int D>
struct Cfg {
  static constexpr int kTile = D / 64 * kChunkBytes;         // a Q, K or V tile
  static constexpr int kSmem = (2 + 2 * kStages) * kTile + 1024 /* alignment */ + sizeof(Bars);
};
static_assert(Cfg<128>::kSmem <= 232448, "shared memory of a block");

// What an item covers.
struct Item {
  int u, b, l, g, split;
  int row0, rows;              // first packed row, packed rows of the item (<= 256)
  int count, next, prefix;     // cached rows, position of the first nodes, visible prefix
  int cached, i0, i1;          // tiles of cached rows; tiles [i0, i1) of them and the tree's are this split's
  int nodes;                   // of the tree, as far as this item's rows see
};

__device__ __forceinline__ Item make_item(const TreeArgs& a, int id) {
  Item t;
  uint32_t split, u, g, l;
  const int qb = static_cast<int>(a.by_units.divmod(a.by_splits.divmod(id, &split), &u));
  t.split = static_cast<int>(split);
  t.u = static_cast<int>(u);
  t.b = static_cast<int>(a.by_layers.divmod(a.by_heads.divmod(u, &g), &l));
  t.l = static_cast<int>(l);
  t.g = static_cast<int>(g);
  t.count = clamp_count(a.rows.count[t.u], a.rows.capacity);
  t.next = a.rows.next_pos[t.u];
  t.prefix = a.mods.prefix_len ? a.mods.prefix_len[t.b] : INT32_MIN;
  const int n = a.n_nodes ? clamp_count(a.n_nodes[t.b], a.n) : a.n;
  t.row0 = qb * a.block_rows;
  t.rows = max(0, min(a.block_rows, n * a.G - t.row0));
  t.nodes = t.rows > 0 ? (t.row0 + t.rows - 1) / a.G + 1 : 0;
  t.cached = (t.count + kKeys - 1) / kKeys;
  const int64_t all = t.cached + (t.nodes + kKeys - 1) / kKeys;
  t.i0 = static_cast<int>(all * split / a.splits);
  t.i1 = static_cast<int>(all * (split + 1) / a.splits);
  return t;
}

// The parent of node i, -1: none (also for what is no earlier node).
__device__ __forceinline__ int parent_of(const int32_t* parent, int i, bool* bad) {
  const int p = parent[i];
  if (p >= -1 && p < i) return p;
  *bad = true;
  return -1;
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(max(-126, min(127, e)) + 127) << 23); }

// x 2^e for |e| up to 252, in two exact steps.
__device__ __forceinline__ float times_pow2(float x, int e) { return x * pow2(e >> 1) * pow2(e - (e >> 1)); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Elements (0,4), (1,5), (2,6), (3,7) of a word of codes times the scale in both halves of s; m = -24 s.
__device__ __forceinline__ uint4 codes_to_half(uint32_t w, uint32_t s, uint32_t m) {
  uint32_t x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t y = k == 0 ? w << 6 : k == 1 ? w << 2 : k == 2 ? w >> 2 : w >> 6;
    asm("lop3.b32 %0, %1, 0x03c003c0, 0x4e004e00, 0x6a;" : "=r"(x[k]) : "r"(y));      // (y & mask) ^ magic = 24 + code
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(x[k]) : "r"(s), "r"(m));
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// Eight bf16 elements times 2^-e in the same order.
__device__ __forceinline__ uint4 bf16_to_half(const uint4& w, int e) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  auto at = [&](int i) { return times_pow2(__uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16), -e); };
  return make_uint4(pack_half2(at(0), at(4)), pack_half2(at(1), at(5)), pack_half2(at(2), at(6)), pack_half2(at(3), at(7)));
}

// Largest magnitude of eight bf16 elements, as bits.
__device__ __forceinline__ uint32_t max_bits(const uint4& w) {
  uint32_t r = 0;
  for (uint32_t x : {w.x, w.y, w.z, w.w}) r = max(r, max(x & 0x7fffu, (x >> 16) & 0x7fffu));
  return r;
}

// Exponent of a bf16 number's bits (subnormals count as the smallest normal).
__device__ __forceinline__ int exponent_of(uint32_t bits) { return static_cast<int>(max(1u, bits >> 7)) - 127; }

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 16-byte piece c of row r of an operand tile of 64-element chunks in 128-byte swizzle.
__device__ __forceinline__ uint4* piece(uint8_t* tile, int r, int c) {
  return reinterpret_cast<uint4*>(tile + (c >> 3) * kChunkBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------- operand warps

// Turns the item's rows into operand tiles, keys one tile ahead of values.
template <int D, bool ROW, bool MODS>
__device__ __forceinline__ void make_operands(const TreeArgs& a, const Item& t, Bars& s, uint8_t* sk, uint8_t* sv) {
  using C = Cfg<D>;
  constexpr int CH = D / 32;                     // 16-byte pieces of codes per row
  constexpr int N = CH;                          // pieces of a thread per tile (128 threads, 128 rows)
  const int tid = threadIdx.x - kOperandWarp * 32, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &s.abort_flag;
  const int64_t base = static_cast<int64_t>(t.u) * a.rows.capacity;
  const uint8_t* codes[2] = {static_cast<const uint8_t*>(a.rows.k) + base * (D / 2), static_cast<const uint8_t*>(a.rows.v) + base * (D / 2)};
  const uint16_t* scales[2] = {static_cast<const uint16_t*>(a.rows.k_scale) + base * (ROW ? 1 : CH),
                               static_cast<const uint16_t*>(a.rows.v_scale) + base * (ROW ? 1 : CH)};
  const int64_t new_at = t.b * a.news.batch + t.l * a.news.layer + t.g * a.news.head;
  const bool windowed = MODS && a.mods.window;
  struct Raw {
    uint4 w[N];
    uint16_t sc[N];
  };
  // codes and scales of this thread's pieces of cached tile i; nothing behind the rows in use is read
  auto load = [&](int which, int i, Raw& raw) {
    const int left = t.count - i * kKeys;
    const uint4* src = reinterpret_cast<const uint4*>(codes[which] + static_cast<int64_t>(i) * (kKeys * D / 2)) + tid;
    const uint16_t* sc = scales[which] + static_cast<int64_t>(i) * (ROW ? kKeys : kKeys * CH);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int p = k * 128 + tid;
      const bool ok = p / CH < left;
      raw.w[k] = ok ? src[k * 128] : make_uint4(0, 0, 0, 0);
      raw.sc[k] = ok ? sc[ROW ? p / CH : p] : static_cast<uint16_t>(0);
      // a piece of zeros tells nothing about the sizes of the others, whatever its scale
      if ((raw.w[k].x | raw.w[k].y | raw.w[k].z | raw.w[k].w) == 0) raw.sc[k] = 0;
    }
  };
  auto prefetch = [&](int i) {
    if (i >= min(t.cached, t.i1)) return;
    const int left = min(kKeys, t.count - i * kKeys);
    // a line of codes per thread (64 lines of keys, 64 of values at d = 128), and the scales' lines
    const int line = tid & 63, which = tid >> 6;
    if (line * 128 < left * (D / 2)) prefetch_l2(codes[which] + static_cast<int64_t>(i) * (kKeys * D / 2) + line * 128);
    if (line * 64 < left * (ROW ? 1 : CH)) prefetch_l2(scales[which] + static_cast<int64_t>(i) * (ROW ? kKeys : kKeys * CH) + line * 64);
  };
  auto store = [&](uint8_t* tile, const Raw& raw, int e) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int p = k * 128 + tid, key = p / CH, chunk = p % CH;
      uint32_t sc = 0x3c003c00u;                 // a scale per row: the codes alone
      if (!ROW) {
        const float f = times_pow2(bf16_bits_to_float(raw.sc[k]), -e);
        sc = pack_half2(f, f);
      }
      uint32_t m;
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(m) : "r"(sc), "r"(0xce00ce00u));          // -24
      // lanes of the second 64 columns take their words in another order: eight lanes then meet every bank once
      const bool far = D == 128 && (chunk & 2);
      const uint32_t w[4] = {far ? raw.w[k].z : raw.w[k].x, far ? raw.w[k].w : raw.w[k].y, far ? raw.w[k].x : raw.w[k].z,
                             far ? raw.w[k].y : raw.w[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) *piece(tile, key, chunk * 4 + (far ? j ^ 2 : j)) = codes_to_half(w[j], sc, m);
    }
  };
  // a tile of the tree: 16-byte pieces of bf16, each thread those of one column
  constexpr int BP = D / 8;
  auto tree_piece = [&](const __nv_bfloat16* x, int j0, int k) -> uint4 {
    const int p = k * 128 + tid, key = j0 + p / BP;
    if (key >= t.nodes) return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4*>(x + new_at + static_cast<int64_t>(key) * a.news.token + (p % BP) * 8);
  };
  auto tree_top = [&](const __nv_bfloat16* x, int j0) {
    uint32_t top = 0;
#pragma unroll 8
    for (int k = 0; k < BP; ++k) top = max(top, max_bits(tree_piece(x, j0, k)));
    return top;
  };
  auto tree_store = [&](uint8_t* tile, const __nv_bfloat16* x, int j0, int e) {
#pragma unroll 4
    for (int k = 0; k < BP; ++k) {
      const int p = k * 128 + tid;
      *piece(tile, p / BP, p % BP) = bf16_to_half(tree_piece(x, j0, k), e);
    }
  };
  // the walk over the item's tiles: cached ones in order, then the tree's from the last to the first
  int at = t.i0, pos_here = 0;
  auto next = [&]() -> int {
    for (; at < t.i1; ++at) {
      if (!MODS || at >= t.cached) return at++;
      const int j = at * kKeys + tid;
      const bool mine = j < t.count;
      const int p = mine ? a.rows.pos[base + j] : INT32_MAX;
      if (windowed) {
        // every warp looks at every position: four of them are four keys of a lane
        bool seen = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int jj = at * kKeys + k * 32 + lane;
          if (jj < t.count) {
            const int q = a.rows.pos[base + jj];
            seen |= t.next - q < a.mods.window || q < t.prefix;
          }
        }
        if (!__any_sync(kFull, seen)) continue;
      }
      pos_here = p;
      return at++;
    }
    return -1;
  };
  // distance of the prefetches: without a window the tiles that follow each other
  if (!windowed)
    for (int i = 0; i < kAhead; ++i) prefetch(t.i0 + 1 + i);

  Raw rk, rv[2];
  int cur = next();                              // the tile whose codes are in rk and rv[0]
  int cur_pos = pos_here;
  if (cur >= 0 && cur < t.cached) load(0, cur, rk), load(1, cur, rv[0]);
  bool fail = false;
  int e_v[2] = {0, 0}, id[2] = {-1, -1};         // of the tiles in flight between keys and values
  // tile n's keys are made, then the values of tile n - 1
#pragma unroll 1
  for (int n0 = 0;; n0 += 2) {
    bool end = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = n0 + h, slot = n & (kSlots - 1), st = n & 1;
      const bool more = cur >= 0, tree = more && cur >= t.cached;
      const int j0 = !more ? 0 : tree ? ((t.nodes + kKeys - 1) / kKeys - 1 - (cur - t.cached)) * kKeys : cur * kKeys;
      // the largest scales of the tile, and with modifiers its smallest position
      uint32_t tk = 0, tv = 0;
      if (tree) {
        tk = tree_top(a.k_new, j0);
        tv = tree_top(a.v_new, j0);
      } else if (more) {
#pragma unroll
        for (int k = 0; k < N; ++k) tk = max(tk, static_cast<uint32_t>(rk.sc[k])), tv = max(tv, static_cast<uint32_t>(rv[h].sc[k]));
      }
      tk = __reduce_max_sync(kFull, tk);
      tv = __reduce_max_sync(kFull, tv);
      if (lane == 0) s.top[slot][warp][0] = tk, s.top[slot][warp][1] = tv;
      fail = named_bar_or(2, 128, fail);         // one answer for the four warps
      if (fail) return;
#pragma unroll
      for (int w = 0; w < 4; ++w) tk = max(tk, s.top[slot][w][0]), tv = max(tv, s.top[slot][w][1]);
      int ek = 0, ev = 0;
      if (tree) {
        ek = tk ? exponent_of(tk) - 13 : 0;      // the largest element below 2^14
        ev = tv ? exponent_of(tv) - 13 : 0;
      } else if (ROW) {
        // 2^ev above the largest row scale
        ev = tv ? static_cast<int>(max(1u, tv >> 10)) - 14 : 0;
      } else {
        ek = tk ? exponent_of(tk) - 10 : 0;      // the largest scale below 2^11: 24 of it and 7 of it fit
        ev = tv ? exponent_of(tv) - 10 : 0;
      }
      if (more) {
        if (!warp_wait(smem_u32(&s.kempty[st]), ((n >> 1) & 1) ^ 1, abort_flag)) fail = true;
        if (!fail) {
          if (tid == 0) {
            s.tile[slot] = {j0, tree ? 1 : 0, ek, ev, 0};
            if (n == 0) s.e_ref = ev;
          }
          if (MODS) {
            int p = cur_pos;
            if (tree) {
              bool bad = false;
              p = t.next;
              if (j0 + tid < t.nodes)
                for (int i = parent_of(a.parent + static_cast<int64_t>(t.b) * a.n, j0 + tid, &bad); i >= 0;
                     i = parent_of(a.parent + static_cast<int64_t>(t.b) * a.n, i, &bad))
                  ++p;
            }
            s.pos[slot][tid] = p;
          }
          if (ROW && !tree) {
            const int j = j0 + tid;
            s.ks[slot][tid] = j < t.count ? __half2float(__ushort_as_half(scales[0][j])) : 0.f;
            // a row of zeros may have a scale above the others'
            s.vs[slot][tid] = j < t.count ? fminf(__half2float(__ushort_as_half(scales[1][j])) * pow2(-ev), 2.f) : 0.f;
          }
          if (tree) tree_store(sk + st * C::kTile, a.k_new, j0, ek);
          else store(sk + st * C::kTile, rk, ek);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.kfull[st]));
        }
        id[h] = tree ? -2 - j0 : cur;
        e_v[h] = ev;
        if (!windowed && !tree) prefetch(cur + 1 + kAhead);
        cur = next();
        cur_pos = pos_here;
        if (cur >= 0 && cur < t.cached) load(0, cur, rk);
      } else {
        id[h] = -1;
        if (tid == 0) s.total = n;
        // one more phase, without keys: the end
        if (!warp_wait(smem_u32(&s.kempty[st]), ((n >> 1) & 1) ^ 1, abort_flag)) fail = true;
        __syncwarp();
        if (!fail && lane == 0) mbar_arrive(smem_u32(&s.kfull[st]));
        end = true;
      }
      // values of the tile before
      const int was = id[h ^ 1];
      if (n > 0 && was != -1 && !fail) {
        const int vst = (n - 1) & 1;
        if (!warp_wait(smem_u32(&s.vempty[vst]), (((n - 1) >> 1) & 1) ^ 1, abort_flag)) {
          fail = true;
        } else {
          if (was < -1) tree_store(sv + vst * C::kTile, a.v_new, -2 - was, e_v[h ^ 1]);
          else store(sv + vst * C::kTile, rv[h ^ 1], e_v[h ^ 1]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.vfull[vst]));
        }
      }
      if (cur >= 0 && cur < t.cached) load(1, cur, rv[h ^ 1]);
      if (end) return;
    }
  }
}

// ---------------------------------------------------------------- MMA issuer

template <int D>
__device__ __forceinline__ void issue(const Item& t, Bars& s, uint8_t* sq, uint8_t* sk, uint8_t* sv, uint32_t tmem, bool share) {
  using C = Cfg<D>;
  volatile int* abort_flag = &s.abort_flag;
  constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(128 >> 4) << 24);           // fp16 x fp16 -> fp32, M = 128
  const uint32_t idesc_s = kIdesc | (static_cast<uint32_t>(kKeys >> 3) << 17);
  const uint32_t idesc_o = kIdesc | (static_cast<uint32_t>(D >> 3) << 17) | (1u << 16);     // B (values) MN-major
  bool ok = warp_wait(smem_u32(&s.qfull[0]), 0, abort_flag);
  if (ok && share) ok = warp_wait(smem_u32(&s.qfull[1]), 0, abort_flag);
  const uint32_t elected = elect_one();
  const uint64_t q_desc = sw128_desc(smem_u32(sq)), k_desc = sw128_desc(smem_u32(sk)), val_desc = v_desc(smem_u32(sv));
  int n_k = 0, n_v = 0;                // K and V tiles taken up
  bool k_more = true;
  // the scores of step x (stream x & 1); false when there is no such step
  auto scores = [&](int x) -> bool {
    const int h = x & 1;
    if (!k_more) return false;
    if (!share || h == 0) {
      if (!warp_wait(smem_u32(&s.kfull[n_k & 1]), (n_k >> 1) & 1, abort_flag)) return ok = k_more = false;
      if (n_k >= uniform(*reinterpret_cast<volatile int*>(&s.total))) return k_more = false;
      ++n_k;
    }
    tc_fence_after();
    const uint32_t st = (n_k - 1) & 1;
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
      if (!warp_wait(smem_u32(&s.vfull[n_v & 1]), (n_v >> 1) & 1, abort_flag)) return false;
      ++n_v;
    }
    if (!warp_wait(smem_u32(&s.phalf[h]), (x >> 1) & 1, abort_flag)) return false;
    tc_fence_after();
    const uint32_t st = (n_v - 1) & 1;
    const uint64_t vd = val_desc + st * (C::kTile >> 4);
    const uint32_t more = x > 1 ? 1u : 0u;
#pragma unroll
    for (int ks = 0; ks < kKeys / 32; ++ks)
      mma_ts(tmem + kOCol + h * 128, tmem + h * 128 + ks * 8, vd + ((ks * 16 * 128) >> 4), idesc_o, ks > 0 ? 1u : more, elected);
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
  // the streams' next scores are none (after an abort they find that by themselves)
  if (ok && elected) {
    mbar_arrive(smem_u32(&s.sfull[0]));
    mbar_arrive(smem_u32(&s.sfull[1]));
  }
  __syncwarp();
  // all MMAs issued above complete before tensor memory is freed
  commit(smem_u32(&s.done), elected);
  drain(smem_u32(&s.done), 0);
}

// ---------------------------------------------------------------- softmax

template <int D, bool ROW, bool MODS>
__device__ __forceinline__ void softmax(const TreeArgs& a, const Item& t, Bars& s, uint8_t* sq, uint32_t tmem, bool share) {
  using C = Cfg<D>;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* abort_flag = &s.abort_flag;
  const int h = warp >> 2, quarter = warp & 3;
  const int r = quarter * 32 + lane;
  const int row = (share ? h * kTileRows : 0) + r;
  const bool valid = row < t.rows;
  uint32_t in_group;                             // head of the group
  const int node = static_cast<int>(a.by_group.divmod(t.row0 + (valid ? row : 0), &in_group));
  const int head = t.g * a.G + static_cast<int>(in_group);

  // Queries of this warp's 32 rows: 16 lanes a row (8 at d = 64), scaled to fp16 by a power of two per row.  One row tile
  // is loaded by the first stream's warps.
  if (share || h == 0) {
    constexpr int LPR = D / 8, PER = 32 / LPR;
    const __nv_bfloat16* q = a.q + t.b * a.qs.batch + t.l * a.qs.layer;
    const int64_t own = static_cast<int64_t>(head) * a.qs.head + static_cast<int64_t>(node) * a.qs.token;
    const int chunk = lane % LPR;
#pragma unroll 1
    for (int i0 = 0; i0 < LPR; i0 += 8) {
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = (i0 + i) * PER + lane / LPR;
        const int64_t at = __shfl_sync(kFull, own, rr);
        w[i] = row - lane + rr < t.rows ? reinterpret_cast<const uint4*>(q + at)[chunk] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = (i0 + i) * PER + lane / LPR;
        uint32_t top = max_bits(w[i]);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        const int e = top ? exponent_of(top) - 14 : 0;       // the largest element below 2^15
        // (bounded so that it fits a byte: queries below 2^-100 lose bits, and no score)
        const int eb = max(-114, min(113, e));
        *piece(sq + (share ? h : 0) * C::kTile, quarter * 32 + rr, chunk) = bf16_to_half(w[i], eb);
        if (chunk == 0) s.q_exp[(share ? h * kTileRows : 0) + quarter * 32 + rr] = static_cast<int8_t>(eb);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.qfull[share ? h : 0]));
  }
  bool fail = false;
  if (!share && h == 1 && !warp_wait(smem_u32(&s.qfull[0]), 0, abort_flag)) fail = true;
  const int q_exp = s.q_exp[row];
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_col = tmem + lanes + h * 128, o_col = tmem + lanes + kOCol + h * 128;
  const bool warp_valid = __any_sync(kFull, valid);
  const int32_t* parent = a.parent + static_cast<int64_t>(t.b) * a.n;
  bool bad = false;
  int p_q = t.next;
  const bool capped = MODS && a.mods.softcap > 0.f, biased = MODS && a.mods.slopes, windowed = MODS && a.mods.window;
  if (MODS && (biased || windowed) && valid)
    for (int i = parent_of(parent, node, &bad); i >= 0; i = parent_of(parent, i, &bad)) ++p_q;
  const float slope = biased ? a.mods.slopes[head] * kLog2e : 0.f;
  const float cap = MODS ? a.mods.softcap : 0.f, inv_cap = capped ? fminf(1.f / cap, 1e30f) : 0.f;
  const float scale = capped ? a.scale : a.scale * kLog2e;
  int up = node;                                 // the lowest ancestor (or the node) that no tile has shown yet
  float m = -INFINITY, l = 0.f;                  // reference of y + ev (base 2), and sum of 2^(y + e_ref - m)
  int n = 0;                                     // tiles of this stream
  int e_ref = 0;
#pragma unroll 1
  for (int i = share ? 0 : h; !fail; i += share ? 1 : 2) {
    if (!warp_wait(smem_u32(&s.sfull[h]), n & 1, abort_flag)) {
      fail = true;
      break;
    }
    if (i >= uniform(*reinterpret_cast<volatile int*>(&s.total))) break;
    ++n;
    tc_fence_after();
    if (!warp_valid) {                           // nothing of this warp is a row: the product's result is not read
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
    const int slot = i & (kSlots - 1);
    const Tile tile = s.tile[slot];
    e_ref = s.e_ref;
    // keys of the tile that this row sees
    const bool tree = tile.tree != 0;
    uint32_t bits[4] = {0, 0, 0, 0};
    bool whole = false;
    if (tree) {
      while (up >= tile.j0 + kKeys) up = parent_of(parent, up, &bad);
      while (up >= tile.j0) {
        const int j = up - tile.j0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j >> 5 == c) bits[c] |= 1u << (j & 31);
        up = parent_of(parent, up, &bad);
      }
    } else {
      whole = tile.j0 + kKeys <= t.count;
#pragma unroll
      for (int c = 0; c < 4; ++c) bits[c] = bit_range(0, t.count - tile.j0 - c * 32);
    }
    // y = scores in base 2 = acc f (scores themselves with a cap)
    float f = fmaxf(scale * pow2(min(120, q_exp + tile.ek)), 0x1p-126f);
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
    float (&y)[4][32] = reinterpret_cast<float (&)[4][32]>(sr);
    const bool rows = ROW && !tree;              // a scale per key
    if (rows) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 k = *reinterpret_cast<const float4*>(&s.ks[slot][c * 32 + e]);
          y[c][e] *= k.x, y[c][e + 1] *= k.y, y[c][e + 2] *= k.z, y[c][e + 3] *= k.w;
        }
    }
    if (MODS) {
      if (capped) {
        float big = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) big = fmaxf(big, fabsf(y[c][e]));
        if (__all_sync(kFull, big * f * inv_cap <= kTanhRange || !valid)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = y[c][e] * f;
              y[c][e] = x * tanh_over_z(x * inv_cap) * kLog2e;
            }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float x = y[c][e] * f;
              y[c][e] = capped_base2(x, x * inv_cap, cap);
            }
        }
        f = 1.f;
      } else if (biased) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) y[c][e] *= f;
        f = 1.f;
      }
      if (biased || windowed) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int p = s.pos[slot][c * 32 + e], far = p_q - p;
            if (biased) y[c][e] = fmaf(-slope, fabsf(static_cast<float>(far)), y[c][e]);
            if (windowed && far >= a.mods.window && p >= t.prefix) y[c][e] = -INFINITY;
          }
      }
    }
    if (!whole) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (!(bits[c] & (1u << e))) y[c][e] = -INFINITY;
    }
    float mx[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mx[c] = fmaxf(y[c][0], y[c][1]);
#pragma unroll
      for (int e = 2; e < 32; e += 2) mx[c] = fmaxf(mx[c], fmaxf(y[c][e], y[c][e + 1]));
    }
    const float ev = static_cast<float>(tile.ev);
    const float top = fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), f, ev);
    const bool grow = top - m > kGrow;           // also from -inf
    if (__any_sync(kFull, grow)) {
      float by = 1.f;
      if (grow) {
        by = m == -INFINITY ? 0.f : ex2_approx(m - top);
        m = top;
        l *= by;
      }
      if (n > 1) {
        if (!warp_wait(smem_u32(&s.odone[h]), n & 1, abort_flag)) {       // the product of tile n - 2
          fail = true;
          break;
        }
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(o_col + c * 16, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
          tmem_st16(o_col + c * 16, o);
        }
      }
    }
    const float sub = m == -INFINITY ? 0.f : m - ev;
    const uint64_t f2 = pair(f, f), sub2 = pair(-sub, -sub);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float p0, p1;
        unpair(fma2(pair(y[c][e], y[c][e + 1]), f2, sub2), &p0, &p1);
        p0 = ex2_approx(p0);
        p1 = ex2_approx(p1);
        sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(p0, p1));
        if (rows) {
          const float2 v = *reinterpret_cast<const float2*>(&s.vs[slot][c * 32 + e]);
          p0 *= v.x;
          p1 *= v.y;
        }
        pk[e / 2] = pack_half2(p0, p1);
      }
      tmem_st16(s_col + c * 16, pk);
      if (c == 1) {                              // the product may start on the first half of the keys
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.phalf[h]));
      }
    }
    float s0, s1;
    unpair(add2(sum[0], sum[1]), &s0, &s1);
    l = fmaf(s0 + s1, pow2(e_ref - tile.ev), l);
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.pfull[h]));
  }
  if (bad && valid && a.unit_status) a.unit_status[t.u] = KVC_UNIT_BAD_INDEX;
  // statistics of the row, once they are those of all its keys in this item
  const bool part = a.splits > 1;
  const int64_t prow = static_cast<int64_t>(t.u) * a.n * a.G + t.row0 + (valid ? row : 0);
  auto write_stats = [&](float top, float sum) {
    if (part)
      a.part_ml[prow * a.splits + t.split] = make_float2(top, sum);
    else if (a.lse)
      a.lse[((static_cast<int64_t>(t.b) * a.L + t.l) * (a.Hkv * a.G) + head) * a.n + node] =
          sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
  };
  float m2 = m == -INFINITY ? -INFINITY : m - static_cast<float>(e_ref);
  if (share && valid) write_stats(m2, l);        // while the last product of this stream runs
  if (!fail && n > 0 && !warp_wait(smem_u32(&s.odone[h]), (n - 1) & 1, abort_flag)) fail = true;
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
    fail = named_bar_or(1, 256, fail);                       // both streams' products are done
    tc_fence_after();
    n_other = uniform(s.tiles[h ^ 1]);
    e_ref = s.e_ref;                                         // (a stream without tiles has not read it)
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
    const float inv = part ? 1.f : l > 0.f ? 1.f / l : 0.f;
    const float back = pow2(e_ref);                          // outputs are 2^e_ref times what is accumulated
    f0 = f0 * inv * back;
    f1 = f1 * inv * back;
    const int64_t own = static_cast<int64_t>(head) * a.os.head + static_cast<int64_t>(node) * a.os.token;
    // this stream's columns, staged in shared memory in 16-byte chunks (Q is not read any more)
    const int cols = share ? D : D / 2, col0 = share ? 0 : h * (D / 2);
    const int chunks = cols / 8, flip = min(chunks - 1, 7);
    uint8_t* stage = sq + h * C::kTile + (share ? 0 : h * 4096) + quarter * (32 * chunks * 16);
    const int pitch = min(chunks, 8) * 16;
    float* part_o = a.part_o + (prow * a.splits + t.split) * D + col0;
    const uint32_t mine = o_col + col0, other = tmem + lanes + kOCol + (h ^ 1) * 128 + col0;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      if (c * 32 >= cols) break;
      uint32_t o0[32] = {}, o1[32] = {};
      if (n > 0) tmem_ld32_issue(mine + c * 32, o0);
      if (!share && n_other > 0) tmem_ld32_issue(other + c * 32, o1);
      tmem_ld_wait(o0);
      tmem_ld_wait(o1);
      float x[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        // element e of its eight lies at place 2 e (0..3) or 2 e - 7 (4..7)
        const int at = (e & ~7) + ((e & 7) < 4 ? 2 * (e & 7) : 2 * (e & 7) - 7);
        x[e] = __uint_as_float(o0[at]) * f0;
        if (!share) x[e] = fmaf(__uint_as_float(o1[at]), f1, x[e]);
      }
      if (!valid) continue;
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
    }
    if (!part) {
      // from shared memory, whole rows (or halves) per store
      __syncwarp();
      const int row0 = (share ? h * kTileRows : 0) + quarter * 32;
      const int chunk = lane & (chunks - 1), per = 32 / chunks;           // rows per instruction
      __nv_bfloat16* out = a.out + t.b * a.os.batch + t.l * a.os.layer + col0;
#pragma unroll 4
      for (int i = 0; i < chunks; ++i) {
        const int rr = i * per + lane / chunks;
        const int64_t at = __shfl_sync(kFull, own, rr);
        if (row0 + rr < t.rows)
          *(reinterpret_cast<uint4*>(out + at) + chunk) =
              *reinterpret_cast<const uint4*>(stage + (chunk >> 3) * 4096 + rr * pitch + (((chunk & 7) ^ (rr & flip)) << 4));
      }
    }
  }
  if (fail && lane == 0 && a.unit_status) a.unit_status[t.u] = KVC_UNIT_TIMEOUT;
}

template <int D, bool ROW, bool MODS>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TreeArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sq = base;                                  // two Q tiles
  uint8_t* sk = sq + 2 * C::kTile;
  uint8_t* sv = sk + kStages * C::kTile;
  Bars& s = *reinterpret_cast<Bars*>(sv + kStages * C::kTile);
  const int warp = uniform(threadIdx.x >> 5);
  wait_for_previous_kernel();
  let_next_kernel_start();
  const Item t = make_item(a, blockIdx.x);
  if (t.rows == 0) return;                             // rows past the tree's nodes
  const bool share = t.rows > kTileRows;               // two Q tiles, or two streams over one
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      // (a.stall_unit: a test makes the first key tile's wait expect an arrival that never comes)
      mbar_init(smem_u32(&s.kfull[i]), i == 0 && t.u == a.stall_unit ? 5 : 4);
      mbar_init(smem_u32(&s.kempty[i]), 1);
      mbar_init(smem_u32(&s.vfull[i]), 4);
      mbar_init(smem_u32(&s.vempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.sfull[i]), 1);
      mbar_init(smem_u32(&s.phalf[i]), 4);
      mbar_init(smem_u32(&s.pfull[i]), 4);
      mbar_init(smem_u32(&s.odone[i]), 1);
      mbar_init(smem_u32(&s.qfull[i]), 4);
    }
    mbar_init(smem_u32(&s.done), 1);
    s.abort_flag = 0;
    s.total = INT32_MAX;
    s.e_ref = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s.tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(s.tmem);
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kMmaWarp) issue<D>(t, s, sq, sk, sv, tmem, share);
  } else if (warp >= kOperandWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    make_operands<D, ROW, MODS>(a, t, s, sk, sv);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    softmax<D, ROW, MODS>(a, t, s, sq, tmem, share);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.n_blocks) * a.U * a.splits);
  const bool mods = a.mods.softcap > 0.f || a.mods.slopes || a.mods.window;
  auto go = [&](auto kernel) -> cudaError_t {
    const int bytes = a.d == 128 ? Cfg<128>::kSmem : Cfg<64>::kSmem;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e != cudaSuccess ? e : launch_after(kernel, dim3(grid), kThreads, bytes, stream, a);
  };
  auto go_mods = [&](auto d, auto row) -> cudaError_t {
    constexpr int D = decltype(d)::value;
    constexpr bool R = decltype(row)::value;
    return mods ? go(tree_kernel<D, R, true>) : go(tree_kernel<D, R, false>);
  };
  auto go_row = [&](auto d) -> cudaError_t {
    return a.rows.quant_mode == KVC_QUANT_ROW_FP16 ? go_mods(d, std::true_type{}) : go_mods(d, std::false_type{});
  };
  const cudaError_t e = a.d == 128 ? go_row(std::integral_constant<int, 128>{}) : go_row(std::integral_constant<int, 64>{});
  if (e != cudaSuccess || a.splits == 1) return e;
  PromptArgs m = {};                               // what joining the splits of a row needs
  m.U = a.U, m.L = a.L, m.Hkv = a.Hkv, m.B = a.B, m.G = a.G, m.d = a.d, m.n_q = a.n;
  m.q_len = a.n_nodes;
  m.os = a.os;
  m.out = a.out;
  m.lse = a.lse;
  m.splits = a.splits;
  m.part_o = a.part_o;
  m.part_ml = a.part_ml;
  return launch_prompt_merge(m, stream);
}

}  // namespace kvc
