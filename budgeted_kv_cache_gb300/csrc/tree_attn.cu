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
// scaled by a power of two per 32 rows that keeps them within its range (2^-ek for
// keys, 2^-ev for values; it is taken back in fp32: 2^ek goes into the softmax
// scale, 2^ev into the running maximum).  Elements more than 2^24 below the
// largest of their 32 rows lose bits to the format's end.  A scale per row in fp16 has 11
// bits itself: there the operands are the plain codes (beside which the tree's
// values are kept below 2^3, and lose bits from 2^20 below the largest on), and
// the scales multiply the scores and the weights in fp32.  Queries are scaled to fp16 per row alike;
// they, and the tree's rows, come in 8 bits.
//   S = Q K^T      tcgen05, both operands in shared memory, S in tensor memory
//   softmax        128 threads, one row each, in base 2; the weights are rounded
//                  to fp16 (2^-11 of a weight, and 2^-25 of the largest product
//                  of weight and value) and stored over S in tensor memory; the
//                  row's sum is that of the unrounded weights (formed anew, key by
//                  key, where the values' sizes leave no common reference for it and
//                  the outputs: kSpread).  The accumulator is rescaled only when
//                  the maximum grew by more than 2^8
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
// Warp roles (20 warps): 0-3 and 4-7 softmax of stream 0 and 1 (152 registers),
// 8-11 make the keys' operands and 12-15 the values' (64; a quarter of every tile
// each), 16 tensor memory and MMA issuer (48): 2 x 152 + 2 x 64 + 48 = 5 x 96, what
// the block was launched with.  Every wait is bounded; one that gives up raises a
// shared abort flag, the unit is marked KVC_UNIT_TIMEOUT and the block ends.
//
// Up to 16 query rows (32 at d = 64) kvc_i4_attn's warps take over (launch_tree).
//
// Measured, replayed from a graph (d = 128, 32 heads over 8, a scale per 32
// elements): 64 nodes, 64 units of 20K to 32K rows 245 us = 50 % of the measured
// tensor rate (263 without the longest units' blocks first); 32 nodes, 8 units of 131,072 rows 81 us = 1.9 TB/s; 13 nodes,
// 8 units of 2,304 rows 13 us, two kernels' latencies.  With a scale per row,
// d = 64, cap, slopes and a window of 4,096, up to 37 nodes and 9,001 rows: 26 us.
// No unit is full: the chain scores - maximum - weights - product of 64 keys
// bounds it (a scheduler issues in 55 % of its cycles, tensor pipe 46 %, ALU 34 %,
// exponentials 23 %; without the exponentials 9 %, without turning codes into
// operands 8 % less time).  64 keys a step, so that a stream's next scores are in
// the making meanwhile.  Each operand warp turns its own 32 rows of every tile:
// with a named barrier that joined four of them at every tile 503 us, not 310.
#include <algorithm>
#include <type_traits>

#include "i4_codes.cuh"
#include "kvc_internal.cuh"
#include "packed_math.cuh"
#include "tc_attn.cuh"

namespace kvc {

namespace {

constexpr int kThreads = 640;
constexpr int kTileRows = 128;
constexpr int kKeys = 128;                       // keys per tile
constexpr uint32_t kTmemCols = 512;              // S0, S1, O0, O1 of 128 columns each
constexpr uint32_t kOCol = 256;
constexpr int kKeyWarp = 8, kValueWarp = 12, kMmaWarp = 16;        // four, four, one
constexpr int kStages = 2;                       // key tiles, and value tiles, in shared memory
constexpr int kSlots = 4;                        // tiles whose description is held
constexpr int kAhead = 4;                        // tiles prefetched to L2 behind the one on its way
constexpr int kEnd = INT32_MIN;
constexpr int kLeast = -100;                     // least exponent: rows below 2^-90 lose bits, and 2^-ev stays in range
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;                     // log2 growth of the maximum that forces a rescale
// The row sum shares the outputs' reference m, the maximum of y + ev.  A weight 2^(y + ev - m) is lost below 2^-126: with the
// values' exponents no further apart than kSpread that is less than 2^-34 of the sum (m <= max y + max ev).  From +-kSizes on
// the sum itself would leave fp32's range (2^31 weights beside exponents of -kSizes do not).
constexpr int kSpread = 92, kSizes = 85;
constexpr int kFar = 40;                         // exponents from which on a block's reference is brought back to the scores'
// Exponents of 32 rows that hold nothing but zeros (below any that matters), and of 32 places without rows (no further than
// kSpread from any others; nothing is seen there).
constexpr int kNoValues = -kSizes, kNoRows = kSpread + kLeast;

// What an item covers.
struct Item {
  int u, b, l, g, split;
  int row0, rows;              // first packed row, packed rows of the item (<= 256)
  int count, next, prefix;     // cached rows, position of the first nodes, visible prefix
  int cached;                  // tiles of cached rows
  int i0, i1, step;            // of those and the tree's this split takes i0, i0 + step, .. below i1
  int nodes;                   // of the tree, as far as this item's rows see
};

struct Bars {
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t efull[kStages], sfull[2][2], pfull[2][2], odone[2], qfull[2], done, sizes;      // [stream][half of a tile's keys]
  uint32_t tmem;
  int abort_flag;
  int ev_min, ev_max;          // of the values' exponents (once `sizes` is complete)
  Item item;                   // (for sum_alone)
  int tiles[2];                // of each stream
  int j0[2 * kSlots];          // a tile's first slot, or -1 - its first node; kEnd: no more tiles (for either stream)
  // operands are keys times 2^-ek and values times 2^-ev, per 32 rows: 2^ek; ev and 2^-ev
  alignas(16) float k_by[kSlots][4];
  alignas(16) float2 v_by[kSlots][4];
  int16_t parent[KVC_TREE_MAX_NODES], depth[KVC_TREE_MAX_NODES];      // of the nodes that the item's rows see
  int32_t counts[kTreeRanked], unit;   // rows in use of every unit; the one that this block takes
  float2 ml[2][kTileRows];     // of each stream's rows: reference of the sum, and the sum
  float m[2][kTileRows];       // reference of the outputs
  int8_t q_exp[128];           // queries are rows times 2^-q_exp (one row tile)
  // with modifiers: smallest position of 32 rows; positions, and how far they lie behind the first nodes
  alignas(16) int32_t p_min[kSlots][4], pos[kSlots][kKeys];
  alignas(16) float behind[kSlots][kKeys];
  alignas(16) float ks[kSlots][kKeys], vs[kSlots][kKeys];    // scale per row: of keys; of values times 2^-ev
};

template <int D>
struct Cfg {
  static constexpr int kTile = D / 64 * kChunkBytes;         // a Q, K or V tile
  static constexpr int kRaw = 32 * (D / 2);                  // codes of 32 rows
  static constexpr int kSmem = (2 + 2 * kStages) * kTile + 8 * kRaw + 1024 /* alignment */ + sizeof(Bars);
};
static_assert(Cfg<128>::kSmem <= 232448, "shared memory of a block");

// Block `id` of the grid: the splits of an item, the items of a unit and the units follow each other.  All threads call.
__device__ __forceinline__ Item make_item(const TreeArgs& a, int id, Bars& s) {
  Item t;
  uint32_t split, qb, g, l, u = a.by_blocks.divmod(a.by_splits.divmod(id, &split), &qb);
  if (a.longest_first) {
    // the unit that u others precede
    const int i = threadIdx.x;
    const int own = i < a.U ? clamp_count(a.rows.count[i], a.rows.capacity) : 0;
    if (i < a.U) s.counts[i] = own;
    __syncthreads();
    uint32_t rank = 0;
#pragma unroll 8
    for (int v = 0; v < a.U; ++v) rank += s.counts[v] > own || (s.counts[v] == own && v < i);
    if (i < a.U && rank == u) s.unit = i;
    __syncthreads();
    u = s.unit;
  }
  t.split = static_cast<int>(split);
  t.u = static_cast<int>(u);
  t.b = static_cast<int>(a.by_layers.divmod(a.by_heads.divmod(u, &g), &l));
  t.l = static_cast<int>(l);
  t.g = static_cast<int>(g);
  t.count = clamp_count(a.rows.count[t.u], a.rows.capacity);
  t.next = a.rows.next_pos[t.u];
  t.prefix = a.mods.prefix_len ? a.mods.prefix_len[t.b] : INT32_MIN;
  const int n = a.n_nodes ? clamp_count(a.n_nodes[t.b], a.n) : a.n;
  t.row0 = static_cast<int>(qb) * a.block_rows;
  t.rows = max(0, min(a.block_rows, n * a.G - t.row0));
  t.nodes = t.rows > 0 ? static_cast<int>(a.by_group.div(t.row0 + t.rows - 1)) + 1 : 0;
  t.cached = (t.count + kKeys - 1) / kKeys;
  const uint32_t all = t.cached + (t.nodes + kKeys - 1) / kKeys;
  t.i0 = static_cast<int>(a.by_splits.div(all * split));             // tiles < 2^24 + 8, splits < 256
  t.i1 = static_cast<int>(a.by_splits.div(all * (split + 1)));
  t.step = 1;
  if (a.mods.window) t.i0 = split, t.i1 = all, t.step = a.splits;    // every split has a part of what is seen
  return t;
}

// Distance back to a position that lies at or before p (up to 2^32 - 1: positions are any 32-bit integers).
__device__ __forceinline__ uint32_t behind(int p, int before) { return static_cast<uint32_t>(p) - static_cast<uint32_t>(before); }

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(max(-126, min(127, e)) + 127) << 23); }

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

// Eight bf16 elements in the same order, times a power of two.
__device__ __forceinline__ uint4 bf16_to_half(const uint4& w, float by) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  auto at = [&](int i) { return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16) * by; };
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

// What seldom happens is told to the compiler, which puts it out of the way: the roles' loops are long, and a jump over
// code that is not there yet costs more than what it skips.
#define SELDOM(x) (__builtin_expect(static_cast<bool>(x), 0))

// Natural logarithm of 2^top times the sum: -inf for a row that saw nothing, NaN for one whose scores are no numbers.
__device__ __forceinline__ float row_statistic(float top, float sum) { return sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2; }

// warp_wait, its first test in line.
__device__ __forceinline__ bool wait_for(const uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t at = smem_u32(bar);
  if (SELDOM(!__all_sync(kFull, try_once(at, parity)))) return warp_wait(at, parity, abort);
  return true;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ uint4 load_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void store_shared(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 16-byte piece c of row r of an operand tile of 64-element chunks in 128-byte swizzle.
__device__ __forceinline__ uint4* piece(uint8_t* tile, int r, int c) {
  return reinterpret_cast<uint4*>(tile + (c >> 3) * kChunkBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// ---------------------------------------------------------------- operand warps

// One warp turns a quarter (32 rows) of every tile of the item's keys (v = false) or values into operands; nothing but
// the tiles' barriers joins it with others.  The next tile's codes are on their way to the warp's own shared memory
// while those in registers are turned, and tiles behind that one to L2.
template <int D, bool ROW, bool MODS>
__device__ __forceinline__ void make_operands(const TreeArgs& a, const Item& t, Bars& s, uint8_t* ring, uint8_t* raw, bool v) {
  using C = Cfg<D>;
  constexpr int CH = D / 32;                     // 16-byte pieces of codes per row; a lane turns one row
  using Scales = typename std::conditional<ROW, uint16_t, typename std::conditional<D == 128, uint2, uint32_t>::type>::type;
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, first = quarter * 32;
  volatile int* abort_flag = &s.abort_flag;
  uint64_t* const full = v ? s.vfull : s.kfull;
  uint64_t* const empty = v ? s.vempty : s.kempty;
  const int64_t base = static_cast<int64_t>(t.u) * a.rows.capacity;
  const uint8_t* const codes = static_cast<const uint8_t*>(v ? a.rows.v : a.rows.k) + (base + first) * (D / 2);
  const Scales* const scales = static_cast<const Scales*>(v ? a.rows.v_scale : a.rows.k_scale) + base + first;
  const bool windowed = MODS && a.mods.window;
  // Copies of the quarter's codes of cached tile i, and its scales to a register: a row a lane.  Nothing behind the rows
  // in use is read.
  Scales sc = {};
  int32_t pos = 0;
  auto spot = [&](int r, int c) { return raw + r * (D / 2) + ((c ^ (D == 128 ? (r >> 1) & 3 : (r >> 2) & 1)) << 4); };
  const uint32_t spot0 = smem_u32(spot(lane / CH, lane % CH)), own_raw = smem_u32(raw) + lane * (D / 2);
  const int flip = D == 128 ? (lane >> 1) & 3 : (lane >> 2) & 1;
  constexpr int kStep = 32 / CH;                 // rows of one copy of the warp; the swizzle repeats with them
  auto load = [&](int i) {
    const int left = t.count - i * kKeys - first;
    const uint8_t* src = codes + static_cast<int64_t>(i) * (kKeys * D / 2) + lane * 16;
    const int64_t j = static_cast<int64_t>(i) * kKeys + lane;
    if (__builtin_expect(left >= 32, 1)) {
#pragma unroll
      for (int k = 0; k < CH; ++k) cp_async16(spot0 + k * 512, src + k * 512, true);
      sc = scales[j];
      if (MODS) pos = a.rows.pos[base + first + j];
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const bool ok = k * kStep + lane / CH < left;
        cp_async16(spot0 + k * 512, ok ? src + k * 512 : codes - first * (D / 2), ok);
      }
      sc = Scales{};
      if (lane < left) {
        sc = scales[j];
        if (MODS) pos = a.rows.pos[base + first + j];
      }
    }
    cp_async_commit();
  };
  auto prefetch = [&](int i) {
    const int left = min(32, t.count - i * kKeys - first);
    if (i >= min(t.cached, t.i1) || left <= 0) return;
    if (lane * 128 < left * (D / 2)) prefetch_l2(codes + static_cast<int64_t>(i) * (kKeys * D / 2) + lane * 128);
    if (lane >= 30 && (lane - 30) * 128 < left * static_cast<int>(sizeof(Scales)))
      prefetch_l2(reinterpret_cast<const uint8_t*>(scales + static_cast<int64_t>(i) * kKeys) + (lane - 30) * 128);
  };
  // The walk over the item's tiles: cached ones in order (with a window those that some node sees), then the tree's from
  // the last to the first.  Every warp walks alike.
  int at = t.i0;
  auto next = [&]() -> int {
    for (; at < t.i1; at += t.step) {
      if (!windowed || at >= t.cached) {
        at += t.step;
        return at - t.step;
      }
      bool seen = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = at * kKeys + k * 32 + lane;
        if (j < t.count) {
          const int p = a.rows.pos[base + j];
          seen |= behind(t.next, p) < static_cast<uint32_t>(a.mods.window) || p < t.prefix;
        }
      }
      if (__any_sync(kFull, seen)) {
        at += t.step;
        return at - t.step;
      }
    }
    return -1;
  };
  int cur = next();
  if (cur >= 0 && cur < t.cached) load(cur);
  // without a window the tiles follow each other
  if (!windowed)
    for (int i = 1; i <= kAhead; ++i) prefetch(t.i0 + i);

#pragma unroll 1
  for (int n = 0;; ++n) {
    const int slot = n & (kSlots - 1), st = n & 1;
    const bool tree = cur >= t.cached;
    auto wait_empty = [&] { return wait_for(&empty[st], ((n >> 1) & 1) ^ 1, abort_flag); };
    if (SELDOM(cur < 0)) {                               // the end: one more phase of the keys, without any
      if (v || !wait_empty()) break;
      if (threadIdx.x == kKeyWarp * 32) s.j0[n & (2 * kSlots - 1)] = s.j0[(n + 1) & (2 * kSlots - 1)] = kEnd;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.kfull[st]));
      break;
    }
    uint8_t* const to = ring + st * C::kTile;
    const int j0 = tree ? ((t.nodes + kKeys - 1) / kKeys - 1 - (cur - t.cached)) * kKeys : cur * kKeys;
    auto publish = [&](int e, Scales own, int32_t p) {      // what the softmax needs of this quarter
      if (v) {
        if (ROW) {
          const float f = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(&own)));
          s.vs[slot][first + lane] = tree ? 1.f : fminf(f * pow2(-e), 2.f);      // a row of zeros may have a scale above the others'
        }
        if (lane == 0) s.v_by[slot][quarter] = make_float2(static_cast<float>(e), pow2(-e));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.efull[st]));
        // (a test makes a unit's values late: the softmax is done with the tile by then)
        if (SELDOM(t.u == a.late_unit))
          for (int i = 0; i < 20; ++i) __nanosleep(1000);
        return;
      }
      if (lane == 0) {
        s.k_by[slot][quarter] = pow2(e);
        if (quarter == 0) s.j0[n & (2 * kSlots - 1)] = tree ? -1 - j0 : j0;
      }
      const int j = j0 + first + lane;
      if (MODS) {
        if (tree && j < t.nodes) p = t.next + s.depth[j];
        s.pos[slot][first + lane] = p;
        s.behind[slot][first + lane] = tree ? -static_cast<float>(p - t.next) : static_cast<float>(behind(t.next, p));
        const int low = __reduce_min_sync(kFull, j < (tree ? t.nodes : t.count) ? p : INT32_MAX);
        if (lane == 0) s.p_min[slot][quarter] = low;
      }
      if (ROW) s.ks[slot][first + lane] = tree ? 1.f : __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t*>(&own)));
    };
    if (__builtin_expect(!tree, 1)) {
      // this tile's codes to registers, the next one's on their way
      cp_async_wait<0>();
      const Scales own = sc;
      const int32_t own_pos = pos;
      __syncwarp();
      uint4 w[CH];
      uint32_t top = 0;
      auto scale = [&](int k) -> uint32_t {
        if constexpr (ROW) return own;
        else if constexpr (D == 128) return k == 0 ? own.x & 0xffffu : k == 1 ? own.x >> 16 : k == 2 ? own.y & 0xffffu : own.y >> 16;
        else return k == 0 ? own & 0xffffu : own >> 16;
      };
      // A group of zeros tells nothing about the sizes of the others, whatever its scale (the quantiser writes 1)
      auto zeros = [](const uint4& x) { return (x.x | x.y | x.z | x.w) == 0; };
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        w[k] = load_shared(own_raw + ((k ^ flip) << 4));
        if (v || !ROW) top = max(top, zeros(w[k]) ? 0u : scale(k));
      }
      __syncwarp();
      if (!windowed) prefetch(cur + 1 + kAhead);
      cur = next();
      if (cur >= 0 && cur < t.cached) load(cur);
      int e = !v ? 0 : j0 + first < t.count ? kNoValues : kNoRows;             // rows times 2^-e:
      if (v || !ROW) {
        top = __reduce_max_sync(kFull, top);
        if (top && !ROW) e = max(exponent_of(top) - 10, kLeast);               // the largest scale below 2^11
        else if (top) e = static_cast<int>(max(1u, top >> 10)) - 14;           // the largest row scale below 1
      }
      if (!wait_empty()) break;
      publish(e, own, own_pos);
      const float by = pow2(-e);
      const int key = first + lane, x = key & 7;
      const uint32_t row = smem_u32(to) + key * 128;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        uint32_t f = 0x3c003c00u, m;             // a scale per row: the codes alone
        if (!ROW) {
          const float g = zeros(w[k]) ? 0.f : __uint_as_float(scale(k) << 16) * by;
          f = pack_half2(g, g);
        }
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(m) : "r"(f), "r"(0xce00ce00u));         // -24
        const uint32_t word[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store_shared(row + (k >> 1) * kChunkBytes + ((((k & 1) * 4 + j) ^ x) << 4), codes_to_half(word[j], f, m));
      }
    } else {
      // the tree's rows, bf16, straight to their places; then turned there, each lane its own pieces
      if (!wait_empty()) break;
      const __nv_bfloat16* src = (v ? a.v_new : a.k_new) + t.b * a.news.batch + t.l * a.news.layer + t.g * a.news.head;
      constexpr int BP = D / 8;
      {
        const int c = lane % BP, r0 = first + lane / BP;
#pragma unroll 4
        for (int r = 0; r < 32; r += 32 / BP) {
          const bool ok = j0 + r0 + r < t.nodes;
          cp_async16(smem_u32(piece(to, r0 + r, c)), ok ? src + static_cast<int64_t>(j0 + r0 + r) * a.news.token + c * 8 : src, ok);
        }
      }
      cp_async_commit();
      cur = next();
      cp_async_wait<0>();
      __syncwarp();
      uint32_t top = 0;
#pragma unroll 4
      for (int c = 0; c < BP; ++c) top = max(top, max_bits(*piece(to, first + lane, c)));
      top = __reduce_max_sync(kFull, top);
      // the largest element below 2^14, as a group's code times its scale; below 2^3, as a plain code, with a scale per
      // row: what the weights are multiplied by is of one size in all tiles, so that none is smaller than it has to be
      const int e = top ? max(exponent_of(top) - (v && ROW ? 2 : 13), kLeast) : !v ? 0 : j0 + first < t.nodes ? kNoValues : kNoRows;
      publish(e, Scales{}, 0);
      const float by = pow2(-e);
#pragma unroll 2
      for (int c = 0; c < BP; ++c) {
        uint4* x = piece(to, first + lane, c);
        *x = bf16_to_half(*x, by);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&full[st]));
  }
  cp_async_wait<0>();                            // of a tile that an abort left
}

// ---------------------------------------------------------------- MMA issuer

// A stream's scores of 64 keys are in the making while its softmax works on the 64 before: S of half b lies in columns
// 64 b of the stream's 128, its weights over the first 32 of them.
template <int D>
__device__ __forceinline__ void issue(const Item& t, Bars& s, uint8_t* sq, uint8_t* sk, uint8_t* sv, uint32_t tmem, bool share, bool stall) {
  using C = Cfg<D>;
  volatile int* abort_flag = &s.abort_flag;
  constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(128 >> 4) << 24);           // fp16 x fp16 -> fp32, M = 128
  constexpr uint32_t kHalf = kKeys / 2 * 128 >> 4;                 // half of a tile's rows
  const uint32_t idesc_s = kIdesc | (static_cast<uint32_t>(kKeys / 2 >> 3) << 17);
  const uint32_t idesc_o = kIdesc | (static_cast<uint32_t>(D >> 3) << 17) | (1u << 16);     // B (values) MN-major
  bool ok = wait_for(&s.qfull[0], 0, abort_flag);
  if (ok && share) ok = wait_for(&s.qfull[1], 0, abort_flag);
  const uint32_t elected = elect_one();
  const uint64_t q_desc = sw128_desc(smem_u32(sq)), k_desc = sw128_desc(smem_u32(sk)), val_desc = v_desc(smem_u32(sv));
  // stream h's tile of round j
  auto tile_of = [&](int j, int h) { return share ? j : 2 * j + h; };
  bool over = false;
  // waits for the keys of that tile; false: there is none, or the wait gave up
  auto has = [&](int j, int h) -> bool {
    if (over || !ok) return false;
    const int n = tile_of(j, h);
    if (SELDOM(!wait_for(stall ? &s.done : &s.kfull[n & 1], (n >> 1) & 1, abort_flag))) return ok = false;
    over = uniform(*reinterpret_cast<volatile int*>(&s.j0[n & (2 * kSlots - 1)])) == kEnd;
    return !over;
  };
  auto scores = [&](int j, int h, int b) {
    const uint32_t st = tile_of(j, h) & 1;
    const uint64_t qd = q_desc + (share ? h : 0) * (C::kTile >> 4), kd = k_desc + st * (C::kTile >> 4) + b * kHalf;
    tc_fence_after();
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const uint32_t off = (ks >> 2) * (kChunkBytes >> 4) + (ks & 3) * 2;
      mma_ss(tmem + h * 128 + b * 64, qd + off, kd + off, idesc_s, ks > 0 ? 1u : 0u, elected);
    }
    commit(smem_u32(&s.sfull[h][b]), elected);
    if (b == 1 && (!share || h == 1)) commit(smem_u32(&s.kempty[st]), elected);
  };
  float ev_min = INFINITY, ev_max = -INFINITY;   // of the values' exponents: the issuer has the time to look after them
  auto values = [&](int j, int h, int b) -> bool {
    const int n = tile_of(j, h);
    const uint32_t st = n & 1;
    if (b == 0 && (!share || h == 0) && SELDOM(!wait_for(&s.vfull[st], (n >> 1) & 1, abort_flag))) return false;
    if (SELDOM(!wait_for(&s.pfull[h][b], j & 1, abort_flag))) return false;
    tc_fence_after();
    const uint64_t vd = val_desc + st * (C::kTile >> 4) + b * kHalf;
    const uint32_t more = j + b > 0 ? 1u : 0u;
#pragma unroll
    for (int ks = 0; ks < kKeys / 32; ++ks)
      mma_ts(tmem + kOCol + h * 128, tmem + h * 128 + b * 64 + ks * 8, vd + ((ks * 16 * 128) >> 4), idesc_o, ks > 0 ? 1u : more, elected);
    commit(smem_u32(&s.odone[h]), elected);
    if (b == 1 && (!share || h == 1)) {
      commit(smem_u32(&s.vempty[st]), elected);
      const float ev = *const_cast<volatile float*>(&s.v_by[n & (kSlots - 1)][threadIdx.x & 3].x);
      ev_min = fminf(ev_min, ev);
      ev_max = fmaxf(ev_max, ev);
    }
    return true;
  };
  bool live0 = has(0, 0), live1 = false;
  if (live0) scores(0, 0, 0);
  if (live0) live1 = share || has(0, 1);
  if (live1) scores(0, 1, 0);
  if (live0) scores(0, 0, 1);
  if (live1) scores(0, 1, 1);
#pragma unroll 1
  for (int j = 0; ok && live0; ++j) {
    bool next0 = false, next1 = false;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (!(ok = ok && values(j, 0, b))) break;
      if (b == 0) next0 = has(j + 1, 0);
      if (next0) scores(j + 1, 0, b);
      if (!live1) continue;
      if (!(ok = ok && values(j, 1, b))) break;
      if (b == 0) next1 = next0 && (share || has(j + 1, 1));
      if (next1) scores(j + 1, 1, b);
    }
    live0 = next0;
    live1 = next1;
  }
  // The streams' next scores are none (after an abort they find that by themselves), told by the tensor core once every
  // product above is done: whoever learns of the end may read the outputs.  A wait for odone could not tell the last
  // product from the last but one of the same parity, and the values of both halves may be late.
  if (ok) {
    commit(smem_u32(&s.sfull[0][0]), elected);
    commit(smem_u32(&s.sfull[1][0]), elected);
  }
  // (and the values' exponents, while those products run)
  for (int k = 1; k < 4; k <<= 1) {
    ev_min = fminf(ev_min, __shfl_xor_sync(kFull, ev_min, k));
    ev_max = fmaxf(ev_max, __shfl_xor_sync(kFull, ev_max, k));
  }
  if (elected) {
    const bool any = ev_max > -INFINITY;
    s.ev_min = any ? static_cast<int>(ev_min) : 0;
    s.ev_max = any ? static_cast<int>(ev_max) : 0;
    mbar_arrive(smem_u32(&s.sizes));
  }
  __syncwarp();
  // all MMAs issued above complete before tensor memory is freed
  commit(smem_u32(&s.done), elected);
  drain(smem_u32(&s.done), 0);
}

// ---------------------------------------------------------------- softmax

// The sum of a row's 2^y (and its reference) over every `parts`-th tile of the item, a key after the other on the CUDA cores:
// where the sizes of values differ so much that weights relative to the outputs' reference cannot hold it.  Slow (64 units of
// 20K to 32K rows x 256 query rows 24 ms, not 226 us), for values that no model has; code for them in the loop of the tiles
// cost everyone 1 to 5 %, not taken.
template <int D, bool ROW, bool MODS>
__device__ __noinline__ float2 sum_alone(const TreeArgs& a, const Bars& s, int node, int head, int part, int parts) {
  const Item& t = s.item;
  const int64_t base = static_cast<int64_t>(t.u) * a.rows.capacity;
  const uint4* const q = reinterpret_cast<const uint4*>(a.q + t.b * a.qs.batch + t.l * a.qs.layer + static_cast<int64_t>(head) * a.qs.head +
                                                        static_cast<int64_t>(node) * a.qs.token);
  auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
  auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
  const float cap = MODS ? a.mods.softcap : 0.f, slope = MODS && a.mods.slopes ? a.mods.slopes[head] * kLog2e : 0.f;
  const int p_q = t.next + (MODS && (a.mods.slopes || a.mods.window) ? s.depth[node] : 0);
  float m = -INFINITY, l = 0.f;
  auto add = [&](float x, int p) {
    const uint32_t dist = behind(p_q, p);
    if (MODS && a.mods.window && dist >= static_cast<uint32_t>(a.mods.window) && p >= t.prefix) return;
    x *= a.scale;
    x = cap > 0.f ? capped_base2(x, x * fminf(1.f / cap, 1e30f), cap) : x * kLog2e;
    if (MODS && a.mods.slopes) x = fmaf(-slope, static_cast<float>(dist), x);
    if (x - m > kGrow) {                         // also from -inf
      l *= m == -INFINITY ? 0.f : ex2_approx(m - x);
      m = x;
    }
    l += ex2_approx(x - m);
  };
  int n = 0;
#pragma unroll 1
  for (int at = t.i0; at < t.i1; at += t.step, ++n) {
    if (n % parts != part) continue;
    if (at < t.cached) {
#pragma unroll 1
      for (int j = at * kKeys; j < min(t.count, (at + 1) * kKeys); ++j) {
        const uint32_t* codes = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.rows.k) + (base + j) * (D / 2));
        const uint16_t* scales = static_cast<const uint16_t*>(a.rows.k_scale) + (base + j) * (ROW ? 1 : D / 32);
        float x = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = q[c];
          const uint32_t v[4] = {w.x, w.y, w.z, w.w}, code = codes[c];
          const uint16_t f = scales[ROW ? 0 : c / 4];
          float y = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y = fmaf(e & 1 ? hi(v[e / 2]) : lo(v[e / 2]), static_cast<float>(static_cast<int32_t>(code << (28 - 4 * e)) >> 28), y);
          x = fmaf(y, ROW ? __half2float(__ushort_as_half(f)) : __uint_as_float(static_cast<uint32_t>(f) << 16), x);
        }
        add(x, MODS ? a.rows.pos[base + j] : 0);
      }
    } else {
      const int j0 = ((t.nodes + kKeys - 1) / kKeys - 1 - (at - t.cached)) * kKeys;
      for (int j = node; j >= j0; j = s.parent[j]) {
        if (j >= j0 + kKeys) continue;
        const uint4* k = reinterpret_cast<const uint4*>(a.k_new + t.b * a.news.batch + t.l * a.news.layer + t.g * a.news.head + j * a.news.token);
        float x = 0.f;
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          const uint4 w = k[c], y = q[c];
          x = fmaf(lo(y.x), lo(w.x), fmaf(hi(y.x), hi(w.x), x));
          x = fmaf(lo(y.y), lo(w.y), fmaf(hi(y.y), hi(w.y), x));
          x = fmaf(lo(y.z), lo(w.z), fmaf(hi(y.z), hi(w.z), x));
          x = fmaf(lo(y.w), lo(w.w), fmaf(hi(y.w), hi(w.w), x));
        }
        add(x, MODS && (a.mods.slopes || a.mods.window) ? t.next + s.depth[j] : t.next);
      }
    }
  }
  return make_float2(m, l);
}

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

  // Queries of this warp's 32 rows, straight to their places in whole rows; then each lane scales its own to fp16 by a
  // power of two.  One row tile is made by the first stream's warps.
  int q_exp = 0;
  if (share || h == 0) {
    constexpr int LPR = D / 8, PER = 32 / LPR;
    uint8_t* const tile = sq + (share ? h : 0) * C::kTile;
    const __nv_bfloat16* q = a.q + t.b * a.qs.batch + t.l * a.qs.layer;
    const int64_t own = static_cast<int64_t>(head) * a.qs.head + static_cast<int64_t>(node) * a.qs.token;
#pragma unroll 8
    for (int i = 0; i < 32; i += PER) {
      const int rr = i + lane / LPR;
      const int64_t at = __shfl_sync(kFull, own, rr);
      const bool ok = row - lane + rr < t.rows;
      cp_async16(smem_u32(piece(tile, quarter * 32 + rr, lane % LPR)), ok ? q + at + (lane % LPR) * 8 : q, ok);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    uint32_t top = 0;
#pragma unroll 8
    for (int c = 0; c < LPR; ++c) top = max(top, max_bits(*piece(tile, r, c)));
    // the largest element below 2^15 (bounded: queries below 2^-100 lose bits, and no score)
    q_exp = top ? max(-112, min(113, exponent_of(top) - 14)) : 0;
    const float by = pow2(-q_exp);
#pragma unroll 4
    for (int c = 0; c < LPR; ++c) {
      uint4* x = piece(tile, r, c);
      *x = bf16_to_half(*x, by);
    }
    if (!share) s.q_exp[r] = static_cast<int8_t>(q_exp);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.qfull[share ? h : 0]));
  }
  bool fail = false;
  if (!share && h == 1) {
    if (SELDOM(!wait_for(&s.qfull[0], 0, abort_flag))) fail = true;
    q_exp = s.q_exp[r];
  }
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t s_col = tmem + lanes + h * 128, o_col = tmem + lanes + kOCol + h * 128;
  const bool warp_valid = __any_sync(kFull, valid);
  const bool capped = MODS && a.mods.softcap > 0.f, biased = MODS && a.mods.slopes, windowed = MODS && a.mods.window;
  const int depth = biased || windowed ? s.depth[node] : 0, p_q = t.next + depth;
  const float slope = biased ? a.mods.slopes[head] * kLog2e : 0.f;
  const float cap = MODS ? a.mods.softcap : 0.f, inv_cap = capped ? fminf(1.f / cap, 1e30f) : 0.f;
  const float scale = (capped ? a.scale : a.scale * kLog2e) * pow2(q_exp);
  int up = node;                                 // the lowest ancestor (or the node) that no tile has shown yet
  float m = -INFINITY, l = 0.f;                  // reference of y + ev (base 2), and sum of 2^(y - m)
  int n = 0;                                     // tiles of this stream
#pragma unroll 1
  for (; !fail; ++n) {
    if (SELDOM(!wait_for(&s.sfull[h][0], n & 1, abort_flag))) {
      fail = true;
      break;
    }
    const int i = share ? n : 2 * n + h, slot = i & (kSlots - 1);
    const int j0_or = *reinterpret_cast<volatile int*>(&s.j0[i & (2 * kSlots - 1)]);
    if (SELDOM(j0_or == kEnd)) break;
    if (SELDOM(!warp_valid)) {                           // nothing of this warp is a row: the products' results are not read
      tc_fence_after();
      tc_fence_before();
      if (lane == 0) mbar_arrive(smem_u32(&s.pfull[h][0]));
      if (SELDOM(!wait_for(&s.sfull[h][1], n & 1, abort_flag))) {
        fail = true;
        break;
      }
      tc_fence_after();
      tc_fence_before();
      if (lane == 0) mbar_arrive(smem_u32(&s.pfull[h][1]));
      continue;
    }
    const bool tree = j0_or < 0;
    const int j0 = tree ? -1 - j0_or : j0_or;
    uint32_t met[4] = {0, 0, 0, 0};              // keys of a tree's tile that this row sees
    if (SELDOM(tree)) {
      while (up >= j0 + kKeys) up = s.parent[up];
      while (up >= j0) {
        const int j = up - j0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j >> 5 == c) met[c] |= 1u << (j & 31);
        up = s.parent[up];
      }
    }
#pragma unroll 1
    for (int b = 0; b < 2; ++b) {
      if (b == 1 && SELDOM(!wait_for(&s.sfull[h][1], n & 1, abort_flag))) {
        fail = true;
        break;
      }
      tc_fence_after();
      uint32_t sr[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c) tmem_ld32_issue(s_col + b * 64 + c * 32, sr[c]);
      // y = scores in base 2 = acc f (scores themselves with a cap)
      const float2 k_by = *reinterpret_cast<const float2*>(&s.k_by[slot][2 * b]);
      auto factor = [&](float by) { return fminf(fmaxf(scale * by, 0x1p-126f), 0x1p120f); };
      float f[2] = {factor(k_by.x), factor(k_by.y)};
      const int left = t.count - j0 - b * 64;
      const bool whole = !tree && left >= 64;
#pragma unroll
      for (int c = 0; c < 2; ++c) tmem_ld_wait(sr[c]);
      float (&y)[2][32] = reinterpret_cast<float (&)[2][32]>(sr);
      // every four scores through one function of packed operations on pairs, with what lies at their keys' places
      auto each = [&](const float* at, auto change) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          ulonglong2 x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = at ? *reinterpret_cast<const ulonglong2*>(at + c * 32 + 4 * k) : make_ulonglong2(0, 0);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            unpair(change(pair(y[c][e], y[c][e + 1]), x[e / 4].x, c), &y[c][e], &y[c][e + 1]);
            unpair(change(pair(y[c][e + 2], y[c][e + 3]), x[e / 4].y, c), &y[c][e + 2], &y[c][e + 3]);
          }
        }
      };
      if (ROW) each(&s.ks[slot][b * 64], [&](uint64_t x, uint64_t k, int) { return mul2(x, k); });
      if (MODS) {
        if (capped) {
          float big = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) big = fmaxf(big, fabsf(y[c][e] *= f[c]));
          if (__all_sync(kFull, big * inv_cap <= kTanhRange || !valid)) {
            const uint64_t z2 = pair(inv_cap, inv_cap);
            each(nullptr, [&](uint64_t x, uint64_t, int) {
              const uint64_t z = mul2(x, z2), w = mul2(z, z);
              uint64_t p = pair(kTanh[4] * kLog2e, kTanh[4] * kLog2e);
#pragma unroll
              for (int k = 3; k >= 0; --k) p = fma2(p, w, pair(kTanh[k] * kLog2e, kTanh[k] * kLog2e));
              return mul2(x, p);
            });
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e) y[c][e] = capped_base2(y[c][e], y[c][e] * inv_cap, cap);
          }
          f[0] = f[1] = 1.f;
        }
        if (biased) {
          // whoever is seen lies behind the row: -slope (p_q - p) = -slope (next - p) - slope depth
          const float at = -slope * static_cast<float>(depth);
          const uint64_t at2 = pair(at, at), slope2 = pair(-slope, -slope);
          each(&s.behind[slot][b * 64],
               [&](uint64_t x, uint64_t behind, int c) { return fma2(slope2, behind, fma2(x, pair(f[c], f[c]), at2)); });
          f[0] = f[1] = 1.f;
        }
        if (windowed) {
          const int2 low = *reinterpret_cast<const int2*>(&s.p_min[slot][2 * b]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int p = c == 0 ? low.x : low.y;          // what lies furthest back
            if (__all_sync(kFull, p == INT32_MAX || behind(p_q, p) < static_cast<uint32_t>(a.mods.window))) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int k = s.pos[slot][b * 64 + c * 32 + e];
              if (behind(p_q, k) >= static_cast<uint32_t>(a.mods.window) && k >= t.prefix) y[c][e] = -INFINITY;
            }
          }
        }
      }
      if (SELDOM(!whole)) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t bits = tree ? (b ? met[2 + c] : met[c]) : bit_range(0, left - c * 32);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(bits & (1u << e))) y[c][e] = -INFINITY;
        }
      }
      float mx[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mx[c] = fmaxf(y[c][0], y[c][1]);
#pragma unroll
        for (int e = 2; e < 32; e += 2) mx[c] = fmax3(mx[c], y[c][e], y[c][e + 1]);
      }
      if (b == 0 && SELDOM(!wait_for(&s.efull[i & 1], (i >> 1) & 1, abort_flag))) {       // how far the values were scaled
        fail = true;
        break;
      }
      const float4 v_by = *reinterpret_cast<const float4*>(&s.v_by[slot][2 * b]);
      const float ev[2] = {v_by.x, v_by.z};
      const float top = fmaxf(fmaf(mx[0], f[0], ev[0]), fmaf(mx[1], f[1], ev[1]));
      const bool grow = top - m > kGrow;         // also from -inf
      if (SELDOM(__any_sync(kFull, grow))) {
        float by = 1.f;
        if (grow) {
          by = m == -INFINITY ? 0.f : ex2_approx(m - top);
          if (SELDOM(m - top < -100.f)) {        // (l may be so large that more of it is left than of `by`)
            const float half = ex2_approx(0.5f * (m - top));
            l = l * half * half;
          } else {
            l *= by;
          }
          m = top;
        }
        if (n + b > 0) {
          if (SELDOM(!wait_for(&s.odone[h], (b ^ 1) & 1, abort_flag))) {       // the product of the 64 keys before
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
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float sub = ev[c] - ref;
        const uint64_t f2 = pair(f[c], f[c]), sub2 = pair(sub, sub);
        uint64_t sum[2] = {0, 0};
        uint32_t pk[16];
        ulonglong2 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[k] = ROW ? *reinterpret_cast<const ulonglong2*>(&s.vs[slot][b * 64 + c * 32 + 4 * k]) : make_ulonglong2(0, 0);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float p0, p1;
            unpair(fma2(pair(y[c][e + 2 * k], y[c][e + 2 * k + 1]), f2, sub2), &p0, &p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            sum[k] = add2(sum[k], pair(p0, p1));
            if (ROW) unpair(mul2(pair(p0, p1), k ? v[e / 4].y : v[e / 4].x), &p0, &p1);
            pk[e / 2 + k] = pack_half2(p0, p1);
          }
        }
        float s0, s1;
        unpair(add2(sum[0], sum[1]), &s0, &s1);
        l = fmaf(s0 + s1, c == 0 ? v_by.y : v_by.w, l);
        tmem_st16(s_col + b * 64 + c * 16, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.pfull[h][b]));
    }
  }
  // statistics of the row, once they are those of all its keys in this item
  const bool part = a.splits > 1;
  const int64_t prow = static_cast<int64_t>(t.u) * a.n * a.G + t.row0 + (valid ? row : 0);
  auto write_stats = [&](float top, float sum) {
    if (part)
      a.part_ml[prow * a.splits + t.split] = make_float2(top, sum);
    else if (a.lse)
      a.lse[((static_cast<int64_t>(t.b) * a.L + t.l) * (a.Hkv * a.G) + head) * a.n + node] = row_statistic(top, sum);
  };
  // Where values are far from 1 the sum's reference m2 is brought near the largest score (splits are joined by it): by their
  // exponent, or, where they lie far apart, by a sum formed anew.
  float m2 = m;
  if (!fail && SELDOM(!wait_for(&s.sizes, 0, abort_flag))) fail = true;
  if (!fail && warp_valid) {
    const int lo = *const_cast<volatile int*>(&s.ev_min), hi = *const_cast<volatile int*>(&s.ev_max);
    if (SELDOM(abs(hi) > kFar || hi - lo > kSpread || lo < -kSizes)) {
      if (hi - lo > kSpread || hi > kSizes || (lo < -kSizes && t.i1 - t.i0 > 4096)) {
        s.item = t;                              // (the same from all)
        __syncwarp();
        const float2 own = sum_alone<D, ROW, MODS>(a, s, node, head, share ? 0 : h, share ? 1 : 2);
        m2 = own.x, l = own.y;
      } else {
        m2 -= static_cast<float>(hi);
        l *= pow2(hi);
      }
    }
    if (share && valid) write_stats(m2, l);
  }
  tc_fence_after();                              // the end is told behind the last product
  // One row tile: both streams hold an output for the same rows, in the same lanes of tensor memory.  They exchange
  // (m, l) and their outputs' references, and each joins and writes one half of the columns.
  int n_other = 0;
  // factors of the outputs, those of this stream and of the other
  auto factor = [](float m, float to) { return m == -INFINITY ? 0.f : ex2_approx(m - to); };
  float f0 = m2 == m ? 1.f : factor(m, m2), f1 = 0.f;
  if (!share) {
    s.ml[h][r] = make_float2(m2, l);
    s.m[h][r] = m;
    if (r == 0) s.tiles[h] = n;
    tc_fence_before();
    fail = named_bar_or(1, 256, fail);                       // both streams' products are done
    tc_fence_after();
    n_other = uniform(s.tiles[h ^ 1]);
    const float2 o = s.ml[h ^ 1][r];
    const float m_other = s.m[h ^ 1][r], mm = fmaxf(m2, o.x);
    f0 = factor(m2, mm);
    f1 = factor(o.x, mm);
    // the same order of the sum on both sides
    l = h == 0 ? fmaf(l, f0, o.y * f1) : fmaf(o.y, f1, l * f0);
    if (SELDOM(m2 != m)) f0 = factor(m, mm);
    if (SELDOM(o.x != m_other)) f1 = factor(m_other, mm);
    m2 = mm;
    if (valid && h == 0) write_stats(m2, l);
  }
  if (!fail && warp_valid) {
    const float inv = part ? 1.f : l > 0.f ? 1.f / l : 0.f;
    f0 *= inv;
    f1 *= inv;
    const int64_t own = static_cast<int64_t>(head) * a.os.head + static_cast<int64_t>(node) * a.os.token;
    // this stream's columns, staged in shared memory in 16-byte chunks (Q is not read any more)
    const int cols = share ? D : D / 2, col0 = share ? 0 : h * (D / 2);
    const int chunks = cols / 8, flip = min(chunks - 1, 7);
    uint8_t* stage = sq + h * C::kTile + quarter * (part ? 4096 : 32 * chunks * 16);
    const int pitch = min(chunks, 8) * 16;
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
      if (part) {
        // 32 rows x 32 columns through shared memory, four whole rows per store
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(stage + lane * 128 + (((e >> 2) ^ (lane & 7)) << 4)) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        __syncwarp();
        const int row0 = (share ? h * kTileRows : 0) + quarter * 32, at = lane & 7;
        float* dst = a.part_o + (static_cast<int64_t>(t.u) * a.n * a.G + t.row0 + row0) * a.splits * D + t.split * D + col0 + c * 32 + at * 4;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const int rr = k + (lane >> 3);
          if (row0 + rr < t.rows)
            *reinterpret_cast<float4*>(dst + static_cast<int64_t>(rr) * a.splits * D) =
                *reinterpret_cast<const float4*>(stage + rr * 128 + ((at ^ (rr & 7)) << 4));
        }
      } else if (valid) {
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
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sq = base;                                  // two Q tiles
  uint8_t* sk = sq + 2 * C::kTile;
  uint8_t* sv = sk + kStages * C::kTile;
  uint8_t* raw = sv + kStages * C::kTile;              // the operand warps' own
  Bars& s = *reinterpret_cast<Bars*>(raw + 8 * C::kRaw);
  const int warp = uniform(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.kfull[i]), 4);
      mbar_init(smem_u32(&s.kempty[i]), 1);
      mbar_init(smem_u32(&s.vfull[i]), 4);
      mbar_init(smem_u32(&s.vempty[i]), 1);
      mbar_init(smem_u32(&s.efull[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&s.sfull[i][b]), 1);
        mbar_init(smem_u32(&s.pfull[i][b]), 4);
      }
      mbar_init(smem_u32(&s.odone[i]), 1);
      mbar_init(smem_u32(&s.qfull[i]), 4);
    }
    mbar_init(smem_u32(&s.done), 1);
    mbar_init(smem_u32(&s.sizes), 1);
    s.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s.tmem), kTmemCols);
    tmem_relinquish();
  }
  wait_for_previous_kernel();
  let_next_kernel_start();
  const Item t = make_item(a, blockIdx.x, s);
  bool bad = false;
  for (int i = threadIdx.x; i < t.nodes; i += kThreads) {
    const int p = a.parent[static_cast<int64_t>(t.b) * a.n + i];
    const bool fine = p >= -1 && p < i;
    s.parent[i] = static_cast<int16_t>(fine ? p : -1);
    bad |= !fine;
  }
  if (bad && a.unit_status) a.unit_status[t.u] = KVC_UNIT_BAD_INDEX;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (MODS && (a.mods.slopes || a.mods.window)) {
    for (int i = threadIdx.x; i < t.nodes; i += kThreads) {
      int n = 0;
      for (int p = s.parent[i]; p >= 0; p = s.parent[p]) ++n;
      s.depth[i] = static_cast<int16_t>(n);
    }
    __syncthreads();
  }
  const uint32_t tmem = uniform(s.tmem);
  if (t.rows == 0) {                                   // rows past the tree's nodes
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  const bool share = t.rows > kTileRows;               // two Q tiles, or two streams over one
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    // (a.stall_unit: a test makes the MMA warp wait for key tiles that never come)
    if (warp == kMmaWarp) issue<D>(t, s, sq, sk, sv, tmem, share, t.u == a.stall_unit);
  } else if (warp >= kKeyWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const bool v = warp >= kValueWarp;
    make_operands<D, ROW, MODS>(a, t, s, v ? sv : sk, raw + (warp - kKeyWarp) * C::kRaw, v);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    softmax<D, ROW, MODS>(a, t, s, sq, tmem, share);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the splits of every row (PASK Eq. 15): W warps a row, each every W-th split, eight splits' outputs on their way
// together and with the statistics.  One warp a row up to eight splits, else four.
constexpr int kMergeThreads = 256;

template <int D, int W>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeArgs a) {
  using Vec = typename std::conditional<D == 128, float4, float2>::type;
  constexpr int kRows = kMergeThreads / 32 / W;
  __shared__ float part[W > 1 ? kMergeThreads / 32 : 1][D];
  __shared__ float2 part_ml[kMergeThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, own = warp % W;
  const uint32_t R = a.n * a.G, at = blockIdx.x * kRows + warp / W;
  const bool there = at < a.U * R;                 // (the last block may have fewer rows)
  uint32_t r, g, l, in_group;
  const uint32_t u = a.by_rows.divmod(there ? at : 0, &r);
  const uint32_t b = a.by_layers.divmod(a.by_heads.divmod(u, &g), &l), node = a.by_group.divmod(r, &in_group);
  const int64_t row = static_cast<int64_t>(u) * R + r;
  const float2* ml = a.part_ml + row * a.splits;
  const float* src = a.part_o + row * a.splits * D + lane * (D / 32);
  wait_for_previous_kernel();
  let_next_kernel_start();
  const bool live = there && (!a.n_nodes || static_cast<int>(node) < clamp_count(a.n_nodes[b], a.n));
  float x[D / 32] = {}, top = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int i0 = live ? own : a.splits; i0 < a.splits; i0 += 8 * W) {
    Vec o[8] = {};
    float2 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + W * k;
      v[k] = make_float2(-INFINITY, 0.f);
      if (i < a.splits) {
        o[k] = *reinterpret_cast<const Vec*>(src + static_cast<int64_t>(i) * D);
        v[k] = ml[i];
      }
    }
    float most = top;
#pragma unroll
    for (int k = 0; k < 8; ++k) most = fmaxf(most, v[k].x);
    const float f = top == -INFINITY ? 0.f : ex2_approx(top - most);
    top = most;
    sum *= f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) x[c] *= f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = v[k].x == -INFINITY ? 0.f : ex2_approx(v[k].x - top);
      sum = fmaf(v[k].y, w, sum);
      const float* e = reinterpret_cast<const float*>(&o[k]);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) x[c] = fmaf(e[c], w, x[c]);
    }
  }
  if (W > 1) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) part[warp][lane * (D / 32) + c] = x[c];
    if (lane == 0) part_ml[warp] = make_float2(top, sum);
    __syncthreads();
    if (own != 0) return;
    float2 v[W];
    top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      v[k] = part_ml[warp + k];
      top = fmaxf(top, v[k].x);
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) x[c] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float w = v[k].x == -INFINITY ? 0.f : ex2_approx(v[k].x - top);
      sum = fmaf(v[k].y, w, sum);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) x[c] = fmaf(part[warp + k][lane * (D / 32) + c], w, x[c]);
    }
  }
  if (!live) return;
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const int64_t head = g * a.G + in_group;
  __nv_bfloat16* out = a.out + b * a.os.batch + l * a.os.layer + head * a.os.head + node * a.os.token + lane * (D / 32);
#pragma unroll
  for (int c = 0; c < D / 32; c += 2) *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(x[c] * inv, x[c + 1] * inv);
  if (lane == 0 && a.lse)
    a.lse[((static_cast<int64_t>(b) * a.L + l) * (a.Hkv * a.G) + head) * a.n + node] = row_statistic(top, sum);
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
  cudaError_t e;
  if (a.few) {
    I4AttnArgs f = {};
    f.U = a.U, f.L = a.L, f.Hkv = a.Hkv, f.B = a.B, f.G = a.G, f.d = a.d, f.n_q = a.n;
    f.scale = a.scale;
    f.rows = a.rows;
    f.qs = a.qs, f.os = a.os;
    f.q = a.q;
    f.mods = a.mods;
    f.out = a.out;
    f.lse = a.lse;
    f.splits = a.splits;
    f.part_o = a.part_o;
    f.part_ml = a.part_ml;
    f.tree = {a.parent, a.n_nodes, a.k_new, a.v_new, a.news, a.unit_status};
    e = launch_i4_tree(f, stream);
  } else {
    e = a.d == 128 ? go_row(std::integral_constant<int, 128>{}) : go_row(std::integral_constant<int, 64>{});
  }
  if (e != cudaSuccess || a.splits == 1) return e;
  const int64_t rows = static_cast<int64_t>(a.U) * a.n * a.G;
  auto join = [&](auto kernel, int per_block) {
    return launch_after(kernel, dim3(static_cast<unsigned>((rows + per_block - 1) / per_block)), kMergeThreads, 0, stream, a);
  };
  if (a.splits <= 8) return a.d == 128 ? join(tree_merge_kernel<128, 1>, 8) : join(tree_merge_kernel<64, 1>, 8);
  return a.d == 128 ? join(tree_merge_kernel<128, 4>, 2) : join(tree_merge_kernel<64, 4>, 2);
}

}  // namespace kvc
