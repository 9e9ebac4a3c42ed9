// The growing 4-bit cache: append (quantise), read (dequantise) and eviction
// in place.  The stored row is that of the compaction's int4 pool (PASK App.
// B.5): symmetric codes -7..7, element 2j in the low nibble, a bf16 scale
// per 32 elements or an fp16 scale per row.
//
// append and read move each byte once (bound by HBM, and by the launch for
// the rows of a single token): a row takes d / 8 lanes, each with one 16-byte
// piece of bf16 on the one side and four bytes of codes on the other, so a
// warp's accesses are whole rows on both sides.  Four rows of a thread are in
// flight together.  Measured (d = 128, g32 scales, 96 units of up to 30,011
// rows): append 235 us and read 192 us, 428 us together = 6.1 TB/s, 91 % of the
// measured bandwidth, the quantiser's instructions (59 % of the ALU cycles)
// under the copies; one token's rows of 288 units appended and read back 5.8 us.
#include <algorithm>

#include "i4_codes.cuh"
#include "kvc_internal.cuh"
#include "packed_math.cuh"

namespace kvc {

namespace {

constexpr int kRowThreads = 256;
constexpr int kBatch = 4;                        // rows of a thread whose loads are in flight together

// The first free slot and number of new rows of unit u; n = 0 with `status`
// set if they cannot be appended.
struct Room {
  int slot, n, status;
};

__device__ __forceinline__ Room room_of(const I4AppendArgs& a, int u) {
  const int b = u / (a.L * a.Hkv);
  Room r;
  r.slot = a.rows.count[u];
  r.n = a.n_new ? clamp_count(a.n_new[b], a.n) : a.n;
  r.status = KVC_UNIT_OK;
  if (r.slot < 0 || r.slot > a.rows.capacity) r.status = KVC_UNIT_BAD_INDEX;
  else if (r.n > a.rows.capacity - r.slot) r.status = KVC_UNIT_FULL;
  if (r.status != KVC_UNIT_OK) r.n = 0;
  return r;
}

__device__ __forceinline__ void advance(const I4AppendArgs& a, int u, const Room& r) {
  if (r.status != KVC_UNIT_OK) {
    if (a.unit_status) a.unit_status[u] = r.status;
  } else if (r.n > 0) {
    a.rows.count[u] = r.slot + r.n;
    a.rows.next_pos[u] += r.n;
  }
}

// Row block blockIdx.x of unit blockIdx.y (+ 65535 blockIdx.z).  A unit of
// one block advances its own counters; those of several blocks are advanced
// by the next kernel, after every block has read them.
template <int D, bool ROW, int THREADS>
__global__ void __launch_bounds__(THREADS) i4_append_kernel(const I4AppendArgs a) {
  wait_for_previous_kernel();
  constexpr int LPR = D / 8, RPB = THREADS / LPR, NS = ROW ? 1 : D / 32;
  const int u = blockIdx.y + blockIdx.z * 65535;
  if (u >= a.U) return;
  const Room r = room_of(a, u);
  const int h = u % a.Hkv, l = u / a.Hkv % a.L, b = u / (a.Hkv * a.L);
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int i_end = min(r.n, static_cast<int>((blockIdx.x + 1) * a.rows_per_block));
  const int first = blockIdx.x * a.rows_per_block;
  const int64_t src = b * a.st.batch + l * a.st.layer + h * a.st.head + (first + sub) * a.st.token + lane * 8;
  const int64_t step = RPB * a.st.token;
  const uint16_t* ks = reinterpret_cast<const uint16_t*>(a.k) + src;
  const uint16_t* vs = reinterpret_cast<const uint16_t*>(a.v) + src;
  const int64_t row = static_cast<int64_t>(u) * a.rows.capacity + r.slot + first + sub;
  uint32_t* codes[2] = {static_cast<uint32_t*>(a.rows.k) + row * LPR + lane, static_cast<uint32_t*>(a.rows.v) + row * LPR + lane};
  const bool has_scale = ROW ? lane == 0 : (lane & 3) == 0;
  uint16_t* scales[2] = {static_cast<uint16_t*>(a.rows.k_scale) + row * NS + (ROW ? 0 : lane / 4),
                         static_cast<uint16_t*>(a.rows.v_scale) + row * NS + (ROW ? 0 : lane / 4)};
  int32_t* pos = a.rows.pos + row;
  float* mass = a.rows.mass + row;
  int32_t p = a.rows.next_pos[u] + first + sub;
#pragma unroll 1
  for (int left = i_end - first; left > 0; left -= RPB * kBatch) {       // rows of the block still to do
    uint4 w[kBatch][2] = {};
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (k * RPB + sub < left) {
        w[k][0] = __ldcs(reinterpret_cast<const uint4*>(ks + k * step));
        w[k][1] = __ldcs(reinterpret_cast<const uint4*>(vs + k * step));
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k * RPB >= left) break;                  // for the whole block
      const bool ok = k * RPB + sub < left;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        uint16_t bits;
        const uint32_t pk = quantise8<ROW, ROW ? LPR : 4>(w[k][v], &bits);
        if (ok) {
          codes[v][k * RPB * LPR] = pk;
          if (has_scale) scales[v][k * RPB * NS] = bits;
        }
      }
      if (ok && lane == 0) {
        pos[k * RPB] = p + k * RPB;
        if (a.rows.mass) mass[k * RPB] = 0.f;
      }
    }
    ks += kBatch * step;
    vs += kBatch * step;
    pos += kBatch * RPB;
    mass += kBatch * RPB;
    p += kBatch * RPB;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      codes[v] += kBatch * RPB * LPR;
      scales[v] += kBatch * RPB * NS;
    }
  }
  if (gridDim.x == 1) {
    __syncthreads();
    if (threadIdx.x == 0) advance(a, u, r);
  }
}

__global__ void i4_advance_kernel(const I4AppendArgs a) {
  wait_for_previous_kernel();
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u < a.U) advance(a, u, room_of(a, u));
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) i4_read_kernel(const I4ReadArgs a) {
  wait_for_previous_kernel();
  constexpr int LPR = D / 8, RPB = kRowThreads / LPR;
  const int u = blockIdx.y + blockIdx.z * 65535;
  if (u >= a.U) return;
  const int n = min(clamp_count(a.rows.count[u], a.rows.capacity), a.n);
  const int h = u % a.Hkv, l = u / a.Hkv % a.L, b = u / (a.Hkv * a.L);
  const int64_t dst0 = b * a.st.batch + l * a.st.layer + h * a.st.head;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const bool row_mode = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  const int i_end = min(n, static_cast<int>((blockIdx.x + 1) * a.rows_per_block));
  const int64_t row0 = static_cast<int64_t>(u) * a.rows.capacity;
  for (int i0 = blockIdx.x * a.rows_per_block + sub; i0 < i_end; i0 += RPB * kBatch) {
    uint32_t pk[kBatch][2];
    uint16_t sb[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int64_t row = row0 + min(i0 + k * RPB, i_end - 1);
        pk[k][v] = static_cast<const uint32_t*>(v ? a.rows.v : a.rows.k)[row * LPR + lane];
        sb[k][v] = static_cast<const uint16_t*>(v ? a.rows.v_scale : a.rows.k_scale)[row_mode ? row : row * (D / 32) + lane / 4];
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * RPB;
      if (i >= i_end) break;
#pragma unroll
      for (int v = 0; v < 2; ++v)
        __stcs(reinterpret_cast<uint4*>((v ? a.v : a.k) + dst0 + static_cast<int64_t>(i) * a.st.token + lane * 8),
               dequantise8(pk[k][v], sb[k][v], row_mode));
    }
  }
}

// ----------------------------------------------------------------------------
// Eviction.  One block per unit.  A row that may leave has the 64-bit key
// (mass, -pos); the `over` rows of smallest key leave.
//   * over = 1 (a token in, a row out): one reduction finds the row, and the
//     row in slot `budget` takes its place.
//   * else a radix select by 8-bit digits finds the `over`-th smallest key:
//     four passes over the mass, which stops as soon as a digit's rows leave
//     all together, and four over the positions where rows of equal mass have
//     to be told apart.  Then every 32 slots give a word of leaving rows, and
//     one prefix sum over the words lists the holes below the budget and the
//     remaining rows behind it; hole i takes row i.
// Bound by the latency of its few dependent steps for the caches it is meant
// for (thousands of rows per unit): 8 units of 2,049 rows 6.6 us, 288 units of
// 2,148 rows, 100 of which leave, 18 us; marks and lists in the workspace
// instead of shared memory took 26 us.
// ----------------------------------------------------------------------------
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kHeld = 8;                         // mass keys of a thread kept in registers
constexpr uint32_t kStays = 0xffffffffu;         // no key: above that of +inf

__device__ __forceinline__ uint32_t mass_key(float mass) {
  uint32_t b = __float_as_uint(mass);
  if (mass != mass) b = 0xff800000u;            // NaN: -inf
  if (b == 0x80000000u) b = 0u;                 // -0: +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t pos_key(int32_t pos) { return ~(static_cast<uint32_t>(pos) ^ 0x80000000u); }

// Exclusive prefix sum of v over the block, and the total.  A barrier has to
// separate two calls' use of `sums`; the call ends with one.
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int s = lane < kEvictWarps ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(kFull, s, 31);
  const int before = warp ? __shfl_sync(kFull, s, warp - 1) : 0;
  __syncthreads();
  return before + x - v;
}

constexpr int kEvictWords = 1024, kEvictMoves = 1024;        // kept in shared memory up to here, else in the workspace

struct EvictSmem {
  uint32_t words[kEvictWords];
  int lists[2][kEvictMoves];
  int hist[256];
  int sums[kEvictWarps];
  unsigned long long best[kEvictWarps];
  int slot[kEvictWarps];
  int bin, before, count;
};

// The digit of the `need`-th smallest among hist, and the number of keys
// below it (warp 0; hist holds at least `need`).
__device__ __forceinline__ void find_bin(EvictSmem& s, int need) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int h[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += h[k] = s.hist[lane * 8 + k];
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    int before = x - sum;
    if (before < need && need <= x) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (before < need && need <= before + h[k]) {
          s.bin = lane * 8 + k;
          s.before = before;
          s.count = h[k];
        }
        before += h[k];
      }
    }
    if (lane == 31 && x < need) s.bin = -1;
  }
}

// What one lane moves of a row: words of the codes, a scale, the position or
// the mass.
struct RowPart {
  uint32_t k, v;
};

__device__ __forceinline__ RowPart load_part(const I4EvictArgs& a, int64_t row) {
  const int lane = threadIdx.x & 31, words = a.d / 8;
  const int sb = a.rows.quant_mode == KVC_QUANT_ROW_FP16 ? 1 : a.d / 32;
  RowPart p = {0, 0};
  if (lane < words) {
    p.k = static_cast<const uint32_t*>(a.rows.k)[row * words + lane];
    p.v = static_cast<const uint32_t*>(a.rows.v)[row * words + lane];
  } else if (lane >= 16 && lane < 16 + sb) {
    p.k = static_cast<const uint16_t*>(a.rows.k_scale)[row * sb + lane - 16];
    p.v = static_cast<const uint16_t*>(a.rows.v_scale)[row * sb + lane - 16];
  } else if (lane == 31) {
    p.k = static_cast<uint32_t>(a.rows.pos[row]);
    p.v = __float_as_uint(a.rows.mass[row]);
  }
  return p;
}

__device__ __forceinline__ void store_part(const I4EvictArgs& a, int64_t row, const RowPart& p) {
  const int lane = threadIdx.x & 31, words = a.d / 8;
  const int sb = a.rows.quant_mode == KVC_QUANT_ROW_FP16 ? 1 : a.d / 32;
  if (lane < words) {
    static_cast<uint32_t*>(a.rows.k)[row * words + lane] = p.k;
    static_cast<uint32_t*>(a.rows.v)[row * words + lane] = p.v;
  } else if (lane >= 16 && lane < 16 + sb) {
    static_cast<uint16_t*>(a.rows.k_scale)[row * sb + lane - 16] = static_cast<uint16_t>(p.k);
    static_cast<uint16_t*>(a.rows.v_scale)[row * sb + lane - 16] = static_cast<uint16_t>(p.v);
  } else if (lane == 31) {
    a.rows.pos[row] = static_cast<int32_t>(p.k);
    a.rows.mass[row] = __uint_as_float(p.v);
  }
}

__global__ void __launch_bounds__(kEvictThreads, 2) i4_evict_kernel(const I4EvictArgs a) {
  wait_for_previous_kernel();
  __shared__ EvictSmem s;
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = a.rows.capacity;
  const int cnt = a.rows.count[u];
  const int64_t first_recent = static_cast<int64_t>(a.rows.next_pos[u]) - a.n_recent;
  if (cnt < 0 || cnt > cap) {
    if (tid == 0 && a.unit_status) a.unit_status[u] = KVC_UNIT_BAD_INDEX;
    return;
  }
  const int over = cnt - a.budget;
  if (over <= 0) return;
  const int64_t base = static_cast<int64_t>(u) * cap;
  const int32_t* pos = a.rows.pos + base;
  const float* mass = a.rows.mass + base;
  auto key_of = [&](int i) -> uint32_t {
    const int32_t p = pos[i];
    const float m = mass[i];
    return p >= a.n_sink && p < first_recent ? mass_key(m) : kStays;
  };

  if (over == 1) {
    unsigned long long best = ~0ull;
    int at = -1;
    for (int i = tid; i < cnt; i += kEvictThreads) {
      const int32_t p = pos[i];
      const float m = mass[i];
      if (!(p >= a.n_sink && p < first_recent)) continue;
      const unsigned long long key = static_cast<unsigned long long>(mass_key(m)) << 32 | pos_key(p);
      if (key < best || at < 0) best = key, at = i;          // ascending slots: the lower of equal keys stays first
    }
    auto merge = [&](unsigned long long k2, int a2) {
      if (a2 >= 0 && (at < 0 || k2 < best || (k2 == best && a2 < at))) best = k2, at = a2;
    };
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long k2 = __shfl_xor_sync(kFull, best, o);
      const int a2 = __shfl_xor_sync(kFull, at, o);
      merge(k2, a2);
    }
    if (lane == 0) s.best[warp] = best, s.slot[warp] = at;
    __syncthreads();
    if (warp) return;
    best = ~0ull, at = -1;
    if (lane < kEvictWarps) best = s.best[lane], at = s.slot[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const unsigned long long k2 = __shfl_xor_sync(kFull, best, o);
      const int a2 = __shfl_xor_sync(kFull, at, o);
      merge(k2, a2);
    }
    if (at < 0) {
      if (lane == 0 && a.unit_status) a.unit_status[u] = KVC_UNIT_OVER_BUDGET;
      return;
    }
    if (at < a.budget) store_part(a, base + at, load_part(a, base + a.budget));
    if (lane == 0) a.rows.count[u] = a.budget;
    return;
  }

  const bool held = cnt <= kEvictThreads * kHeld;
  uint32_t key[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) key[k] = held && k * kEvictThreads + tid < cnt ? key_of(k * kEvictThreads + tid) : kStays;

  // the threshold: rows whose key's top bits are below thr leave, and `need` of those that equal it
  uint32_t thr = 0, thr_pos = 0;
  int need = over, shift = 32, shift_pos = 32;
  bool whole = false;
#pragma unroll 1
  while (shift > 0 && !whole) {
    shift -= 8;
    if (tid < 256) s.hist[tid] = 0;
    __syncthreads();
    auto count = [&](uint32_t x) {
      if (x != kStays && (shift == 24 || x >> (shift + 8) == thr)) atomicAdd(&s.hist[(x >> shift) & 255], 1);
    };
    if (held) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) count(key[k]);
    } else {
#pragma unroll 4
      for (int i = tid; i < cnt; i += kEvictThreads) count(key_of(i));
    }
    __syncthreads();
    find_bin(s, need);
    __syncthreads();
    if (s.bin < 0) {                    // only at the first digit: too few rows may leave
      if (tid == 0 && a.unit_status) a.unit_status[u] = KVC_UNIT_OVER_BUDGET;
      return;
    }
    thr = thr << 8 | static_cast<uint32_t>(s.bin);
    need -= s.before;
    whole = s.count == need;
    __syncthreads();
  }
  // equal mass: the later positions
#pragma unroll 1
  while (shift_pos > 0 && !whole) {
    shift_pos -= 8;
    if (tid < 256) s.hist[tid] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < cnt; i += kEvictThreads) {
      if (key_of(i) != thr) continue;
      const uint32_t x = pos_key(pos[i]);
      if (shift_pos == 24 || x >> (shift_pos + 8) == thr_pos) atomicAdd(&s.hist[(x >> shift_pos) & 255], 1);
    }
    __syncthreads();
    find_bin(s, need);
    __syncthreads();
    thr_pos = thr_pos << 8 | static_cast<uint32_t>(s.bin);
    need -= s.before;
    whole = s.count == need;
    __syncthreads();
  }
  const bool by_pos = shift_pos < 32;
  auto below = [&](uint32_t x, int i) { return x != kStays && ((x >> shift) < thr || (by_pos && x == thr && (pos_key(pos[i]) >> shift_pos) < thr_pos)); };
  auto equal = [&](uint32_t x, int i) { return x != kStays && (x >> shift) == thr && (!by_pos || (pos_key(pos[i]) >> shift_pos) == thr_pos); };

  // a word of leaving rows per 32 slots; rows of one key and position leave in slot order
  const int words = (cnt + 31) / 32;
  uint32_t* leaves = words <= kEvictWords ? s.words : a.words + static_cast<int64_t>(u) * a.n_words;
  const bool own_lists = over <= kEvictMoves;      // no list is longer than the rows that leave
  int32_t* holes = own_lists ? s.lists[0] : a.lists + static_cast<int64_t>(u) * 2 * a.max_moves;
  int32_t* donors = own_lists ? s.lists[1] : holes + a.max_moves;
  int n_eq = 0;
  auto mark = [&](int i0, uint32_t x) {
    const int i = i0 + tid;
    bool gone = i < cnt && below(x, i);
    const bool eq = i < cnt && equal(x, i);
    if (whole) {
      gone |= eq;
    } else {
      int total;
      const int rank = n_eq + block_scan(eq, s.sums, &total);
      n_eq += total;
      gone |= eq && rank < need;
    }
    const uint32_t word = __ballot_sync(kFull, gone);
    if (lane == 0 && i < cnt) leaves[i >> 5] = word;
  };
  if (held) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (k * kEvictThreads < cnt) mark(k * kEvictThreads, key[k]);
  } else {
#pragma unroll 1
    for (int i0 = 0; i0 < cnt; i0 += kEvictThreads) mark(i0, i0 + tid < cnt ? key_of(i0 + tid) : kStays);
  }
  __syncthreads();
  int n_holes = 0, n_donors = 0;
#pragma unroll 1
  for (int w0 = 0; w0 < words; w0 += kEvictThreads) {
    const int w = w0 + tid, i0 = w * 32;
    uint32_t h = 0, d = 0;
    if (w < words) {
      const uint32_t gone = leaves[w];
      const int used = min(32, cnt - i0);
      const uint32_t in_use = used == 32 ? ~0u : (1u << used) - 1;
      const int below_budget = max(0, min(32, a.budget - i0));
      const uint32_t front = below_budget == 32 ? ~0u : (1u << below_budget) - 1;
      h = gone & front;
      d = ~gone & in_use & ~front;
    }
    int total;
    int at = n_holes + block_scan(__popc(h), s.sums, &total);
    n_holes += total;
    for (; h; h &= h - 1) holes[at++] = i0 + __ffs(h) - 1;
    at = n_donors + block_scan(__popc(d), s.sums, &total);
    n_donors += total;
    for (; d; d &= d - 1) donors[at++] = i0 + __ffs(d) - 1;
  }
  __syncthreads();
  // four rows of a warp on their way together
  for (int m0 = warp; m0 < n_holes; m0 += kEvictWarps * 4) {
    RowPart p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = load_part(a, base + donors[min(m0 + k * kEvictWarps, n_holes - 1)]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (m0 + k * kEvictWarps < n_holes) store_part(a, base + holes[m0 + k * kEvictWarps], p[k]);
  }
  if (tid == 0) a.rows.count[u] = a.budget;
}

}  // namespace

namespace {

template <int D, bool ROW>
cudaError_t append(const I4AppendArgs& a, dim3 grid, bool wide, cudaStream_t stream) {
  return wide ? launch_after(i4_append_kernel<D, ROW, 512>, grid, 512, 0, stream, a)
              : launch_after(i4_append_kernel<D, ROW, 256>, grid, 256, 0, stream, a);
}

}  // namespace

cudaError_t launch_i4_append(const I4AppendArgs& a0, cudaStream_t stream) {
  I4AppendArgs a = a0;
  // up to 256 rows of a unit in one block, which advances the counters itself
  // (one launch), 512 threads from 64 rows on; longer ones in blocks of 128
  // rows and a second launch.  Measured (288 units, with the read): 200 rows
  // 17.4 us, 19.0 with 256 threads, 20.1 in blocks of 128; one row 5.8 us, 6.9
  // with 512 threads.
  a.rows_per_block = a.n <= 256 ? 256 : 128;
  const bool wide = a.n > 64 && a.n <= 256, row = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  const dim3 grid((a.n + a.rows_per_block - 1) / a.rows_per_block, std::min(a.U, 65535), (a.U + 65534) / 65535);
  const cudaError_t e = a.d == 128 ? (row ? append<128, true>(a, grid, wide, stream) : append<128, false>(a, grid, wide, stream))
                                   : (row ? append<64, true>(a, grid, wide, stream) : append<64, false>(a, grid, wide, stream));
  if (e != cudaSuccess || grid.x == 1) return e;
  return launch_after(i4_advance_kernel, dim3((a.U + 255) / 256), 256, 0, stream, a);
}

cudaError_t launch_i4_read(const I4ReadArgs& a0, cudaStream_t stream) {
  I4ReadArgs a = a0;
  // one batch of rows per thread: blocks of 64 rows (128 at d = 64)
  a.rows_per_block = kRowThreads / (a.d / 8) * kBatch;
  const dim3 grid((a.n + a.rows_per_block - 1) / a.rows_per_block, std::min(a.U, 65535), (a.U + 65534) / 65535);
  return launch_after(a.d == 128 ? i4_read_kernel<128> : i4_read_kernel<64>, grid, kRowThreads, 0, stream, a);
}

cudaError_t launch_i4_evict(const I4EvictArgs& a, cudaStream_t stream) {
  return launch_after(i4_evict_kernel, dim3(a.U), kEvictThreads, 0, stream, a);
}

}  // namespace kvc
