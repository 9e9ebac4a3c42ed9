// The growing 4-bit cache: append (quantise), read (dequantise) and eviction
// in place.  The stored row is that of the compaction's int4 pool (PASK App.
// B.5): symmetric codes -7..7, element 2j in the low nibble, a bf16 scale
// per 32 elements or an fp16 scale per row.
//
// append and read move each byte once (bound by HBM, and by the launch for
// the rows of a single token): a row takes d / 8 lanes, each with one 16-byte
// piece of bf16 on the one side and four bytes of codes on the other, so a
// warp's accesses are whole rows on both sides.
#include <algorithm>

#include "kvc_internal.cuh"

namespace kvc {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRowThreads = 256;

__device__ __forceinline__ float scale_of(uint16_t bits, bool row_mode) {
  return row_mode ? __half2float(__ushort_as_half(bits)) : bf16_bits_to_float(bits);
}

// Quantises the 8 elements of this lane (lanes_per_group adjacent lanes share
// a scale): packed codes, and the scale's bits.
__device__ __forceinline__ uint32_t quantise8(const uint4& w, bool row_mode, int lanes_per_group, uint16_t* bits) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
  float x[8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r[i] << 16);
    x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    amax = fmaxf(amax, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
  }
  for (int o = 1; o < lanes_per_group; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
  float sc = 1.f;
  if (amax > 0.f) {
    const float s = __fdiv_rn(amax, 7.f);
    if (row_mode) sc = fmaxf(fminf(__half2float(__float2half_rn(s)), 65504.f), 0x1p-24f);
    else sc = fmaxf(bf16_bits_to_float(float_to_bf16_bits(s)), __uint_as_float(0x00010000u));   // 2^-133
  }
  *bits = row_mode ? __half_as_ushort(__float2half_rn(sc)) : float_to_bf16_bits(sc);
  const bool fast = recip_div_ok(sc);
  const float y = __fdiv_rn(1.f, sc);
  uint32_t pk = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int q = __float2int_rn(fast ? div_by_recip(x[i], sc, y) : __fdiv_rn(x[i], sc));
    q = max(-7, min(7, amax > 0.f ? q : 0));
    pk |= static_cast<uint32_t>(q & 0xf) << (4 * i);
  }
  return pk;
}

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
template <int D>
__global__ void __launch_bounds__(kRowThreads) i4_append_kernel(const I4AppendArgs a) {
  constexpr int LPR = D / 8, RPB = kRowThreads / LPR;
  const int u = blockIdx.y + blockIdx.z * 65535;
  if (u >= a.U) return;
  const Room r = room_of(a, u);
  const int32_t p0 = a.rows.next_pos[u];
  const int h = u % a.Hkv, l = u / a.Hkv % a.L, b = u / (a.Hkv * a.L);
  const int64_t src0 = b * a.st.batch + l * a.st.layer + h * a.st.head;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const bool row_mode = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  const int i_end = (min(r.n, static_cast<int>((blockIdx.x + 1) * a.rows_per_block)) + RPB - 1) / RPB * RPB;
  for (int i = blockIdx.x * a.rows_per_block + sub; i < i_end; i += RPB) {
    const bool ok = i < r.n;
    const int64_t src = src0 + static_cast<int64_t>(ok ? i : 0) * a.st.token + lane * 8;
    const int64_t row = static_cast<int64_t>(u) * a.rows.capacity + r.slot + i;
    uint4 w[2] = {};
    if (ok) {
      w[0] = __ldg(reinterpret_cast<const uint4*>(a.k + src));
      w[1] = __ldg(reinterpret_cast<const uint4*>(a.v + src));
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint16_t bits;
      const uint32_t pk = quantise8(w[v], row_mode, row_mode ? LPR : 4, &bits);
      if (ok) {
        static_cast<uint32_t*>(v ? a.rows.v : a.rows.k)[row * LPR + lane] = pk;
        uint16_t* sp = static_cast<uint16_t*>(v ? a.rows.v_scale : a.rows.k_scale);
        if (row_mode) {
          if (lane == 0) sp[row] = bits;
        } else if ((lane & 3) == 0) {
          sp[row * (D / 32) + lane / 4] = bits;
        }
      }
    }
    if (ok && lane == 0) {
      a.rows.pos[row] = p0 + i;
      if (a.rows.mass) a.rows.mass[row] = 0.f;
    }
  }
  if (gridDim.x == 1) {
    __syncthreads();
    if (threadIdx.x == 0) advance(a, u, r);
  }
}

__global__ void i4_advance_kernel(const I4AppendArgs a) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u < a.U) advance(a, u, room_of(a, u));
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) i4_read_kernel(const I4ReadArgs a) {
  constexpr int LPR = D / 8, RPB = kRowThreads / LPR;
  const int u = blockIdx.y + blockIdx.z * 65535;
  if (u >= a.U) return;
  const int n = min(clamp_count(a.rows.count[u], a.rows.capacity), a.n);
  const int h = u % a.Hkv, l = u / a.Hkv % a.L, b = u / (a.Hkv * a.L);
  const int64_t dst0 = b * a.st.batch + l * a.st.layer + h * a.st.head;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const bool row_mode = a.rows.quant_mode == KVC_QUANT_ROW_FP16;
  const int i_end = min(n, static_cast<int>((blockIdx.x + 1) * a.rows_per_block));
  for (int i = blockIdx.x * a.rows_per_block + sub; i < i_end; i += RPB) {
    const int64_t row = static_cast<int64_t>(u) * a.rows.capacity + i;
    const int64_t dst = dst0 + static_cast<int64_t>(i) * a.st.token + lane * 8;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint32_t pk = __ldg(static_cast<const uint32_t*>(v ? a.rows.v : a.rows.k) + row * LPR + lane);
      const uint16_t* sp = static_cast<const uint16_t*>(v ? a.rows.v_scale : a.rows.k_scale);
      const float sc = scale_of(__ldg(sp + (row_mode ? row : row * (D / 32) + lane / 4)), row_mode);
      uint32_t o[4];
#pragma unroll
      for (int i2 = 0; i2 < 4; ++i2) {
        const float lo = static_cast<float>(static_cast<int32_t>(pk << (28 - 8 * i2)) >> 28) * sc;
        const float hi = static_cast<float>(static_cast<int32_t>(pk << (24 - 8 * i2)) >> 28) * sc;
        o[i2] = float_to_bf16_bits(lo) | static_cast<uint32_t>(float_to_bf16_bits(hi)) << 16;
      }
      *reinterpret_cast<uint4*>((v ? a.v : a.k) + dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// ----------------------------------------------------------------------------
// Eviction.  One block per unit.  The key of a row that may leave is (mass,
// -pos) as one 64-bit number, so the rows that leave are the `over` smallest:
// a radix select by 8-bit digits finds the `over`-th, and one ordered pass
// over the slots lists the holes below the budget and the remaining rows
// behind it.  Both lists have the same length; hole i takes row i.
// ----------------------------------------------------------------------------
constexpr int kEvictThreads = 1024;

__device__ __forceinline__ uint64_t evict_key(float mass, int32_t pos) {
  uint32_t b = __float_as_uint(mass);
  if (mass != mass) b = 0xff800000u;            // NaN: -inf
  if (b == 0x80000000u) b = 0u;                 // -0: +0
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return static_cast<uint64_t>(b) << 32 | ~(static_cast<uint32_t>(pos) ^ 0x80000000u);
}

// Exclusive prefix sum of v over the block, and the total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[32 + lane] = s;
  }
  __syncthreads();
  *total = warp_sums[63];
  const int before = x - v + (warp ? warp_sums[32 + warp - 1] : 0);
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kEvictThreads) i4_evict_kernel(const I4EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int warp_sums[64];
  __shared__ int s_bin, s_before, s_free;
  const int u = blockIdx.x, tid = threadIdx.x;
  const int cap = a.rows.capacity;
  const int cnt = a.rows.count[u];
  if (cnt < 0 || cnt > cap) {
    if (tid == 0 && a.unit_status) a.unit_status[u] = KVC_UNIT_BAD_INDEX;
    return;
  }
  const int over = cnt - a.budget;
  if (over <= 0) return;
  const int64_t base = static_cast<int64_t>(u) * cap;
  int32_t* pos = a.rows.pos + base;
  float* mass = a.rows.mass + base;
  const int64_t first_recent = static_cast<int64_t>(a.rows.next_pos[u]) - a.n_recent;
  auto may_leave = [&](int32_t p) { return p >= a.n_sink && p < first_recent; };

  uint64_t prefix = 0;
  int need = over;                     // rank of the threshold key among those that match the prefix
  int shift = 56;
#pragma unroll 1
  for (; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kEvictThreads) hist[i] = 0;
    if (tid == 0) s_free = 0;
    __syncthreads();
    int mine = 0;
    for (int i = tid; i < cnt; i += kEvictThreads) {
      const int32_t p = pos[i];
      if (!may_leave(p)) continue;
      const uint64_t key = evict_key(mass[i], p);
      if (shift < 56 && (key >> (shift + 8)) != (prefix >> (shift + 8))) continue;
      atomicAdd(&hist[(key >> shift) & 255], 1);
      ++mine;
    }
    if (mine) atomicAdd(&s_free, mine);
    __syncthreads();
    if (s_free < need) {               // only at the first digit: too few rows may leave
      if (tid == 0 && a.unit_status) a.unit_status[u] = KVC_UNIT_OVER_BUDGET;
      return;
    }
    if (tid == 0) {
      int before = 0, bin = 0;
      while (before + hist[bin] < need) before += hist[bin++];
      s_bin = bin;
      s_before = before;
    }
    __syncthreads();
    prefix |= static_cast<uint64_t>(s_bin) << shift;
    need -= s_before;
    const bool whole = hist[s_bin] == need;
    __syncthreads();
    if (whole) break;
  }
  // rows with key >> shift below the threshold's leave, and the first `need` that equal it
  if (shift < 0) shift = 0;
  const uint64_t thr = prefix >> shift;
  int32_t* holes = a.lists + static_cast<int64_t>(u) * 2 * a.max_moves;
  int32_t* donors = holes + a.max_moves;
  int n_eq = 0, n_holes = 0, n_donors = 0;
  for (int i0 = 0; i0 < cnt; i0 += kEvictThreads) {
    const int i = i0 + tid;
    bool less = false, eq = false;
    if (i < cnt) {
      const int32_t p = pos[i];
      if (may_leave(p)) {
        const uint64_t key = evict_key(mass[i], p) >> shift;
        less = key < thr;
        eq = key == thr;
      }
    }
    int total;
    const int rank = n_eq + block_scan(eq, warp_sums, &total);
    n_eq += total;
    const bool leaves = less || (eq && rank < need);
    const bool hole = leaves && i < a.budget, donor = i < cnt && !leaves && i >= a.budget;
    const int at_h = n_holes + block_scan(hole, warp_sums, &total);
    n_holes += total;
    if (hole) holes[at_h] = i;
    const int at_d = n_donors + block_scan(donor, warp_sums, &total);
    n_donors += total;
    if (donor) donors[at_d] = i;
  }
  __syncthreads();
  const int half = a.d / 2, lane = tid & 31;
  const int sb = a.rows.quant_mode == KVC_QUANT_ROW_FP16 ? 1 : a.d / 32;
  for (int m = tid >> 5; m < n_holes; m += kEvictThreads / 32) {
    const int64_t to = base + holes[m], from = base + donors[m];
    const uint32_t* ks = static_cast<const uint32_t*>(a.rows.k) + from * (half / 4);
    const uint32_t* vs = static_cast<const uint32_t*>(a.rows.v) + from * (half / 4);
    if (lane < half / 4) {
      static_cast<uint32_t*>(a.rows.k)[to * (half / 4) + lane] = ks[lane];
      static_cast<uint32_t*>(a.rows.v)[to * (half / 4) + lane] = vs[lane];
    } else if (lane >= 16 && lane < 16 + sb) {
      const int g = lane - 16;
      static_cast<uint16_t*>(a.rows.k_scale)[to * sb + g] = static_cast<const uint16_t*>(a.rows.k_scale)[from * sb + g];
      static_cast<uint16_t*>(a.rows.v_scale)[to * sb + g] = static_cast<const uint16_t*>(a.rows.v_scale)[from * sb + g];
    } else if (lane == 30) {
      a.rows.pos[to] = a.rows.pos[from];
    } else if (lane == 31) {
      a.rows.mass[to] = a.rows.mass[from];
    }
  }
  if (tid == 0) a.rows.count[u] = a.budget;
}

}  // namespace

cudaError_t launch_i4_append(const I4AppendArgs& a0, cudaStream_t stream) {
  I4AppendArgs a = a0;
  // up to 256 rows per block: enough blocks to fill the device from a few
  // thousand rows on, and the rows of a short append in one launch
  a.rows_per_block = 256;
  const dim3 grid((a.n + a.rows_per_block - 1) / a.rows_per_block, std::min(a.U, 65535), (a.U + 65534) / 65535);
  if (a.d == 128) i4_append_kernel<128><<<grid, kRowThreads, 0, stream>>>(a);
  else i4_append_kernel<64><<<grid, kRowThreads, 0, stream>>>(a);
  if (grid.x > 1) i4_advance_kernel<<<(a.U + 255) / 256, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_i4_read(const I4ReadArgs& a0, cudaStream_t stream) {
  I4ReadArgs a = a0;
  a.rows_per_block = 256;
  const dim3 grid((a.n + a.rows_per_block - 1) / a.rows_per_block, std::min(a.U, 65535), (a.U + 65534) / 65535);
  if (a.d == 128) i4_read_kernel<128><<<grid, kRowThreads, 0, stream>>>(a);
  else i4_read_kernel<64><<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_i4_evict(const I4EvictArgs& a, cudaStream_t stream) {
  i4_evict_kernel<<<a.U, kEvictThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kvc
