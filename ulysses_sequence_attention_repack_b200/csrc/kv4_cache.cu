// Kernels that fill, read back and compact the 4-bit K/V cache (kv4.cuh).
//
// All three move bytes: per (token, head) the append reads 512 bytes of bf16
// and writes 144 + 8, the load reads 144 and writes 512, and the eviction
// reads the 4-byte weight of every cached slot and moves 152 bytes of those it
// keeps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bounds.cuh"
#include "internal.h"
#include "kv4.cuh"

namespace ulysses {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 8;   // consecutive tokens of one head a warp has in flight

__device__ __forceinline__ int4 ld_stream(const int4* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The sequence of packed row i: the last b with cu[b] <= i, or -1 when i lies
// behind the last sequence (or before the first).  cu is read inside
// [0, batch] only, whatever it holds.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int64_t i) {
  if (i < cu[0] || i >= cu[batch]) return -1;
  int lo = 0, hi = batch;   // cu[lo] <= i < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Where rows i0 .. i0 + 7 live: lane u < 8 holds the pair (sequence, slot) of
// row i0 + u, slot -1 for a row of no sequence or a slot outside the cache.
struct RowPlace {
  int b;
  int64_t slot;
};

__device__ __forceinline__ RowPlace place_row(const Kv4Rows& r, int64_t i, int batch, int64_t capacity,
                                              unsigned int* err) {
  RowPlace p{0, -1};
  if (i >= r.rows) return p;
  const int b = find_sequence(r.cu, batch, i);
  if (b < 0) return p;
  p.b = b;
  p.slot = static_cast<int64_t>(r.start[b]) + (i - r.cu[b]);
  if (p.slot < 0 || p.slot >= capacity) {
    if (err) atomicOr(err, kErrCacheIndex);
    p.slot = -1;
  }
  return p;
}

__device__ __forceinline__ int64_t row_offset(const Kv4Rows& r, int64_t i, int h) {
  const int rank = h / r.heads_per_rank;
  return i * r.token_stride + rank * r.rank_stride + (h - rank * r.heads_per_rank) * r.head_stride;
}

// Append: one warp takes 8 consecutive tokens of one head (neighbouring warps
// the neighbouring heads, whose rows are neighbours in memory).  Half a warp
// holds a row, 8 dims a lane: lanes 0-15 the K row, 16-31 the V row, so a
// group of 64 is 8 lanes and its minimum and maximum three shuffles.
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4RowsLaunch a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t groups = (a.r.rows + kTokens - 1) / kTokens;
  if (item >= groups * a.H) return;
  const int64_t i0 = item / a.H * kTokens;
  const int h = static_cast<int>(item - item / a.H * a.H);
  const RowPlace mine = lane < kTokens ? place_row(a.r, i0 + lane, a.B, a.cap, a.err) : RowPlace{0, -1};
  const int plane = lane >> 4, l16 = lane & 15;
  const uint16_t* src = static_cast<const uint16_t*>(plane ? a.r.v : a.r.k);

  int64_t slot[kTokens];
  int4 x[kTokens];
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    slot[u] = __shfl_sync(0xffffffffu, mine.slot, u);
    x[u] = make_int4(0, 0, 0, 0);
    if (slot[u] >= 0)
      x[u] = ld_stream(reinterpret_cast<const int4*>(src + row_offset(a.r, i0 + u, h) + l16 * 8));
  }
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    const int b = __shfl_sync(0xffffffffu, mine.b, u);
    const uint32_t w[4] = {static_cast<uint32_t>(x[u].x), static_cast<uint32_t>(x[u].y),
                           static_cast<uint32_t>(x[u].z), static_cast<uint32_t>(x[u].w)};
    float f[8];
    bool nan = false;
    float lo = __int_as_float(0x7f800000), hi = __int_as_float(0xff800000);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = bf16_lo(w[e]);
      f[2 * e + 1] = bf16_hi(w[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      nan |= f[e] != f[e];
      lo = fminf(lo, f[e]);
      hi = fmaxf(hi, f[e]);
    }
    if (nan) hi = lo = __int_as_float(0x7fc00000);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      const float ol = __shfl_xor_sync(0xffffffffu, lo, d), oh = __shfl_xor_sync(0xffffffffu, hi, d);
      // a NaN in any lane stays: fminf and fmaxf alone would drop it
      lo = (ol != ol || lo != lo) ? __int_as_float(0x7fc00000) : fminf(lo, ol);
      hi = (oh != oh || hi != hi) ? __int_as_float(0x7fc00000) : fmaxf(hi, oh);
    }
    // IEEE subtraction, division and rounding.  m and s have 8-bit mantissas
    // and the borders (n + 1/2) s at most 12, so a quotient that is not on a
    // border is further from it than the division's rounding.
    const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)));
    const bool finite = fabsf(s) <= 3.4e38f && fabsf(lo) <= 3.4e38f;
    uint32_t code = 0;
    if (finite && s > 0.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(f[e], lo), s)), 0.f), 15.f);
        code |= static_cast<uint32_t>(n) << (4 * e);
      }
    }
    const uint32_t sb = __float_as_uint(s) >> 16, mb = __float_as_uint(lo) >> 16;
    const uint32_t meta = finite ? (sb | (mb << 16)) : 0x7fc07fc0u;
    if (slot[u] < 0) continue;
    const int64_t bh = static_cast<int64_t>(b) * a.H + h;
    const int64_t blk = kv4_block_offset(bh, a.cap, slot[u]);
    const int at = static_cast<int>(slot[u] % kKv4BlockSlots);
    const int64_t c_off = blk + plane * kKv4VOffset + at * 64 + (l16 & 7) * 8 + (l16 >> 3) * 4;
    if (in_bounds(c_off, 4, a.blocks_bytes, a.err)) *reinterpret_cast<uint32_t*>(a.cache + c_off) = code;
    if ((lane & 7) == 0) {
      const int64_t m_off = blk + kKv4MetaOffset + at * 16 + (lane >> 3) * 4;
      if (in_bounds(m_off, 4, a.blocks_bytes, a.err)) *reinterpret_cast<uint32_t*>(a.cache + m_off) = meta;
    }
    if (lane == 1) a.weight[bh * a.cap + slot[u]] = 0.f;
    if (lane == 2)
      a.pos[bh * a.cap + slot[u]] =
          a.r.pos0 ? static_cast<int32_t>(a.r.pos0[b] + (slot[u] - a.r.start[b])) : static_cast<int32_t>(slot[u]);
  }
}

// Load: the same split; a lane turns one 32-bit word of codes into 8 bf16.
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const Kv4RowsLaunch a) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t groups = (a.r.rows + kTokens - 1) / kTokens;
  if (item >= groups * a.H) return;
  const int64_t i0 = item / a.H * kTokens;
  const int h = static_cast<int>(item - item / a.H * a.H);
  const RowPlace mine = lane < kTokens ? place_row(a.r, i0 + lane, a.B, a.cap, a.err) : RowPlace{0, -1};
  const int plane = lane >> 4, l16 = lane & 15;
  uint16_t* dst = static_cast<uint16_t*>(plane ? a.r.v : a.r.k);
  int64_t slot[kTokens];
  uint32_t code[kTokens], meta[kTokens];
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    slot[u] = __shfl_sync(0xffffffffu, mine.slot, u);
    const int b = __shfl_sync(0xffffffffu, mine.b, u);
    code[u] = meta[u] = 0;
    if (slot[u] >= 0) {
      const int64_t blk = kv4_block_offset(static_cast<int64_t>(b) * a.H + h, a.cap, slot[u]);
      const int at = static_cast<int>(slot[u] % kKv4BlockSlots);
      const int64_t c_off = blk + plane * kKv4VOffset + at * 64 + (l16 & 7) * 8 + (l16 >> 3) * 4;
      const int64_t m_off = blk + kKv4MetaOffset + at * 16 + plane * 8 + (l16 >> 3) * 4;
      if (in_bounds(c_off, 4, a.blocks_bytes, a.err)) code[u] = *reinterpret_cast<const uint32_t*>(a.cache + c_off);
      if (in_bounds(m_off, 4, a.blocks_bytes, a.err)) meta[u] = *reinterpret_cast<const uint32_t*>(a.cache + m_off);
    }
  }
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    if (slot[u] < 0) continue;
    const float s = bf16_lo(meta[u]), m = bf16_hi(meta[u]);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // s n is exact in fp32 (8 + 4 bits): one rounding at the sum, one to bf16
      const float lo = fmaf(s, static_cast<float>((code[u] >> (8 * e)) & 15u), m);
      const float hi = fmaf(s, static_cast<float>((code[u] >> (8 * e + 4)) & 15u), m);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[e]) : "f"(hi), "f"(lo));
    }
    *reinterpret_cast<uint4*>(dst + row_offset(a.r, i0 + u, h) + l16 * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ---------------------------------------------------------------- eviction

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

// Larger key = larger weight; equal weights (also -0 and +0) have equal keys;
// NaN ranks below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Block-wide inclusive scan of v (every thread calls it); *total gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  if (w == 0) {
    uint32_t s = lane < static_cast<int>(blockDim.x >> 5) ? warp_sums[lane] : 0u;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const uint32_t before = w ? warp_sums[w - 1] : 0u;
  *total = warp_sums[(blockDim.x >> 5) - 1];
  __syncthreads();
  return before + x;
}

// The slots that one (sequence, head) pair keeps, in their order, written into
// the destination's position array (the gather replaces them by positions).
// The k-th largest key is found by its digits (11, 11 and 10 bits): a
// histogram of the digit over the keys that agree so far, then the bin in
// which the k-th falls.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4EvictLaunch a) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t s_bin, s_above;
  const int64_t bh = blockIdx.x;
  const int b = static_cast<int>(bh / a.H);
  const int n = kv4_length(a.lengths[b], a.src_cap, threadIdx.x == 0 ? a.err : nullptr);
  const int kept = n < a.keep ? n : a.keep;
  if (bh - static_cast<int64_t>(b) * a.H == 0 && threadIdx.x == 0) a.new_lengths[b] = kept;
  int32_t* idx = a.dst_pos + bh * a.dst_cap;
  if (n <= a.keep) {
    for (int j = threadIdx.x; j < n; j += blockDim.x) idx[j] = j;
    return;
  }
  const float* w = a.src_weight + bh * a.src_cap;
  const int c0 = a.sink, c1 = n - a.recent;   // candidates [c0, c1): more than k of them, since n > keep
  const uint32_t k = static_cast<uint32_t>(a.keep - a.sink - a.recent);
  uint32_t prefix = 0, left = k;              // the k-th largest key's digits so far; its rank among those that agree
  if (k > 0) {
    uint32_t mask = 0;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      for (int i = threadIdx.x; i < kBins; i += blockDim.x) hist[i] = 0;
      __syncthreads();
      for (int i = c0 + threadIdx.x; i < c1; i += blockDim.x) {
        const uint32_t key = weight_key(w[i]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & digit], 1u);
      }
      __syncthreads();
      // bins from the top: thread t holds bins kBins-1-2t and kBins-2-2t
      const uint32_t h0 = hist[kBins - 1 - 2 * threadIdx.x], h1 = hist[kBins - 2 - 2 * threadIdx.x];
      uint32_t total;
      const uint32_t upto = block_scan(h0 + h1, warp_sums, &total);
      const uint32_t before = upto - h0 - h1;
      if (before < left && left <= upto) {
        const bool first = left <= before + h0;
        s_bin = kBins - 1 - 2 * threadIdx.x - (first ? 0 : 1);
        s_above = before + (first ? 0 : h0);
      }
      __syncthreads();
      prefix |= s_bin << shift;
      mask |= digit << shift;
      left -= s_above;
      __syncthreads();
    }
  }
  // Keep the protected slots, the keys above the k-th and the first `left` of
  // its equals.  before(i) of each kind by a running scan; the two counts are
  // scanned together, 16 bits each (a chunk has 1024 slots).
  uint32_t base_keep = 0, base_equal = 0;
  for (int i0 = 0; i0 < n; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    bool sure = false, equal = false;
    if (i < n) {
      if (i < c0 || i >= c1) {
        sure = true;
      } else if (k > 0) {
        const uint32_t key = weight_key(w[i]);
        sure = key > prefix;
        equal = key == prefix;
      }
    }
    uint32_t total;
    const uint32_t upto = block_scan((sure ? 1u : 0u) | (equal ? 0x10000u : 0u), warp_sums, &total);
    const uint32_t keep_before = base_keep + (upto & 0xFFFFu) - (sure ? 1u : 0u);
    const uint32_t equal_before = base_equal + (upto >> 16) - (equal ? 1u : 0u);
    if (sure || (equal && equal_before < left))
      idx[keep_before + (equal_before < left ? equal_before : left)] = i;
    base_keep += total & 0xFFFFu;
    base_equal += total >> 16;
  }
}

// Eight lanes move one kept slot: 16 bytes of K or V codes each, and one of
// them the scales, one the weight, one the position.
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4EvictLaunch a) {
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / a.H);
  const int n = kv4_length(a.lengths[b], a.src_cap, nullptr);
  const int kept = n < a.keep ? n : a.keep;
  const int lane = threadIdx.x & 31, part = lane & 7;
  const int64_t j = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 3;
  if (j - (lane >> 3) >= kept) return;   // the whole warp is behind the end
  const bool on = j < kept;
  int32_t* dpos = a.dst_pos + bh * a.dst_cap;
  const int src = on ? dpos[j] : 0;
  int4 codes = make_int4(0, 0, 0, 0), meta = codes;
  float w = 0.f;
  int32_t pos = 0;
  const int64_t sblk = kv4_block_offset(bh, a.src_cap, src), dblk = kv4_block_offset(bh, a.dst_cap, on ? j : 0);
  const int sat = src % kKv4BlockSlots, dat = static_cast<int>(j % kKv4BlockSlots);
  const int c_at = (part >> 2) * kKv4VOffset + (part & 3) * 16;
  if (on) {
    codes = ld_stream(reinterpret_cast<const int4*>(a.src + sblk + c_at + sat * 64));
    if (part == 0) meta = ld_stream(reinterpret_cast<const int4*>(a.src + sblk + kKv4MetaOffset + sat * 16));
    if (part == 1) w = a.src_weight[bh * a.src_cap + src];
    if (part == 2) pos = a.src_pos[bh * a.src_cap + src];
  }
  __syncwarp();   // every lane has its slot number before the position replaces it
  if (on) {
    *reinterpret_cast<int4*>(a.dst + dblk + c_at + dat * 64) = codes;
    if (part == 0) *reinterpret_cast<int4*>(a.dst + dblk + kKv4MetaOffset + dat * 16) = meta;
    if (part == 1) a.dst_weight[bh * a.dst_cap + j] = w;
    if (part == 2) dpos[j] = pos;
  }
}

}  // namespace

cudaError_t launch_kv4_rows(bool load, const Kv4RowsLaunch& a, cudaStream_t stream) {
  const int64_t items = (a.r.rows + kTokens - 1) / kTokens * a.H;
  if (items == 0) return cudaSuccess;
  const int64_t grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  if (load)
    kv4_load_kernel<<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
  else
    kv4_append_kernel<<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_evict(const Kv4EvictLaunch& a, cudaStream_t stream) {
  const int pairs = a.B * a.H;
  kv4_select_kernel<<<pairs, kSelThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t most = a.keep < a.src_cap ? a.keep : a.src_cap;
  const dim3 grid(static_cast<unsigned>((most * 8 + kThreads - 1) / kThreads), pairs);
  kv4_gather_kernel<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace ulysses
