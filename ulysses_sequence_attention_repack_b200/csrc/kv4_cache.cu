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
#include "sm100_ptx.cuh"

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

// Where rows i0 .. i0 + 7 live: lane u < 8 gets the pair (sequence, slot) of
// row i0 + u, slot -1 for a row of no sequence or a slot outside the cache.
struct RowPlace {
  int b;
  int64_t slot;
};

// Row i belongs to the last b with cu[b] <= i, if i < cu[batch].  The whole
// warp looks for i0's sequence, 32 entries a round (one round below 32
// sequences), then counts the ends that rows i0 + 1 .. pass.  cu is read inside
// [0, batch] only, whatever it holds.
__device__ __forceinline__ RowPlace place_rows(const Kv4Rows& r, int64_t i0, int batch, int64_t capacity,
                                               unsigned int* err) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;
  while (hi - lo >= 32) {
    const int step = (hi - lo) / 32 + 1, j = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, j <= hi && r.cu[min(j, hi)] <= i0));
    lo += max(n - 1, 0) * step;
    hi = min(hi, lo + step - 1);
  }
  const int b0 = lo + __popc(__ballot_sync(0xffffffffu, lo + lane <= hi && r.cu[min(lo + lane, hi)] <= i0)) - 1;
  const int64_t end = b0 + 1 + lane <= batch ? r.cu[b0 + 1 + lane] : INT64_MAX;
  int b = b0;
#pragma unroll
  for (int u = 1; u < kTokens; ++u) {
    const int n = __popc(__ballot_sync(0xffffffffu, end <= i0 + u));
    if (lane == u) b = b0 + n;
  }
  const int64_t i = i0 + lane;
  RowPlace p{0, -1};
  if (lane >= kTokens || i >= r.rows || b < 0 || b >= batch) return p;
  if (b == b0 + 32)   // many empty sequences in a row: go on one by one
    while (b < batch && r.cu[b + 1] <= i) ++b;
  if (b >= batch) return p;
  const int64_t first = r.cu[b];
  if (i < first || i >= r.cu[b + 1]) return p;   // (sums that fall)
  p.b = b;
  p.slot = static_cast<int64_t>(r.start[b]) + (i - first);
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

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The code of d = x - m >= 0 for a step s, by a division: for steps so small
// that their reciprocal is not a number to work with.
__device__ __noinline__ uint32_t code_by_division(float d, float s) {
  return static_cast<uint32_t>(fminf(fmaxf(rintf(__fdiv_rn(d, s)), 0.f), 15.f));
}

// Append: one warp takes 8 consecutive tokens of one head (neighbouring warps
// the neighbouring heads, whose rows are neighbours in memory).  Half a warp
// holds a row, 8 dims a lane: lanes 0-15 the K row, 16-31 the V row, so a
// group of 64 is 8 lanes and its minimum and maximum three shuffles of pairs.
//
// n = round((x - m) / s) without a division: t = d r rounded to an integer by
// adding 1.5 2^23 (r an approximate 1 / s) is the right integer or, next to a
// border, its neighbour.  The residual d - n s is exact (d and s are bf16
// differences and steps: |d - n s| <= s is a multiple of d's last place), so
// comparing it with s / 2 tells which, and finds the ties, which go to even.
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4RowsLaunch a) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t groups = (a.r.rows + kTokens - 1) / kTokens;
  pdl_wait();
  if (item >= groups * a.H) return;
  const int64_t i0 = item / a.H * kTokens;
  const int h = static_cast<int>(item - item / a.H * a.H);
  const int plane = lane >> 4, l16 = lane & 15;
  const uint16_t* src = static_cast<const uint16_t*>(plane ? a.r.v : a.r.k) + row_offset(a.r, i0, h) + l16 * 8;
  int4 x[kTokens];
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    x[u] = make_int4(0, 0, 0, 0);
    if (i0 + u < a.r.rows) x[u] = ld_stream(reinterpret_cast<const int4*>(src + u * a.r.token_stride));
  }
  const RowPlace mine = place_rows(a.r, i0, a.B, a.cap, a.err);
  uint32_t meta[kTokens];
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    const int64_t slot = __shfl_sync(0xffffffffu, mine.slot, u);
    const int64_t bh = static_cast<int64_t>(__shfl_sync(0xffffffffu, mine.b, u)) * a.H + h;
    const uint32_t w[4] = {static_cast<uint32_t>(x[u].x), static_cast<uint32_t>(x[u].y),
                           static_cast<uint32_t>(x[u].z), static_cast<uint32_t>(x[u].w)};
    uint32_t lo2 = min2(min2(w[0], w[1]), min2(w[2], w[3])), hi2 = max2(max2(w[0], w[1]), max2(w[2], w[3]));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      lo2 = min2(lo2, __shfl_xor_sync(0xffffffffu, lo2, d));
      hi2 = max2(hi2, __shfl_xor_sync(0xffffffffu, hi2, d));
    }
    const float lo = min_nan(bf16_lo(lo2), bf16_hi(lo2)), hi = max_nan(bf16_lo(hi2), bf16_hi(hi2));
    // (hi - lo) / 15 by its reciprocal and one correction, which is exact where the quotient is a bf16 border
    const float spread = __fsub_rn(hi, lo);
    const float q0 = spread * (1.0f / 15.0f);
    const float s = __bfloat162float(__float2bfloat16_rn(fmaf(fmaf(-q0, 15.0f, spread), 1.0f / 15.0f, q0)));
    const bool finite = fabsf(s) <= 3.4e38f && fabsf(lo) <= 3.4e38f;
    uint32_t code = 0;
    if (finite && s > 0.f) {
      if (s < 0x1p-100f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          code |= code_by_division(__fsub_rn(e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]), lo), s) << (4 * e);
      } else {
        constexpr float kRound = 12582912.f;   // 1.5 2^23, bits 0x4B400000
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        const float half = 0.5f * s;
        bool border = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = __fsub_rn(e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]), lo);
          const float t = fmaf(d, r, kRound);
          border |= fabsf(fmaf(-(t - kRound), s, d)) >= half;
          code += __float_as_uint(t) << (4 * e);
        }
        // (each t's upper bits: the sum of 0x4B400000 << 4 e)
        constexpr uint32_t kExtra = 0x4B400000u + 0xB4000000u + 0x40000000u;
        code -= kExtra;
        if (border) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float d = __fsub_rn(e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]), lo);
            const uint32_t n = (code >> (4 * e)) & 15u;
            const float rest = fmaf(-static_cast<float>(n), s, d);
            // one step on or back past the border; on it, to the even one
            if (rest > half || (rest == half && (n & 1u))) code += 1u << (4 * e);
            if (rest < -half || (rest == -half && (n & 1u))) code -= 1u << (4 * e);
          }
        }
      }
    }
    meta[u] = finite ? (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xFFFF0000u) : 0x7fc07fc0u;
    if (slot < 0) continue;
    const int64_t c_off = kv4_block_offset(bh, a.cap, slot) + plane * kKv4VOffset +
                          static_cast<int>(slot % kKv4BlockSlots) * 64 + (l16 & 7) * 8 + (l16 >> 3) * 4;
    if (in_bounds(c_off, 4, a.blocks_bytes, a.err)) *reinterpret_cast<uint32_t*>(a.cache + c_off) = code;
  }
  // Scales, weights and positions of the 8 tokens in one store each: lane
  // 4 u + p writes part p of token u's scales, lane u its weight and position.
  {
    const int u = lane >> 2, p = lane & 3;
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < kTokens; ++v) {   // part p is held by lanes 8 p ..
      const uint32_t y = __shfl_sync(0xffffffffu, meta[v], 8 * p);
      if (v == u) m = y;
    }
    const int64_t slot = __shfl_sync(0xffffffffu, mine.slot, u);
    const int64_t bh = static_cast<int64_t>(__shfl_sync(0xffffffffu, mine.b, u)) * a.H + h;
    if (slot >= 0) {
      const int64_t m_off = kv4_block_offset(bh, a.cap, slot) + kKv4MetaOffset +
                            static_cast<int>(slot % kKv4BlockSlots) * 16 + p * 4;
      if (in_bounds(m_off, 4, a.blocks_bytes, a.err)) *reinterpret_cast<uint32_t*>(a.cache + m_off) = m;
    }
  }
  if (mine.slot >= 0) {
    const int64_t at = (static_cast<int64_t>(mine.b) * a.H + h) * a.cap + mine.slot;
    a.weight[at] = 0.f;
    a.pos[at] = static_cast<int32_t>(a.r.pos0 ? a.r.pos0[mine.b] + (mine.slot - a.r.start[mine.b]) : mine.slot);
  }
}

// Load: the same split; a lane turns one 32-bit word of codes into 8 bf16.
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const Kv4RowsLaunch a) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t groups = (a.r.rows + kTokens - 1) / kTokens;
  pdl_wait();
  if (item >= groups * a.H) return;
  const int64_t i0 = item / a.H * kTokens;
  const int h = static_cast<int>(item - item / a.H * a.H);
  const RowPlace mine = place_rows(a.r, i0, a.B, a.cap, a.err);
  const int plane = lane >> 4, l16 = lane & 15;
  uint16_t* dst = static_cast<uint16_t*>(plane ? a.r.v : a.r.k) + row_offset(a.r, i0, h) + l16 * 8;
  uint32_t code[kTokens], meta[kTokens];
  uint32_t there = 0;
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    const int64_t slot = __shfl_sync(0xffffffffu, mine.slot, u);
    const int b = __shfl_sync(0xffffffffu, mine.b, u);
    code[u] = meta[u] = 0;
    if (slot >= 0) {
      there |= 1u << u;
      const int64_t blk = kv4_block_offset(static_cast<int64_t>(b) * a.H + h, a.cap, slot);
      const int at = static_cast<int>(slot % kKv4BlockSlots);
      const int64_t c_off = blk + plane * kKv4VOffset + at * 64 + (l16 & 7) * 8 + (l16 >> 3) * 4;
      const int64_t m_off = blk + kKv4MetaOffset + at * 16 + plane * 8 + (l16 >> 3) * 4;
      if (in_bounds(c_off, 4, a.blocks_bytes, a.err)) code[u] = *reinterpret_cast<const uint32_t*>(a.cache + c_off);
      if (in_bounds(m_off, 4, a.blocks_bytes, a.err)) meta[u] = *reinterpret_cast<const uint32_t*>(a.cache + m_off);
    }
  }
#pragma unroll
  for (int u = 0; u < kTokens; ++u) {
    const float s = bf16_lo(meta[u]), m = bf16_hi(meta[u]);
    const uint32_t even = code[u] & 0x0F0F0F0Fu, odd = (code[u] >> 4) & 0x0F0F0F0Fu;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // a byte under the exponent of 2^23 is that number plus 2^23; s n is
      // exact in fp32 (8 + 4 bits): one rounding at the sum, one to bf16
      const float n0 = __uint_as_float(__byte_perm(even, 0x4B000000u, 0x7440u + e)) - 8388608.f;
      const float n1 = __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7440u + e)) - 8388608.f;
      const float lo = fmaf(s, n0, m), hi = fmaf(s, n1, m);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[e]) : "f"(hi), "f"(lo));
    }
    if (there >> u & 1)
      *reinterpret_cast<uint4*>(dst + u * a.r.token_stride) = make_uint4(o[0], o[1], o[2], o[3]);
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

__device__ __forceinline__ uint32_t ld_cluster(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

// The slots that one (sequence, head) pair keeps, in their order, written into
// the destination's position array (the gather replaces them by positions).
//
// A cluster of blocks shares a pair, each block a run of its slots.  The k-th
// largest key is found by its digits (11, 11 and 10 bits): every block makes a
// histogram of the digit over its keys that agree so far, and all add up the
// cluster's histograms through distributed shared memory.  Their own
// histograms then say how many slots each block keeps, so the kept slots are
// numbered without another pass.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4EvictLaunch a, int cluster) {
  __shared__ __align__(8) uint32_t hist[3][kBins];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t s_bin, s_above;
  __shared__ uint32_t s_sure, s_equal;   // slots of this block's run: kept for sure, equal to the k-th
  pdl_launch_dependents();
  const int rank = static_cast<int>(blockIdx.x) % cluster;
  const int64_t bh = blockIdx.x / cluster;
  const int b = static_cast<int>(bh / a.H);
  for (int i = threadIdx.x; i < 3 * kBins; i += blockDim.x) (&hist[0][0])[i] = 0;
  if (threadIdx.x == 0) s_sure = s_equal = 0;
  __syncthreads();
  pdl_wait();
  const int n = kv4_length(a.lengths[b], a.src_cap, threadIdx.x == 0 ? a.err : nullptr);
  const int kept = n < a.keep ? n : a.keep;
  if (bh - static_cast<int64_t>(b) * a.H == 0 && rank == 0 && threadIdx.x == 0) a.new_lengths[b] = kept;
  int32_t* idx = a.dst_pos + bh * a.dst_cap;
  const int run = ((n + cluster - 1) / cluster + 3) / 4 * 4;   // a multiple of 4: 16-byte loads of weights
  const int i_begin = min(n, rank * run), i_end = min(n, i_begin + run);
  if (n <= a.keep) {   // (the whole cluster)
    for (int j = i_begin + threadIdx.x; j < i_end; j += blockDim.x) idx[j] = j;
    return;
  }
  const float* w = a.src_weight + bh * a.src_cap;
  const int c0 = a.sink, c1 = n - a.recent;   // candidates [c0, c1): more than k of them, since n > keep
  const uint32_t k = static_cast<uint32_t>(a.keep - a.sink - a.recent);
  uint32_t prefix = 0, left = k;              // the k-th largest key's digits so far; its rank among those that agree
  if (k > 0) {
    uint32_t mask = 0, above = 0;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      for (int i = i_begin + 4 * threadIdx.x; i < i_end; i += 4 * blockDim.x) {
        // (capacities are multiples of 4: the load stays inside the pair)
        const float4 v = *reinterpret_cast<const float4*>(w + i);
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t key = weight_key(x[e]);
          if (i + e < i_end && i + e >= c0 && i + e < c1 && (key & mask) == prefix)
            atomicAdd(&hist[pass][(key >> shift) & digit], 1u);
        }
      }
      __syncwarp();
      cluster_sync();
      // bins from the top: thread t holds bins kBins-1-2t and kBins-2-2t
      const uint32_t top = kBins - 2 - 2 * threadIdx.x;
      uint32_t h0 = 0, h1 = 0;
      for (int r = 0; r < cluster; ++r) {
        h1 += ld_cluster(&hist[pass][top], r);
        h0 += ld_cluster(&hist[pass][top + 1], r);
      }
      uint32_t total;
      const uint32_t upto = block_scan(h0 + h1, warp_sums, &total);
      const uint32_t before = upto - h0 - h1;
      if (before < left && left <= upto) {
        const bool first = left <= before + h0;
        s_bin = top + (first ? 1 : 0);
        s_above = before + (first ? 0 : h0);
      }
      __syncthreads();
      const uint32_t bin = s_bin;
      left -= s_above;
      prefix |= bin << shift;
      mask |= digit << shift;
      above += (top > bin ? hist[pass][top] : 0u) + (top + 1 > bin ? hist[pass][top + 1] : 0u);   // this block's own
      if (pass == 2 && threadIdx.x == 0) s_equal = hist[pass][bin];
      __syncthreads();
    }
    if (above) atomicAdd(&s_sure, above);
  }
  __syncthreads();
  if (threadIdx.x == 0)   // the protected slots of this run
    s_sure += static_cast<uint32_t>(max(0, min(i_end, c0) - i_begin) + max(0, i_end - max(i_begin, c1)));
  __syncwarp();
  cluster_sync();
  uint32_t base_keep = 0, base_equal = 0;
  for (int r = 0; r < rank; ++r) {
    base_keep += ld_cluster(&s_sure, r);
    base_equal += ld_cluster(&s_equal, r);
  }
  // Keep the protected slots, the keys above the k-th and the first `left` of
  // its equals, numbered by a running scan; the two counts are scanned
  // together, 16 bits each (a chunk has 4096 slots).
  for (int i0 = i_begin; i0 < i_end; i0 += 4 * blockDim.x) {
    const int i = i0 + 4 * threadIdx.x;
    uint32_t sure = 0, equal = 0;   // bit e: slot i + e
    if (i < i_end) {
      const float4 v = *reinterpret_cast<const float4*>(w + i);
      const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (i + e >= i_end) continue;
        if (i + e < c0 || i + e >= c1) {
          sure |= 1u << e;
        } else if (k > 0) {
          const uint32_t key = weight_key(x[e]);
          if (key > prefix) sure |= 1u << e;
          if (key == prefix) equal |= 1u << e;
        }
      }
    }
    const uint32_t mine = __popc(sure) | (__popc(equal) << 16);
    uint32_t total;
    const uint32_t upto = block_scan(mine, warp_sums, &total) - mine;
    uint32_t keep_before = base_keep + (upto & 0xFFFFu), equal_before = base_equal + (upto >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool is_sure = sure >> e & 1, is_equal = equal >> e & 1;
      if (is_sure || (is_equal && equal_before < left)) idx[keep_before + min(equal_before, left)] = i + e;
      keep_before += is_sure;
      equal_before += is_equal;
    }
    base_keep += total & 0xFFFFu;
    base_equal += total >> 16;
  }
  __syncwarp();
  cluster_sync();   // no block ends while another may read its shared memory
}

// Eight lanes move a kept slot: 16 bytes of K or V codes each, and one of them
// the scales, one the weight, one the position.  Each takes kMoves slots, 4
// kMoves apart in a warp, so that their loads are in flight together.
constexpr int kMoves = 4;
constexpr int kGatherSlots = kThreads / 8 * kMoves;

__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4EvictLaunch a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t bh = blockIdx.y;
  const int b = static_cast<int>(bh / a.H);
  const int n = kv4_length(a.lengths[b], a.src_cap, nullptr);
  const int kept = n < a.keep ? n : a.keep;
  const int lane = threadIdx.x & 31, part = lane & 7;
  const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kGatherSlots + (threadIdx.x >> 5) * 4 * kMoves + (lane >> 3);
  int32_t* dpos = a.dst_pos + bh * a.dst_cap;
  const int c_at = (part >> 2) * kKv4VOffset + (part & 3) * 16;
  int32_t src[kMoves];
#pragma unroll
  for (int u = 0; u < kMoves; ++u) src[u] = j0 + 4 * u < kept ? dpos[j0 + 4 * u] : -1;
  int4 codes[kMoves], meta[kMoves];
  int32_t word[kMoves];
#pragma unroll
  for (int u = 0; u < kMoves; ++u) {
    codes[u] = meta[u] = make_int4(0, 0, 0, 0);
    word[u] = 0;
    if (src[u] < 0) continue;
    const uint8_t* blk = a.src + kv4_block_offset(bh, a.src_cap, src[u]);
    const int at = src[u] % kKv4BlockSlots;
    codes[u] = ld_stream(reinterpret_cast<const int4*>(blk + c_at + at * 64));
    if (part == 0) meta[u] = ld_stream(reinterpret_cast<const int4*>(blk + kKv4MetaOffset + at * 16));
    if (part == 1) word[u] = __float_as_int(a.src_weight[bh * a.src_cap + src[u]]);
    if (part == 2) word[u] = a.src_pos[bh * a.src_cap + src[u]];
  }
  __syncwarp();   // every lane has its slot numbers before positions replace them
#pragma unroll
  for (int u = 0; u < kMoves; ++u) {
    if (src[u] < 0) continue;
    const int64_t j = j0 + 4 * u;
    uint8_t* blk = a.dst + kv4_block_offset(bh, a.dst_cap, j);
    const int at = static_cast<int>(j % kKv4BlockSlots);
    *reinterpret_cast<int4*>(blk + c_at + at * 64) = codes[u];
    if (part == 0) *reinterpret_cast<int4*>(blk + kKv4MetaOffset + at * 16) = meta[u];
    if (part == 1) a.dst_weight[bh * a.dst_cap + j] = __int_as_float(word[u]);
    if (part == 2) dpos[j] = word[u];
  }
}

}  // namespace

cudaError_t launch_kv4_rows(bool load, const Kv4RowsLaunch& a, cudaStream_t stream) {
  const int64_t items = (a.r.rows + kTokens - 1) / kTokens * a.H;
  if (items == 0) return cudaSuccess;
  const int64_t grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_after(load ? kv4_load_kernel : kv4_append_kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, 1,
                      stream, a);
}

cudaError_t launch_kv4_evict(const Kv4EvictLaunch& a, cudaStream_t stream) {
  const int pairs = a.B * a.H;
  // blocks that share a pair: about 8,192 slots of the longest each
  int cluster = 1;
  while (cluster < 8 && a.src_cap > 8192ll * cluster) cluster *= 2;
  cudaError_t e = launch_after(kv4_select_kernel, dim3(static_cast<unsigned>(pairs) * cluster), kSelThreads, 0, cluster,
                               stream, a, cluster);
  if (e != cudaSuccess) return e;
  const int64_t most = a.keep < a.src_cap ? a.keep : a.src_cap;
  return launch_after(kv4_gather_kernel,
                      dim3(static_cast<unsigned>((most + kGatherSlots - 1) / kGatherSlots), static_cast<unsigned>(pairs)),
                      kThreads, 0, 1, stream, a);
}

}  // namespace ulysses
