// Kernels that fill, read back and compact the 4-bit K/V cache (kv4.cuh).
//
// All three move bytes: per (token, head) the append reads 512 bytes of bf16
// and writes 144 + 8, the load reads 144 and writes 512, and the eviction
// reads the 4-byte weight of every cached slot and moves 152 bytes of those it
// keeps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "bounds.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "sm100_ptx.cuh"

namespace ulysses {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 8;   // consecutive tokens of one head a warp takes together

__device__ __forceinline__ int4 ld_stream(const int4* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Where row i0 + lane lives, for lanes below T: its sequence and slot; slot -1
// for a row of no sequence or a slot outside the cache.
struct RowPlace {
  int b;
  int64_t slot;
};

// Row i belongs to the last b with cu[b] <= i, if i < cu[batch].  The whole
// warp looks for i0's sequence, 32 entries a round (one round below 32
// sequences), then counts the ends that rows i0 + 1 .. pass.  cu is read inside
// [0, batch] only, whatever it holds.
template <int T>
__device__ __forceinline__ RowPlace place_rows(const Kv4Rows& r, int rows, int i0, int batch, int64_t capacity,
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
  int b = b0;
  if (T > 1) {
    const int end = b0 + 1 + lane <= batch ? r.cu[b0 + 1 + lane] : 0x7fffffff;
#pragma unroll
    for (int u = 1; u < T; ++u) {
      const int n = __popc(__ballot_sync(0xffffffffu, end <= i0 + u));
      if (lane == u) b = b0 + n;
    }
  }
  const int i = i0 + lane;
  RowPlace p{0, -1};
  if (lane >= T || i >= rows || b < 0 || b >= batch) return p;
  if (b == b0 + 32)   // many empty sequences in a row: go on one by one
    while (b < batch && r.cu[b + 1] <= i) ++b;
  if (b >= batch) return p;
  const int first = r.cu[b];
  if (i < first || i >= r.cu[b + 1]) return p;   // (sums that fall)
  p.b = b;
  p.slot = static_cast<int64_t>(r.start[b]) + i - first;
  if (p.slot < 0 || p.slot >= capacity) {
    if (err) atomicOr(err, kErrCacheIndex);
    p.slot = -1;
  }
  return p;
}

// Whether rows i0 .. i0 + T - 1 fill consecutive slots of one sequence.
template <int T>
__device__ __forceinline__ bool one_run(const RowPlace& p) {
  if (T == 1) return __shfl_sync(0xffffffffu, p.slot, 0) >= 0;
  const int lane = threadIdx.x & 31;
  const int b = __shfl_sync(0xffffffffu, p.b, 0);
  const int64_t slot = __shfl_sync(0xffffffffu, p.slot, 0);
  return __all_sync(0xffffffffu, lane >= T || (slot >= 0 && p.b == b && p.slot == slot + lane));
}

// Offset of the slot `at` slots on from the start of a block: from its code
// row and its scales.  (at < 64: in this block or the pair's next.)
__device__ __forceinline__ int code_row(int at) { return at * 64 + (at >> 5) * (kKv4BlockBytes - 32 * 64); }
__device__ __forceinline__ int meta_row(int at) {
  return kKv4MetaOffset + at * 16 + (at >> 5) * (kKv4BlockBytes - 32 * 16);
}

__device__ __forceinline__ int64_t row_offset(const Kv4Rows& r, int64_t i, int h, int H) {
  const int rank = r.heads_per_rank < H ? h / r.heads_per_rank : 0;
  return i * r.token_stride + rank * r.rank_stride + (h - rank * r.heads_per_rank) * r.head_stride;
}

// Elements from the first row's to the last one's end, and slots of the cache (for the bounds-checked build).
__device__ __forceinline__ int64_t row_extent(const Kv4Rows& r, int H) {
  return (r.rows - 1) * r.token_stride + (r.heads_per_rank - 1) * r.head_stride +
         (H / r.heads_per_rank - 1) * r.rank_stride + kKv4Dim;
}
__device__ __forceinline__ int64_t slots_of(int B, int H, int64_t capacity) {
  return static_cast<int64_t>(B) * H * capacity;
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

// Value e of 16, given as bf16 pairs.
__device__ __forceinline__ float value_of(const uint32_t (&w)[8], int e) {
  return e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
}

// Codes by divisions: for steps so small that their reciprocal is not a number
// to work with.
__device__ __noinline__ uint2 codes_by_division(uint4 w0, uint4 w1, float lo, float s) {
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint2 code = make_uint2(0, 0);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float n = fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(value_of(w, e), lo), s)), 0.f), 15.f);
    (e < 8 ? code.x : code.y) |= static_cast<uint32_t>(n) << (4 * (e & 7));
  }
  return code;
}

// The codes of this lane's 16 values of a group, whose other values the lanes
// of its quad hold; *meta gets the group's step and minimum.
//
// n = round(d / s) of d = x - m by a quotient from an approximate reciprocal r
// and one correction by its exact residual, which is the division's result;
// above all it is exact where the quotient is half way between two codes (one
// value in some 300 of bf16 data), so that adding 1.5 2^23 rounds those to even.
__device__ __forceinline__ uint2 quantise(const uint32_t (&w)[8], uint32_t* meta) {
  uint32_t lo2 = w[0], hi2 = w[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo2 = min2(lo2, w[i]);
    hi2 = max2(hi2, w[i]);
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    lo2 = min2(lo2, __shfl_xor_sync(0xffffffffu, lo2, d));
    hi2 = max2(hi2, __shfl_xor_sync(0xffffffffu, hi2, d));
  }
  const float lo = min_nan(bf16_lo(lo2), bf16_hi(lo2)), hi = max_nan(bf16_lo(hi2), bf16_hi(hi2));
  // (hi - lo) / 15 in the same way; it is exact where the quotient is a bf16 border
  const float spread = __fsub_rn(hi, lo);
  const float q0 = spread * (1.0f / 15.0f);
  const float s = __bfloat162float(__float2bfloat16_rn(fmaf(fmaf(-q0, 15.0f, spread), 1.0f / 15.0f, q0)));
  const bool finite = spread <= 3.402823466e38f;   // then hi, lo and s are, too (false for NaN)
  *meta = finite ? __byte_perm(__float_as_uint(s), __float_as_uint(lo), 0x7632u) : 0x7fc07fc0u;
  if (!(finite && s > 0.f)) return make_uint2(0, 0);
  if (s < 0x1p-100f)
    return codes_by_division(make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]), lo, s);
  constexpr float kRound = 12582912.f;   // 1.5 2^23, bits 0x4B400000
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  uint32_t code[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    code[j] = 0u - (0x4B400000u + 0xB4000000u + 0x40000000u);   // less the sum of 0x4B400000 << 4 e
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = __fsub_rn(value_of(w, 8 * j + e), lo);
      const float q = d * r;
      code[j] += __float_as_uint(__fadd_rn(fmaf(fmaf(-q, s, d), r, q), kRound)) * (1u << (4 * e));
    }
  }
  return make_uint2(code[0], code[1]);
}

// Append: one warp takes 8 consecutive tokens of one head (neighbouring warps
// the neighbouring heads, whose rows are neighbours in memory), their K rows
// and then their V rows.  Four lanes hold a row, 16 values of each group a
// lane: few lanes a group make its minimum and maximum cheap (two shuffles),
// and with 8 dims a lane the kernel spent twice the instructions, 295 us for
// 19,394 tokens x 56 heads.  A lane's token has a place of its own, so tokens
// of many sequences (a decoding step) go side by side.
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4RowsLaunch a) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  // (row numbers and items fit 32 bits: the launch sees to it)
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5), group = item / a.H;
  const int i0 = static_cast<int>(group) * kRun, h = static_cast<int>(item - group * a.H);
  pdl_wait();
  if (item >= a.items) return;
  const int u = lane >> 2, q = lane & 3;   // token; which 8 of every 32 dims
  const int64_t row = row_offset(a.r, i0 + u, h, a.H) + q * 8;
  uint4 x[2][4];
#pragma unroll
  for (int plane = 0; plane < 2; ++plane)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[plane][i] = make_uint4(0, 0, 0, 0);
      if (i0 + u < a.rows32 && in_bounds(row + 32 * i, 8, row_extent(a.r, a.H), a.err)) {
        const int4 v = ld_stream(reinterpret_cast<const int4*>(static_cast<const uint16_t*>(plane ? a.r.v : a.r.k) +
                                                               row + 32 * i));
        x[plane][i] = make_uint4(v.x, v.y, v.z, v.w);
      }
    }
  const RowPlace mine = place_rows<kRun>(a.r, a.rows32, i0, a.B, a.cap, a.err);
  const int64_t slot = __shfl_sync(0xffffffffu, mine.slot, u);
  const int b = __shfl_sync(0xffffffffu, mine.b, u);
  const int64_t bh = static_cast<int64_t>(b) * a.H + h;
  const int64_t blk = kv4_block_offset(bh, a.cap, max(slot, int64_t(0)));
  const int at = static_cast<int>(max(slot, int64_t(0)) % kKv4BlockSlots);
  uint32_t meta[2][2];
#pragma unroll
  for (int plane = 0; plane < 2; ++plane) {
    uint2 code[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint4 y = x[plane][2 * g], z = x[plane][2 * g + 1];
      const uint32_t w[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
      code[g] = quantise(w, &meta[plane][g]);
    }
    // chunks q and q + 4 of the row: the words of both groups
    const int64_t off = blk + plane * kKv4VOffset + at * 64 + q * 8;
    if (slot >= 0 && in_bounds(off, 40, a.blocks_bytes, a.err)) {
      *reinterpret_cast<uint2*>(a.cache + off) = make_uint2(code[0].x, code[1].x);
      *reinterpret_cast<uint2*>(a.cache + off + 32) = make_uint2(code[0].y, code[1].y);
    }
  }
  if (slot < 0) return;
  const int64_t m_off = blk + kKv4MetaOffset + at * 16;
  if (q == 0 && in_bounds(m_off, 16, a.blocks_bytes, a.err))
    *reinterpret_cast<uint4*>(a.cache + m_off) = make_uint4(meta[0][0], meta[0][1], meta[1][0], meta[1][1]);
  const int64_t slots = slots_of(a.B, a.H, a.cap);
  if (q == 1) store_at(a.weight, bh * a.cap + slot, slots, 0.f, a.err);
  if (q == 2)
    store_at(a.pos, bh * a.cap + slot, slots,
             static_cast<int32_t>(a.r.pos0 ? a.r.pos0[b] + (slot - a.r.start[b]) : slot), a.err);
}

// bf16(m + s n) of the 8 codes of a word: a nibble under the exponent of 2^7 is
// that number plus 128; the fused multiply-add rounds once.
__device__ __forceinline__ uint4 dequantise(uint32_t code, uint32_t meta) {
  const uint32_t s2 = __byte_perm(meta, 0, 0x1010u), m2 = __byte_perm(meta, 0, 0x3232u), up = code >> 4;
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // byte e of the codes and of the codes shifted down by a nibble: dims 2 e and 2 e + 1
    uint32_t n = (__byte_perm(code, up, 0x0400u + e * 0x0101u) & 0x000F000Fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(n) : "r"(0x43004300u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[e]) : "r"(s2), "r"(n), "r"(m2));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Load: the same split; a lane turns one 32-bit word of codes into 8 bf16.
template <int T>
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const Kv4RowsLaunch a) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5), group = item / a.H;
  const int i0 = static_cast<int>(group) * T, h = static_cast<int>(item - group * a.H);
  pdl_wait();
  if (item >= a.items) return;
  const int plane = lane >> 4, l16 = lane & 15;
  const int c_at = plane * kKv4VOffset + (l16 & 7) * 8 + (l16 >> 3) * 4, m_at = plane * 8 + (l16 >> 3) * 4;
  uint4* dst = static_cast<uint4*>(plane ? a.r.v : a.r.k);
  const int64_t to = row_offset(a.r, i0, h, a.H) / 8 + l16, step = a.r.token_stride / 8;
  const int64_t extent = row_extent(a.r, a.H) / 8;
  const RowPlace mine = place_rows<T>(a.r, a.rows32, i0, a.B, a.cap, a.err);
  if (one_run<T>(mine)) {
    const int64_t slot0 = __shfl_sync(0xffffffffu, mine.slot, 0);
    const int64_t blk = kv4_block_offset(static_cast<int64_t>(__shfl_sync(0xffffffffu, mine.b, 0)) * a.H + h, a.cap,
                                         slot0);
    const int at = static_cast<int>(slot0 % kKv4BlockSlots);
    uint32_t code[T], meta[T];
#pragma unroll
    for (int u = 0; u < T; ++u) {
      const int64_t off = blk + (code_row(at + u) + c_at), m_off = blk + (meta_row(at + u) + m_at);
      code[u] = meta[u] = 0;
      if (in_bounds(off, 4, a.blocks_bytes, a.err)) code[u] = *reinterpret_cast<const uint32_t*>(a.cache + off);
      if (in_bounds(m_off, 4, a.blocks_bytes, a.err)) meta[u] = *reinterpret_cast<const uint32_t*>(a.cache + m_off);
    }
#pragma unroll
    for (int u = 0; u < T; ++u)
      store_at(dst, to + u * step, extent, dequantise(code[u], meta[u]), a.err);
  } else if (T > 1) {
#pragma unroll 1
    for (int u = 0; u < T; ++u) {
      const int64_t slot = __shfl_sync(0xffffffffu, mine.slot, u);
      const int b = __shfl_sync(0xffffffffu, mine.b, u);
      if (slot < 0) continue;
      const int64_t blk = kv4_block_offset(static_cast<int64_t>(b) * a.H + h, a.cap, slot);
      const int at = static_cast<int>(slot % kKv4BlockSlots);
      const int64_t off = blk + (code_row(at) + c_at), m_off = blk + (meta_row(at) + m_at);
      if (in_bounds(off, 4, a.blocks_bytes, a.err) && in_bounds(m_off, 4, a.blocks_bytes, a.err))
        store_at(dst, to + u * step, extent,
                 dequantise(*reinterpret_cast<const uint32_t*>(a.cache + off),
                            *reinterpret_cast<const uint32_t*>(a.cache + m_off)),
                 a.err);
    }
  }
}

// ---------------------------------------------------------------- eviction

constexpr int kSelThreads = 1024;
constexpr int kBins = 256;
constexpr int kColumns = 16;
constexpr int kMaxCluster = 8;
constexpr int kHeldKeys = 22528;   // 88 KB

// Larger key = larger weight; equal weights (also -0 and +0) have equal keys;
// NaN ranks below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Inclusive scan over the lanes of a warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ uint32_t ld_cluster(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

// The slots that one (sequence, head) pair keeps, in their order, written into
// the destination's position array (the gather replaces them by positions):
// those of the `keep` largest keys, where a protected slot's key is above that
// of any weight and equal keys count from the lowest slot.
//
// A cluster of blocks shares a pair, each block a run of its slots whose keys
// it holds in shared memory (or, past kHeldKeys, makes anew from the weights
// each time).  The keep-th largest key is found digit by digit (four of 8
// bits): every block makes a histogram of the digit over its keys that agree
// so far, and all add up the cluster's histograms through distributed shared
// memory.  A histogram has 16 columns, so that at most two lanes of a warp meet
// in a counter: weights share few exponents, and many are equal (with one
// counter a bin the first digit's collisions alone took 100 us for 56 pairs of
// 104,448 slots; 32 columns take twice as long to clear and add up).  Their own histograms then say how many slots each block keeps, so
// the kept slots are numbered without another exchange.
template <bool kHeld>
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const Kv4EvictLaunch a, int cluster) {
  constexpr int kSelWarps = kSelThreads / 32;
  extern __shared__ __align__(16) uint32_t held[];
  __shared__ __align__(16) uint32_t hist[kBins][kColumns];
  __shared__ uint32_t sums[4][kBins];
  __shared__ uint32_t scan_sums[kBins / 32], warp_sure[kSelWarps], warp_equal[kSelWarps];
  __shared__ uint32_t s_bin, s_above;
  __shared__ uint32_t s_sure, s_equal;   // slots of this block's run: above the keep-th key, equal to it
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, column = lane & (kColumns - 1);
  const int rank = static_cast<int>(blockIdx.x) % cluster;
  const int64_t bh = blockIdx.x / cluster;
  const int b = static_cast<int>(bh / a.H);
  uint4* const cells = reinterpret_cast<uint4*>(&hist[0][0]) + threadIdx.x;   // 4 counters of bin threadIdx.x / 4
  static_assert(kBins * kColumns == 4 * kSelThreads, "a thread has 4 counters");
  *cells = make_uint4(0, 0, 0, 0);
  if (threadIdx.x == 0) s_sure = 0;
  pdl_wait();
  const int n = kv4_length(a.lengths[b], a.src_cap, threadIdx.x == 0 ? a.err : nullptr);
  const int kept = n < a.keep ? n : a.keep;
  if (bh - static_cast<int64_t>(b) * a.H == 0 && rank == 0 && threadIdx.x == 0) a.new_lengths[b] = kept;
  const auto put = [&](int64_t j, int i) {   // the pair's kept slot j is slot i
    if (in_bounds(j, 1, a.keep, a.err))
      store_at(a.dst_pos, bh * a.dst_cap + j, slots_of(a.B, a.H, a.dst_cap), i, a.err);
  };
  const int run = ((n + cluster - 1) / cluster + 3) / 4 * 4;   // a multiple of 4: 16-byte loads of weights
  const int i_begin = min(n, rank * run), i_end = min(n, i_begin + run);
  if (n <= a.keep) {   // (the whole cluster)
    for (int j = i_begin + threadIdx.x; j < i_end; j += blockDim.x) put(j, j);
    return;
  }
  const int64_t w = bh * a.src_cap, slots = slots_of(a.B, a.H, a.src_cap);   // the pair's weights
  const int c0 = a.sink, c1 = n - a.recent;   // slots outside [c0, c1) are protected
  // The keys of slots i .. i + 3 (capacities are multiples of 4: the load stays
  // inside the pair).  Slots behind the length, which follow the very last
  // one only, get the lowest key: the first of its equals are kept, and there
  // are enough of them before these.
  const auto make_keys = [&](int i) {
    const float4 v = load_at(reinterpret_cast<const float4*>(a.src_weight), (w + i) / 4, slots / 4,
                             make_float4(0.f, 0.f, 0.f, 0.f), a.err);
    uint32_t k[4] = {weight_key(v.x), weight_key(v.y), weight_key(v.z), weight_key(v.w)};
    if (i < c0 || i + 3 >= c1) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < c0 || i + e >= c1) k[e] = i + e < n ? 0xffffffffu : 0u;
    }
    return make_uint4(k[0], k[1], k[2], k[3]);
  };
  const auto keys = [&](int i) {
    if constexpr (kHeld)
      return *reinterpret_cast<const uint4*>(held + (i - i_begin));
    else
      return make_keys(i);
  };
  const auto key_of = [&](int i) {
    if constexpr (kHeld)
      return held[i - i_begin];
    else
      return i < c0 || i >= c1 ? 0xffffffffu : weight_key(load_at(a.src_weight, w + i, slots, 0.f, a.err));
  };
  __syncthreads();

  uint32_t prefix = 0, left = a.keep;   // the key's digits so far; its rank among the keys that agree
  uint32_t above = 0;
#pragma unroll
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    if (pass == 0) {
#pragma unroll 2
      for (int i = i_begin + 4 * threadIdx.x; i < i_end; i += 4 * kSelThreads) {
        const uint4 v = make_keys(i);
        if constexpr (kHeld) *reinterpret_cast<uint4*>(held + (i - i_begin)) = v;
        atomicAdd(&hist[v.x >> 24][column], 1u);
        atomicAdd(&hist[v.y >> 24][column], 1u);
        atomicAdd(&hist[v.z >> 24][column], 1u);
        atomicAdd(&hist[v.w >> 24][column], 1u);
      }
    } else {
      const uint32_t want = prefix >> (shift + 8);
#pragma unroll 2
      for (int i = i_begin + 4 * threadIdx.x; i < i_end; i += 4 * kSelThreads) {
        const uint4 v = keys(i);
        const bool x = v.x >> (shift + 8) == want, y = v.y >> (shift + 8) == want, z = v.z >> (shift + 8) == want,
                   w4 = v.w >> (shift + 8) == want;
        if (!(x || y || z || w4)) continue;   // few keys agree with a digit or two
        if (x) atomicAdd(&hist[(v.x >> shift) & 255u][column], 1u);
        if (y) atomicAdd(&hist[(v.y >> shift) & 255u][column], 1u);
        if (z) atomicAdd(&hist[(v.z >> shift) & 255u][column], 1u);
        if (w4) atomicAdd(&hist[(v.w >> shift) & 255u][column], 1u);
      }
    }
    __syncthreads();
    const uint4 y = *cells;
    *cells = make_uint4(0, 0, 0, 0);
    uint32_t own = y.x + y.y + y.z + y.w;
    own += __shfl_xor_sync(0xffffffffu, own, 1);
    own += __shfl_xor_sync(0xffffffffu, own, 2);
    if ((threadIdx.x & 3) == 0) sums[pass][threadIdx.x >> 2] = own;
    __syncwarp();
    cluster_sync();
    // the first 8 warps: bins from the top, one a thread
    const int bin = kBins - 1 - static_cast<int>(threadIdx.x);
    uint32_t all = 0, upto = 0;
    if (warp < kBins / 32) {
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < cluster) all += ld_cluster(&sums[pass][bin], r);
      upto = warp_scan(all);
      if (lane == 31) scan_sums[warp] = upto;
    }
    __syncthreads();
    if (warp < kBins / 32) {
      for (int v = 0; v < warp; ++v) upto += scan_sums[v];
      if (upto - all < left && left <= upto) {
        s_bin = bin;
        s_above = upto - all;
      }
    }
    __syncthreads();
    left -= s_above;
    prefix |= s_bin << shift;
    if (bin > static_cast<int>(s_bin)) above += sums[pass][bin];   // this block's own
  }
  if (above) atomicAdd(&s_sure, above);
  if (threadIdx.x == 0) s_equal = sums[3][prefix & 255u];

  // each warp's part of the run: how many of its slots are above the key, and equal to it
  const int part = ((run + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int p_begin = min(i_end, i_begin + warp * part), p_end = min(i_end, p_begin + part);
  uint32_t sure = 0, equal = 0;
  for (int i = p_begin + 4 * lane; i < p_end; i += 128) {
    const uint4 v = keys(i);
    const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sure += k[e] > prefix;
      equal += k[e] == prefix;
    }
  }
  sure = __reduce_add_sync(0xffffffffu, sure);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    warp_sure[warp] = sure;
    warp_equal[warp] = equal;
  }
  __syncthreads();
  cluster_sync();   // (also s_sure and s_equal)
  uint32_t keep_before = 0, equal_before = 0;
  // lane r: block r's counts, and warp r's of this block
  keep_before = (lane < rank ? ld_cluster(&s_sure, lane) : 0u) + (lane < warp ? warp_sure[lane] : 0u);
  equal_before = (lane < rank ? ld_cluster(&s_equal, lane) : 0u) + (lane < warp ? warp_equal[lane] : 0u);
  keep_before = __reduce_add_sync(0xffffffffu, keep_before);
  equal_before = __reduce_add_sync(0xffffffffu, equal_before);
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i0 = p_begin; i0 < p_end; i0 += 32) {   // (a part is a multiple of 32)
    const int i = i0 + lane;
    const uint32_t k = i < p_end ? key_of(i) : 0u;
    const bool equal_here = k == prefix && i < p_end;
    const uint32_t is_sure = __ballot_sync(0xffffffffu, k > prefix);
    const uint32_t is_equal = __ballot_sync(0xffffffffu, equal_here);
    const uint32_t q = equal_before + __popc(is_equal & below);
    if (k > prefix || (equal_here && q < left))
      put(keep_before + __popc(is_sure & below) + min(q, left), i);
    keep_before += __popc(is_sure);
    equal_before += __popc(is_equal);
  }
  // (not earlier: blocks of the gather that waited beside these took 25 us from them)
  pdl_launch_dependents();
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
  const int64_t to = bh * a.dst_cap, from = bh * a.src_cap;   // the pair's first slots
  const int64_t src_slots = slots_of(a.B, a.H, a.src_cap), dst_slots = slots_of(a.B, a.H, a.dst_cap);
  const int c_at = (part >> 2) * kKv4VOffset + (part & 3) * 16;
  int32_t src[kMoves];
#pragma unroll
  for (int u = 0; u < kMoves; ++u) {
    src[u] = j0 + 4 * u < kept ? load_at(a.dst_pos, to + j0 + 4 * u, dst_slots, -1, a.err) : -1;
    if (src[u] >= 0 && !in_bounds(src[u], 1, a.src_cap, a.err)) src[u] = -1;
  }
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
    if (part == 1) word[u] = __float_as_int(load_at(a.src_weight, from + src[u], src_slots, 0.f, a.err));
    if (part == 2) word[u] = load_at(a.src_pos, from + src[u], src_slots, 0, a.err);
  }
  __syncwarp();   // every lane has its slot numbers before positions replace them
#pragma unroll
  for (int u = 0; u < kMoves; ++u) {
    const int64_t j = j0 + 4 * u;
    if (src[u] < 0 || !in_bounds(j, 1, a.dst_cap, a.err)) continue;
    uint8_t* blk = a.dst + kv4_block_offset(bh, a.dst_cap, j);
    const int at = static_cast<int>(j % kKv4BlockSlots);
    *reinterpret_cast<int4*>(blk + c_at + at * 64) = codes[u];
    if (part == 0) *reinterpret_cast<int4*>(blk + kKv4MetaOffset + at * 16) = meta[u];
    if (part == 1) store_at(a.dst_weight, to + j, dst_slots, __int_as_float(word[u]), a.err);
    if (part == 2) store_at(a.dst_pos, to + j, dst_slots, word[u], a.err);
  }
}

}  // namespace

cudaError_t launch_kv4_rows(bool load, Kv4RowsLaunch a, cudaStream_t stream) {
  if (a.r.rows == 0) return cudaSuccess;
  // The load takes runs of tokens where sequences bring enough of them to fill
  // runs and the launch enough of those to fill the GPU, else a warp a token
  // (a run that crosses sequences goes one by one, and few runs are a longer
  // wait than more warps).  Tokens a sequence x sequences x heads, us a token
  // at a time / in runs: 4 x 256 x 8 3.7 / 4.7, 8 x 48 x 8 2.8 / 3.1, 16 x 48 x 8
  // 3.6 / 3.3, 8 x 256 x 8 5.3 / 4.9, 16 x 48 x 56 11.5 / 8.0, 32 x 1024 x 8
  // 72 / 32; 128 x 1 x 8 2.1 / 2.9, 64 x 1 x 56 3.1 / 3.0.
  const bool runs =
      !load || (a.r.rows >= static_cast<int64_t>(kRun) * a.B && a.r.rows * a.H >= 4096);
  const int64_t items = runs ? (a.r.rows + kRun - 1) / kRun * a.H : a.r.rows * a.H;
  const int64_t grid = (items + kWarps - 1) / kWarps;
  if (grid * kWarps > 0xffffffffll || grid > 0x7fffffff) return cudaErrorInvalidValue;
  a.items = static_cast<uint32_t>(items);
  a.rows32 = static_cast<int32_t>(a.r.rows);   // (at most 2^31 - 4096)
  const auto kernel = !load ? kv4_append_kernel : (runs ? kv4_load_kernel<kRun> : kv4_load_kernel<1>);
  return launch_after(kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, 1, stream, a);
}

cudaError_t launch_kv4_evict(const Kv4EvictLaunch& a, cudaStream_t stream) {
  const int pairs = a.B * a.H;
  // Blocks that share a pair: as many as leave all pairs resident at once (two
  // blocks an SM: 56 pairs of 104,448 slots take 5 each; 8 took two rounds and
  // half as long again), but 4,096 slots each at least.  A block holds its keys
  // where two blocks' fit an SM, else makes them anew each time.
  int dev = 0, sms = 1;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  int cluster = std::max(1, std::min(kMaxCluster, 2 * sms / pairs));
  cluster = static_cast<int>(std::min<int64_t>(cluster, (a.src_cap + 4095) / 4096));
  const int64_t run = (a.src_cap + 4 * cluster - 1) / (4 * cluster) * 4;
  const bool held = run <= kHeldKeys;
  static PerDeviceOnce once;
  e = once.run(dev, [] {
    return cudaFuncSetAttribute(kv4_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldKeys * 4);
  });
  if (e != cudaSuccess) return e;
  e = launch_after(held ? kv4_select_kernel<true> : kv4_select_kernel<false>,
                   dim3(static_cast<unsigned>(pairs) * cluster), kSelThreads, held ? run * 4 : 0, cluster, stream, a,
                   cluster);
  if (e != cudaSuccess) return e;
  const int64_t most = a.keep < a.src_cap ? a.keep : a.src_cap;
  return launch_after(kv4_gather_kernel,
                      dim3(static_cast<unsigned>((most + kGatherSlots - 1) / kGatherSlots), static_cast<unsigned>(pairs)),
                      kThreads, 0, 1, stream, a);
}

}  // namespace ulysses
