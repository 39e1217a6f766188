// Attention of new tokens over a 4-bit K/V cache (kv4.cuh).
//
// Row r of a K/V head is query token r / G of the sequence and its query head
// h * G + r % G.  With a slot's K row held as m_w + s_w n (group w = d / 64),
//
//   z_rt = scale q_r . k_t = scale sum_w ( s_tw (q_rw . n_tw) + m_tw sum_d q_rwd )
//   o_r  = sum_t p_rt v_t  = sum_t (p_rt s_tw) n_t + sum_t p_rt m_tw,   p = softmax z
//
// so the products run on the codes, and scales and minima are applied to
// their fp32 results.  The work is bound by the cache's bytes (144 a slot), so
// what counts is that a slot's 256 codes cost few instructions:
//
// - A code becomes an fp16 number by one AND: fp16 bits 0 .. 15 are the
//   subnormal n 2^-24, and bits n << 4 are 16 n 2^-24 (both exact, and the
//   tensor core multiplies subnormals exactly).  The factors 16 are taken out
//   of the query (K) and of the finished sums (V), and 2^-24 with the scale.
// - z^T = K q^T is a 16 x 8 x 16 product with slots as rows: 8 query rows a
//   product, so that up to 8 rows (one query head, or a group of them) cost
//   the same.  The lanes that hold z^T hold the same two query rows as those
//   of o^T = V^T p^T, so the running maximum and sums need no exchange, and p
//   becomes an operand of the second product by one 8 x 8 transpose.
// - The maximum in the exponent is replaced only when a row's grows by more
//   than 2^8, and the power of two that keeps a row's p s inside fp16 with it or
//   when p s has grown by 2^10, so most steps neither exchange nor rescale
//   anything.  Both are the row's own, from the slots that it sees: a step
//   that is large in a slot with hardly any weight, or in one that the row does
//   not see, costs its other slots nothing.
//
// Roundings: codes, scales and minima enter exactly, and q by a power of two
// that takes its row's largest just below fp16's end: 8 bits down to 2^-28 of
// that (of its power of two; a sixteenth of an odd value is 2^-17 there, whose
// last bit is fp16's least, 2^-24), fewer below; z, p, maxima and sums are fp32; p s is rounded to fp16 for the second product, off by at most
// 2^-11 of itself (bf16's 2^-8 would show in o) and, since the row's largest p s
// sits at 2^5 or more, by 2^-30 of that for the smallest; o is rounded once, to
// bf16.
//
// Work split: the tiles of 128 slots of all (sequence, K/V head, block of
// query rows) are one list, cut into equal runs, one a CTA, so ragged lengths
// and few heads fill the GPU alike.  Each of a CTA's four warps takes one
// 32-slot block of a tile.  Where a run ends inside a pair the CTA leaves an
// unfinished sum with its maximum in the workspace, and a second kernel joins
// them.  The lists are found from the lengths on the device, so that a
// captured launch stays right when they change.
//
// Measured (one B200, device time): 104,448 slots x 56 heads, one query row,
// 842 MB: 140 us (6.0 TB/s of 6.55 measured) at 1.95 GHz, 158 us in a loop of
// half a second, where the 1000 W cap holds 1.76 GHz; its copies alone take 125.
// Memory and the ALU share the time: of 384 instructions a warp spends on a
// block, 176 are the ANDs, shifts and byte moves that make operands of codes,
// and the ALU, at half rate, is 58% busy.  With more rows neither is the bound:
// with 8 (495 instructions a block, 8 heads x 313,344 slots: 79 us, 4.5 TB/s)
// issue slots and ALU are half busy and each warp waits on its own results, three
// warps a scheduler; with 16 (662, two warps a scheduler, 14 heads x 104,448: 73
// us, 2.9 TB/s) issue slots are 43% busy and the ALU 36%.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "bounds.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "sm100_ptx.cuh"

namespace ulysses {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kTile = kWarps * kKv4BlockSlots;   // slots of a tile
constexpr int kStages = 2;                       // blocks a warp has in flight
constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;
constexpr int kSmsMax = 148;
constexpr int kCtasPerSm = 3;
constexpr int kMaxCtas = kSmsMax * kCtasPerSm;   // sizes the workspace; the grid never passes it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;                     // log2 by which a maximum may be passed before it moves
// The second product's operand is p s 2^(5 - c), at most 2^15; c follows the row's largest p s.
constexpr int kHeadroom = 5;
constexpr int kGrowSteps = 10;                   // powers of two by which p s may outgrow 2^c before c moves
constexpr int kLeastExp = -114, kMostExp = 124;  // of c: p <= 2^8 times 2^(5 - c) is finite; no step passes 2^125
constexpr float kMost = 32768.f;

struct Args {
  const uint8_t* cache;
  float* weight;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t* lengths;
  float* part_o;      // [2 * CTAs][rows of a block][128]: unfinished sums
  float2* part_ml;    // [2 * CTAs][rows of a block]: their maxima and sums of p
  float2* row_ml;     // [B * H][R]: maxima and sums of rows that one CTA finished, for the weights
  float* logits;      // [B * H][R][cap]: z log2 e of the slots, for the weights
  int64_t cap, q_token_stride, q_head_stride;
  int32_t B, H, G, Lq, R, RB;
  float scale_log2;
  int32_t causal;
  unsigned int* err;

  // extents, for the bounds-checked build
  __device__ int64_t slots() const { return static_cast<int64_t>(B) * H * cap; }
  __device__ int64_t blocks_bytes() const { return slots() / kKv4BlockSlots * kKv4BlockBytes; }
  __device__ int64_t rows() const { return static_cast<int64_t>(B) * H * R; }
  __device__ int64_t q_extent() const {
    return (static_cast<int64_t>(B) * Lq - 1) * q_token_stride + (static_cast<int64_t>(H) * G - 1) * q_head_stride +
           kKv4Dim;
  }
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Both halves at once, in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 x, x, y, z; "
      "mov.b64 {%0, %1}, x;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127
__device__ __forceinline__ int exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }   // x >= 0

// A row's factor u = 2^(5 - c) of a group's p s, after a block whose largest p s is y, for a maximum whose move makes f
// of what was summed before (1: it did not move; 0: nothing counted before).  Returns what the finished sums of
// p s 2^(5 - c) are to be multiplied by.
__device__ __forceinline__ float move_power(float& u, float f, float y) {
  const int c = kHeadroom - exponent(u), top = exponent(y);
  int to = c;
  if (f != 1.f || top >= c + kGrowSteps)
    to = min(kMostExp, max(kLeastExp, max(f > 0.f ? c + exponent(f) : kLeastExp, top)));
  u = pow2(kHeadroom - to);
  return f * pow2(max(-126, min(126, c - to)));
}

// Slots below this are seen by row r of a sequence of len slots.
__device__ __forceinline__ int row_limit(const Args& a, int len, int r) {
  return a.causal ? max(0, len - a.Lq + r / a.G + 1) : len;
}

constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
#define NEG_INF __int_as_float(0xff800000)

// ---------------------------------------------------------------- the list of tiles

// The list runs over sequences, then heads, then blocks of query rows, then
// tiles.  Every warp finds its way by itself from the lengths, 32 at a time,
// without a barrier: this is what a launch does before its first copy.

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Tiles in the list.  report: flag lengths outside the cache.
__device__ __forceinline__ int total_tiles(const Args& a, bool report) {
  const int lane = threadIdx.x & 31;
  unsigned int* err = report ? a.err : nullptr;
  if (a.B == 1) return tiles_of(kv4_length(a.lengths[0], a.cap, lane == 0 ? err : nullptr)) * a.H * a.RB;
  int n = 0;
  for (int b = lane; b < a.B; b += 32) n += tiles_of(kv4_length(a.lengths[b], a.cap, err));
  return __reduce_add_sync(0xffffffffu, n) * a.H * a.RB;
}

// First tile of sequence b's in the list.
__device__ __forceinline__ int first_tile(const Args& a, int b) {
  if (b == 0) return 0;
  int n = 0;
  for (int i = threadIdx.x & 31; i < b; i += 32) n += tiles_of(kv4_length(a.lengths[i], a.cap, nullptr));
  return __reduce_add_sync(0xffffffffu, n) * a.H * a.RB;
}

// Rows of unfinished sums in the workspace: two of a block of RPB a CTA.
template <int RPB>
__host__ __device__ constexpr int64_t part_rows() {
  return static_cast<int64_t>(2) * kMaxCtas * RPB;
}

// A place in the list: tile `lo` of `ntiles` of unit (head, row block) `unit` of sequence b.
struct Place {
  int b, len, ntiles, unit, lo;

  // Tile number `tile`, below the total.
  __device__ __forceinline__ void find(const Args& a, int tile) {
    const int lane = threadIdx.x & 31, per = a.H * a.RB;
    b = 0;
    len = 0;
    if (a.B == 1) {
      len = kv4_length(a.lengths[0], a.cap, nullptr);
    } else {
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int l = b0 + lane < a.B ? kv4_length(a.lengths[b0 + lane], a.cap, nullptr) : 0;
        const int n = tiles_of(l) * per;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, upto > tile);
        if (past) {
          const int at = __ffs(past) - 1;
          b = b0 + at;
          len = __shfl_sync(0xffffffffu, l, at);
          tile -= __shfl_sync(0xffffffffu, upto - n, at);
          break;
        }
        tile -= __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    // (the bounds hold even if the lengths were changed meanwhile)
    ntiles = max(tiles_of(len), 1);
    unit = min(tile / ntiles, per - 1);
    lo = min(tile - unit * ntiles, ntiles - 1);
  }

  // The first tile of the next unit; there is one.
  __device__ __forceinline__ void next_unit(const Args& a) {
    lo = 0;
    if (++unit < a.H * a.RB) return;
    unit = 0;
    len = 0;
    while (len == 0 && b < a.B - 1) len = kv4_length(a.lengths[++b], a.cap, nullptr);
    ntiles = max(tiles_of(len), 1);
  }
};

__device__ __forceinline__ int tiles_per_cta(int total, int ctas) { return (total + ctas - 1) / ctas; }

// The blocks that one warp takes of a CTA's run, copied ahead into its ring.
struct Feed {
  Place at;
  int tile, end;
  const uint8_t* pair;
  uint32_t issued, ring, bars;

  __device__ __forceinline__ void locate(const Args& a) {
    pair = a.cache + (static_cast<int64_t>(at.b) * a.H + at.unit / a.RB) * (a.cap / kKv4BlockSlots) * kKv4BlockBytes;
  }
  // Starts the copy of the next block, if there is one.  A whole block is
  // copied even where the length ends inside it: it lies in the cache.
  __device__ __forceinline__ void next(const Args& a, int warp, int lane) {
    while (tile < end) {
      const int block = at.lo * kWarps + warp;
      const bool exists = block * kKv4BlockSlots < at.len;
      if (exists) {
        if (lane == 0) {
          const uint32_t s = issued % kStages, bar = bars + 8 * s;
          const uint8_t* from = pair + static_cast<int64_t>(block) * kKv4BlockBytes;
          if (in_bounds(from - a.cache, kKv4BlockBytes, a.blocks_bytes(), a.err)) {
            mbar_arrive_expect_tx(bar, kKv4BlockBytes);
            bulk_load(ring + s * kKv4BlockBytes, from, kKv4BlockBytes, bar);
          } else {
            mbar_arrive(bar);
          }
        }
        ++issued;
      }
      ++tile;
      if (++at.lo == at.ntiles && tile < end) {
        at.next_unit(a);
        locate(a);
      }
      if (exists) return;
    }
  }
};

// The log-sum of row r of a sequence of len slots, from its sum of p and its
// maximum.  A sum of 0 is a row that sees no slot, or one whose logits are all
// -infinity, past the range of fp32: that one has no softmax.
__device__ __forceinline__ float row_log2(const Args& a, int len, int r, float sum, float M) {
  if (sum == 0.f) return row_limit(a, len, r) > 0 ? __int_as_float(0x7fc00000) : NEG_INF;
  return M + log2f(sum);
}

// Row r of (sequence b of len slots, K/V head h): four dims a lane of the warp,
// from its sum o, its sum of p and its maximum.
__device__ __forceinline__ void finish_row(const Args& a, int b, int len, int h, int r, int lane, float4 o, float sum,
                                           float M) {
  const int i = r / a.G, hq = h * a.G + (r - i * a.G);
  const float log_sum = row_log2(a, len, r, sum, M);
  const float f = sum == 0.f ? (log_sum == NEG_INF ? 0.f : log_sum) : 1.f / sum;
  uint2 y;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.x) : "f"(o.y * f), "f"(o.x * f));
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y.y) : "f"(o.w * f), "f"(o.z * f));
  const int64_t row = (static_cast<int64_t>(b) * a.Lq + i) * a.H * a.G + hq;
  store_at(reinterpret_cast<uint2*>(a.out), row * (kKv4Dim / 4) + lane, a.rows() * (kKv4Dim / 4), y, a.err);
  if (a.lse && lane == 0)
    store_at(a.lse, (static_cast<int64_t>(b) * a.H * a.G + hq) * a.Lq + i, a.rows(), log_sum, a.err);
}

// ---------------------------------------------------------------- main kernel

__host__ __device__ inline int smem_rows(int R, int RPB) { return R < RPB ? R : RPB; }

// Dynamic shared memory: the warps' rings, then their sums [warp][row][128],
// maxima and sums of p [warp][row], then a warp's scratch: with kR > 0 its products' results [slot][row][group] in
// fp32, p s of a block [row][group][32 slots] in fp16 and 16 bytes of zeros;
// else a block's K scales and minima, and V's, 16 bytes a slot.
__host__ __device__ constexpr int scratch_bytes(int kR) { return kR ? kR * (256 + 128) + 16 : 1024; }
__host__ __device__ inline int64_t smem_bytes(int R, int RPB, int kR) {
  return kWarps * (kStages * kKv4BlockBytes + smem_rows(R, RPB) * (kKv4Dim * 4 + 8) + scratch_bytes(kR));
}

// NT: 8 or 16 query rows in a product.  kR: with 1 or 2 rows most columns of
// z^T are empty, so its lanes would spend the softmax's instructions on
// nothing; then z^T goes through shared memory and a lane takes one slot and
// its kR rows (0: more rows; a lane takes 4 slots and 2 rows as the products
// leave them).  104,448 slots x 56 heads: 1 row 164 -> 141 us, 2 rows 164 -> 148;
// with 4 rows it gains nothing (164 -> 167).
template <int NT, int kR, bool kWeights>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) kv4_attn_kernel(const Args a) {
  static_assert(kR == 0 || NT == 1, "few rows are one product wide");
  constexpr int RPB = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bar_mem[kWarps][kStages];
  __shared__ int abort_mem, drain_mem;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int mrows = smem_rows(a.R, RPB);
  uint8_t* ring = smem + warp * kStages * kKv4BlockBytes;
  float* mo = reinterpret_cast<float*>(smem + kWarps * kStages * kKv4BlockBytes);   // [warp][mrows][128]
  float* mM = mo + kWarps * mrows * kKv4Dim;
  float* ml = mM + kWarps * mrows;
  constexpr int kRows = kR ? kR : 1;
  uint8_t* zbuf = reinterpret_cast<uint8_t*>(ml + kWarps * mrows) + warp * scratch_bytes(kR);   // [slot][row][group] fp32
  uint8_t* wbuf = zbuf + kRows * 256;                                                           // [row][group][slot] fp16
  float4* kput = reinterpret_cast<float4*>(zbuf);
  // this lane's column of p s as the second operand (all 32 slots of row g), or zeros
  const uint8_t* wcol = g < kR ? wbuf + g * 128 + t * 16 : wbuf + kRows * 128;
  const int wstep = g < kR ? 64 : 0;
  // slot `lane`: pair (slot & 7) / 2 of register 2 (slot / 16) + (slot / 8 & 1) of a column
  uint8_t* wput = wbuf + ((lane & 7) >> 1) * 16 + (lane >> 3) * 4 + (lane & 1) * 2;
  if (kR && lane < 4) reinterpret_cast<uint32_t*>(wbuf + kRows * 128)[lane] = 0u;

  if (threadIdx.x == 0) {
    abort_mem = drain_mem = 0;
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(&bar_mem[0][0]) + 8 * i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  const WaitGuard guard{&abort_mem, a.err, kWaitLimitNs};
  const int total = total_tiles(a, blockIdx.x == 0 && warp == 0);
  const int chunk = tiles_per_cta(total, gridDim.x);
  const int64_t first64 = static_cast<int64_t>(blockIdx.x) * chunk;
  if (first64 >= total) return;
  int tile = static_cast<int>(first64);
  const int tile_end = min(total, tile + chunk);
  const int run_begin = tile;

  Place at;
  at.find(a, tile);
  Feed feed;
  feed.at = at;
  feed.tile = tile;
  feed.end = tile_end;
  feed.locate(a);
  feed.issued = 0;
  feed.ring = smem_u32(ring);
  feed.bars = smem_u32(&bar_mem[warp][0]);
#pragma unroll
  for (int i = 0; i < kStages; ++i) feed.next(a, warp, lane);
  uint32_t used = 0;        // blocks this warp has taken from its ring
  uint32_t left_at = 0;     // the block whose copy did not come
  bool alive = true;        // false once a wait has given up: nothing more is issued or waited for

  while (tile < tile_end) {
    // the fragment: tiles [lo, hi) of one (sequence, head, row block)
    const int b = at.b, len = at.len, ntiles = at.ntiles, lo = at.lo;
    const int hi = min(ntiles, lo + tile_end - tile);
    const int h = at.unit / a.RB, rb = at.unit - h * a.RB;
    const int64_t bh = static_cast<int64_t>(b) * a.H + h;
    const int row0 = rb * RPB;

    // the query as the second operand of z^T = K q^T: this lane holds, of row
    // row0 + 8 nt + g, dims 16t .. 16t + 15 of each group, scaled by a power of
    // two that takes the row's largest into [2^15, 2^16) (65,280 at most)
    uint32_t qf[NT][16];
    float qscale[NT][2], qsum[NT][2][2];
    int limit[NT][2];
    int lowest = len, highest = 0;             // of the rows' limits
    float rq[kRows], rq0[kRows], rq1[kRows];   // kR: scale and group sums of every row, and its limit
    int rlimit[kRows];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + 8 * nt + g;
      float f[2][16];
      if (r < a.R) {
        const int i = r / a.G;
        const int64_t at = (static_cast<int64_t>(b) * a.Lq + i) * a.q_token_stride +
                           static_cast<int64_t>(h * a.G + (r - i * a.G)) * a.q_head_stride + 16 * t;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint4 x = load_at(reinterpret_cast<const uint4*>(a.q), at / 8 + 8 * w + v, a.q_extent() / 8,
                                    make_uint4(0, 0, 0, 0), a.err);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[w][8 * v + 2 * e] = bf16_lo(u[e]);
              f[w][8 * v + 2 * e + 1] = bf16_hi(u[e]);
            }
          }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) f[0][e] = f[1][e] = 0.f;
      }
      uint32_t top = 0;   // bits of the largest magnitude: NaN and infinity rank above every number
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(f[w][e]) & 0x7fffffffu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int k = static_cast<int>(top >> 23) - 127;
      const int e = max(-100, min(126, 15 - k));
      const float up = pow2(e);
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f[w][i] *= up;
          sum[w] += f[w][i];
        }
      // word v of the lane's 16-byte K load: group v & 1, dims 16t + 8 (v >> 1) + 0 .. 7
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float* x = &f[v & 1][8 * (v >> 1)];
        qf[nt][4 * v] = pack_f16(x[0], x[4]);
        qf[nt][4 * v + 1] = pack_f16(x[1] * 0.0625f, x[5] * 0.0625f);
        qf[nt][4 * v + 2] = pack_f16(x[2], x[6]);
        qf[nt][4 * v + 3] = pack_f16(x[3] * 0.0625f, x[7] * 0.0625f);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 1);
        sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 2);
        sum[w] *= 0x1p-24f;
      }
      // a row with an infinity or a NaN has no softmax: its logits are NaN; so are those of a row that reaches 2^115,
      // which the powers of two do not
      const float qs = top >= (115u + 127u) << 23 ? __int_as_float(0x7fc00000) : a.scale_log2 * pow2(24 - e);
#pragma unroll
      for (int c = 0; c < 2; ++c) {   // to the lanes that hold this row's z: rows 2t and 2t + 1
        const int from = 4 * (2 * t + c);
        qscale[nt][c] = __shfl_sync(0xffffffffu, qs, from);
        qsum[nt][c][0] = __shfl_sync(0xffffffffu, sum[0], from);
        qsum[nt][c][1] = __shfl_sync(0xffffffffu, sum[1], from);
        const int rr = row0 + 8 * nt + 2 * t + c;
        limit[nt][c] = rr < a.R ? row_limit(a, len, rr) : 0;
        if (rr < a.R) {
          lowest = min(lowest, limit[nt][c]);
          highest = max(highest, limit[nt][c]);
        }
      }
      if constexpr (kR > 0) {
#pragma unroll
        for (int rr = 0; rr < kR; ++rr) {
          rq[rr] = __shfl_sync(0xffffffffu, qs, 4 * rr);
          rq0[rr] = __shfl_sync(0xffffffffu, sum[0], 4 * rr);
          rq1[rr] = __shfl_sync(0xffffffffu, sum[1], 4 * rr);
          rlimit[rr] = rr < a.R ? row_limit(a, len, rr) : 0;
        }
      }
    }
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    highest = __reduce_max_sync(0xffffffffu, highest);

    float acc[NT][8][4];
    float M[NT][2], Ms[NT][2], l[NT][2];   // Ms: M, or 0 while M is -inf
    float2 z0[NT][2], u[NT][2];            // of both groups: sums of p m, the rows' factors of p s
    // a step that takes no row's p s past its bound, whatever p is: 2^(c + 2) of the least c of the rows with a maximum
    // (infinity before any has one: a row's first slot moves its own)
    float s_limit[2] = {INFINITY, INFINITY};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][i][c] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        M[nt][c] = NEG_INF;
        Ms[nt][c] = l[nt][c] = 0.f;
        z0[nt][c] = make_float2(0.f, 0.f);
        u[nt][c] = make_float2(pow2(kHeadroom - kLeastExp), pow2(kHeadroom - kLeastExp));
      }
    }

    // z^T = K q^T on the codes: d[row block][16-slot half][group].  Neighbouring
    // products go to different sums, so none waits for the one before.
    auto scores = [&](const uint8_t* blk, float (&d)[NT][2][2][4]) {
      uint32_t wa[2][4], wb[2][4];   // the codes of slots g and g + 8
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint4 ka = *reinterpret_cast<const uint4*>(blk + (16 * mt + g) * 64 + t * 16);
        const uint4 kb = *reinterpret_cast<const uint4*>(blk + (16 * mt + g + 8) * 64 + t * 16);
        wa[mt][0] = ka.x;
        wa[mt][1] = ka.y;
        wa[mt][2] = ka.z;
        wa[mt][3] = ka.w;
        wb[mt][0] = kb.x;
        wb[mt][1] = kb.y;
        wb[mt][2] = kb.z;
        wb[mt][3] = kb.w;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 8; ++c) (&d[nt][mt][0][0])[c] = 0.f;
      }
#pragma unroll
      for (int v = 0; v < 4; v += 2)
#pragma unroll
        for (int up = 0; up < 2; ++up)   // nibbles 0, 1, 4, 5 of a word, then 2, 3, 6, 7
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t xa = wa[mt][v + w] >> (8 * up), xb = wb[mt][v + w] >> (8 * up);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma(d[nt][mt][w], xa & kLow, xb & kLow, xa & kHigh, xb & kHigh, qf[nt][4 * (v + w) + 2 * up],
                    qf[nt][4 * (v + w) + 2 * up + 1]);
            }
    };

    // o^T += V^T p^T for the p s of a block
    uint32_t pb[2][NT][2][2];   // [group][row block][half][operand register]
    auto values = [&](const uint8_t* blk) {
      // this lane holds dims 8g .. 8g + 7 of each group, and
      // slots 2t, 2t + 1 and 2t + 8, 2t + 9 of the half are the pairs of its registers
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint8_t* vrow = blk + kKv4VOffset + (16 * mt + 2 * t) * 64 + g * 8;
        const uint2 v0 = *reinterpret_cast<const uint2*>(vrow), v1 = *reinterpret_cast<const uint2*>(vrow + 64);
        const uint2 v8 = *reinterpret_cast<const uint2*>(vrow + 512), v9 = *reinterpret_cast<const uint2*>(vrow + 576);
        const uint32_t A[2] = {v0.x, v0.y}, B[2] = {v1.x, v1.y}, C[2] = {v8.x, v8.y}, D[2] = {v9.x, v9.y};
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            uint32_t x = __byte_perm(A[w], B[w], sel), y = __byte_perm(C[w], D[w], sel);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int i = 4 * w + 2 * half + j;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma(acc[nt][i], x & kLow, x & kHigh, y & kLow, y & kHigh, pb[w][nt][mt][0], pb[w][nt][mt][1]);
              x >>= 8;
              y >>= 8;
            }
          }
      }
    };

    // kR: the same of every row; sums over this lane's slots
    float rM[kRows], rMs[kRows], rl[kRows], rz[kRows][2], ru[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      rM[r] = NEG_INF;
      rMs[r] = rl[r] = rz[r][0] = rz[r][1] = 0.f;
      ru[r][0] = ru[r][1] = pow2(kHeadroom - kLeastExp);
    }

    // One block, a slot a lane.
    auto step_few = [&](auto edge_tag, const uint8_t* blk, int slot0) {
      constexpr bool kEdge = decltype(edge_tag)::value;
      float d[NT][2][2][4];
      scores(blk, d);
      if (2 * t < kR) {   // the lanes with columns of rows
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint8_t* to = zbuf + (16 * mt + g + 8 * i) * (8 * kRows) + t * 16;
            const float(&x)[2][4] = d[0][mt];
            if constexpr (kR == 1)
              *reinterpret_cast<float2*>(to) = make_float2(x[0][2 * i], x[1][2 * i]);
            else
              *reinterpret_cast<float4*>(to) = make_float4(x[0][2 * i], x[1][2 * i], x[0][2 * i + 1], x[1][2 * i + 1]);
          }
      }
      __syncwarp();
      const int slot = slot0 + lane;
      uint4 m = *reinterpret_cast<const uint4*>(blk + kKv4MetaOffset + lane * 16);
      if (kEdge && slot >= highest) m = make_uint4(0, 0, 0, 0);   // no row sees it; anything may be held there
      const float vs[2] = {bf16_lo(m.z), bf16_lo(m.w)}, vm[2] = {bf16_hi(m.z), bf16_hi(m.w)};
      float z[kRows] = {}, p[kRows], ps[kRows][2];
      const auto weigh = [&](int r) {   // p, and p s as the operand
        p[r] = ex2(z[r] - rMs[r]);
#pragma unroll
        for (int w = 0; w < 2; ++w)   // (whatever the steps of an unseen slot are)
          ps[r][w] = kEdge && slot >= rlimit[r] ? 0.f : p[r] * ru[r][w] * vs[w];
      };
      bool move = false;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float2 d = *reinterpret_cast<const float2*>(zbuf + lane * (8 * kRows) + r * 8);
        float x = bf16_lo(m.x) * d.x;
        x = fmaf(bf16_hi(m.x), rq0[r], x);
        x = fmaf(bf16_lo(m.y), d.y, x);
        x = fmaf(bf16_hi(m.y), rq1[r], x);
        x *= rq[r];
        if (kEdge && slot >= rlimit[r]) x = NEG_INF;
        z[r] = x;
        weigh(r);
        move |= x > rM[r] + kGrow || ps[r][0] > kMost || ps[r][1] > kMost;
        if (kWeights && r < a.R && (!kEdge || slot < len))
          store_at(a.logits, (bh * a.R + r) * a.cap + slot, a.rows() * a.cap, x, a.err);
      }
      if (__any_sync(0xffffffffu, move)) {
        float fac[2][2] = {{1.f, 1.f}, {1.f, 1.f}};   // of this lane's columns of o^T, in each group
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          float top = z[r];
#pragma unroll
          for (int dlt = 16; dlt; dlt >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, dlt));
          const float m_new = top > rM[r] + kGrow ? top : rM[r];
          const float f = m_new == rM[r] ? 1.f : ex2(rM[r] - m_new);
          rM[r] = m_new;
          rMs[r] = m_new == NEG_INF ? 0.f : m_new;
          rl[r] *= f;
          rz[r][0] *= f;
          rz[r][1] *= f;
          const float now = kEdge && slot >= rlimit[r] ? 0.f : ex2(z[r] - rMs[r]);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            // (what is no number takes no part: as the largest it would take the others' to zero)
            const uint32_t y = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(now * vs[w], 0.f)));
            const float down = move_power(ru[r][w], f, __uint_as_float(y));
            if (t == (r >> 1)) fac[r & 1][w] = down;
          }
          weigh(r);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[0][i][c] *= fac[c & 1][i >> 2];
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        rl[r] += p[r];
        const bool unseen = kEdge && slot >= rlimit[r];
        rz[r][0] = fmaf(p[r], unseen ? 0.f : vm[0], rz[r][0]);
        rz[r][1] = fmaf(p[r], unseen ? 0.f : vm[1], rz[r][1]);
        const uint32_t both = pack_f16(ps[r][0], ps[r][1]);
        *reinterpret_cast<uint16_t*>(wput + r * 128) = static_cast<uint16_t>(both);
        *reinterpret_cast<uint16_t*>(wput + r * 128 + 64) = static_cast<uint16_t>(both >> 16);
      }
      __syncwarp();
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint4 x = *reinterpret_cast<const uint4*>(wcol + w * wstep);
        pb[w][0][0][0] = x.x;
        pb[w][0][0][1] = x.y;
        pb[w][0][1][0] = x.z;
        pb[w][0][1][1] = x.w;
      }
      values(blk);
    };

    // One block of 32 slots at blk.  kEdge: some row does not see all of them.
    auto step = [&](auto edge_tag, const uint8_t* blk, int slot0) {
      constexpr bool kEdge = decltype(edge_tag)::value;
      // each lane turns one slot's scales and minima into fp32 for all
      bool big;   // a step that may take a p s past its bound
      {
        uint4 m = *reinterpret_cast<const uint4*>(blk + kKv4MetaOffset + lane * 16);
        // slots that no row sees hold anything: nothing of them may reach a sum
        if (kEdge && slot0 + lane >= highest) m = make_uint4(0, 0, 0, 0);
        const float vs[2] = {bf16_lo(m.z), bf16_lo(m.w)};
        big = __any_sync(0xffffffffu, vs[0] > s_limit[0] || vs[1] > s_limit[1]);
        kput[lane] = make_float4(bf16_lo(m.x), bf16_hi(m.x), bf16_lo(m.y), bf16_hi(m.y));
        kput[32 + lane] = make_float4(vs[0], vs[1], bf16_hi(m.z), bf16_hi(m.w));
      }
      __syncwarp();
      float s[NT][2][4];   // z / qscale: [16-slot half][slot g row 2t, g 2t+1, g+8 2t, g+8 2t+1]
      float d[NT][2][2][4];
      scores(blk, d);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 k = kput[16 * mt + g + 8 * i];
          const int slot = slot0 + 16 * mt + g + 8 * i;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int row = 0; row < 2; ++row) {
              const int c = 2 * i + row;
              float x = k.x * d[nt][mt][0][c];
              x = fmaf(k.y, qsum[nt][row][0], x);
              x = fmaf(k.z, d[nt][mt][1][c], x);
              x = fmaf(k.w, qsum[nt][row][1], x);
              if (kEdge && slot >= limit[nt][row]) x = NEG_INF;
              s[nt][mt][c] = x;
              if (kWeights) {
                const int r = row0 + 8 * nt + 2 * t + row;
                const float z = kEdge && slot >= limit[nt][row] ? NEG_INF : x * qscale[nt][row];
                if (r < a.R && (!kEdge || slot < len))
                  store_at(a.logits, (bh * a.R + r) * a.cap + slot, a.rows() * a.cap, z, a.err);
              }
            }
        }
      }
      float top[NT][2];
      bool move = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[nt][c] = fmaxf(fmaxf(s[nt][0][c], s[nt][0][c + 2]), fmaxf(s[nt][1][c], s[nt][1][c + 2])) * qscale[nt][c];
          move |= top[nt][c] > M[nt][c] + kGrow;
        }
      if (big) {   // by the rows' largest p in this block
        const float4 mine = kput[32 + lane];
        const float s0 = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(mine.x, 0.f))));
        const float s1 = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(mine.y, 0.f))));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float p = ex2(top[nt][c] - Ms[nt][c]);
            move |= p * u[nt][c].x * s0 > kMost || p * u[nt][c].y * s1 > kMost;
          }
      }
      if (__any_sync(0xffffffffu, move)) {
        // Where the block's steps are within 2^8 of each other, the least of them stands for the largest p s of a row whose
        // maximum it moves (p is 1 there); else every row finds its own.
        uint32_t least[2];
        bool own = big;
        {
          const float4 mine = kput[32 + lane];
          const float vs[2] = {fmaxf(mine.x, 0.f), fmaxf(mine.y, 0.f)};   // (what is no number takes no part)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t step = __float_as_uint(vs[w]);
            least[w] = __reduce_min_sync(0xffffffffu, kEdge && slot0 + lane >= highest ? 0x7f800000u : step);
            own |= (__reduce_max_sync(0xffffffffu, step) >> 23) >= (least[w] >> 23) + 8 || least[w] == 0;
          }
        }
        float f[NT][2], y[NT][2][2];   // what the moves make of sums so far; the rows' largest p s
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = top[nt][c];
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float m_new = m > M[nt][c] + kGrow ? m : M[nt][c];
            f[nt][c] = m_new == M[nt][c] ? 1.f : ex2(M[nt][c] - m_new);
            M[nt][c] = m_new;
            Ms[nt][c] = m_new == NEG_INF ? 0.f : m_new;
            l[nt][c] *= f[nt][c];
            z0[nt][c].x *= f[nt][c];
            z0[nt][c].y *= f[nt][c];
#pragma unroll
            for (int w = 0; w < 2; ++w) y[nt][c][w] = f[nt][c] != 1.f ? __uint_as_float(least[w]) : 0.f;
          }
        if (own) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float y0 = 0.f, y1 = 0.f;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float4 v = kput[32 + 8 * k + g];
                float p = ex2(fmaf(s[nt][k >> 1][2 * (k & 1) + c], qscale[nt][c], -Ms[nt][c]));
                if (kEdge && slot0 + 8 * k + g >= limit[nt][c]) p = 0.f;
                y0 = fmaxf(y0, p * v.x);
                y1 = fmaxf(y1, p * v.y);
              }
              // both groups' in one word: their leading halves, whose order is theirs
              uint32_t both = __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x7632u);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, d));
              y[nt][c][0] = bf16_lo(both);
              y[nt][c][1] = bf16_hi(both);
            }
        }
        if (s_limit[0] == INFINITY && !own) {
          // nothing is summed yet, and all rows get one power: most fragments' first block (5 ragged sequences of 14 x 2
          // heads, 8 tokens: 55.4 us the long way, 54.2 so)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int e = max(kLeastExp, min(kMostExp, exponent(__uint_as_float(least[w]))));
            s_limit[w] = pow2(e + 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) (w ? u[nt][c].y : u[nt][c].x) = pow2(kHeadroom - e);
          }
        } else {
          float up[2] = {pow2(kHeadroom - kMostExp), pow2(kHeadroom - kMostExp)};   // largest factor of a row with slots
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float down0 = move_power(u[nt][c].x, f[nt][c], y[nt][c][0]);
              const float down1 = move_power(u[nt][c].y, f[nt][c], y[nt][c][1]);
              if (M[nt][c] != NEG_INF) {
                up[0] = fmaxf(up[0], u[nt][c].x);
                up[1] = fmaxf(up[1], u[nt][c].y);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                acc[nt][i][c] *= i < 4 ? down0 : down1;
                acc[nt][i][c + 2] *= i < 4 ? down0 : down1;
              }
            }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(up[w]));
            s_limit[w] = pow2(kHeadroom + 2 - exponent(__uint_as_float(most)));
          }
        }
      }
      // p, its sums, and p s as the operand of the second product
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float4 va = kput[32 + 16 * mt + g], vb = kput[32 + 16 * mt + g + 8];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w0[4], w1[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int i = c >> 1, row = c & 1;
            const float4& v = i ? vb : va;
            float p = ex2(fmaf(s[nt][mt][c], qscale[nt][row], -Ms[nt][row]));
            // (0 by the limit, not by s = -inf alone: the row's scale is NaN where its query is, and may be 0)
            const bool unseen = kEdge && slot0 + 16 * mt + g + 8 * i >= limit[nt][row];
            if (unseen) p = 0.f;
            l[nt][row] += p;
            // both groups in one (104,448 slots x 56 heads, 4 rows: 187 us one by one, 178 in pairs)
            const float2 pp = make_float2(p, p);
            float2 ps = mul2(mul2(pp, u[nt][row]), make_float2(v.x, v.y)), vm = make_float2(v.z, v.w);
            if (unseen) ps = vm = make_float2(0.f, 0.f);   // (whatever the slot's steps are)
            w0[c] = ps.x;
            w1[c] = ps.y;
            z0[nt][row] = fma2(pp, vm, z0[nt][row]);
          }
          pb[0][nt][mt][0] = transpose8x8(pack_f16(w0[0], w0[1]));
          pb[0][nt][mt][1] = transpose8x8(pack_f16(w0[2], w0[3]));
          pb[1][nt][mt][0] = transpose8x8(pack_f16(w1[0], w1[1]));
          pb[1][nt][mt][1] = transpose8x8(pack_f16(w1[2], w1[3]));
        }
      }
      values(blk);
    };

    for (int tl = lo; tl < hi; ++tl) {
      const int slot0 = tl * kTile + warp * kKv4BlockSlots;
      if (slot0 >= len) break;
      const uint32_t stage = used % kStages;
      if (alive && !mbar_wait_warp(feed.bars + 8 * stage, (used / kStages) & 1u, guard)) {
        alive = false;
        left_at = used;
      }
      ++used;
      const uint8_t* blk = ring + stage * kKv4BlockBytes;
      if constexpr (kR > 0) {
        if (slot0 + kKv4BlockSlots > lowest)
          step_few(std::true_type{}, blk, slot0);
        else
          step_few(std::false_type{}, blk, slot0);
      } else {
        if (slot0 + kKv4BlockSlots > lowest)
          step(std::true_type{}, blk, slot0);
        else
          step(std::false_type{}, blk, slot0);
      }
      __syncwarp();   // every lane has read the block before it is replaced
      if (alive) feed.next(a, warp, lane);
    }

    // the fragment's sums: over the lanes that hold the same rows, then over the warps
    if constexpr (kR > 0) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
#pragma unroll
        for (int dlt = 1; dlt < 32; dlt <<= 1) {
          rl[r] += __shfl_xor_sync(0xffffffffu, rl[r], dlt);
          rz[r][0] += __shfl_xor_sync(0xffffffffu, rz[r][0], dlt);
          rz[r][1] += __shfl_xor_sync(0xffffffffu, rz[r][1], dlt);
        }
        if (t == (r >> 1)) {
          M[0][r & 1] = rM[r];
          l[0][r & 1] = rl[r];
          z0[0][r & 1] = make_float2(rz[r][0], rz[r][1]);
          u[0][r & 1] = make_float2(ru[r][0], ru[r][1]);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int dlt = 4; dlt < 32 && kR == 0; dlt <<= 1) {
          l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], dlt);
          z0[nt][c].x += __shfl_xor_sync(0xffffffffu, z0[nt][c].x, dlt);
          z0[nt][c].y += __shfl_xor_sync(0xffffffffu, z0[nt][c].y, dlt);
        }
        const int row = 8 * nt + 2 * t + c;
        if (row >= mrows) continue;
        if (g == 0) {
          mM[warp * mrows + row] = M[nt][c];
          ml[warp * mrows + row] = l[nt][c];
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          // codes 2^-24, p s 2^(5 - c); the odd nibbles carry a further 16.  (In two factors: together they may pass
          // the range of fp32 where the values do not.)
          const float even = pow2(24 - kHeadroom), odd = even * 0.0625f, zz = w ? z0[nt][c].y : z0[nt][c].x;
          const float up = pow2(kHeadroom - exponent(w ? u[nt][c].y : u[nt][c].x));
          float4* dst = reinterpret_cast<float4*>(mo + (warp * mrows + row) * kKv4Dim + 64 * w + 8 * g);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            dst[i] = make_float4(fmaf(acc[nt][4 * w + 2 * i][c] * even, up, zz),
                                 fmaf(acc[nt][4 * w + 2 * i][c + 2] * odd, up, zz),
                                 fmaf(acc[nt][4 * w + 2 * i + 1][c] * even, up, zz),
                                 fmaf(acc[nt][4 * w + 2 * i + 1][c + 2] * odd, up, zz));
        }
      }
    __syncthreads();
    // a warp takes every fourth row, a lane four of its dims
    const bool whole = lo == 0 && hi == ntiles;
    const int part = 2 * blockIdx.x + (tile == run_begin ? 0 : 1);
    for (int row = warp; row < RPB && row0 + row < a.R; row += kWarps) {
      float Mt = NEG_INF;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) Mt = fmaxf(Mt, mM[w * mrows + row]);
      const float base = Mt == NEG_INF ? 0.f : Mt;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(mM[w * mrows + row] - base);
        const float4 x = reinterpret_cast<const float4*>(mo + (w * mrows + row) * kKv4Dim)[lane];
        o.x = fmaf(f, x.x, o.x);
        o.y = fmaf(f, x.y, o.y);
        o.z = fmaf(f, x.z, o.z);
        o.w = fmaf(f, x.w, o.w);
        sum = fmaf(f, ml[w * mrows + row], sum);
      }
      const int r = row0 + row;
      if (whole) {
        finish_row(a, b, len, h, r, lane, o, sum, Mt);
        if (kWeights && lane == 0) store_at(a.row_ml, bh * a.R + r, a.rows(), make_float2(Mt, sum), a.err);
      } else {
        store_at(reinterpret_cast<float4*>(a.part_o), (static_cast<int64_t>(part) * RPB + row) * (kKv4Dim / 4) + lane,
                 part_rows<RPB>() * (kKv4Dim / 4), o, a.err);
        if (lane == 0) store_at(a.part_ml, part * RPB + row, part_rows<RPB>(), make_float2(Mt, sum), a.err);
      }
    }
    __syncthreads();
    tile += hi - lo;
    if (tile < tile_end) at.next_unit(a);
  }
  pdl_launch_dependents();   // (not earlier: waiting blocks of the next kernel would hold this one's places)
  // a warp that gave up has copies in flight: wait for them (again with a limit) before the memory is freed
  if (!alive) {
    const WaitGuard drain{&drain_mem, a.err, kWaitLimitNs};
    for (; left_at < feed.issued; ++left_at)
      if (!mbar_wait_warp(feed.bars + 8 * (left_at % kStages), (left_at / kStages) & 1u, drain)) break;
  }
}

// ---------------------------------------------------------------- joining the parts

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kWeightSlots = kJoinThreads * 8;   // slots of a block that adds weights

// The parts that one unit's tiles were cut into: those of CTAs c0 .. c1.  A
// unit that one CTA held is whole.
struct Parts {
  int c0, c1, chunk, t0;
  bool empty;   // no tile at all
  // chunk: tiles a CTA; first: the first tile of the unit's sequence.  (No CTA
  // past the last, even if the lengths were changed meanwhile.)
  __device__ __forceinline__ Parts(int chunk_, int ctas, int first, int unit, int ntiles) {
    chunk = max(chunk_, 1);
    empty = ntiles == 0;
    t0 = first + unit * ntiles;
    c0 = min(t0 / chunk, ctas - 1);
    c1 = min((t0 + ntiles - 1) / chunk, ctas - 1);
  }
  // a CTA's run begins with this unit, or it is the run's last
  __device__ __forceinline__ int part(int c) const { return 2 * c + (c * chunk >= t0 ? 0 : 1); }
};

// One warp: the maximum over the parts of a row, and the sum of p for it.
template <int RPB>
__device__ __forceinline__ float2 join_ml(const Args& a, const Parts& p, int row) {
  const int lane = threadIdx.x & 31;
  float M = NEG_INF, sum = 0.f;
  for (int c = p.c0 + lane; c <= p.c1; c += 32) {
    const float2 x = load_at(a.part_ml, p.part(c) * RPB + row, part_rows<RPB>(), make_float2(NEG_INF, 0.f), a.err);
    const float m = fmaxf(M, x.x);
    const float base = m == NEG_INF ? 0.f : m;
    sum = sum * ex2(M - base) + x.y * ex2(x.x - base);
    M = m;
  }
  float top = M;
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  sum *= ex2(M - (top == NEG_INF ? 0.f : top));
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return make_float2(top, sum);
}

// A row's sum over some of its parts: four dims a lane, and for all lanes the
// maximum and the sum of p.
struct Sum {
  float4 o;
  float M, p;
  __device__ __forceinline__ void scale(float f) {
    o.x *= f;
    o.y *= f;
    o.z *= f;
    o.w *= f;
    p *= f;
  }
  __device__ __forceinline__ void add(float f, const float4& y, float q) {
    o.x = fmaf(f, y.x, o.x);
    o.y = fmaf(f, y.y, o.y);
    o.z = fmaf(f, y.z, o.z);
    o.w = fmaf(f, y.w, o.w);
    p = fmaf(f, q, p);
  }
};

// The parts c0 + first, c0 + first + step, ..: eight at a time, so that one
// wait covers their loads (8 heads x 104,448 slots, 7 rows: 36.6 -> 34.1 us
// against reading the maxima first).
template <int RPB>
__device__ __forceinline__ Sum join_parts(const Args& a, const Parts& p, int row, int first, int step) {
  constexpr int kBatch = 8;
  const int lane = threadIdx.x & 31;
  Sum s{make_float4(0.f, 0.f, 0.f, 0.f), NEG_INF, 0.f};
  for (int c = p.c0 + first; c <= p.c1; c += kBatch * step) {
    float2 ml[kBatch];
    float4 y[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      ml[u] = make_float2(NEG_INF, 0.f);
      y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c + u * step <= p.c1) {
        const int64_t at = static_cast<int64_t>(p.part(c + u * step)) * RPB + row;
        ml[u] = load_at(a.part_ml, at, part_rows<RPB>(), ml[u], a.err);
        y[u] = load_at(reinterpret_cast<const float4*>(a.part_o), at * (kKv4Dim / 4) + lane,
                       part_rows<RPB>() * (kKv4Dim / 4), y[u], a.err);
      }
    }
    float m = s.M;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) m = fmaxf(m, ml[u].x);
    const float base = m == NEG_INF ? 0.f : m;
    s.scale(ex2(s.M - base));
    s.M = m;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) s.add(ex2(ml[u].x - base), y[u], ml[u].y);
  }
  return s;
}

// Blocks below `row_blocks` join `rpb` rows each: a warp a row, or, where a row
// was cut into more than kWarpParts parts, all warps one after another.
// Further blocks: kWeightSlots slots of a pair each,
// weight_t += sum_r 2^(z_rt - lse_r), the rows in their order.  Four blocks an SM
// (64 registers; with 74 and three, 24 ragged sequences x 8 heads with 7 rows
// and weights: 50.2 -> 53.7 us).
constexpr int kWarpParts = 8;

template <int RPB>
__global__ void __launch_bounds__(kJoinThreads, 4) kv4_join_kernel(const Args a, int ctas, int rpb, int64_t rows,
                                                                int64_t row_blocks) {
  __shared__ __align__(16) float so[kJoinWarps][kKv4Dim];
  __shared__ float2 sml[kJoinWarps];
  __shared__ float slse[kJoinWarps];
  __shared__ int shared_row[kJoinWarps];   // this warp's row is for all
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int64_t x = blockIdx.x;
  const int chunk = tiles_per_cta(total_tiles(a, false), ctas);
  if (x < row_blocks) {
    const auto parts_of = [&](int64_t i, int* b, int* len, int* h, int* r) {   // of row i
      const int64_t bh = i / a.R;
      *r = static_cast<int>(i - bh * a.R);
      *b = static_cast<int>(bh / a.H);
      *h = static_cast<int>(bh - static_cast<int64_t>(*b) * a.H);
      *len = kv4_length(a.lengths[*b], a.cap, nullptr);
      return Parts(chunk, ctas, first_tile(a, *b), *h * a.RB + *r / RPB, tiles_of(*len));
    };
    const auto all_warps = [&](const Parts& p, int b, int len, int h, int r) {
      const Sum mine = join_parts<RPB>(a, p, r % RPB, warp, kJoinWarps);
      reinterpret_cast<float4*>(so[warp])[lane] = mine.o;
      if (lane == 0) sml[warp] = make_float2(mine.M, mine.p);
      __syncthreads();
      if (warp == 0) {
        Sum all{make_float4(0.f, 0.f, 0.f, 0.f), NEG_INF, 0.f};
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) all.M = fmaxf(all.M, sml[w].x);
        const float base = all.M == NEG_INF ? 0.f : all.M;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w)
          all.add(ex2(sml[w].x - base), reinterpret_cast<const float4*>(so[w])[lane], sml[w].y);
        finish_row(a, b, len, h, r, lane, all.o, all.p, all.M);
      }
    };
    const int64_t i0 = x * rpb, mine = rpb == 1 ? i0 : i0 + warp;
    int b, len, h, r;
    if (lane == 0) shared_row[warp] = 0;
    if (mine < rows) {
      const Parts p = parts_of(mine, &b, &len, &h, &r);
      const int n = p.c1 - p.c0 + 1;
      if (p.empty) {
        if (rpb > 1 || warp == 0) finish_row(a, b, 0, h, r, lane, make_float4(0.f, 0.f, 0.f, 0.f), 0.f, NEG_INF);
      } else if (rpb == 1) {
        if (n > 1) all_warps(p, b, len, h, r);
      } else if (n > kWarpParts) {
        if (lane == 0) shared_row[warp] = 1;
      } else if (n > 1) {
        const Sum s = join_parts<RPB>(a, p, r % RPB, 0, 1);
        finish_row(a, b, len, h, r, lane, s.o, s.p, s.M);
      }
    }
    if (rpb == 1) return;
    __syncthreads();
    for (int v = 0; v < rpb; ++v) {
      if (!shared_row[v]) continue;
      const Parts p = parts_of(i0 + v, &b, &len, &h, &r);
      all_warps(p, b, len, h, r);
      __syncthreads();
    }
    return;
  }
  const int64_t per = (a.cap + kWeightSlots - 1) / kWeightSlots, y = x - row_blocks;
  const int64_t bh = y / per;
  const int64_t slot0 = (y - bh * per) * kWeightSlots + threadIdx.x * 4;   // and kWeightSlots / 2 further on
  const int b = static_cast<int>(bh / a.H), h = static_cast<int>(bh - static_cast<int64_t>(b) * a.H);
  const int len = kv4_length(a.lengths[b], a.cap, nullptr);
  if ((y - bh * per) * kWeightSlots >= len) return;
  const int ntiles = tiles_of(len);
  const int first = first_tile(a, b);
  float4 sum[2] = {};
  for (int r0 = 0; r0 < a.R; r0 += kJoinWarps) {
    const int r = r0 + warp;   // each warp finds one row's log-sum
    if (r < a.R) {
      const Parts p(chunk, ctas, first, h * a.RB + r / RPB, ntiles);
      const float2 ml = p.c0 == p.c1
                            ? load_at(a.row_ml, bh * a.R + r, a.rows(), make_float2(NEG_INF, 0.f), a.err)
                            : join_ml<RPB>(a, p, r % RPB);
      if (lane == 0) slse[warp] = row_log2(a, len, r, ml.y, ml.x);
    }
    __syncthreads();
#pragma unroll 2
    for (int i = 0; i < min(kJoinWarps, a.R - r0); ++i) {
      const float lse = slse[i];
      const int64_t z = ((bh * a.R + r0 + i) * a.cap + slot0) / 4;
      float4 v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (slot0 + k * (kWeightSlots / 2) < len)
          v[k] = load_at(reinterpret_cast<const float4*>(a.logits), z + k * (kWeightSlots / 8), a.rows() * a.cap / 4,
                         make_float4(0.f, 0.f, 0.f, 0.f), a.err);
      if (lse == NEG_INF) continue;
      if (lse != lse) {   // a row without a softmax: no number for the slots it sees, nothing for the others
        const int limit = row_limit(a, len, r0 + i);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int64_t slot = slot0 + k * (kWeightSlots / 2);
          if (slot < limit) sum[k].x = lse;
          if (slot + 1 < limit) sum[k].y = lse;
          if (slot + 2 < limit) sum[k].z = lse;
          if (slot + 3 < limit) sum[k].w = lse;
        }
        continue;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        sum[k].x += ex2(v[k].x - lse);
        sum[k].y += ex2(v[k].y - lse);
        sum[k].z += ex2(v[k].z - lse);
        sum[k].w += ex2(v[k].w - lse);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t slot = slot0 + k * (kWeightSlots / 2);
    if (slot < len && !in_bounds(bh * a.cap + slot, 4, a.slots(), a.err)) continue;
    float* f = a.weight + bh * a.cap + slot;   // (16-byte aligned: capacities are multiples of 32)
    if (slot + 3 < len) {
      const float4 v = *reinterpret_cast<float4*>(f);
      *reinterpret_cast<float4*>(f) = make_float4(v.x + sum[k].x, v.y + sum[k].y, v.z + sum[k].z, v.w + sum[k].w);
    } else if (slot < len) {   // the slots behind the length keep what they hold
      f[0] += sum[k].x;
      if (slot + 1 < len) f[1] += sum[k].y;
      if (slot + 2 < len) f[2] += sum[k].z;
    }
  }
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

int rows_of_block(int64_t R) { return R <= 8 ? 8 : 16; }

template <int NT, int kR, bool kWeights>
cudaError_t launch_main(const Args& a, int* ctas, cudaStream_t stream) {
  static PerDeviceOnce once;
  int dev = 0, sms = 1;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  e = once.run(dev, [&] {
    return cudaFuncSetAttribute(kv4_attn_kernel<NT, kR, kWeights>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem_bytes(8 * NT, 8 * NT, kR)));
  });
  if (e != cudaSuccess) return e;
  const int64_t bytes = smem_bytes(a.R, 8 * NT, kR);
  // as many CTAs as an SM holds: registers allow 3 (2 with 16 rows), shared memory (1 KB a CTA is the system's) may
  // allow fewer
  const int64_t fit = 228 * 1024 / (bytes + 1024 + 256);
  *ctas = std::min(sms, kSmsMax) * static_cast<int>(std::min<int64_t>(NT == 1 ? 3 : 2, fit));
  return launch_after(kv4_attn_kernel<NT, kR, kWeights>, dim3(*ctas), kThreads, bytes, 1, stream, a);
}

template <bool kWeights>
cudaError_t launch_rows(const Args& a, int* ctas, cudaStream_t stream) {
  if (a.R == 1) return launch_main<1, 1, kWeights>(a, ctas, stream);
  if (a.R == 2) return launch_main<1, 2, kWeights>(a, ctas, stream);
  if (a.R <= 8) return launch_main<1, 0, kWeights>(a, ctas, stream);
  return launch_main<2, 0, kWeights>(a, ctas, stream);
}

}  // namespace

// Parts and their (maximum, sum) pairs; with weights also each row's log-sum
// and the logits of every slot.
int64_t kv4_attn_workspace_bytes(int32_t B, int32_t H, int32_t G, int32_t Lq, int64_t cap, bool weights) {
  const int64_t R = static_cast<int64_t>(G) * Lq, rpb = rows_of_block(R);
  int64_t n = up256(2 * kMaxCtas * rpb * kKv4Dim * 4) + up256(2 * kMaxCtas * rpb * 8);
  if (weights) n += up256(static_cast<int64_t>(B) * H * R * 8) + static_cast<int64_t>(B) * H * R * cap * 4;
  return n;
}

cudaError_t launch_kv4_attn(const Kv4AttnLaunch& p, cudaStream_t stream) {
  const int64_t R = static_cast<int64_t>(p.G) * p.Lq;
  const int rpb = rows_of_block(R);
  Args a;
  a.cache = p.cache;
  a.weight = p.weight;
  a.q = static_cast<const uint16_t*>(p.q);
  a.out = static_cast<uint16_t*>(p.out);
  a.lse = p.lse;
  a.lengths = p.lengths;
  uint8_t* w = p.workspace;
  a.part_o = reinterpret_cast<float*>(w);
  w += up256(static_cast<int64_t>(2) * kMaxCtas * rpb * kKv4Dim * 4);
  a.part_ml = reinterpret_cast<float2*>(w);
  w += up256(static_cast<int64_t>(2) * kMaxCtas * rpb * 8);
  a.row_ml = p.weight ? reinterpret_cast<float2*>(w) : nullptr;
  w += up256(static_cast<int64_t>(p.B) * p.H * R * 8);
  a.logits = p.weight ? reinterpret_cast<float*>(w) : nullptr;
  a.cap = p.cap;
  a.q_token_stride = p.q_token_stride;
  a.q_head_stride = p.q_head_stride;
  a.B = p.B;
  a.H = p.H;
  a.G = p.G;
  a.Lq = p.Lq;
  a.R = static_cast<int32_t>(R);
  a.RB = static_cast<int32_t>((R + rpb - 1) / rpb);
  a.scale_log2 = p.scale * kLog2e;
  a.causal = p.causal;
  a.err = p.err;
  int ctas = 0;
  cudaError_t e;
  e = p.weight ? launch_rows<true>(a, &ctas, stream) : launch_rows<false>(a, &ctas, stream);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.B) * p.H * R;
  const int64_t weight_blocks =
      p.weight ? static_cast<int64_t>(p.B) * p.H * ((p.cap + kWeightSlots - 1) / kWeightSlots) : 0;
  // a warp a row where there are more rows than blocks fit the GPU at once (1,344 rows of a ragged batch: 8 us with a
  // block each, 5 with a warp); fewer rows were cut into more parts each
  int dev = 0, sms = 1;
  if ((e = current_device_sms(&dev, &sms)) != cudaSuccess) return e;
  const int per_block = rows > 4 * sms ? kJoinWarps : 1;
  const int64_t row_blocks = (rows + per_block - 1) / per_block;
  if (row_blocks + weight_blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_after(rpb == 8 ? kv4_join_kernel<8> : kv4_join_kernel<16>,
                      dim3(static_cast<unsigned>(row_blocks + weight_blocks)), kJoinThreads, 0, 1, stream, a, ctas,
                      per_block, rows, row_blocks);
}

}  // namespace ulysses
