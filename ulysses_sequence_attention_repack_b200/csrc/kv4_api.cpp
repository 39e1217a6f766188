// C ABI of the 4-bit K/V cache: argument checks and launches.  Declarations
// and argument contracts are in include/ulysses.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <new>

#include "api_util.h"
#include "internal.h"

using ulysses::aligned16;
using ulysses::NvtxRange;
using ulysses::overlap;
using ulysses::status_of;

namespace {

constexpr int32_t kHeadDim = 128;
constexpr int32_t kMaxBatch = 1024;
constexpr int32_t kMaxHeads = 1024;
constexpr int64_t kMaxPairs = 65535;                            // grid.y
constexpr int64_t kMaxSlots = (int64_t(1) << 31) - 4096;        // kernels number slots with int32
constexpr int64_t kMaxInt32 = std::numeric_limits<int32_t>::max();
constexpr int64_t kMaxElements = int64_t(1) << 48;              // strides and row counts beyond it are mistakes
constexpr int64_t kBlockSlots = 32, kBlockBytes = 4608;

int64_t slots(const ulysses_kv4_t* kv) { return static_cast<int64_t>(kv->B) * kv->H * kv->cap; }
int64_t blocks_bytes(const ulysses_kv4_t* kv) { return slots(kv) / kBlockSlots * kBlockBytes; }
int64_t cache_bytes(const ulysses_kv4_t* kv) { return blocks_bytes(kv) + 8 * slots(kv); }

int device_ready(const ulysses_kv4_t* kv) {
  if (!kv->dev_err) return ULYSSES_ERR_CUDA;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return ULYSSES_ERR_CUDA;
  }
  return dev == kv->device ? ULYSSES_OK : ULYSSES_ERR_ARG;
}

float* weights_of(const ulysses_kv4_t* kv, void* cache) {
  return reinterpret_cast<float*>(static_cast<uint8_t*>(cache) + blocks_bytes(kv));
}
int32_t* positions_of(const ulysses_kv4_t* kv, void* cache) {
  return reinterpret_cast<int32_t*>(static_cast<uint8_t*>(cache) + blocks_bytes(kv) + 4 * slots(kv));
}

// Checks of the bf16 K and V rows of an append (write = false) or a load.
int check_rows(const ulysses_kv4_t* kv, const void* cache, const void* k, const void* v, int64_t rows,
               int64_t token_stride, int64_t head_stride, int64_t rank_stride, int32_t heads_per_rank,
               const void* cu, const void* start, bool write) {
  if (!kv || !cache || !k || !v || !cu || !start || rows < 0) return ULYSSES_ERR_ARG;
  if (heads_per_rank < 1 || kv->H % heads_per_rank != 0) return ULYSSES_ERR_DIVISIBILITY;
  if (token_stride < 0 || head_stride < 0 || rank_stride < 0) return ULYSSES_ERR_ARG;
  if (rows > kMaxSlots) return ULYSSES_ERR_UNSUPPORTED;
  const int64_t ranks = kv->H / heads_per_rank;
  if (token_stride > kMaxElements / std::max<int64_t>(rows, 1) || head_stride > kMaxElements / heads_per_rank ||
      rank_stride > kMaxElements / ranks)
    return ULYSSES_ERR_ARG;
  if (token_stride % 8 || head_stride % 8 || rank_stride % 8) return ULYSSES_ERR_ALIGN;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v)) return ULYSSES_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(cu) | reinterpret_cast<uintptr_t>(start)) & 3u) return ULYSSES_ERR_ALIGN;
  if (rows == 0) return ULYSSES_OK;
  const int64_t span = ((rows - 1) * token_stride + (heads_per_rank - 1) * head_stride + (ranks - 1) * rank_stride +
                        kHeadDim) * 2;
  if (overlap(k, span, cache, cache_bytes(kv)) || overlap(v, span, cache, cache_bytes(kv))) return ULYSSES_ERR_ARG;
  if (write) {
    // No two destination rows may share an element.  The rows form a lattice
    // of up to four (stride, count) steps -- the planes' distance is one where
    // K and V interleave -- and are apart when, by rising stride, each stride
    // passes the extent of the steps inside it.
    const uintptr_t x = reinterpret_cast<uintptr_t>(k), y = reinterpret_cast<uintptr_t>(v);
    struct Step {
      int64_t stride, count;
    } s[4] = {{head_stride, heads_per_rank}, {token_stride, rows}, {rank_stride, ranks}, {0, 1}};
    if (overlap(k, span, v, span)) s[3] = {static_cast<int64_t>((x < y ? y - x : x - y) / 2), 2};
    std::sort(s, s + 4, [](const Step& a, const Step& b) { return a.stride < b.stride; });
    int64_t extent = kHeadDim;
    for (const Step& d : s) {
      if (d.count == 1) continue;
      if (d.stride < extent) return ULYSSES_ERR_ARG;
      extent += (d.count - 1) * d.stride;
    }
    const int64_t idx = static_cast<int64_t>(kv->B) * 4;
    if (overlap(cu, idx + 4, k, span) || overlap(cu, idx + 4, v, span) || overlap(start, idx, k, span) ||
        overlap(start, idx, v, span))
      return ULYSSES_ERR_ARG;
  }
  return ULYSSES_OK;
}

ulysses::Kv4RowsLaunch rows_launch(const ulysses_kv4_t* kv, void* cache, void* k, void* v, int64_t rows,
                                   int64_t token_stride, int64_t head_stride, int64_t rank_stride,
                                   int32_t heads_per_rank, const int32_t* cu, const int32_t* start,
                                   const int32_t* pos0) {
  ulysses::Kv4RowsLaunch a;
  a.r = {k, v, rows, token_stride, head_stride, rank_stride, heads_per_rank, cu, start, pos0};
  a.B = kv->B;
  a.H = kv->H;
  a.cap = kv->cap;
  a.cache = static_cast<uint8_t*>(cache);
  a.weight = weights_of(kv, cache);
  a.pos = positions_of(kv, cache);
  a.blocks_bytes = blocks_bytes(kv);
  a.err = kv->dev_err;
  return a;
}

}  // namespace

extern "C" {

int ulysses_kv4_plan(ulysses_kv4_t** out, int32_t batch, int32_t heads, int32_t D, int64_t capacity) {
  if (!out) return ULYSSES_ERR_ARG;
  *out = nullptr;
  if (D != kHeadDim) return ULYSSES_ERR_UNSUPPORTED;
  if (batch < 1 || heads < 1 || capacity < 1) return ULYSSES_ERR_ARG;
  if (capacity % kBlockSlots) return ULYSSES_ERR_ALIGN;
  if (batch > kMaxBatch || heads > kMaxHeads || static_cast<int64_t>(batch) * heads > kMaxPairs ||
      capacity > kMaxSlots)
    return ULYSSES_ERR_UNSUPPORTED;
  ulysses_kv4_t* kv = new (std::nothrow) ulysses_kv4_t;
  if (!kv) return ULYSSES_ERR_ARG;
  kv->B = batch;
  kv->H = heads;
  kv->cap = capacity;
  kv->device = -1;
  kv->dev_err = nullptr;
  int dev = -1;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    void* e = nullptr;
    if (cudaMalloc(&e, 16) == cudaSuccess) {
      if (cudaMemset(e, 0, 16) == cudaSuccess) {
        kv->dev_err = static_cast<unsigned int*>(e);
        kv->device = dev;
      } else {
        cudaFree(e);
      }
    }
  }
  cudaGetLastError();   // a missing device is not an error of plan creation
  *out = kv;
  return ULYSSES_OK;
}

void ulysses_kv4_plan_destroy(ulysses_kv4_t* kv) {
  if (!kv) return;
  if (kv->dev_err) {
    int cur = -1;
    cudaGetDevice(&cur);
    if (cur != kv->device) cudaSetDevice(kv->device);
    cudaFree(kv->dev_err);
    if (cur >= 0 && cur != kv->device) cudaSetDevice(cur);
    cudaGetLastError();
  }
  delete kv;
}

size_t ulysses_kv4_cache_bytes(const ulysses_kv4_t* kv) { return kv ? static_cast<size_t>(cache_bytes(kv)) : 0; }

size_t ulysses_kv4_weight_offset(const ulysses_kv4_t* kv) { return kv ? static_cast<size_t>(blocks_bytes(kv)) : 0; }

size_t ulysses_kv4_position_offset(const ulysses_kv4_t* kv) {
  return kv ? static_cast<size_t>(blocks_bytes(kv) + 4 * slots(kv)) : 0;
}

int ulysses_kv4_append(const ulysses_kv4_t* kv, void* cache, const void* k, const void* v, int64_t rows,
                       int64_t token_stride, int64_t head_stride, int64_t rank_stride, int32_t heads_per_rank,
                       const int32_t* dev_cu, const int32_t* dev_start, const int32_t* dev_pos0, void* stream) {
  NvtxRange range("ulysses_kv4_append");
  int s = check_rows(kv, cache, k, v, rows, token_stride, head_stride, rank_stride, heads_per_rank, dev_cu, dev_start,
                     false);
  if (s != ULYSSES_OK) return s;
  if (reinterpret_cast<uintptr_t>(dev_pos0) & 3u) return ULYSSES_ERR_ALIGN;
  const int64_t idx = static_cast<int64_t>(kv->B) * 4;
  if (overlap(dev_cu, idx + 4, cache, cache_bytes(kv)) || overlap(dev_start, idx, cache, cache_bytes(kv)) ||
      (dev_pos0 && overlap(dev_pos0, idx, cache, cache_bytes(kv))))
    return ULYSSES_ERR_ARG;
  if ((s = device_ready(kv)) != ULYSSES_OK) return s;
  return status_of(ulysses::launch_kv4_rows(
      false,
      rows_launch(kv, cache, const_cast<void*>(k), const_cast<void*>(v), rows, token_stride, head_stride, rank_stride,
                  heads_per_rank, dev_cu, dev_start, dev_pos0),
      static_cast<cudaStream_t>(stream)));
}

int ulysses_kv4_load(const ulysses_kv4_t* kv, const void* cache, void* k, void* v, int64_t rows, int64_t token_stride,
                     int64_t head_stride, int64_t rank_stride, int32_t heads_per_rank, const int32_t* dev_cu,
                     const int32_t* dev_start, void* stream) {
  NvtxRange range("ulysses_kv4_load");
  int s = check_rows(kv, cache, k, v, rows, token_stride, head_stride, rank_stride, heads_per_rank, dev_cu, dev_start,
                     true);
  if (s != ULYSSES_OK) return s;
  if ((s = device_ready(kv)) != ULYSSES_OK) return s;
  return status_of(ulysses::launch_kv4_rows(true,
                                            rows_launch(kv, const_cast<void*>(cache), k, v, rows, token_stride,
                                                        head_stride, rank_stride, heads_per_rank, dev_cu, dev_start,
                                                        nullptr),
                                            static_cast<cudaStream_t>(stream)));
}

// Whether an attention call of this shape can be numbered by the kernels.
static int check_attn_shape(const ulysses_kv4_t* kv, int32_t q_heads, int32_t q_len) {
  if (!kv || q_heads < 1 || q_len < 1) return ULYSSES_ERR_ARG;
  if (q_heads % kv->H != 0) return ULYSSES_ERR_DIVISIBILITY;
  const int64_t pairs = static_cast<int64_t>(kv->B) * kv->H;
  const int64_t R = static_cast<int64_t>(q_heads / kv->H) * q_len;
  if (R > kMaxInt32 / pairs) return ULYSSES_ERR_UNSUPPORTED;
  const int64_t tiles = (kv->cap + 127) / 128 * pairs;   // < 2^24 * 2^16
  if (tiles > kMaxInt32 / 2 / ((R + 7) / 8)) return ULYSSES_ERR_UNSUPPORTED;
  return ULYSSES_OK;
}

size_t ulysses_kv4_attn_workspace_bytes(const ulysses_kv4_t* kv, int32_t q_heads, int32_t q_len, uint32_t flags) {
  if (check_attn_shape(kv, q_heads, q_len) != ULYSSES_OK) return 0;
  return static_cast<size_t>(ulysses::kv4_attn_workspace_bytes(kv->B, kv->H, q_heads / kv->H, q_len, kv->cap,
                                                               (flags & ULYSSES_KV4_WEIGHTS) != 0));
}

int ulysses_kv4_attn(const ulysses_kv4_t* kv, void* cache, const void* q, int32_t q_heads, int32_t q_len,
                     int64_t q_token_stride, int64_t q_head_stride, void* out, void* lse, const int32_t* dev_lengths,
                     float softmax_scale, uint32_t flags, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("ulysses_kv4_attn");
  if (!kv || !cache || !q || !out || !dev_lengths) return ULYSSES_ERR_ARG;
  if (flags & ~(ULYSSES_KV4_CAUSAL | ULYSSES_KV4_WEIGHTS)) return ULYSSES_ERR_ARG;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return ULYSSES_ERR_ARG;
  int s = check_attn_shape(kv, q_heads, q_len);
  if (s != ULYSSES_OK) return s;
  const int64_t q_rows = static_cast<int64_t>(kv->B) * q_len;
  if (q_token_stride < 0 || q_head_stride < 0 || q_token_stride > kMaxElements / q_rows ||
      q_head_stride > kMaxElements / q_heads)
    return ULYSSES_ERR_ARG;
  if (q_token_stride % 8 || q_head_stride % 8) return ULYSSES_ERR_ALIGN;
  if (!aligned16(cache) || !aligned16(q) || !aligned16(out) || !aligned16(workspace)) return ULYSSES_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(dev_lengths)) & 3u) return ULYSSES_ERR_ALIGN;
  const size_t need = ulysses_kv4_attn_workspace_bytes(kv, q_heads, q_len, flags);
  if (!workspace || workspace_bytes < need) return ULYSSES_ERR_WORKSPACE;
  struct Range {
    const void* p;
    int64_t n;
    bool written;
  } r[] = {{cache, cache_bytes(kv), (flags & ULYSSES_KV4_WEIGHTS) != 0},
           {q, ((q_rows - 1) * q_token_stride + (q_heads - 1) * q_head_stride + kHeadDim) * 2, false},
           {out, q_rows * q_heads * kHeadDim * 2, true},
           {lse, q_rows * q_heads * 4, true},
           {dev_lengths, static_cast<int64_t>(kv->B) * 4, false},
           {workspace, static_cast<int64_t>(need), true}};
  for (int i = 0; i < 6; ++i)
    for (int j = 0; j < i; ++j)
      if (r[i].p && r[j].p && (r[i].written || r[j].written) && overlap(r[i].p, r[i].n, r[j].p, r[j].n))
        return ULYSSES_ERR_ARG;
  if ((s = device_ready(kv)) != ULYSSES_OK) return s;
  ulysses::Kv4AttnLaunch a;
  a.B = kv->B;
  a.H = kv->H;
  a.G = q_heads / kv->H;
  a.Lq = q_len;
  a.cap = kv->cap;
  a.cache = static_cast<const uint8_t*>(cache);
  a.weight = (flags & ULYSSES_KV4_WEIGHTS) ? weights_of(kv, cache) : nullptr;
  a.q = q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.out = out;
  a.lse = static_cast<float*>(lse);
  a.lengths = dev_lengths;
  a.scale = softmax_scale;
  a.causal = (flags & ULYSSES_KV4_CAUSAL) ? 1 : 0;
  a.workspace = static_cast<uint8_t*>(workspace);
  a.err = kv->dev_err;
  return status_of(ulysses::launch_kv4_attn(a, static_cast<cudaStream_t>(stream)));
}

int ulysses_kv4_evict(const ulysses_kv4_t* src_kv, const void* src_cache, const ulysses_kv4_t* dst_kv, void* dst_cache,
                      const int32_t* dev_lengths, int32_t* dev_new_lengths, int32_t keep, int32_t sink, int32_t recent,
                      void* stream) {
  NvtxRange range("ulysses_kv4_evict");
  if (!src_kv || !dst_kv || !src_cache || !dst_cache || !dev_lengths || !dev_new_lengths) return ULYSSES_ERR_ARG;
  if (src_kv->B != dst_kv->B || src_kv->H != dst_kv->H) return ULYSSES_ERR_ARG;
  if (keep < 1 || keep > dst_kv->cap || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > keep)
    return ULYSSES_ERR_ARG;
  if (!aligned16(src_cache) || !aligned16(dst_cache)) return ULYSSES_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(dev_lengths) | reinterpret_cast<uintptr_t>(dev_new_lengths)) & 3u)
    return ULYSSES_ERR_ALIGN;
  const int64_t idx = static_cast<int64_t>(src_kv->B) * 4;
  if (overlap(src_cache, cache_bytes(src_kv), dst_cache, cache_bytes(dst_kv)) ||
      overlap(dev_lengths, idx, dev_new_lengths, idx) || overlap(dev_lengths, idx, dst_cache, cache_bytes(dst_kv)) ||
      overlap(dev_new_lengths, idx, dst_cache, cache_bytes(dst_kv)) ||
      overlap(dev_new_lengths, idx, src_cache, cache_bytes(src_kv)))
    return ULYSSES_ERR_ARG;
  int s = device_ready(src_kv);
  if (s == ULYSSES_OK) s = device_ready(dst_kv);
  if (s != ULYSSES_OK) return s;
  ulysses::Kv4EvictLaunch a;
  a.B = src_kv->B;
  a.H = src_kv->H;
  a.src_cap = src_kv->cap;
  a.dst_cap = dst_kv->cap;
  void* src = const_cast<void*>(src_cache);
  a.src = static_cast<const uint8_t*>(src_cache);
  a.src_weight = weights_of(src_kv, src);
  a.src_pos = positions_of(src_kv, src);
  a.dst = static_cast<uint8_t*>(dst_cache);
  a.dst_weight = weights_of(dst_kv, dst_cache);
  a.dst_pos = positions_of(dst_kv, dst_cache);
  a.lengths = dev_lengths;
  a.new_lengths = dev_new_lengths;
  a.keep = keep;
  a.sink = sink;
  a.recent = recent;
  a.err = src_kv->dev_err;
  return status_of(ulysses::launch_kv4_evict(a, static_cast<cudaStream_t>(stream)));
}

int ulysses_kv4_last_device_error(const ulysses_kv4_t* kv, void* stream) {
  if (!kv || !kv->dev_err) return -1;
  unsigned int v = 0;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(&v, kv->dev_err, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess ||
      (v != 0 && cudaMemset(kv->dev_err, 0, sizeof(v)) != cudaSuccess)) {
    cudaGetLastError();
    return -1;
  }
  return static_cast<int>(v);
}

}  // extern "C"
