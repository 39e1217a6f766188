// The 4-bit K/V cache: layout and device helpers shared by its kernels.
//
// A (sequence, head) pair has `capacity` slots in blocks of 32; a block is
// 4608 contiguous bytes:
//
//   [0, 2048)      K codes, 64 bytes a slot
//   [2048, 4096)   V codes, 64 bytes a slot
//   [4096, 4608)   32 x 8 bf16: ks0, km0, ks1, km1, vs0, vm0, vs1, vm1
//
// so one block is one bulk copy, and what a slot holds never straddles a
// 16-byte boundary.  A row of 128 values is two groups of 64 (group w holds
// d = 64 w .. 64 w + 63); in a group
//
//   x ~ m + s n,   m = min x,   s = bf16((max x - min x) / 15),
//   n = round((x - m) / s) in 0..15 (0 where s = 0)
//
// with m and s in bf16: m is one of the row's bf16 values, so it is held
// exactly, and s has the range of the values whatever their size.  A group
// whose spread is not finite is held as s = m = NaN.
//
// The 64 bytes of a row are eight 8-byte chunks; chunk g is the 32-bit word of
// dims 8g .. 8g + 7, then that of dims 64 + 8g .. 64 + 8g + 7, and nibble j of
// a word is dim j of its eight.  With this order the lanes of a warp read the
// fragments of a 16 x 8 x 16 product straight from 16-byte (K) and 8-byte (V)
// loads, and every product stays inside one group.
//
// After the blocks of all pairs: accumulated weights fp32 [batch, heads,
// capacity], token positions int32 [batch, heads, capacity].
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ulysses {

constexpr int kKv4BlockSlots = 32;
constexpr int kKv4BlockBytes = 4608;
constexpr int kKv4VOffset = 2048;
constexpr int kKv4MetaOffset = 4096;
constexpr int kKv4Dim = 128;

// Bit set in the device error word: a length, a start or a slot outside the cache.
enum : uint32_t { kErrCacheIndex = 16u };

// Byte offset of slot `slot` of pair bh (its K row is at +64 * (slot % 32)).
__device__ __forceinline__ int64_t kv4_block_offset(int64_t bh, int64_t capacity, int64_t slot) {
  return (bh * (capacity / kKv4BlockSlots) + slot / kKv4BlockSlots) * kKv4BlockBytes;
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Wait for, and allow, the programmatic launch of the next kernel on the
// stream: a kernel launched with the stream-serialization attribute may start
// before its predecessor has ended and must not touch the predecessor's
// results before pdl_wait().
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches a kernel that may start before its predecessor on the stream has
// ended (it calls pdl_wait before it touches global memory), in clusters of
// `cluster` blocks.  Clusters do not start early: whole SMs of waiting blocks
// cost the predecessor more than the early start gains (eviction of 104,448
// slots x 56 heads: 92 us with it, 77 without).
template <class... P, class... V>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int64_t smem, int cluster, cudaStream_t stream,
                         V... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = static_cast<size_t>(smem);
  c.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = cluster > 1 ? 0 : 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  c.attrs = at;
  c.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// The current device and its SMs (asked for once a device: the call is on the
// way of every launch).
inline cudaError_t current_device_sms(int* dev, int* sms) {
  static std::atomic<int> known[64] = {};
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  const bool tracked = *dev >= 0 && *dev < 64;
  *sms = tracked ? known[*dev].load(std::memory_order_relaxed) : 0;
  if (*sms > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
  if (e == cudaSuccess && tracked) known[*dev].store(*sms, std::memory_order_relaxed);
  return e;
}

// A device-side length, held inside 0 .. capacity (and reported if it was not).
__device__ __forceinline__ int kv4_length(int n, int64_t capacity, unsigned int* err) {
  if (n < 0 || n > capacity) {
    if (err) atomicOr(err, kErrCacheIndex);
    return n < 0 ? 0 : static_cast<int>(capacity);
  }
  return n;
}

}  // namespace ulysses
