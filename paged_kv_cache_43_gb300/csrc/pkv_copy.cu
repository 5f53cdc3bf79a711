// pkv_copy.cu -- copies whole pages (blocks) of many buffers at once: the
// device side of forking a sequence (its last, partly filled block) and of
// compacting a pool.
//
// A buffer is [num_blocks, page bytes]: a layer's K or V cache of any dtype,
// or its scales.  One launch carries up to kCopyPairs (from, to) pairs and
// kCopyBuffers buffers in its arguments (5.6 KB), so a call needs no copy of
// the pairs to the device first.  The launch is cut into units of about
// kCopyUnit bytes: a part of a page, or several pages where they are small
// (scales).  Bound by HBM: every byte read once and written once; the loads
// of a thread are all in flight before its first store.  512 pages of 16 int8
// layers with their scales, 538 MB moved: 84 us, 6.4 TB/s (256 pairs a launch,
// so two launches: 88 us; units of 32 KB: 95 us); 16 pages of one layer 2 us.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kCopyThreads = 256;

template <typename V>
__device__ __forceinline__ void copy_unit(const CopyArgs& a, const CopyBuffer& b, int64_t unit) {
  constexpr int kVec = sizeof(V);
  constexpr int kDepth = kCopyUnit / (kCopyThreads * 16);   // 16-byte loads per thread
  char* base = static_cast<char*>(b.base);
  if (b.split > 0) {   // a part of one page
    const int pair = static_cast<int>(unit / b.split);
    const int64_t begin = (unit - static_cast<int64_t>(pair) * b.split) * kCopyUnit;
    const int64_t len = min(static_cast<int64_t>(kCopyUnit), b.page_bytes - begin) / kVec;
    const V* src = reinterpret_cast<const V*>(base + a.pairs[pair].x * b.page_bytes + begin);
    V* dst = reinterpret_cast<V*>(base + a.pairs[pair].y * b.page_bytes + begin);
    for (int64_t i0 = threadIdx.x; i0 < len; i0 += kDepth * kCopyThreads) {
      V v[kDepth];
#pragma unroll
      for (int k = 0; k < kDepth; ++k)
        if (i0 + k * kCopyThreads < len) v[k] = __ldcs(src + i0 + k * kCopyThreads);
#pragma unroll
      for (int k = 0; k < kDepth; ++k)
        if (i0 + k * kCopyThreads < len) dst[i0 + k * kCopyThreads] = v[k];
    }
  } else {             // several small pages
    const int per_page = static_cast<int>(b.page_bytes / kVec);
    const int pair0 = static_cast<int>(unit) * -b.split;
    const int n = min(-b.split, a.num_pairs - pair0) * per_page;
    for (int i = threadIdx.x; i < n; i += kCopyThreads) {
      const int p = i / per_page, c = i - p * per_page;
      const V v = __ldcs(reinterpret_cast<const V*>(base + a.pairs[pair0 + p].x * b.page_bytes) + c);
      reinterpret_cast<V*>(base + a.pairs[pair0 + p].y * b.page_bytes)[c] = v;
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads)
    pkv_copy_blocks_kernel(const __grid_constant__ CopyArgs a) {
  // the buffer of this unit: the last one that begins at or before it
  int lo = 0, hi = a.num_buffers;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.buffers[mid].unit_begin <= blockIdx.x) lo = mid;
    else hi = mid;
  }
  const CopyBuffer& b = a.buffers[lo];
  const int64_t unit = blockIdx.x - b.unit_begin;
  if (((reinterpret_cast<uintptr_t>(b.base) | b.page_bytes) & 15) == 0) copy_unit<uint4>(a, b, unit);
  else copy_unit<uint32_t>(a, b, unit);
}

}  // namespace

cudaError_t launch_copy_blocks(const CopyArgs& a, unsigned units, cudaStream_t stream) {
  if (units == 0) return cudaSuccess;
  pkv_copy_blocks_kernel<<<units, kCopyThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
