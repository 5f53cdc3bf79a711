// pkv_accept.cu -- what is kept of a batch's drafted tokens: the K and V rows of each
// sequence's accepted path move to the places right behind the keys that were there
// before the drafts, in every layer's caches at once.
//
// A sequence of L keys, the last n of them drafted, accepts the drafts path[0] < path[1] <
// ... < path[m - 1]: row L - n + path[j] becomes row L - n + j.  Since path[j] >= j, a
// row is overwritten only after it was moved, if one thread moves its 16 bytes of every
// row in the order of j; a batch of kRowsInFlight rows is loaded before the first of them is
// stored (a later batch's rows lie behind every place that an earlier one wrote).
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kAcceptThreads = 128;
constexpr int kRowsInFlight = 8;

template <typename V>
__device__ __forceinline__ void move_rows(const AcceptArgs& a, const AcceptBuffer& b,
                                          const int32_t* path, const int32_t* table, int first,
                                          int count) {
  char* base = static_cast<char*>(b.base);
  const int64_t cols = b.row_bytes / static_cast<int64_t>(sizeof(V));
  auto row_at = [&](int p) -> char* {
    const int block = __ldg(table + p / kBlock);
    return block >= 0 && block < a.num_blocks
               ? base + (static_cast<int64_t>(block) * kBlock + p % kBlock) * b.row_bytes : nullptr;
  };
  for (int64_t col = threadIdx.x; col < cols; col += kAcceptThreads) {
    for (int j0 = 0; j0 < count; j0 += kRowsInFlight) {
      V v[kRowsInFlight];
      char* to[kRowsInFlight];
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u) {
        to[u] = nullptr;
        const int j = j0 + u;
        if (j >= count) continue;
        const int p = __ldg(path + j);
        if (p == j) continue;
        const char* from = row_at(first + p);
        char* dst = row_at(first + j);
        if (from == nullptr || dst == nullptr) continue;   // (a bad block id: the row stays)
        v[u] = *(reinterpret_cast<const V*>(from) + col);
        to[u] = dst;
      }
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u)
        if (to[u] != nullptr) *(reinterpret_cast<V*>(to[u]) + col) = v[u];
    }
  }
}

__global__ void __launch_bounds__(kAcceptThreads)
    pkv_accept_kernel(const __grid_constant__ AcceptArgs a) {
  const int s = blockIdx.x;
  const AcceptBuffer& b = a.buffers[blockIdx.y];
  const bool reporter = a.report != 0 && blockIdx.y == 0 && threadIdx.x == 0;
  const int L = __ldg(a.context_lens + s);
  const int n = __ldg(a.query_start_loc + s + 1) - __ldg(a.query_start_loc + s);
  const int count = __ldg(a.num_accepted + s);
  const int32_t* path = a.accepted + static_cast<int64_t>(s) * a.max_accepted;
  const int32_t* table = a.block_tables + s * a.bt_stride;
  int32_t bad = 0;
  if (n < 0 || n > L) bad = PKV_ERR_QUERY_LEN;
  else if (static_cast<int64_t>(L) > a.bt_stride * kBlock) bad = PKV_ERR_CONTEXT_LEN;
  else if (count < 0 || count > n || count > a.max_accepted) bad = PKV_ERR_ACCEPTED;
  else {
    // a rising path inside the drafts (each thread looks at some of it)
    bool fine = true;
    for (int j = threadIdx.x; j < count; j += kAcceptThreads) {
      const int p = __ldg(path + j);
      fine = fine && p >= 0 && p < n && (j == 0 || __ldg(path + j - 1) < p);
    }
    if (!__syncthreads_and(fine)) bad = PKV_ERR_ACCEPTED;
  }
  if (reporter && a.new_lens != nullptr) a.new_lens[s] = bad != 0 ? L : L - n + count;
  if (bad != 0) {
    if (reporter) raise_error(a.err, bad);
    return;
  }
  if (a.num_buffers == 0) return;   // (the lengths alone)
  const int first = L - n;
  if (reporter) {
    for (int j = 0; j < count; ++j) {
      const int p = __ldg(path + j);
      const int x = __ldg(table + (first + p) / kBlock), y = __ldg(table + (first + j) / kBlock);
      if (p != j && (x < 0 || x >= a.num_blocks || y < 0 || y >= a.num_blocks))
        raise_error(a.err, PKV_ERR_BLOCK_ID);
    }
  }
  if (((reinterpret_cast<uintptr_t>(b.base) | b.row_bytes) & 15) == 0)
    move_rows<uint4>(a, b, path, table, first, count);
  else
    move_rows<uint32_t>(a, b, path, table, first, count);
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0) return cudaSuccess;
  pkv_accept_kernel<<<dim3(a.num_seqs, a.num_buffers > 0 ? a.num_buffers : 1), kAcceptThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
