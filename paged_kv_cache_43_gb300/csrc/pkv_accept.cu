// pkv_accept.cu -- what is kept of a batch's drafted tokens: the K and V rows of each
// sequence's accepted path move to the places right behind the keys that were there
// before the drafts, in every layer's caches at once.
//
// A sequence of L keys, the last n of them drafted, accepts the drafts path[0] < path[1] <
// ... < path[m - 1]: row L - n + path[j] becomes row L - n + j.  Since path[j] >= j, a
// row is overwritten only after it was moved, if one thread moves its 16 bytes of every
// row in the order of j; a batch of kRowsInFlight rows is loaded before the first of them is
// stored (a later batch's rows lie behind every place that an earlier one wrote).
//
// Bound by loads that wait for one another: lengths and path, then the tables' ids, then the rows, 8
// of them in flight (1 sequence in 32 buffers 3.7 us; 256 sequences of up to 8 accepted drafts in 32
// buffers 16.7 us, 83 MB read and written at 5.0 TB/s, much of it in L2: from a cold L2 20 us and
// 45 MB of HBM traffic, 2.2 TB/s, with 36 % of the issue slots used).  A CTA has 4 buffers, so that the
// path's lookups are gone once for them.
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kAcceptThreads = 256;
constexpr int kRowsInFlight = 8;
constexpr int kCtaBuffers = 4;   // buffers of a CTA, for which a path is looked up once
constexpr int kChunk = 64;       // drafts of a path looked up at a time

// Moves rows[u].x to rows[u].y, u < count (below zero: none), of buffers [b0, b0 + nb).
template <typename V>
__device__ __forceinline__ void move_rows(const AcceptArgs& a, int b0, int nb, const int2* rows,
                                          int count) {
  int cols[kCtaBuffers], total = 0;   // vectors of a row
#pragma unroll
  for (int i = 0; i < kCtaBuffers; ++i) {
    cols[i] = i < nb ? static_cast<int>(a.buffers[b0 + i].row_bytes / static_cast<int64_t>(sizeof(V))) : 0;
    total += cols[i];
  }
  for (int at = threadIdx.x; at < total; at += kAcceptThreads) {
    int col = at, i = 0;
#pragma unroll
    for (int k = 0; k + 1 < kCtaBuffers; ++k)
      if (i == k && col >= cols[k]) {
        col -= cols[k];
        ++i;
      }
    const AcceptBuffer& b = a.buffers[b0 + i];
    char* base = static_cast<char*>(b.base) + static_cast<int64_t>(col) * static_cast<int64_t>(sizeof(V));
    for (int j0 = 0; j0 < count; j0 += kRowsInFlight) {
      V v[kRowsInFlight];
      int to[kRowsInFlight];
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u) {
        const int2 r = j0 + u < count ? rows[j0 + u] : make_int2(-1, -1);
        to[u] = r.y;
        if (r.y >= 0) v[u] = *reinterpret_cast<const V*>(base + r.x * b.row_bytes);
      }
#pragma unroll
      for (int u = 0; u < kRowsInFlight; ++u)
        if (to[u] >= 0) *reinterpret_cast<V*>(base + to[u] * b.row_bytes) = v[u];
    }
  }
}

__global__ void __launch_bounds__(kAcceptThreads)
    pkv_accept_kernel(const __grid_constant__ AcceptArgs a) {
  __shared__ int2 rows[kChunk];
  const int s = blockIdx.x;
  const bool first_cta = a.report != 0 && blockIdx.y == 0;
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
  if (first_cta && threadIdx.x == 0) {
    if (a.new_lens != nullptr) a.new_lens[s] = bad != 0 ? L : L - n + count;
    if (bad != 0) raise_error(a.err, bad);
  }
  if (bad != 0 || a.num_buffers == 0) return;
  const int first = L - n, b0 = blockIdx.y * kCtaBuffers, nb = min(a.num_buffers - b0, kCtaBuffers);
  bool wide = true;
  for (int i = 0; i < nb; ++i)
    wide = wide && ((reinterpret_cast<uintptr_t>(a.buffers[b0 + i].base) | a.buffers[b0 + i].row_bytes) & 15) == 0;
  for (int c0 = 0; c0 < count; c0 += kChunk) {
    const int m = min(count - c0, kChunk);
    if (c0 > 0) __syncthreads();
    if (threadIdx.x < m) {
      const int j = c0 + threadIdx.x, p = __ldg(path + j);
      int2 r = make_int2(-1, -1);
      if (p != j) {
        const int x = __ldg(table + (first + p) / kBlock), y = __ldg(table + (first + j) / kBlock);
        if (x >= 0 && x < a.num_blocks && y >= 0 && y < a.num_blocks)
          r = make_int2(x * kBlock + (first + p) % kBlock, y * kBlock + (first + j) % kBlock);
        else if (first_cta)
          raise_error(a.err, PKV_ERR_BLOCK_ID);   // (the row stays)
      }
      rows[threadIdx.x] = r;
    }
    __syncthreads();
    if (wide) move_rows<uint4>(a, b0, nb, rows, m);
    else move_rows<uint32_t>(a, b0, nb, rows, m);
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t stream) {
  if (a.num_seqs == 0) return cudaSuccess;
  pkv_accept_kernel<<<dim3(a.num_seqs, a.num_buffers > kCtaBuffers ? (a.num_buffers + kCtaBuffers - 1) / kCtaBuffers : 1),
                      kAcceptThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
