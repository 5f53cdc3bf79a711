// pkv_tree.cuh -- what the tree-attention kernels share: a sequence's checks and the
// bits of a query row's mask.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

struct TreeSeq {
  int q0, n, L;      // first query row, drafted rows, keys with them
  int first;         // the first drafted key: keys before it are seen by every row
  int32_t err;       // what is wrong (PKV_ERR_* bits, 0: nothing)
  bool skip;         // nothing to do, nothing to write
};

// n > 0 and err != 0 without skip: the sequence's rows are zeroed.
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int s) {
  TreeSeq q;
  q.L = __ldg(a.context_lens + s);
  q.q0 = __ldg(a.query_start_loc + s);
  q.n = __ldg(a.query_start_loc + s + 1) - q.q0;
  q.first = q.L - q.n;
  q.err = 0;
  q.skip = q.n == 0;
  if (q.n < 0 || q.q0 < 0 || static_cast<int64_t>(q.q0) + q.n > a.num_tokens) {
    q.err = PKV_ERR_QUERY_LEN;
    q.skip = true;
  } else if (q.n > 0) {
    if (q.L < 1 || static_cast<int64_t>(q.L) > a.bt_stride * kBlock || q.L > a.max_context_len)
      q.err = PKV_ERR_CONTEXT_LEN;
    else if (q.n > q.L || q.n > a.max_query_len) q.err = PKV_ERR_QUERY_LEN;
  }
  return q;
}

// The sequence that computes query row t, -1: none; a whole warp together.  query_start_loc ascends
// unless some sequence's entry is bad, and the search for t may end at such a one: then all
// sequences are looked at, as those that are right are not to suffer.
__device__ __forceinline__ int tree_seq_of_row(const TreeArgs& a, int t, TreeSeq& q) {
  const int lane = threadIdx.x & 31;
  int s = seq_of_row(a.query_start_loc, a.num_seqs, t);
  if (s >= 0) {
    q = tree_seq(a, s);
    if (!q.skip && q.err == 0) return s;
  }
  for (int at = 0; at < a.num_seqs; at += 32) {
    q = tree_seq(a, min(at + lane, a.num_seqs - 1));
    const uint32_t has = __ballot_sync(0xffffffffu, !q.skip && q.err == 0 && t >= q.q0 && t < q.q0 + q.n);
    if (has == 0) continue;
    s = min(at + __ffs(has) - 1, a.num_seqs - 1);
    q = tree_seq(a, s);
    return s;
  }
  return -1;
}

// Bits of the keys [key0, key0 + 64) that the row whose mask words are `mask` sees: every
// key before the sequence's first draft, and the drafts whose bits are set.
__device__ __forceinline__ uint64_t tree_bits(const uint64_t* mask, const TreeSeq& q, int key0) {
  const int j0 = key0 - q.first;             // draft of the first key
  if (j0 <= -64) return ~0ull;
  if (j0 >= q.n) return 0ull;
  uint64_t bits;
  if (j0 < 0) {
    bits = ((1ull << -j0) - 1) | (__ldg(mask) << -j0);
  } else {
    const int w = j0 >> 6, sh = j0 & 63;
    bits = __ldg(mask + w) >> sh;
    if (sh != 0 && (w + 1) * 64 < q.n) bits |= __ldg(mask + w + 1) << (64 - sh);
  }
  const int left = q.n - j0;                 // keys of the sequence from key0 on
  return left < 64 ? bits & ((1ull << left) - 1) : bits;
}

}  // namespace pkv
