// pkv_tree.cu -- attention of a tree of drafted tokens over the paged cache: the fp32
// kernel, and the merge of split keys.
//
// Mathematics.  A sequence has L keys, the last n of them its drafted tokens, and n query
// rows.  Row i sees every key before the drafts, and draft j where bit j of its mask is
// set; out = sum_p w_p V_p / sum_p w_p, w_p = 2^(scale log2(e) (q . k_p) - m), m the running
// maximum, a row that sees no key is zero.  Keys are cut into splits; a split writes O_i =
// (sum w V) / (sum w) and lse_i = m + log2(sum w), and the merge forms
// sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M).
//
// The fp32 kernel: a CTA has 32 rows (drafted token, q head of one kv head), walks its
// split 32 keys at a time, K and V in shared memory, scores on CUDA cores (fp32 scores
// cannot go through the tensor core's types at the accuracy that fp32 is held to).  It is
// bound by its multiplications out of shared memory (8 sequences of 16 drafts over 2000 keys, 32 / 8 heads of
// 128: 539 us, 136 MB of keys, the shared-memory pipe 56 % busy, the issue slots 26 %): as the first kernel
// for every type it took 4478 us where the bf16 kernel of pkv_tree_tc.cu takes 66 (8 sequences of 64
// drafts over 2K to 8K keys).
#include "pkv_tree.cuh"

namespace pkv {

namespace {

constexpr int kRows = 32, kKeys = 32, kThreads = 128;

// The row of the partials of query row t, head hq.
__device__ __forceinline__ int64_t tree_partial(const TreeArgs& a, int64_t t, int hq, int split) {
  return (t * a.num_q_heads + hq) * a.max_splits + split;
}

// Splits that a sequence's keys are cut into.
__device__ __forceinline__ int tree_splits(const TreeArgs& a, int L) {
  return ((L + kBlock - 1) / kBlock + a.split_blocks - 1) / a.split_blocks;
}

template <int D>
__global__ void __launch_bounds__(kThreads) pkv_tree_kernel(const TreeArgs a) {
  constexpr int LD = D + 4;
  extern __shared__ float sm[];
  float* sQ = sm;                        // [kRows][LD]
  float* sK = sQ + kRows * LD;           // [kKeys][LD]
  float* sV = sK + kKeys * LD;           // [kKeys][LD]
  float* sP = sV + kKeys * LD;           // [kRows][kKeys + 1]
  const int s = blockIdx.z, kvh = blockIdx.y % a.num_kv_heads, tile = blockIdx.y / a.num_kv_heads;
  const int split = blockIdx.x, G = a.group, Hq = a.num_q_heads;
  const TreeSeq q = tree_seq(a, s);
  const bool reporter = split == 0 && blockIdx.y == 0 && threadIdx.x == 0;
  if (q.err != 0 && reporter) raise_error(a.err, q.err);
  const int row0 = tile * kRows;   // (more drafts than the stated most: the first are zeroed)
  const int rows = min(min(q.n, a.max_query_len) * G - row0, kRows);
  if (q.skip || rows <= 0) return;
  float* out = static_cast<float*>(a.out);
  auto at = [&](int r) {   // row r of the tile in q and out
    return (static_cast<int64_t>(q.q0 + (row0 + r) / G) * Hq + kvh * G + (row0 + r) % G) * D;
  };
  if (q.err != 0) {
    if (split == 0)
      for (int i = threadIdx.x; i < rows * D; i += kThreads) out[at(i / D) + i % D] = 0.f;
    return;
  }
  const int nsplit = tree_splits(a, q.L);
  if (split >= nsplit) return;
  const int key_begin = split * a.split_blocks * kBlock;
  const int key_end = min(q.L, key_begin + a.split_blocks * kBlock);
  for (int i = threadIdx.x; i < kRows * D; i += kThreads)
    sQ[i / D * LD + i % D] =
        i / D < rows ? __ldg(static_cast<const float*>(a.q) + at(i / D) + i % D) : 0.f;

  // scores: thread = row of 4 neighbours, 8 keys 4 apart; output: the same row, D / 4 elements
  const int row = threadIdx.x / 4, part = threadIdx.x % 4;
  const uint64_t* mask = a.tree_mask +
      static_cast<int64_t>(q.q0 + (row0 + min(row, rows - 1)) / G) * a.mask_words;
  float o[D / 4];
#pragma unroll
  for (int i = 0; i < D / 4; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  const int32_t* bt = a.block_tables + s * a.bt_stride;
  for (int k0 = key_begin; k0 < key_end; k0 += kKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * D; i += kThreads) {
      const int p = k0 + i / D;
      float k = 0.f, v = 0.f;
      if (p < key_end) {
        const int b = __ldg(bt + p / kBlock);
        if (b >= 0 && b < a.num_blocks) {
          const int64_t src = ((static_cast<int64_t>(b) * kBlock + p % kBlock) * a.num_kv_heads + kvh) * D + i % D;
          k = __ldg(static_cast<const float*>(a.k_cache) + src);
          v = __ldg(static_cast<const float*>(a.v_cache) + src);
        } else if (i % D == 0) {
          raise_error(a.err, PKV_ERR_BLOCK_ID);
        }
      }
      sK[i / D * LD + i % D] = k;
      sV[i / D * LD + i % D] = v;
    }
    __syncthreads();
    // bits of these 32 keys (the tree's bits come by 64)
    const uint64_t bits = tree_bits(mask, q, k0);
    float x[kKeys / 4], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kKeys / 4; ++j) {
      const int c = part + 4 * j;
      float dot = 0.f;
#pragma unroll 8
      for (int d = 0; d < D; d += 4) {
        const float4 u = *reinterpret_cast<const float4*>(sQ + row * LD + d);
        const float4 w = *reinterpret_cast<const float4*>(sK + c * LD + d);
        dot = fmaf(u.x, w.x, fmaf(u.y, w.y, fmaf(u.z, w.z, fmaf(u.w, w.w, dot))));
      }
      x[j] = k0 + c < key_end && (bits >> c & 1) ? dot * a.scale_log2 : -INFINITY;
      top = fmaxf(top, x[j]);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float mn = fmaxf(m, top), mu = mn == -INFINITY ? 0.f : mn;
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - mn);
    m = mn;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kKeys / 4; ++j) {
      const int c = part + 4 * j;
      const bool seen = k0 + c < key_end && (bits >> c & 1);
      const float w = exp2f(x[j] - mu);
      // (a key that the row does not see is marked, so that whatever its V holds stays out)
      sP[row * (kKeys + 1) + c] = seen ? w : -1.f;
      sum += seen ? w : 0.f;
    }
    l = l * alpha + sum;
    __syncwarp();   // (a row's weights are written and read by four neighbours)
#pragma unroll
    for (int i = 0; i < D / 4; ++i) o[i] *= alpha;
    for (int c = 0; c < kKeys; ++c) {
      const float w = sP[row * (kKeys + 1) + c];
      if (w < 0.f) continue;   // (a NaN is a weight)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(sV + c * LD + 16 * i + 4 * part);
        o[4 * i] = fmaf(w, v.x, o[4 * i]);
        o[4 * i + 1] = fmaf(w, v.y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(w, v.z, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(w, v.w, o[4 * i + 3]);
      }
    }
  }
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (row >= rows) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t dst = at(row);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 16 * i + 4 * part + e;
      const float r = o[4 * i + e] * inv;
      if (nsplit == 1) {
        out[dst + d] = r;
      } else {
        const int64_t w = tree_partial(a, q.q0 + (row0 + row) / G, kvh * G + (row0 + row) % G, split);
        a.ws_o[w * D + d] = r;
        if (d == 0) a.ws_lse[w] = l == 0.f ? -INFINITY : m + log2f(l);
      }
    }
}

// One warp per (query row, q head) of a sequence with several splits.
template <int D>
__global__ void __launch_bounds__(128) pkv_tree_merge_kernel(const TreeArgs a) {
  constexpr int PER = D / 32;
  constexpr int kUnroll = 8;   // partials in flight
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = w / a.num_q_heads;
  if (t >= a.num_tokens) return;
  TreeSeq q;
  const int s = tree_seq_of_row(a, static_cast<int>(t), q);
  if (s < 0) return;   // a row of no sequence, or of a bad one
  const int nsplit = tree_splits(a, q.L);
  if (nsplit <= 1) return;
  const int64_t row = w * a.max_splits;
  const float* lse = a.ws_lse + row;
  float M = -INFINITY;
  bool nan = false;
  for (int i = lane; i < nsplit; i += 32) {
    M = fmaxf(M, lse[i]);
    nan = nan || lse[i] != lse[i];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if (__any_sync(0xffffffffu, nan)) M = NAN;
  float acc[PER] = {}, den = 0.f;
  if (M != -INFINITY) {
    const float* o = a.ws_o + row * D + lane * PER;
    for (int i0 = 0; i0 < nsplit; i0 += kUnroll) {
      float v[kUnroll][PER], e[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        e[u] = -INFINITY;
#pragma unroll
        for (int k = 0; k < PER; ++k) v[u][k] = 0.f;
        if (i0 + u < nsplit) {
          e[u] = lse[i0 + u];
          const float* src = o + static_cast<int64_t>(i0 + u) * D;
          if constexpr (PER == 4) *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(src);
          else *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(src);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (e[u] == -INFINITY) continue;   // a split that the row sees nothing of
        const float f = exp2f(e[u] - M);
        den += f;
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[k] = fmaf(f, v[u][k], acc[k]);
      }
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  float* out = static_cast<float*>(a.out) + w * D + lane * PER;
#pragma unroll
  for (int k = 0; k < PER; ++k) out[k] = acc[k] * inv;
}

template <int D>
cudaError_t launch_t(const TreeArgs& a, cudaStream_t stream) {
  constexpr int smem = (3 * 32 * (D + 4) + kRows * (kKeys + 1)) * 4;
  auto kfn = pkv_tree_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.max_query_len * a.group + kRows - 1) / kRows;
  kfn<<<dim3(a.max_splits, a.num_kv_heads * tiles, a.num_seqs), kThreads, smem, stream>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.max_splits <= 1) return e;
  const int64_t warps = static_cast<int64_t>(a.num_tokens) * a.num_q_heads;
  pkv_tree_merge_kernel<D><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace


cudaError_t launch_tree_f32(const TreeArgs& a, int head_size, cudaStream_t stream) {
  return head_size == 128 ? launch_t<128>(a, stream) : launch_t<64>(a, stream);
}

}  // namespace pkv
