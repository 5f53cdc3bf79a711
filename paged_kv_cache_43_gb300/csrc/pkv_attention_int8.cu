// pkv_attention_int8.cu -- paged attention over int8 caches whose codes are
// scaled by one fp32 number for each (block of 16 tokens, kv head).
//
// out[t][hq] = sum_p w_p V_p / sum_p w_p, w_p = exp(scale q . K_p - max), with
// K_p = code * k_scale[block of p][kv head] (likewise V), over the keys that
// row t sees (causal inside a chunk, optional window).
//
// The path of chunk rows with more than 128 q heads on a kv head, which a query
// tile of the tcgen05 kernel cannot hold: one CTA per (query row, q head), 4
// warps taking every 4th key, a warp-wide dot product per key, the running
// maximum and sum in fp32.  Bound by its instructions (5 TFLOP/s; K and V come
// from L1 and L2 again for every row).
#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) pkv_attention_int8_kernel(const AttnInt8Args a) {
  constexpr int PER = D / 32;
  __shared__ float sm_m[kWarps], sm_l[kWarps];
  __shared__ float sm_o[kWarps][D];
  const int t = blockIdx.x;
  const int hq = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = seq_of_row(a.query_start_loc, a.num_seqs, t);
  if (s < a.seq_begin) return;   // a row of no sequence, or of a decode sequence
  const int q0 = __ldg(a.query_start_loc + s);
  const int qn = __ldg(a.query_start_loc + s + 1) - q0;
  const int L = __ldg(a.context_lens + s);
  if (q0 < 0 || static_cast<int64_t>(q0) + qn > a.num_tokens) {   // rows that there are not
    if (threadIdx.x == 0 && hq == 0 && (t == q0 || t == 0)) raise_error(a.err, PKV_ERR_QUERY_LEN);
    return;
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                       (static_cast<int64_t>(t) * a.num_q_heads + hq) * D;
  const bool bad_len = L < 1 || static_cast<int64_t>(L) > a.bt_stride * kBlock;
  if (bad_len || qn > L || qn > a.max_query_len) {
    if (threadIdx.x == 0 && hq == 0 && t == q0)
      raise_error(a.err, bad_len ? PKV_ERR_CONTEXT_LEN : PKV_ERR_QUERY_LEN);
    for (int d = threadIdx.x; d < D; d += blockDim.x) out[d] = __float2bfloat16(0.f);
    return;
  }
  const int kvh = hq / (a.num_q_heads / a.num_kv_heads);
  const int pos = L - qn + (t - q0);
  const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(a.q) +
                              (static_cast<int64_t>(t) * a.num_q_heads + hq) * D;
  float qv[PER], acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    qv[e] = __bfloat162float(qrow[lane * PER + e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int32_t* bt = a.block_tables + static_cast<int64_t>(s) * a.bt_stride;
  const int first = (a.window > 0 && pos + 1 > a.window) ? pos + 1 - a.window : 0;
  for (int p = first + warp; p <= pos; p += kWarps) {
    const int bid = __ldg(bt + p / kBlock);
    if (bid < 0 || bid >= a.num_blocks) {
      if (lane == 0) raise_error(a.err, PKV_ERR_BLOCK_ID);
      continue;
    }
    const int64_t sc = static_cast<int64_t>(bid) * a.num_kv_heads + kvh;
    const float ks = int8_scale(__ldg(a.k_scales + sc)), vs = int8_scale(__ldg(a.v_scales + sc));
    const float vs_down = vs * (1.f / kTwoSumBias);   // (many V of about 2^127 add up below infinity)
    const int64_t row =
        ((static_cast<int64_t>(bid) * kBlock + p % kBlock) * a.num_kv_heads + kvh) * D + lane * PER;
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e)
      dot = fmaf(qv[e], static_cast<float>(static_cast<const int8_t*>(a.k_cache)[row + e]), dot);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    const float x = dot * (ks * a.scale_log2);
    const float mn = fmaxf(m, x);
    const float alpha = exp2f(m - mn);
    const float w = exp2f(x - mn);
    l = l * alpha + w;
#pragma unroll
    for (int e = 0; e < PER; ++e)
      acc[e] = fmaf(w * vs_down, static_cast<float>(static_cast<const int8_t*>(a.v_cache)[row + e]),
                    acc[e] * alpha);
    m = mn;
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) sm_o[warp][lane * PER + e] = acc[e];
  __syncthreads();
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  float den = 0.f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = (sm_m[w] == -INFINITY) ? 0.f : exp2f(sm_m[w] - M);
    den += f[w] * sm_l[w];
  }
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float r = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) r += f[w] * sm_o[w][d];
    out[d] = __float2bfloat16(den == 0.f ? 0.f : r / den * kTwoSumBias);
  }
}

}  // namespace

cudaError_t launch_attention_int8(const AttnInt8Args& a, int head_size, cudaStream_t stream) {
  dim3 grid(a.num_tokens, a.num_q_heads);
  if (head_size == 128) pkv_attention_int8_kernel<128><<<grid, kWarps * 32, 0, stream>>>(a);
  else pkv_attention_int8_kernel<64><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
