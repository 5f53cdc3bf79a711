// pkv_write_int8.cu -- KV-cache write into int8 caches with one fp32 scale
// for each (block of 16 tokens, kv head), K and V apart.
//
// Mathematics.  For a block and head, a = max |x| over the finite elements of
// the rows this call puts there, want = max(a / 127, 2^-60).  If the call's
// rows include the block's offset 0 the block begins anew, s = want;
// otherwise it already holds earlier tokens under s_old and s = max(s_old,
// want).  New codes are rint(x * (1 / s)); where s grew, the earlier tokens'
// codes become rint(code * (s_old / s)): a re-rounding of at most half a step
// of the new scale, paid only when a later token is the block's largest (the
// chance that the n-th of n like tokens is: 1 / n).  The alternative, keeping
// a bf16 copy of every open block until it is full, costs a second cache and
// a second path in the attention.
//
// Work: one warp per (touched block, kv head, K or V), heads fastest, so that
// consecutive warps read consecutive head rows of the same tokens.  A warp
// holds its up to 16 rows in registers: one pass over the input.  Bound by the
// chain of dependent loads (lengths, block id, old scale) and, for long chunks, by
// issue slots (58 % busy): one row 2.7 us, 256 rows of 8 kv heads of 128 4.3 us,
// 14362 rows of 5 kv heads of 64 in 40 sequences 7.1 us, 3.9 TB/s of the bytes it
// has to move.
#include <cuda_bf16.h>
#include <float.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kWriteWarps = 8;

// Lengths of sequence s: false if they are inconsistent (bits to raise) or
// there is nothing to write (no bits).
struct SeqRows {
  int q0, qn, L;
};

__device__ __forceinline__ bool load_seq(const WriteInt8Args& a, int s, SeqRows* r, int32_t* bad) {
  r->q0 = __ldg(a.query_start_loc + s);
  r->qn = __ldg(a.query_start_loc + s + 1) - r->q0;
  r->L = __ldg(a.context_lens + s);
  *bad = 0;
  if (r->qn == 0) return false;
  if (r->qn < 0 || r->q0 < 0 || static_cast<int64_t>(r->q0) + r->qn > a.num_tokens ||
      r->qn > a.max_query_len)
    *bad |= PKV_ERR_QUERY_LEN;
  if (r->L < 1 || static_cast<int64_t>(r->L) > a.bt_stride * kBlock) *bad |= PKV_ERR_CONTEXT_LEN;
  else if (r->L < r->qn) *bad |= PKV_ERR_QUERY_LEN;
  return *bad == 0;
}

// First unit of sequence s when sequences have several rows: rows / 16 plus
// two units a sequence always leave room for the blocks its rows touch
// (n rows touch at most n / 16 + 2 blocks).
__device__ __forceinline__ int64_t unit_base(const WriteInt8Args& a, int s) {
  return (static_cast<int64_t>(__ldg(a.query_start_loc + s)) >> 4) + 2 * static_cast<int64_t>(s);
}

// The last s < num_seqs with unit_base(s) <= u (0 if none): every step the
// warp's lanes probe 32 evenly spaced sequences, so 1024 sequences take two
// rounds of loads.
__device__ __forceinline__ int find_seq(const WriteInt8Args& a, int64_t u, int lane) {
  int lo = 0, n = a.num_seqs;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int s = lo + lane * step;
    const bool below = lane * step < n && (lane == 0 || unit_base(a, s) <= u);
    const uint32_t votes = __ballot_sync(0xffffffffu, below);
    const int k = 31 - __clz(votes);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Codes of two bf16 pairs (four elements, in order).  FINITE: |x| * inv is at
// most 127 (plus a rounding), and adding 1.5 * 2^23 leaves the product, rounded
// to the nearest even integer, in the sum's low byte (product and sum rounded
// apart: no FMA).  Otherwise infinities
// saturate and NaN becomes 0 (as cvt.rni has it).
template <bool FINITE>
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
  const float x[4] = {__fmul_rn(bf16_lo(w0), inv), __fmul_rn(bf16_hi(w0), inv),
                      __fmul_rn(bf16_lo(w1), inv), __fmul_rn(bf16_hi(w1), inv)};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = FINITE ? __float_as_uint(__fadd_rn(x[i], 12582912.f))
                  : static_cast<uint32_t>(max(-127, min(127, __float2int_rn(x[i]))));
  return prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u);
}

__device__ __forceinline__ uint32_t requantise4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = static_cast<int8_t>((w >> (8 * i)) & 0xffu);
    const int r = __float2int_rn(static_cast<float>(c) * ratio);
    out |= (static_cast<uint32_t>(r) & 0xffu) << (8 * i);
  }
  return out;
}

template <int D>
__global__ void __launch_bounds__(kWriteWarps * 32)
    pkv_write_int8_kernel(const WriteInt8Args a) {
  constexpr int kLanesPerRow = D / 8;             // 8 bf16 (16 bytes) per lane
  constexpr int kRowsPerLoad = 32 / kLanesPerRow;
  constexpr int kLoads = kBlock / kRowsPerLoad;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWriteWarps + (threadIdx.x >> 5);
  const int hkv = a.num_kv_heads;
  const int64_t u = w / (2 * hkv);
  if (u >= a.num_units) return;
  const int rem = static_cast<int>(w - u * 2 * hkv);
  const bool is_v = rem >= hkv;
  const int h = is_v ? rem - hkv : rem;
  if (rem == 0 && u < a.num_seqs && lane == 0) {   // sequence u's lengths, once
    SeqRows r;
    int32_t bad;
    (void)load_seq(a, static_cast<int>(u), &r, &bad);
    if (bad) raise_error(a.err, bad);
  }
  int s, j;   // sequence, touched block of it
  if (a.max_query_len == 1) {
    s = static_cast<int>(u);
    j = 0;
  } else {
    s = find_seq(a, u, lane);
    const int64_t dj = u - unit_base(a, s);
    if (dj < 0 || dj > a.max_query_len) return;   // (a malformed query_start_loc)
    j = static_cast<int>(dj);
  }
  SeqRows r;
  int32_t bad;
  if (!load_seq(a, s, &r, &bad)) return;
  const int p0 = r.L - r.qn;                       // position of the first new row
  const int64_t blk = static_cast<int64_t>(p0 / kBlock) + j;
  if (blk * kBlock >= r.L) return;
  const int begin = max(p0, static_cast<int>(blk * kBlock));
  const int end = min(r.L, static_cast<int>(blk * kBlock) + kBlock);
  const int o0 = begin % kBlock, n = end - begin;
  const int bid = __ldg(a.block_tables + static_cast<int64_t>(s) * a.bt_stride + blk);
  // this warp's rows, 8 elements a lane; on their way before the block id is
  // looked at
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? a.v : a.k) +
                     (static_cast<int64_t>(r.q0 + (begin - p0)) * hkv + h) * kLanesPerRow;
  const int row0 = lane / kLanesPerRow, col = lane % kLanesPerRow;
  uint4 x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = i * kRowsPerLoad + row0;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row < n) x[i] = __ldg(src + static_cast<int64_t>(row) * hkv * kLanesPerRow + col);
  }
  if (bid < 0 || bid >= a.num_blocks) {
    if (rem == 0 && lane == 0) raise_error(a.err, PKV_ERR_BLOCK_ID);
    return;
  }
  float* scale_at = (is_v ? a.v_scales : a.k_scales) + static_cast<int64_t>(bid) * hkv + h;
  float stored = 0.f, old = 0.f;
  if (o0 > 0) {
    stored = *scale_at;
    // (a scale that no write makes, as of a block that was never begun, counts as
    // the floor, and the floor goes to memory if the new rows ask for no more)
    old = stored >= kInt8ScaleFloor && stored <= FLT_MAX ? stored : kInt8ScaleFloor;
  }
  // largest magnitude: bf16 patterns without their sign compare like the values
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t q[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __vmaxu2(top, q[e] & 0x7fff7fffu);
  }
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  const bool finite = top < 0x7f80u;
  if (!finite) {   // infinities or NaN: the largest of the others
    if (lane == 0) raise_error(a.err, PKV_ERR_NONFINITE);
    top = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t q[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = q[e] & 0x7fffu, hi = (q[e] >> 16) & 0x7fffu;
        top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const float amax = __uint_as_float(top << 16);
  const float want = fmaxf(__fdiv_rn(amax, 127.f), kInt8ScaleFloor);
  const float scale = fmaxf(old, want);
  int8_t* cache = static_cast<int8_t*>(is_v ? a.v_cache : a.k_cache) +
                  (static_cast<int64_t>(bid) * kBlock * hkv + h) * D;
  const int64_t row_stride = static_cast<int64_t>(hkv) * D;
  if (o0 > 0 && scale > old) {   // re-round the block's earlier codes
    const float ratio = __fdiv_rn(old, scale);
    constexpr int kVecs = D / 16;
    for (int i = lane; i < o0 * kVecs; i += 32) {
      uint4* at = reinterpret_cast<uint4*>(cache + (i / kVecs) * row_stride) + i % kVecs;
      const uint4 c = *at;
      *at = make_uint4(requantise4(c.x, ratio), requantise4(c.y, ratio), requantise4(c.z, ratio),
                       requantise4(c.w, ratio));
    }
  }
  if (lane == 0 && scale != stored) *scale_at = scale;   // (a NaN differs)
  const float inv = __fdiv_rn(1.f, scale);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = i * kRowsPerLoad + row0;
    if (row >= n) continue;
    const uint2 out = finite
                          ? make_uint2(codes4<true>(x[i].x, x[i].y, inv), codes4<true>(x[i].z, x[i].w, inv))
                          : make_uint2(codes4<false>(x[i].x, x[i].y, inv), codes4<false>(x[i].z, x[i].w, inv));
    *(reinterpret_cast<uint2*>(cache + (o0 + row) * row_stride) + col) = out;
  }
}

}  // namespace

cudaError_t launch_write_int8(const WriteInt8Args& a, cudaStream_t stream) {
  const int64_t warps = a.num_units * 2 * a.num_kv_heads;
  const int64_t blocks = (warps + kWriteWarps - 1) / kWriteWarps;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (a.head_size == 128)
    pkv_write_int8_kernel<128><<<grid, kWriteWarps * 32, 0, stream>>>(a);
  else
    pkv_write_int8_kernel<64><<<grid, kWriteWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
