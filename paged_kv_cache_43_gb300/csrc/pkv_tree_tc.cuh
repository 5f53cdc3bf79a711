// pkv_tree_tc.cuh -- what the tcgen05 tree-attention kernels share: the line of work that
// is cut into equal ranges, and how 16-bit values that are not finite are told.
//
// All units (sequence, group of row tiles, kv head) of the batch lie on one line: a unit is
// kStart steps for its start (its ids, Q and first copies, its rows out) and a step for each
// step_keys of its keys.  Worker w of W has the line's w-th equal part (its sequences'
// lengths are read on the device).  A unit that lies in several parts leaves partials: its
// first worker's in the second of that worker's two places (it ends there), the others'
// in their first; span says which workers those are.  A worker is cta_tiles CTAs, one for
// each row tile of a unit, which walk the same keys side by side and find each other's in L2.
#pragma once

#include <float.h>

#include "pkv_prefill_tc.cuh"
#include "pkv_tree.cuh"

namespace pkv {

namespace {

// What a CTA computes next: steps [step0, step0 + steps) of a unit's rows.
struct alignas(16) Seg {
  int32_t s, kvh, q0, n;
  int32_t L, row0, rows, step0;
  int32_t steps;                                // < 0: nothing more
  int32_t part;                                 // where its partial goes, -1: the whole unit
};
constexpr int kSegs = 4;
// What weights (of 64 keys together, or one) may come to before a row's reference moves.  fp16 weights
// reach 65504; of bf16 ones O holds up to this times a V value for each key in fp32, so |V| x keys
// stays right below 2^113.  (One sequence of 4000 keys, 8 drafts x 4 heads: with 2^60 29.9 us,
// 2^15 29.9, 2^8 33.9; larger batches 0 to 2 % apart.)
constexpr float kTreeMost = 32768.f;
constexpr int kStart = kTreeStart;

// Calls emit(seg) for each segment of this CTA, one warp's lanes together, until it returns
// false; tile rows are (query row, q head) pairs.
template <typename Emit>
__device__ __forceinline__ void tree_walk(const TreeArgs& a, int step_keys, Emit emit) {
  const int lane = threadIdx.x & 31;
  const int ct = a.cta_tiles;
  const int worker = blockIdx.x / ct, tile_c = blockIdx.x - worker * ct;
  const int tile_rows = a.tile_toks * a.group;
  // the 32 sequences that the lanes hold, one each:
  int q0, n, len, steps, groups;
  int64_t unit_cost, cost;
  auto hold = [&](int at) {
    q0 = n = len = steps = groups = 0;
    unit_cost = cost = 0;
    if (at + lane >= a.num_seqs) return;
    const TreeSeq q = tree_seq(a, at + lane);
    if (q.skip || q.err != 0) return;
    q0 = q.q0;
    n = q.n;
    len = q.L;
    steps = (q.L + step_keys - 1) / step_keys;
    groups = ((q.n + a.tile_toks - 1) / a.tile_toks + ct - 1) / ct;
    unit_cost = a.whole ? 1 : steps + kStart;
    cost = unit_cost * groups * a.num_kv_heads;
  };
  // the cost of the 128 sequences from `at` on, four a lane at a time
  auto cost_of = [&](int at) {
    int64_t c = 0;
#pragma unroll
    for (int i = 0; i < 128; i += 32) {
      const int s = at + i + lane;
      TreeSeq q = tree_seq(a, min(s, a.num_seqs - 1));
      if (s >= a.num_seqs || q.skip || q.err != 0) q.n = 0;
      const int64_t uc = a.whole ? 1 : (q.L + step_keys - 1) / step_keys + kStart;
      c += uc * (((q.n + a.tile_toks - 1) / a.tile_toks + ct - 1) / ct) * a.num_kv_heads;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
    return c;
  };
  int64_t total = 0;
  for (int at = 0; at < a.num_seqs; at += 128) total += cost_of(at);
  // This worker's part of the line.  The contexts may be far shorter than max_context_len, which
  // made the number of workers: the first of them share the line then, so that none between
  // a unit's first and last is without a step (the merge reads a partial of each).
  const int W = gridDim.x / ct;
  int64_t range = a.range, begin, end;
  if (a.whole) {
    begin = total * worker / W;
    end = total * (worker + 1) / W;
  } else {
    if (range == 0) range = max((total + W - 1) / W, static_cast<int64_t>(kTreeMinRange));
    begin = range * worker;
    end = min(total, begin + range);
  }
  auto worker_of = [&](int64_t p) { return static_cast<int>(p / range); };
  int64_t before = 0;    // the line up to the sequences that the lanes hold
  int from = 0;          // (128 at a time past those that lie before this part)
  while (from + 128 < a.num_seqs) {
    const int64_t c = cost_of(from);
    if (before + c > begin) break;
    before += c;
    from += 128;
  }
  for (int at = from; at < a.num_seqs && before < end; at += 32) {
    hold(at);
    int64_t upto = cost;   // inclusive sums over the lanes
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += x;
    }
    const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
    for (int j = 0; before + all > begin && j < 32; ++j) {
      const int64_t x1 = before + __shfl_sync(0xffffffffu, upto, j);
      const int64_t c1 = __shfl_sync(0xffffffffu, cost, j), x0 = x1 - c1;
      if (c1 == 0 || x1 <= begin) continue;
      if (x0 >= end) break;
      const int64_t uc = __shfl_sync(0xffffffffu, unit_cost, j);
      const int N = __shfl_sync(0xffffffffu, steps, j);
      const int units = __shfl_sync(0xffffffffu, groups, j) * a.num_kv_heads;
      Seg g;
      g.s = at + j;
      g.q0 = __shfl_sync(0xffffffffu, q0, j);
      g.n = __shfl_sync(0xffffffffu, n, j);
      g.L = __shfl_sync(0xffffffffu, len, j);
      for (int u = begin > x0 ? static_cast<int>((begin - x0) / uc) : 0; u < units; ++u) {
        const int64_t x = x0 + u * uc;
        if (x >= end) break;
        int i0 = 0, i1 = N;   // this worker's steps of the unit
        if (!a.whole) {
          i0 = static_cast<int>(max(begin - x - kStart, int64_t{0}));
          i1 = static_cast<int>(min(end - x - kStart, static_cast<int64_t>(N)));
          if (x >= begin && tile_c == 0 && lane == 0) {
            const int w0 = worker_of(x + kStart), w1 = worker_of(x + kStart + N - 1);
            a.span[(static_cast<int64_t>(g.s) * a.max_groups) * a.num_kv_heads + u] =
                make_int2(w0, w1 - w0 + 1);
          }
        }
        const int tg = u / a.num_kv_heads;
        g.kvh = u - tg * a.num_kv_heads;
        g.row0 = (tg * ct + tile_c) * tile_rows;
        g.rows = min(g.n * a.group - g.row0, tile_rows);
        if (i1 <= i0 || g.rows <= 0) continue;
        g.step0 = i0;
        g.steps = i1 - i0;
        g.part = i0 == 0 && i1 == N ? -1 : worker * 2 + (i0 > 0 ? 0 : 1);
        if (!emit(g)) return;
      }
    }
    before += all;
  }
}

// Sequences with bad lengths: said, and their rows (the first max_query_len) zeroed; `threads`
// threads of each CTA, numbered `thread`.
template <int D>
__device__ __forceinline__ void tree_bad_sequences(const TreeArgs& a, int thread, int threads) {
  for (int s = blockIdx.x; s < a.num_seqs; s += gridDim.x) {
    const TreeSeq q = tree_seq(a, s);
    if (q.err == 0) continue;
    if (thread == 0) raise_error(a.err, q.err);
    if (q.skip) continue;
    const int64_t rows = static_cast<int64_t>(min(q.n, a.max_query_len)) * a.num_q_heads * (D / 8);
    uint4* zero = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                           static_cast<int64_t>(q.q0) * a.num_q_heads * D);
    for (int64_t i = thread; i < rows; i += threads) zero[i] = make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ bool quick_wait(uint32_t bar, uint32_t parity, volatile int32_t* abort,
                                           int32_t* err, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         warp_wait(bar, parity, abort, err, limit_ns);
}

// The sign bits of those 16-bit values in w whose exponent is all ones (adding one to it carries
// into the sign's place).
template <bool FP8>
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  return FP8 ? ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u
             : ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}
template <bool FP8>
__device__ __forceinline__ uint32_t even_value(uint32_t w) {   // those values as zero
  constexpr uint32_t e = FP8 ? 0x7C00u : 0x7F80u;
  if ((w & e) == e) w &= 0xffff0000u;
  if ((w & (e << 16)) == (e << 16)) w &= 0xffffu;
  return w;
}

// Adds to element d of a row that is written (fp32 partial, or bf16 at `out`) the V values that are
// not finite of those drafts among the keys [k0, k1) that the row sees: the products left
// them out.  Rare, and kept apart from the code that every unit runs through.
template <bool FP8, int D>
__device__ __forceinline__ void add_odd_values(const TreeArgs& a, int s, int kvh, int first, int k0, int k1,
                                            const uint64_t* mask, int d, float* part, __nv_bfloat16* out) {
  float sum = part != nullptr ? *part : __bfloat162float(*out);
  const int32_t* bt = a.block_tables + s * a.bt_stride;
#pragma unroll 1
  for (int p = max(first, k0); p < k1; ++p) {
    const int j = p - first, b = __ldg(bt + p / kBlock);
    if (!(__ldg(mask + (j >> 6)) >> (j & 63) & 1) || b < 0 || b >= a.num_blocks) continue;
    const int64_t at = ((static_cast<int64_t>(b) * kBlock + p % kBlock) * a.num_kv_heads + kvh) * D + d;
    float v;
    if constexpr (FP8) v = f16_lo(e4m3x4_to_f16x4(static_cast<const uint8_t*>(a.v_cache)[at]).x);
    else v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.v_cache)[at]);
    if (!(fabsf(v) <= FLT_MAX)) sum += v;
  }
  if (part != nullptr) *part = sum;
  else *out = __float2bfloat16(sum);
}

}  // namespace

}  // namespace pkv
