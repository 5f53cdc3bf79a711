// pkv_decode_int8.cu -- decode attention (one query row per sequence) over
// int8 caches with one fp32 scale per (block of 16 tokens, kv head), for large
// batches; small ones take the split kernel of pkv_decode.cu (make_int8_plan in
// pkv_api.cu has the rule and both sides' times).
//
// Mathematics.  With codes c, block scales sk and sv, and x_p = scale log2(e)
// sk[b(p)] (q . ck_p):
//     out = sum_p 2^x_p sv[b(p)] cv_p / sum_p 2^x_p.
// The weight that meets the V codes on the tensor cores is w_p = 2^(x_p +
// log2 sv[b(p)] - m): the block's V scale rides in the exponent, and m
// follows the largest x_p + log2 sv, so that w_p, rounded to fp16, is at most
// 2^8 and exact to 2^-11 relative to the largest term of the numerator,
// whatever the scales' sizes.  The denominator adds 2^(x_p - m) in fp32 (not
// w_p / sv[b(p)], which is zero where w_p is too small a number beside a far larger
// scale; the kernel waits for HBM, so the second exponential costs nothing).
// Codes are exact in fp16 (|c| <= 127), so K and V are not rounded at all; Q is
// scaled by a power of two into fp16's range.
//
// Split.  The decode sequences' blocks, one sequence after the other, form
// one line (with kSeqCost blocks of nothing before each sequence, for what its
// start and its end cost a team), which is cut into equal ranges, one for every
// team that the GPU holds at a time; a team of up to 8 warps walks a range, whatever sequences
// lie in it, each warp with its own kv head (or group of 8
// q heads of one), over blocks that one TMA copy of K and one of V brings in
// for all their heads.  Where a range ends inside a sequence its warps write
// partials (normalised O and log2-sum-exp); a range holds at most two a head,
// so the workspace does not grow with the context.  A second launch merges
// them (fixed order: the same inputs give the same bits).  The ranges come
// from the lengths on the device: each CTA adds them up when it starts.
//
// Bound by HBM: every code is read once.  What the layout answers to:
//  * a head's 128 bytes of a token lie beside the next head's; read at
//    different times they cost a DRAM row each (a warp per head and nothing
//    that keeps the heads together: 5.1 TB/s, against 7.1 where they happened
//    to run side by side), so a team reads its heads in one copy;
//  * with equal ranges the SMs of some GPCs, which get less bandwidth than the
//    others, are waited for: 64 sequences of 32 heads are done at 150 us on
//    the median and at 153 to 160 on the last SM.  Handing the last third out in small
//    ranges to whoever is done costs more than that (their starts, their
//    partials, and heads read out of step): 173 us against 165.
#include <float.h>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kWarps = kDecInt8Warps;
constexpr int kThreads = kWarps * 32;

// A CTA's rings: NS stages of a K and a V block for each of its heads.
template <int D, int NS>
constexpr int dec8_smem_bytes() {
  return 1024 /* alignment slack */ + kWarps * NS * 2 * D * kBlock + kWarps * NS * 2 * 8 +
         (kThreads + 1) * 8;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Keys [first, L) of decode sequence s, or nothing (*bits: why, 0 if it has no
// rows).
struct DecSeq {
  int q0, L, first;
  __device__ __forceinline__ int blk0() const { return first / kBlock; }
  __device__ __forceinline__ int blocks() const { return (L + kBlock - 1) / kBlock - first / kBlock; }
};

__device__ __forceinline__ bool dec_seq(const TeamDecodeArgs& a, int s, DecSeq* r, int32_t* bits) {
  *bits = 0;
  r->q0 = __ldg(a.query_start_loc + s);
  const int qn = __ldg(a.query_start_loc + s + 1) - r->q0;
  r->L = __ldg(a.context_lens + s);
  if (qn == 0) return false;
  if (qn != 1) *bits = PKV_ERR_DECODE_QLEN;
  else if (r->q0 < 0 || r->q0 >= a.num_tokens) *bits = PKV_ERR_QUERY_LEN;
  else if (r->L < 1 || static_cast<int64_t>(r->L) > a.bt_stride * kBlock ||
           r->L > a.max_context_len)
    *bits = PKV_ERR_CONTEXT_LEN;
  r->first = a.window > 0 && r->L > a.window ? r->L - a.window : 0;
  return *bits == 0;
}

template <int D, int NS>
__global__ void __launch_bounds__(kThreads, kDecInt8CtasPerSm)
    pkv_team_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const TeamDecodeArgs a) {
  constexpr int kTile = D * kBlock;        // one block of one head, K or V: bytes
  // (the merge launch may be scheduled beside this grid's last CTAs; it waits
  // for the grid's completion itself)
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * NS * 2 * kTile);
  int64_t* upto = reinterpret_cast<int64_t*>(bars + kWarps * NS * 2);   // [kThreads + 1]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group, Hq = a.num_q_heads;
  // the team: team_heads kv heads x (team_warps / team_heads) groups of 8 q heads
  const int team_warps = a.team_warps, team_heads = a.team_heads;
  const int team = warp / team_warps, mate = warp - team * team_warps;
  const int mate_cols = team_warps / team_heads;
  const uint32_t stage_bytes = static_cast<uint32_t>(team_heads) * 2 * kTile;
  const uint32_t ring = smem_u32(smem) + team * NS * stage_bytes;
  const uint32_t full = smem_u32(bars) + team * NS * 16, empty = full + NS * 8;
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&kmap);
    prefetch_tensor_map(&vmap);
  }
  if (mate == 0 && lane == 0) {
#pragma unroll
    for (int st = 0; st < NS; ++st) {
      mbar_init(full + 8 * st, 1);
      mbar_init(empty + 8 * st, team_warps);
    }
    fence_barrier_init();
  }

  // ---- the line of blocks: upto[t] = blocks of the sequences before thread
  // t's run of `per` sequences
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  {
    int64_t mine = 0;
    for (int s = threadIdx.x * per; s < min((static_cast<int>(threadIdx.x) + 1) * per, a.num_seqs); ++s) {
      DecSeq q;
      int32_t bits;
      if (dec_seq(a, s, &q, &bits)) {
        mine += kSeqCost + q.blocks();
      } else if (blockIdx.x == 0) {
        // nothing to attend: rows of a sequence with a bad length are zero
        if (a.span != nullptr) a.span[s] = make_int2(0, 0);
        raise_error(a.err, bits);
        if (bits == PKV_ERR_CONTEXT_LEN) {
          uint4* row = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                                static_cast<int64_t>(q.q0) * Hq * D);
          for (int i = 0; i < Hq * D / 8; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    int64_t sum = mine;   // inclusive over the warp, then the CTA
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += y;
    }
    __shared__ int64_t warp_sum[kWarps];
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += warp_sum[w];
    upto[threadIdx.x + 1] = sum;
    if (threadIdx.x == 0) upto[0] = 0;
    __syncthreads();
  }
  // blocks of a range: what the caller asked for, or an equal share (they fit
  // 32 bits: the host sees to it)
  __shared__ int range_blocks;
  int ranges;
  {
    const int64_t total = upto[kThreads];
    const int64_t R = a.range_blocks > 0
                          ? a.range_blocks
                          : max((total + a.num_ranges - 1) / a.num_ranges,
                                static_cast<int64_t>(kMinRangeBlocks));
    ranges = static_cast<int>((total + R - 1) / R);
    if (threadIdx.x == 0) range_blocks = static_cast<int>(R);
    __syncthreads();
  }

  const uint64_t policy = policy_evict_first();
  const uint64_t wlim = wait_limit(a.wait_limit_ns);
  const int t = lane & 3, r0 = lane >> 2;
  const int c0 = 2 * t;                       // this lane's two q-head columns: c0, c0 + 1
  // ---- this warp's work: a range, a kv head, a group of 8 q heads
  const int unit = blockIdx.x * (kWarps / team_warps) + team;   // team's number
  const int range = unit / a.teams_per_range;
  const int rest = unit - range * a.teams_per_range;
  const int col_teams = (a.col_groups + mate_cols - 1) / mate_cols;
  const int kvh0 = rest / col_teams * team_heads;    // the team's first kv head
  const int head_of = mate / mate_cols;              // the warp's, counted from there
  const int kvh = kvh0 + head_of;
  const int gsub = rest % col_teams * mate_cols + mate % mate_cols;   // (past G: zero columns)
  // Fragment addresses of stage 0 (see the loop): K row r0 at its first chunk
  // and, D = 128, its second; V rows 2t and 2t + 1.  Rows 8 further on lie 8 row
  // lengths behind (the swizzle repeats every 8 rows).
  constexpr int KC = D / 64;
  constexpr int kRows8 = 8 * D;
  uint32_t k_at[KC], v_at[2];
#pragma unroll
  for (int c = 0; c < KC; ++c) k_at[c] = ring + head_of * kTile + swz8<D>(r0, KC * t + c);
#pragma unroll
  for (int x = 0; x < 2; ++x)
    v_at[x] = ring + (team_heads + head_of) * kTile +
              (D == 128 ? swz8<D>(2 * t + x, r0) : swz8<D>(2 * t + x, r0 >> 1) + 8 * (r0 & 1));
  // The team counts its blocks through all its segments: block c is in stage c %
  // NS.  A warp of the team starts each copy, in turn: when it has read block c,
  // the one that takes the stage of block c - lag (which the others have
  // probably read by then, too).
  const int lag = team_warps > 1 ? 1 : 0;
  uint32_t seg0 = 0;            // blocks of the segments before
  int st = 0;                   // stage of the next block, parity of its phase
  uint32_t phase = 0;
  uint32_t next_issue = 0;      // blocks below this that are this warp's to start are started
  bool alive = true;
  // Test hook: the team of warp 0 withholds its first block, so that its waits run out.
  const bool withheld = a.debug_stall != 0 && team == 0;

  if (range < ranges) {
    // ---- the sequence in which the range begins, how far into it, and how
    // much of the range is left
    int s, into, left;
    {
      const int64_t begin = static_cast<int64_t>(range) * range_blocks;
      left = static_cast<int>(min(static_cast<int64_t>(range_blocks), upto[kThreads] - begin));
      int64_t base;
      int th = 0;   // the last thread run that begins at or before `begin`
#pragma unroll
      for (int i = 0; i < kThreads; i += 32)
        th += __popc(__ballot_sync(0xffffffffu, upto[i + lane + 1] <= begin));
      s = th * per;
      base = upto[th];
      while (true) {   // 32 sequences of the run at a time
        DecSeq q;
        int32_t bits;
        const int n = s + lane < a.num_seqs && dec_seq(a, s + lane, &q, &bits) ? kSeqCost + q.blocks() : 0;
        int64_t sum = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, sum, off);
          if (lane >= off) sum += y;
        }
        const uint32_t votes = __ballot_sync(0xffffffffu, base + sum > begin);
        if (votes != 0) {
          const int k = __ffs(votes) - 1;
          base += __shfl_sync(0xffffffffu, sum - n, k);
          s += k;
          break;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
        s += 32;
        if (s >= a.num_seqs) return;   // (cannot be: begin < total)
      }
      into = static_cast<int>(begin - base);
    }
    int n, steps;   // blocks of a segment, and its length on the line
    for (; left > 0 && s < a.num_seqs && alive; ++s, left -= steps, into = 0, seg0 += n) {
      DecSeq q;
      int32_t bits;
      n = steps = 0;
      if (!dec_seq(a, s, &q, &bits)) continue;
      const int nblk = q.blocks();
      const int rest_of_seq = kSeqCost + nblk - into;
      steps = min(left, rest_of_seq);
      const int b0 = max(into - kSeqCost, 0);   // the segment: blocks [b0, b0 + n)
      n = max(into + steps - kSeqCost, 0) - b0;
      if (n == 0) continue;   // (the sequence's blocks begin in the next range)
      const int32_t* bt =
          a.block_tables + static_cast<int64_t>(s) * a.bt_stride + q.blk0() + b0;

      // ids of 32 blocks at a time, lane i the i-th; the next 32 a group ahead
      auto ids_of = [&](int i0) { return i0 + lane < n ? __ldg(bt + i0 + lane) : -1; };
      auto valid = [&](int bid) {
        return static_cast<uint32_t>(bid) < static_cast<uint32_t>(a.num_blocks);
      };
      auto scales_of = [&](int bid, float* ks, float* vs) {
        const int64_t i = static_cast<int64_t>(valid(bid) ? bid : 0) * a.num_kv_heads + kvh;
        *ks = __ldg(a.k_scales + i);
        *vs = __ldg(a.v_scales + i);
      };
      int cur = ids_of(0), nxt = ids_of(32);
      // Starts the team's block c, which is block `bid` (lane 0 acts): waits until
      // every warp of the team has read what its stage held.
      auto issue = [&](uint32_t c, int bid) {
        next_issue = c + 1;
        if (lane != 0 || (withheld && c == 0)) return;
        const int stage = c % NS;
        const uint32_t dst = ring + stage * stage_bytes, bar = full + 8 * stage;
        if (c >= NS && !mbar_wait(empty + 8 * stage, (c / NS - 1) & 1, wlim)) {
          mbar_arrive(bar);   // (given up: the wait for this block will see it)
          raise_error(a.err, PKV_ERR_TIMEOUT);
        } else if (valid(bid)) {
          fence_proxy_async();
          mbar_arrive_expect_tx(bar, stage_bytes);
          tma_load_3d(dst, &kmap, bar, 0, bid * kBlock, kvh0, policy);
          tma_load_3d(dst + team_heads * kTile, &vmap, bar, 0, bid * kBlock, kvh0, policy);
        } else {
          mbar_arrive(bar);   // nothing to load: complete the phase empty
        }
      };
      if (mate == 0) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
          if (i < n) issue(seg0 + i, __shfl_sync(0xffffffffu, cur, i));
      }
      float ks_c, lv_c, ks_n = 1.f, vs_n = 1.f;   // K scales, log2 of the V scales
      scales_of(cur, &ks_c, &lv_c);
      ks_c = int8_scale(ks_c);
      lv_c = log2f(int8_scale(lv_c));

      // ---- Q^T as the B operand, over the permutation of d that makes a
      // lane's K codes contiguous: step kk, k-slots {2t, 2t+1, 2t+8, 2t+9} are
      // d = (D/4) t + 4 kk + {0, 1, 2, 3}; heads past the group are zero.
      uint32_t qb[D / 16][2];
      float col_scale[2];
      {
        const int g = gsub * 8 + r0;
        const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
            static_cast<const __nv_bfloat16*>(a.q) +
            (static_cast<int64_t>(q.q0) * Hq + kvh * G + min(g, G - 1)) * D);
        float amax = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w = __ldg(qrow + (D / 8) * t + 2 * kk + j);
            qb[kk][j] = g < G ? w : 0u;
            amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(qb[kk][j])), fabsf(bf16_hi(qb[kk][j]))));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));   // the head's 4 lanes
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int e = f16_fit_exponent(amax);
        const float down = pow2f(-e);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = 0; j < 2; ++j) qb[kk][j] = bf16x2_to_f16x2(qb[kk][j], down);
        col_scale[0] = a.scale_log2 * pow2f(__shfl_sync(0xffffffffu, e, 4 * c0));
        col_scale[1] = a.scale_log2 * pow2f(__shfl_sync(0xffffffffu, e, 4 * c0 + 4));
      }

      float o[D / 16][4];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      // blocks with keys that the row does not see: the first, the last
      const int edge_lo = b0 == 0 && q.first % kBlock != 0 ? 0 : -1;
      const int edge_hi = b0 + n == nblk && q.L % kBlock != 0 ? n - 1 : -1;
      uint32_t ok_mask = 0;
      for (int i = 0; i < n; ++i) {
        if ((i & 31) == 0) {
          if (i > 0) {
            cur = nxt;
            ks_c = int8_scale(ks_n);
            lv_c = log2f(int8_scale(vs_n));
            nxt = ids_of(i + 32);
          }
          ok_mask = __ballot_sync(0xffffffffu, valid(cur));
          if (mate == 0 && !valid(cur) && i + lane < n) raise_error(a.err, PKV_ERR_BLOCK_ID);
        }
        const float ks = __shfl_sync(0xffffffffu, ks_c, i & 31);
        const float lv = __shfl_sync(0xffffffffu, lv_c, i & 31);
        if (!mbar_wait(full + 8 * st, phase, wlim)) {
          alive = false;
          break;
        }
        // The whole block goes to registers first, so that its stage is
        // refilled before the block is computed.  K: rows r0 and r0 + 8, bytes
        // [(D/4) t, (D/4) t + D/4).  V: rows 2t, 2t+1, 2t+8, 2t+9, bytes
        // [(D/8) r0, (D/8) r0 + D/8): the output rows of step dt are d =
        // (D/8) r0 + 2 dt + {0, 1}.
        constexpr int VW = D / 32;
        const uint32_t off = st * stage_bytes;
        uint4 kw[2][KC];
        uint32_t vw[4][VW];
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          kw[0][c] = lds128(k_at[c] + off);
          kw[1][c] = lds128(k_at[c] + off + kRows8);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t at = v_at[x & 1] + off + (x >> 1) * kRows8;
          if constexpr (D == 128) {
            const uint4 u = lds128(at);
            vw[x][0] = u.x; vw[x][1] = u.y; vw[x][2] = u.z; vw[x][3] = u.w;
          } else {
            const uint2 u = lds64(at);
            vw[x][0] = u.x; vw[x][1] = u.y;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * st);
        if (++st == NS) {
          st = 0;
          phase ^= 1;
        }
        {
          const int k = i - lag + NS;   // the segment's block to start now, and whose turn it is
          if (i >= lag && k < n && (i & (team_warps - 1)) == mate)
            issue(seg0 + k, __shfl_sync(0xffffffffu, (k ^ i) < 32 ? cur : nxt, k & 31));
        }
        if ((i & 31) == 8) scales_of(nxt, &ks_n, &vs_n);
        if (!(ok_mask >> (i & 31) & 1)) continue;   // (its stage holds something else)
        // ---- S^T = K . Q^T (16 keys x 8 heads), even and odd steps apart to
        // halve the chain of dependent products
        float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&kw[0][kk / 4]);
          const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&kw[1][kk / 4]);
          const uint2 x = i8x4_to_f16x4(w0[kk % 4]), y = i8x4_to_f16x4(w1[kk % 4]);
          mma_f16_16816((kk & 1) ? sd : sc, x.x, y.x, x.y, y.y, qb[kk][0], qb[kk][1]);
        }
        // ---- weights.  The reference m of a column moves only when an
        // exponent exceeds it by more than 8, so most blocks cost one vote.
        float y[4];
        y[0] = fmaf(sc[0] + sd[0], col_scale[0] * ks, lv);
        y[1] = fmaf(sc[1] + sd[1], col_scale[1] * ks, lv);
        y[2] = fmaf(sc[2] + sd[2], col_scale[0] * ks, lv);
        y[3] = fmaf(sc[3] + sd[3], col_scale[1] * ks, lv);
        if (i == edge_lo || i == edge_hi) {
          const int p0 = (q.blk0() + b0 + i) * kBlock;
          const bool v0 = p0 + r0 < q.L && p0 + r0 >= q.first;
          const bool v1 = p0 + r0 + 8 < q.L && p0 + r0 + 8 >= q.first;
          if (!v0) y[0] = y[1] = -INFINITY;
          if (!v1) y[2] = y[3] = -INFINITY;
        }
        const float lim0 = m[0] + 8.f, lim1 = m[1] + 8.f;
        if (__any_sync(0xffffffffu, y[0] > lim0 || y[1] > lim1 || y[2] > lim0 || y[3] > lim1)) {
          float mx0 = fmaxf(y[0], y[2]), mx1 = fmaxf(y[1], y[3]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
          }
          const float mn0 = fmaxf(m[0], mx0), mn1 = fmaxf(m[1], mx1);
          // (in two steps: the sums may be far above 1 where the factor is below 2^-126)
          const float half0 = mn0 == -INFINITY ? 1.f : ex2(0.5f * (m[0] - mn0));
          const float half1 = mn1 == -INFINITY ? 1.f : ex2(0.5f * (m[1] - mn1));
          const float alpha0 = half0 * half0, alpha1 = half1 * half1;
          m[0] = mn0;
          m[1] = mn1;
          l[0] = l[0] * half0 * half0;
          l[1] = l[1] * half1 * half1;
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            o[dt][0] *= alpha0;
            o[dt][1] *= alpha1;
            o[dt][2] *= alpha0;
            o[dt][3] *= alpha1;
          }
        }
        const float mu0 = m[0] == -INFINITY ? 0.f : m[0];   // every key so far masked
        const float mu1 = m[1] == -INFINITY ? 0.f : m[1];
        const float w0 = ex2(y[0] - mu0), w1 = ex2(y[1] - mu1);
        const float w2 = ex2(y[2] - mu0), w3 = ex2(y[3] - mu1);
        const float d0 = kSumBias - lv - mu0, d1 = kSumBias - lv - mu1;
        l[0] += ex2(y[0] + d0) + ex2(y[2] + d0);
        l[1] += ex2(y[1] + d1) + ex2(y[3] + d1);
        const uint32_t pb0 = movmatrix_trans(pack_f16(w0, w1));   // rows = heads
        const uint32_t pb1 = movmatrix_trans(pack_f16(w2, w3));
        // ---- O^T += V^T . W^T
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          // bytes 2dt, 2dt+1 of rows (2t, 2t+1) interleaved: (k0,d0) (k1,d0) (k0,d1) (k1,d1)
          const uint32_t sel = (dt & 1) ? 0x7362u : 0x5140u;
          const uint2 lo = i8x4_to_f16x4(prmt(vw[0][dt / 2], vw[1][dt / 2], sel));
          const uint2 hi = i8x4_to_f16x4(prmt(vw[2][dt / 2], vw[3][dt / 2], sel));
          mma_f16_16816(o[dt], lo.x, lo.y, hi.x, hi.y, pb0, pb1);
        }
      }

      // ---- the segment's end: denominators over the 8 lanes of a column
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], off);
      }
      // (a row all of whose blocks were bad, or a wait that gave up, has l = 0)
      const bool whole = b0 == 0 && n == nblk;
      if (b0 == 0 && kvh == 0 && gsub == 0 && lane == 0 && a.span != nullptr)
        a.span[s] = make_int2(range, 1 + (rest_of_seq - left + range_blocks - 1) / range_blocks);
      const int64_t slot = 2 * static_cast<int64_t>(range) + (b0 == 0 ? 1 : 0);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int g = gsub * 8 + c0 + c;
        if (g >= G) continue;
        const int hq = kvh * G + g;
        const float inv = l[c] == 0.f ? 0.f : kTwoSumBias / l[c];
        if (whole) {   // D / 8 consecutive d a lane
          uint32_t w[D / 16];
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) w[dt] = pack_bf16(o[dt][c] * inv, o[dt][2 + c] * inv);
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) +
                                                (static_cast<int64_t>(q.q0) * Hq + hq) * D +
                                                (D / 8) * r0);
#pragma unroll
          for (int i = 0; i < D / 64; ++i)
            dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
          float4* dst = reinterpret_cast<float4*>(a.ws_o + (slot * Hq + hq) * D + (D / 8) * r0);
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            dst[i] = make_float4(o[2 * i][c] * inv, o[2 * i][2 + c] * inv, o[2 * i + 1][c] * inv,
                                 o[2 * i + 1][2 + c] * inv);
          // (the exponent reference m carries log2 sv; l has it divided out)
          if (r0 == 0)
            a.ws_lse[slot * Hq + hq] = l[c] == 0.f ? -INFINITY : m[c] + (log2f(l[c]) - kSumBias);
        }
      }
      if (!alive) {
        if (lane == 0) raise_error(a.err, PKV_ERR_TIMEOUT);
        // every copy that this warp started lands before the CTA's memory is
        // released: of the segment's blocks from the one not read on, the first NS
        // are warp 0's, the later ones went round
        for (uint32_t c = seg0; c < next_issue; ++c) {
          const int k = static_cast<int>(c - seg0);
          const int by = k < NS ? 0 : (k - NS + lag) & (team_warps - 1);
          if (by == mate && !(withheld && c == 0) && c + NS >= next_issue)
            (void)mbar_wait(full + 8 * (c % NS), (c / NS) & 1);
        }
      }
    }
  }
}

// WARPS warps per (sequence, q head) with more than one partial:
// out = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M).  Bound by the latency of
// its loads: a warp has those of 8 partials in flight together, and rows of
// many partials (long contexts, few sequences) get 4 warps, which meet in
// shared memory (fixed order: the same inputs give the same bits).
template <int D, int WARPS>
__global__ void __launch_bounds__(128) pkv_team_merge_kernel(const TeamDecodeArgs a) {
  constexpr int PER = D / 32, kUnroll = 8;
  __shared__ float sm_o[WARPS][D], sm_l[WARPS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = WARPS == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + warp : blockIdx.x;
  const int me = WARPS == 1 ? 0 : warp;
  const int s = static_cast<int>(row / a.num_q_heads);
  if (s >= a.num_seqs) return;
  const int hq = static_cast<int>(row - static_cast<int64_t>(s) * a.num_q_heads);
  const int2 span = a.span[s];
  if (span.y <= 1) return;   // nothing, or the decode kernel wrote the row
  if (span.x < 0 || span.y > a.max_ranges - span.x) return;   // (a launch that gave up)
  // partial 0 begins inside its range (the range's second slot), the others
  // at their range's start (its first)
  auto slot = [&](int i) {
    return (2 * static_cast<int64_t>(span.x + i) + (i == 0 ? 1 : 0)) * a.num_q_heads + hq;
  };
  float M = -INFINITY;
  for (int i = lane; i < span.y; i += 32) M = fmaxf(M, a.ws_lse[slot(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float acc[PER] = {}, den = 0.f;
  for (int i0 = me; i0 < span.y; i0 += kUnroll * WARPS) {
    float v[kUnroll][PER], lse[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * WARPS;
      const int64_t k = slot(min(i, span.y - 1));
      lse[u] = i < span.y ? a.ws_lse[k] : -INFINITY;
      const float* src = a.ws_o + k * D + lane * PER;
      if constexpr (PER == 4) *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(src);
      else *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(src);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const float w = lse[u] == -INFINITY ? 0.f : exp2f(lse[u] - M);
      den += w;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = w == 0.f ? acc[e] : fmaf(w, v[u][e], acc[e]);
    }
  }
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int e = 0; e < PER; ++e) sm_o[me][lane * PER + e] = acc[e];
    if (lane == 0) sm_l[me] = den;
    __syncthreads();
    if (me != 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      den += sm_l[w];
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] += sm_o[w][lane * PER + e];
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                       (static_cast<int64_t>(__ldg(a.query_start_loc + s)) * a.num_q_heads + hq) * D +
                       lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(out + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

template <int D, int NS>
cudaError_t launch_t(const CUtensorMap& kmap, const CUtensorMap& vmap, const TeamDecodeArgs& a,
                     bool merge, cudaStream_t stream) {
  constexpr int smem = dec8_smem_bytes<D, NS>();
  auto kfn = pkv_team_decode_kernel<D, NS>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  TeamDecodeArgs b = a;
  debug_wait_settings(&b.wait_limit_ns, &b.debug_stall);
  kfn<<<a.grid, kThreads, smem, stream>>>(kmap, vmap, b);
  e = cudaGetLastError();
  if (e != cudaSuccess || !merge) return e;
  // a programmatic dependent of the decode launch: its CTAs are scheduled
  // beside the decode's last ones and wait for that grid's completion
  cudaLaunchConfig_t cfg{};
  const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.num_q_heads;
  const bool wide = a.max_ranges / a.num_seqs >= 8;   // partials of a row, about
  cfg.gridDim = dim3(static_cast<unsigned>(wide ? rows : (rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return wide ? cudaLaunchKernelEx(&cfg, pkv_team_merge_kernel<D, 4>, b)
              : cudaLaunchKernelEx(&cfg, pkv_team_merge_kernel<D, 1>, b);
}

}  // namespace

cudaError_t launch_team_decode(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const TeamDecodeArgs& a, int head_size, bool merge,
                               cudaStream_t stream) {
  if (head_size == 128) return launch_t<128, 3>(kmap, vmap, a, merge, stream);
  return launch_t<64, 6>(kmap, vmap, a, merge, stream);
}

}  // namespace pkv
