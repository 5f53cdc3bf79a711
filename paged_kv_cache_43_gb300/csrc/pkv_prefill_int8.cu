// pkv_prefill_int8.cu -- chunked-prefill attention over int8 caches with one fp32
// scale per (block of 16 tokens, kv head), on tcgen05.
//
// Mathematics.  With codes c, block scales sk and sv, and x_p = scale log2(e)
// sk[b(p)] (q . ck_p), a row's output is sum_p 2^x_p sv[b(p)] cv_p / sum_p
// 2^x_p.  S = Q CK^T and O += P CV run on fp16 operands: codes are exact in
// fp16, a row of Q is scaled by a power of two into its range.  P = 2^(x + log2
// sv - m): a block's V scale rides in the softmax exponent, and m follows the
// largest x + log2 sv, so P in fp16 is at most 2^15 whatever the scales are;
// the row sum divides sv out again (per block, in fp32; where V scales
// differ by 2^64 and more it is formed without it).  Both scales cost
// nothing per element: they are the factor and the addend of the exponent's one
// FMA.  Every code is finite, so rows no key may see need no zeroing.
//
// Layout.  A CTA (one per SM) has two tiles of 128 (token, q head) rows of one
// kv head, and walks the keys 128 at a time, as pkv_prefill_tc.cu, but its
// products take 64 keys: S of a tile is two buffers of 64 columns (P, 32
// columns of fp16 pairs, over the buffer's own start), so S of the next 64 keys
// is there when a softmax warp has done with these; with one buffer of 128 the
// chain S - softmax - P V - next S, 2.6 us of which the tensor core worked 1.0,
// was what a step took.  N = 64 products are bound by their operands' shared
// memory reads (49 cycles, 32 at full rate): 1.2 us for a step of 128 keys.
// 16 warps:
//   0-3, 4-7  softmax of tile 0, 1: a thread a row
//   8, 9      start the TMA copies of K, of V (one box per cache block)
//   10, 13    widen K codes in place (D = 128: half the rows each; 64: warp 10)
//   11, 14    widen V codes
//   12, 15    issue the products of tile 0, 1
// Starting a tile's copies and widening half of it take a warp 1 us each, and
// issuing a half step's products of one tile 0.5: with fewer warps for them (one
// to start all, two to widen all, one to issue all) those bound the step.
// Measured, 4 x 2048 tokens over 2K to 8K keys (32 q / 8 kv heads, head_size 128):
// 564 us, 1080 TFLOP/s, 0.56 of the measured bf16 peak (the first form, products of
// 128 keys as in pkv_prefill_tc.cu: 737).  A step of 128 keys takes 2.1 us, of
// which the tensor core's reads of shared memory 1.2; an SM is idle or filling
// for 11 us of each CTA (launch and work choice 2.7, the first K landing, widened
// and multiplied 5.4, the last rows out 2.8).
// Weights are first formed against the running reference m, with no pass for
// the row maximum; only if one may have grown past 2^15 is the maximum found and
// the 64 weights formed anew.
#include <float.h>

#include <algorithm>

#include "pkv_prefill_tc.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 512;
constexpr int kHalfKeys = kTcKeys / 2;          // keys of a product
constexpr int kHalfBlocks = kHalfKeys / kBlock;
// The launch gives each thread 128 registers; the other two warpgroups hand 40
// each to the softmax warpgroups.
constexpr int kRegsSoftmax = 168;
constexpr int kRegsOther = 88;
static_assert(2 * 128 * (kRegsSoftmax + kRegsOther) <= kThreads * 128, "register split");

// TMEM columns: S of tile t, half step h at 128t + 64 (h % 2), P over its first
// 32; O of tile t at 256 + 128t.
__device__ __forceinline__ uint32_t col_s(int t, int h) { return 128u * t + 64u * (h & 1); }
__device__ __forceinline__ uint32_t col_o(int t) { return 256u + 128u * t; }

struct Shared {
  uint64_t q_full, q_conv;
  uint64_t drain[kTcTiles];
  uint64_t s_full[kTcTiles][2], p_full[kTcTiles][2];   // of half step h: [h % 2]
  uint64_t pv_done[kTcTiles];    // P V of each half step
  uint64_t o_done[kTcTiles];     // the last one (a phase of its own: a waiter for one of
                                 // pv_done's last two could find it a phase further on)
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint64_t kv_land[2 * kRing];   // ring element e: [e % 10], so that K and V have their own
  uint32_t tmem_base;
  int32_t abort;
  int32_t n_issued[2];           // K / V tiles started, for the drain
  // (K scale, log2 of the V scale, 2^kSumBias / V scale, the tile's largest V scale
  // / 2^kSumBias or, of a marked tile, infinity) of a key tile's blocks, a copy for
  // each softmax warp.
  alignas(16) float4 sc[8][kTcKeys / kBlock];
};

template <int D>
constexpr int smem_bytes() {
  constexpr int need = 1024 + kTcTiles * TcLayout<D>::kQTile + kRing * TcLayout<D>::kTileBytes +
                       static_cast<int>(sizeof(Shared));
  static_assert(need <= 227 * 1024, "shared memory");
  return need > 120 * 1024 ? need : 120 * 1024;   // (one CTA per SM: it owns all of TMEM)
}

template <int R>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// As warp_wait, for waits that are mostly over already.
__device__ __forceinline__ bool quick_wait(uint32_t bar, uint32_t parity, volatile int32_t* abort,
                                           int32_t* err, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         warp_wait(bar, parity, abort, err, limit_ns);
}

// Key parts: the row of q head hq of sequence s's token `tok` among the
// partials, max_query_len rows a sequence.
__device__ __forceinline__ int64_t part_row(const PrefillArgs& a, int s, int tok, int hq) {
  return (static_cast<int64_t>(s - a.seq_begin) * a.max_query_len + tok) * a.num_q_heads + hq;
}

// kLongestFirst: CTAs handed out longest first; kKeyParts: each CTA's keys cut
// into parts (grid.z), whose partials a second kernel merges.
constexpr int kPlain = 0, kLongestFirst = 1, kKeyParts = 2;
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    pkv_prefill_int8_kernel(const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap,
                            const __grid_constant__ CUtensorMap omap, const PrefillArgs a) {
  using Lt = TcLayout<D>;
  constexpr bool PARTS = MODE == kKeyParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                                   // [tile][half][128 rows x 128 B]
  uint8_t* sKV = smem + kTcTiles * Lt::kQTile;          // [slot][half][128 keys x 128 B]
  Shared* sh = reinterpret_cast<Shared*>(sKV + kRing * Lt::kTileBytes);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&qmap);
    prefetch_tensor_map(&kmap);
    prefetch_tensor_map(&vmap);
    prefetch_tensor_map(&omap);
  }
  const int G = a.group;
  const int Hq = a.num_q_heads;
  const int tile_toks = kTcRows / G;                // tokens per query tile (its last rows
  const int toks = kTcTiles * tile_toks;            // idle where G does not divide 128)
  int s, kvh, mtile;
  if constexpr (MODE == kLongestFirst) {
    const TcWork w = pick_work(a, toks, reinterpret_cast<int32_t*>(sKV));
    s = w.s;
    kvh = w.kvh;
    mtile = w.mtile;
  } else {
    s = a.seq_begin + (PARTS ? blockIdx.z / a.key_splits : blockIdx.z);
    kvh = blockIdx.y;
    mtile = a.num_mtiles - 1 - blockIdx.x;  // heaviest pair of each sequence first
  }
  const int L = __ldg(a.context_lens + s);
  const int q0 = __ldg(a.query_start_loc + s);
  const int qn = __ldg(a.query_start_loc + s + 1) - q0;
  const int tok0 = mtile * toks;
  const bool bad_rows = qn < 0 || q0 < 0 || static_cast<int64_t>(q0) + qn > a.num_tokens;
  if (bad_rows || qn == 0 || tok0 >= qn) {
    if (bad_rows && mtile == 0 && kvh == 0 && threadIdx.x == 0)
      raise_error(a.err, PKV_ERR_QUERY_LEN);
    return;
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  const bool bad_len = L < 1 || static_cast<int64_t>(L) > a.bt_stride * kBlock;
  if (bad_len || qn > L || qn > a.max_query_len) {
    if constexpr (PARTS)
      if (blockIdx.z % a.key_splits != 0) return;   // (part 0 does this)
    if (threadIdx.x == 0 && mtile == 0 && kvh == 0)
      raise_error(a.err, bad_len ? PKV_ERR_CONTEXT_LEN : PKV_ERR_QUERY_LEN);
    const int nt = min(toks, qn - tok0);
    for (int i = threadIdx.x; i < nt * G * D; i += blockDim.x) {
      const int r = i / D;
      out[(static_cast<int64_t>(q0 + tok0 + r / G) * Hq + kvh * G + r % G) * D + i % D] =
          __float2bfloat16(0.f);
    }
    return;
  }
  const int tok_last = min(tok0 + toks, qn) - 1;
  const int ntq = (tok0 + tile_toks < qn) ? 2 : 1;  // query tiles holding a valid row
  // The CTA walks the key tiles [j0, ntiles) that some row of it sees.
  const int pos_max = L - qn + tok_last, pos_min = L - qn + tok0;
  const int lo_min = a.window > 0 ? max(pos_min - a.window + 1, 0) : 0;
  int j0 = lo_min / kTcKeys;
  int ntiles = (pos_max + kTcKeys) / kTcKeys;
  [[maybe_unused]] int key_part = 0;   // this CTA's part of the tiles
  if constexpr (PARTS) {
    key_part = blockIdx.z % a.key_splits;
    const int per = (ntiles - j0 + a.key_splits - 1) / a.key_splits;
    j0 += key_part * per;
    ntiles = min(ntiles, j0 + per);
    if (ntiles <= j0) {   // a part without key tiles: its partials count for nothing
      for (int i = threadIdx.x; i < (tok_last + 1 - tok0) * G; i += blockDim.x)
        a.ws_lse[part_row(a, s, tok0 + i / G, kvh * G + i % G) * a.key_splits + key_part] = -INFINITY;
      return;
    }
  }
  const int n_rel = __shfl_sync(0xffffffffu, ntiles - j0, 0);
  // half steps: the last tile's second half only if a row sees it
  const int H = 2 * n_rel - (pos_max - (ntiles - 1) * kTcKeys < kHalfKeys ? 1 : 0);
  // cache blocks with a key that some row (of this part) sees
  const int b_lo = max(lo_min / kBlock, j0 * (kTcKeys / kBlock));
  const int nblk = min((pos_max + kBlock) / kBlock, ntiles * (kTcKeys / kBlock));

  const int32_t* bt = a.block_tables + static_cast<int64_t>(s) * a.bt_stride;
  // Block ids of four consecutive tiles per warp-wide load: lane l holds block
  // l % 8 of ring position 4g + l / 8.  Group g + 1 is loaded while group g is
  // started, the first one before the barriers are up, so no tile waits on its ids.
  auto load_ids4 = [&](int g) {
    const int b = (j0 + 4 * g) * (kTcKeys / kBlock) + lane;
    return b >= b_lo && b < nblk ? __ldg(bt + b) : -1;
  };
  const int first_ids = warp == 8 || warp == 9 ? load_ids4(0) : -1;

  const uint32_t q_full = smem_u32(&sh->q_full), q_conv = smem_u32(&sh->q_conv);
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_conv, 8);   // one arrival per softmax warp
    for (int t = 0; t < kTcTiles; ++t) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&sh->s_full[t][b]), 1);
        mbar_init(smem_u32(&sh->p_full[t][b]), 4);
      }
      mbar_init(smem_u32(&sh->pv_done[t]), 1);
      mbar_init(smem_u32(&sh->o_done[t]), 1);
      mbar_init(smem_u32(&sh->drain[t]), 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&sh->kv_full[i]), D == 128 ? 2 : 1);   // its widening warps
      mbar_init(smem_u32(&sh->kv_empty[i]), ntq);               // the tiles' issuers
    }
    for (int i = 0; i < 2 * kRing; ++i) mbar_init(smem_u32(&sh->kv_land[i]), 1);
    sh->abort = 0;
    fence_barrier_init();
  }
  if (warp == 12) tc::alloc(smem_u32(&sh->tmem_base), kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
  volatile int32_t* abort = &sh->abort;
  const uint64_t wlim = wait_limit(a.wait_limit_ns);
  auto land_bar = [&](int e) { return smem_u32(&sh->kv_land[e % (2 * kRing)]); };
  auto land_phase = [](int e) { return static_cast<uint32_t>((e / (2 * kRing)) & 1); };

  if (warp >= 8) {
    fewer_regs<kRegsOther>();
    if (warp == 8 || warp == 9) {
      // ---------------------------------------------------------- producers
      const bool is_v = warp == 9;
      const uint64_t keep = policy_evict_normal();   // K/V tiles are re-read by the
                                                     // other row tiles
      constexpr int kBlocks = kTcKeys / kBlock;      // cache blocks per tile
      int g_cur = first_ids, g_nxt = load_ids4(1);
      if (!is_v && lane == 0) {
        mbar_arrive_expect_tx(q_full, ntq * Lt::kHalves * tile_toks * G * 128);
        for (int t = 0; t < ntq; ++t)
#pragma unroll
          for (int h = 0; h < Lt::kHalves; ++h)
            tma_load_3d(smem_u32(sQ + t * Lt::kQTile + h * Lt::kQHalf), &qmap, q_full, h * 64,
                        kvh * G, q0 + tok0 + t * tile_toks, keep);
      }
      // Test hook: the K producer withholds the first K tile (no copy, no
      // arrival), so that the waits for it run out.
      const bool withhold_k0 = a.debug_stall != 0 && !is_v;
      int n = 0;   // tiles started
      for (; n < n_rel; ++n) {
        if (n > 0 && (n & 3) == 0) {
          g_cur = g_nxt;
          g_nxt = load_ids4((n >> 2) + 1);
        }
        const int e = 2 * n + (is_v ? 1 : 0);
        if (e >= kRing && !warp_wait(smem_u32(&sh->kv_empty[ring_slot(e)]), ring_phase(e - kRing),
                                     abort, a.err, wlim))
          break;
        if (withhold_k0 && n == 0) continue;
        // the tile's blocks; one with a bad id is left out (K reports it)
        const uint32_t dst = smem_u32(sKV + ring_slot(e) * Lt::kTileBytes), bar = land_bar(e);
        bool ok[kBlocks];
        int bid[kBlocks];
        uint32_t bytes = 0;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          bid[b] = __shfl_sync(0xffffffffu, g_cur, 8 * (n & 3) + b);
          const int blk = (j0 + n) * kBlocks + b;
          const bool in_range = blk < nblk && blk >= b_lo;
          ok[b] = in_range && bid[b] >= 0 && bid[b] < a.num_blocks;
          if (!is_v && in_range && !ok[b] && lane == 0) raise_error(a.err, PKV_ERR_BLOCK_ID);
          bytes += ok[b] ? 16u * D : 0u;
        }
        if (lane == 0) {
          if (bytes == 0) {
            mbar_arrive(bar);
          } else {
            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
              if (ok[b])
                tma_load_3d(dst + b * 16 * D, is_v ? &vmap : &kmap, bar, 0, kvh, bid[b] * kBlock,
                            keep);
          }
        }
      }
      // Before the CTA's shared memory is released every copy must have landed.
      // Only the last use of a slot can still be in flight: element e's slot is
      // refilled by element e + kRing only after e has been read.
      if (lane == 0) sh->n_issued[is_v ? 1 : 0] = n;
      named_barrier(3, 64);   // the two producers: both counts final
      const int n_k = sh->n_issued[0], n_v = sh->n_issued[1];
      for (int i = max(0, n - kRing); i < n; ++i) {
        const int e = 2 * i + (is_v ? 1 : 0), nx = e + kRing;
        if ((withhold_k0 && i == 0) || ((nx & 1) ? (nx >> 1) < n_v : (nx >> 1) < n_k)) continue;
        if (lane == 0) (void)mbar_wait(land_bar(e), land_phase(e));
      }
      if (!is_v && lane == 0) (void)mbar_wait(q_full, 0);   // the query tiles too
      __syncwarp();
    } else if (warp == 10 || warp == 11 || (D == 128 && (warp == 13 || warp == 14))) {
      // ------------------------------------------------------------ widening
      // (D = 64: the in-place widening overwrites later rows' codes with earlier
      // rows' fp16, from the last rows to the first, so one warp takes a tile)
      const int b0 = warp >= 13 ? kTcKeys / 32 : 0;   // batches of 16 rows
      for (int e = warp == 10 || warp == 13 ? 0 : 1; e < 2 * n_rel; e += 2) {
        if (!quick_wait(land_bar(e), land_phase(e), abort, a.err, wlim)) break;
        uint8_t* tile = sKV + ring_slot(e) * Lt::kTileBytes;
        if constexpr (D == 128) widen_tile_fp8<true>(tile, lane, b0, b0 + kTcKeys / 32);
        else widen_tile_fp8_d64<true>(tile, lane);
        fence_proxy_async();   // generic writes, then the tensor core reads
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->kv_full[ring_slot(e)]));
      }
    } else if (warp == 12 || (warp == 15 && ntq > 1)) {
      // ------------------------------------------------------------ products
      constexpr uint32_t idS = tc::idesc_f16_f32(kTcRows, kHalfKeys, 0, 0);
      constexpr uint32_t idO = tc::idesc_f16_f32(kTcRows, D, 0, 1);
      const uint64_t dq0 = tc::smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk0 = tc::smem_desc_sw128(smem_u32(sKV), 16, 1024);
      const uint64_t dv0 = tc::smem_desc_sw128(smem_u32(sKV), Lt::kKvHalf, 1024);
      constexpr int kHalfStep = kHalfKeys * 128 >> 4;   // 64 keys on, in descriptor units
      const int t = warp == 12 ? 0 : 1;
      auto issue_s = [&](int h) {
        const uint64_t da = dq0 + static_cast<uint64_t>((t * Lt::kQTile) >> 4);
        const uint64_t db = dk0 + static_cast<uint64_t>(
                                      ((ring_slot(h & ~1) * Lt::kTileBytes) >> 4) + (h & 1) * kHalfStep);
        const uint32_t d = tmem + col_s(t, h);
        if constexpr (D == 128) {
          tc::mma_ss_x8<2, 4, 6, 1024, 1026, 1028, 1030, 2, 4, 6, 1024, 1026, 1028, 1030>(
              d, da, db, idS, 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_ss(d, da + (kk * 32 >> 4), db + (kk * 32 >> 4), idS, kk > 0 ? 1u : 0u);
        }
        tc::commit(smem_u32(&sh->s_full[t][h & 1]));
      };
      auto issue_pv = [&](int h) {
        const uint64_t db =
            dv0 + static_cast<uint64_t>(((ring_slot((h & ~1) + 1) * Lt::kTileBytes) >> 4) +
                                        (h & 1) * kHalfStep);
#pragma unroll
        for (int kk = 0; kk < kHalfKeys / 16; ++kk)
          tc::mma_ts(tmem + col_o(t), tmem + col_s(t, h) + 8 * kk, db + 128 * kk, idO,
                     h > 0 || kk > 0 ? 1u : 0u);
        tc::commit(smem_u32(h == H - 1 ? &sh->o_done[t] : &sh->pv_done[t]));
      };
      auto full = [&](int e) {   // ring element e is in shared memory, widened
        return quick_wait(smem_u32(&sh->kv_full[ring_slot(e)]), ring_phase(e), abort, a.err, wlim);
      };
      auto empty = [&](int e) { tc::commit(smem_u32(&sh->kv_empty[ring_slot(e)])); };
      bool go = quick_wait(q_conv, 0, abort, a.err, wlim) && full(0);
      if (go) {
        tc::fence_after_sync();
        if (tc::elect_one()) {
          issue_s(0);
          if (H > 1) issue_s(1);
          empty(0);
        }
        __syncwarp();
      }
      // Half step h: P V, then S of half step h + 2, over the columns that P was
      // read from (a thread's products execute in the order of their issue).
      for (int h = 0; go && h < H; ++h) {
        const bool more = h + 2 < H;
        go = quick_wait(smem_u32(&sh->p_full[t][h & 1]), (h >> 1) & 1, abort, a.err, wlim) &&
             ((h & 1) || full(h + 1));   // (V of this tile: element h + 1)
        if (!go) break;
        tc::fence_after_sync();
        if (tc::elect_one()) issue_pv(h);
        __syncwarp();
        if (more) {
          go = (h & 1) || full(h + 2);   // (K of the next tile)
          if (!go) break;
          tc::fence_after_sync();
          if (tc::elect_one()) issue_s(h + 2);
          __syncwarp();
        }
        if ((h & 1) && tc::elect_one()) {   // both halves read: V, then the next K
          empty(h);
          if (more) empty(h + 1);
        }
        __syncwarp();
      }
      if (tc::elect_one()) {   // every product completes before TMEM is freed
        tc::commit(smem_u32(&sh->drain[t]));
        (void)mbar_wait(smem_u32(&sh->drain[t]), 0);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    more_regs<kRegsSoftmax>();
    const int t = warp >> 2;                      // query tile of this warpgroup
    const int quarter = warp & 3;                 // TMEM lanes this warp may touch
    const int row = quarter * 32 + lane;          // tile row == TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int tok = tok0 + t * tile_toks + row / G;
    const int g = row % G;
    const bool valid = tok <= tok_last && row < tile_toks * G;
    const int pos = L - qn + (valid ? tok : tok_last);
    const uint32_t tO = lanes + col_o(t);
    const uint32_t pv_done = smem_u32(&sh->pv_done[t]);
    float sl2 = a.scale_log2;
    // Block scales of a key tile, lanes 0-7 the K, 8-15 the V scales: ids two
    // tiles and scales one tile ahead.
    auto id_of = [&](int j) {
      const int b = (j0 + j) * (kTcKeys / kBlock) + (lane & 7);
      return lane < 16 && b >= b_lo && b < nblk
                 ? __ldg(bt + b) : -1;
    };
    auto scale_of = [&](int id) {   // (a block that is not read: any finite scale)
      return id >= 0 && id < a.num_blocks
                 ? __ldg(((lane & 8) ? a.v_scales : a.k_scales) +
                         static_cast<int64_t>(id) * a.num_kv_heads + kvh) : 1.f;
    };
    float scale_next = scale_of(id_of(0));
    int id_next = id_of(1);
    // this thread's Q row to fp16
    if (quick_wait(q_full, 0, abort, a.err, wlim)) {
      uint8_t* qrow = sQ + t * Lt::kQTile + row * 128;
      uint4 v[Lt::kHalves * 8];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < Lt::kHalves * 8; ++i) {
        v[i] = *reinterpret_cast<const uint4*>(qrow + (i >> 3) * Lt::kQHalf +
                                               (((i & 7) ^ (row & 7)) << 4));
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
      }
      const int ex = f16_fit_exponent(amax);
      float down = pow2f(-ex);
      sl2 *= pow2f(ex);
      if (sl2 < 0.f) {   // a negative scale: its sign goes to the query
        sl2 = -sl2;
        down = -down;
      }
#pragma unroll
      for (int i = 0; i < Lt::kHalves * 8; ++i)
        *reinterpret_cast<uint4*>(qrow + (i >> 3) * Lt::kQHalf + (((i & 7) ^ (row & 7)) << 4)) =
            make_uint4(bf16x2_to_f16x2(v[i].x, down), bf16x2_to_f16x2(v[i].y, down),
                       bf16x2_to_f16x2(v[i].z, down), bf16x2_to_f16x2(v[i].w, down));
      fence_proxy_async();   // generic writes, then the tensor core reads
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_conv);
    float m_used = -INFINITY, l = 0.f;
    float low = kInt8ScaleFloor;   // a V scale outside [low, low * kNearScales] marks its tile
    bool done = t < ntq;
    const int lo = a.window > 0 ? pos - a.window + 1 : 0;   // first key this row sees
    for (int h = 0; done && h < H; ++h) {
      if (!(h & 1)) {   // this tile's scales to shared memory, the next tile's on their way
        // (as int8_scale, but an infinite or NaN scale stays for now)
        const float now = scale_next < kInt8ScaleFloor ? kInt8ScaleFloor : scale_next;
        scale_next = scale_of(id_next);
        id_next = id_of((h >> 1) + 2);
        const float lv = log2f(__shfl_sync(0xffffffffu, now, 8 + (lane & 7)));
        // The largest V scale: patterns of positive numbers compare like the numbers.  A V
        // scale out of range and a K scale that is not finite mark the tile with
        // infinity, which sends its keys to the pass for the maximum.  (Told without a
        // vote or a branch of its own: those cost 2 to 30 us of the 564.)
        const bool is_v = (lane & 24) == 8;
        const bool fine = is_v ? now >= low && now <= low * kNearScales : now <= FLT_MAX;
        const uint32_t bits = !fine ? 0x7f800000u : (is_v ? __float_as_uint(now) : 0u);
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, bits));
        if (lane < 8)
          sh->sc[warp][lane] =
              make_float4(now, lv, ex2(kSumBias - lv), top * (1.f / kTwoSumBias));
        __syncwarp();
      }
      const float4* sc = sh->sc[warp] + (h & 1) * kHalfBlocks;
      const uint32_t tS = lanes + col_s(t, h);
      if (!quick_wait(smem_u32(&sh->s_full[t][h & 1]), (h >> 1) & 1, abort, a.err, wlim)) {
        done = false;
        break;
      }
      tc::fence_after_sync();
      // The weights are first formed against the reference m of the keys before:
      // no pass over the row for its maximum.  Only if one may have grown past
      // 2^15 (fp16 holds it until then; none is above the row sum times the
      // largest V scale), or there is no reference yet, the row is loaded again,
      // the maximum found and the weights formed anew.  P is stored after that
      // is settled, since it lies over S.
      float alpha = 1.f, ls;
      uint32_t pk[kHalfKeys / 2];
      bool find_max = __any_sync(0xffffffffu, valid && m_used == -INFINITY);
#pragma unroll 1
      while (true) {
        float x[kHalfKeys];
#pragma unroll
        for (int c0 = 0; c0 < kHalfKeys; c0 += 32) {
          uint32_t r[32];
          tc::ld32(tS + c0, r);
#pragma unroll
          for (int c = 0; c < 32; ++c) x[c0 + c] = __uint_as_float(r[c]);
        }
        tc::wait_ld();
        // causal mask on raw scores (also hides keys >= L)
        const int key0 = j0 * kTcKeys + h * kHalfKeys;
        // (warp-uniform branches: the votes below need every lane)
        if (__any_sync(0xffffffffu, key0 + kHalfKeys - 1 > pos || key0 < lo)) {
          // visible columns [nlo, nvis) of this row; one compare per element
          // where no row of the warp has a lower bound in these keys
          const int nvis = pos - key0 + 1;
          const int nlo = lo - key0;
          if (__any_sync(0xffffffffu, nlo > 0)) {
#pragma unroll
            for (int c = 0; c < kHalfKeys; ++c) x[c] = (c < nvis && c >= nlo) ? x[c] : -INFINITY;
          } else {
#pragma unroll
            for (int c = 0; c < kHalfKeys; ++c) x[c] = c < nvis ? x[c] : -INFINITY;
          }
        }
        if (find_max && !(sc[0].w <= FLT_MAX)) {   // a marked tile
          // A scale that is not finite becomes 1, where masked keys meet it too; the
          // rows that see a key of its block become NaN through their sums.
          float4 c = sh->sc[warp][lane & 7];
          const bool bad = !(c.x <= FLT_MAX) || !(c.y <= FLT_MAX);
          for (uint32_t left = __ballot_sync(0xffffffffu, bad) & 0xffu; left != 0; left &= left - 1) {
            const int p0 = (j0 + (h >> 1)) * kTcKeys + (__ffs(left) - 1) * kBlock;
            if (p0 <= pos && p0 + kBlock > lo) l = NAN;
          }
          // a V scale above the range moves it, to 2^16 above that scale
          const float up = bad ? 0.f : ex2(c.y + 16.f - 64.f);
          const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(up)));
          if (most > low * 0x1p16f) low = most;
          if (lane < 8) sh->sc[warp][lane] = make_float4(bad ? 1.f : c.x, bad ? 0.f : c.y, 0.f, c.w);
          __syncwarp();
        }
        if (find_max) {   // (the factors are not negative: maxima of raw scores serve)
          float mt = -INFINITY;
#pragma unroll
          for (int b = 0; b < kHalfBlocks; ++b) {
            const float* xb = x + b * kBlock;
            float u = tc::max3(xb[0], xb[1], xb[2]), w = tc::max3(xb[3], xb[4], xb[5]);
            u = tc::max3(u, xb[6], xb[7]);
            w = tc::max3(w, xb[8], xb[9]);
            u = tc::max3(u, xb[10], xb[11]);
            w = tc::max3(w, xb[12], xb[13]);
            u = tc::max3(u, xb[14], xb[15]);
            mt = fmaxf(mt, fmaf(fmaxf(u, w), fmaf(sc[b].x, sl2, FLT_MIN), sc[b].y));
          }
          if (mt > m_used + kLazyRescale) {
            // (l in two steps: it may be far above 1 where the factor is below 2^-126)
            const float half = (m_used == -INFINITY) ? 0.f : ex2(0.5f * (m_used - mt));
            alpha = half * half;
            l = l * half * half;
            m_used = mt;
          }
          // A marked tile's denominators come from the scores themselves (its weights
          // are not added): beside a far larger V scale weights go to zero.
          if (!(sc[0].w <= FLT_MAX)) {
            const float add = (m_used == -INFINITY) ? kSumBias : kSumBias - m_used;
#pragma unroll
            for (int b = 0; b < kHalfBlocks; ++b) {
              const float f = fmaf(sc[b].x, sl2, FLT_MIN);
#pragma unroll
              for (int k = b * kBlock; k < (b + 1) * kBlock; ++k) l += ex2(fmaf(x[k], f, add));
            }
          }
        }
        const float neg_mu = (m_used == -INFINITY) ? 0.f : -m_used;
        float part[2] = {0.f, 0.f}, top = 0.f;
#pragma unroll
        for (int b = 0; b < kHalfBlocks; ++b) {
          const float4 c = sc[b];
          // (above zero, so that a masked -inf stays what it is)
          const float f = fmaf(c.x, sl2, FLT_MIN), add = c.y + neg_mu;
          const uint64_t f2 = tc::pack_f32x2(f, f), a2 = tc::pack_f32x2(add, add);
          uint64_t acc = 0;
#pragma unroll
          for (int k = b * kBlock; k < (b + 1) * kBlock; k += 2) {
            float y0, y1;
            tc::fma_f32x2(x[k], x[k + 1], f2, a2, y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            pk[k / 2] = pack_f16(y0, y1);
            tc::add_f32x2(acc, y0, y1);
          }
          part[b & 1] = fmaf(tc::sum_f32x2(acc), c.z, part[b & 1]);
          if (b == 0) top = c.w;
        }
        ls = part[0] + part[1];
        if (find_max || !__any_sync(0xffffffffu, valid && !(ls * top <= 32768.f))) break;
        find_max = true;
      }
      if (h > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {   // rescale O in TMEM
        // (P V of h - 2 is complete, since S of these keys was issued after it, and
        // that of h waits for this warp)
        if (!warp_wait(pv_done, (h - 1) & 1, abort, a.err, wlim)) {
          done = false;
          break;
        }
        tc::fence_after_sync();
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tc::ld32(tO + c0, o);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
          tc::st32(tO + c0, o);
        }
      }
      tc::st32(tS, pk);
      l += ls;
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[t][h & 1]));
    }
    // ---- outputs
    const bool ok = done && warp_wait(smem_u32(&sh->o_done[t]), 0, abort, a.err, wlim);
    if (t < ntq) {
      tc::fence_after_sync();
      const float inv = l == 0.f ? 0.f : kTwoSumBias / l;   // (a NaN stays)
      // every row of the tile is a query row of this sequence: its rows go out
      // through the tile's Q slot (its products have all completed), in the
      // swizzled layout Q arrived in, and one TMA store per 64-column half (a row
      // per thread written straight to memory would make every store touch 32)
      const bool full_tile = !PARTS && tok0 + (t + 1) * tile_toks - 1 <= tok_last;
      uint8_t* srow = sQ + t * Lt::kQTile + row * 128;
      const int hq = kvh * G + g;
#pragma unroll 1
      for (int c0 = 0; ok && c0 < D; c0 += 32) {
        uint32_t o[32];
        tc::ld32(tO + c0, o);
        tc::wait_ld();
        if constexpr (PARTS) {   // the row's normalised partial
          if (valid) {
            float4* dst = reinterpret_cast<float4*>(
                a.ws_o + (part_row(a, s, tok, hq) * a.key_splits + key_part) * D + c0);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv, __uint_as_float(o[4 * v + 1]) * inv,
                                   __uint_as_float(o[4 * v + 2]) * inv,
                                   __uint_as_float(o[4 * v + 3]) * inv);
          }
        } else {
          __nv_bfloat16* orow = out + (static_cast<int64_t>(q0 + tok) * Hq + hq) * D + c0;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              w[c] = pack_bf16(__uint_as_float(o[8 * v + 2 * c]) * inv,
                               __uint_as_float(o[8 * v + 2 * c + 1]) * inv);
            const uint4 q = make_uint4(w[0], w[1], w[2], w[3]);
            const int j = (c0 % 64) / 8 + v;   // 16-byte chunk of the half
            if (full_tile)
              *reinterpret_cast<uint4*>(srow + (c0 / 64) * Lt::kQHalf + ((j ^ (row & 7)) << 4)) = q;
            else if (valid)
              *reinterpret_cast<uint4*>(orow + 8 * v) = q;
          }
        }
      }
      if constexpr (PARTS) {   // its log2-sum-exp, in the domain of m_used (NaN stays)
        if (ok && valid)
          a.ws_lse[part_row(a, s, tok, hq) * a.key_splits + key_part] =
              l != 0.f ? m_used + (log2f(l) - kSumBias) : -INFINITY;
      } else if (full_tile) {
        fence_proxy_async();   // generic writes, then the TMA engine reads
        // the tile's four warps (named barrier 1 + t); no store unless all wrote
        const bool all = named_barrier_and(1 + t, 128, ok);
        if (all && quarter == 0 && lane == 0) {
#pragma unroll
          for (int h = 0; h < Lt::kHalves; ++h)
            tma_store_3d(&omap, smem_u32(sQ + t * Lt::kQTile + h * Lt::kQHalf), h * 64, kvh * G,
                         q0 + tok0 + t * tile_toks);
          bulk_commit_group();
          bulk_wait_group_read0();   // shared memory stays until the reads are done
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 12) {
    tc::fence_after_sync();
    tc::dealloc(tmem, kTmemCols);
  }
}

// Merges the key_splits partials of every prefill row, one warp per (row, q
// head): out = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M).  Rows of
// sequences with bad lengths (zeroed by the prefill kernel) are left alone.
constexpr int kMaxKeySplits = 8;

template <int D>
__global__ void __launch_bounds__(128) pkv_prefill_merge_kernel(const PrefillArgs a) {
  constexpr int PER = D / 32;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t r = w / a.num_q_heads;   // (sequence, row of max_query_len)
  const int s = a.seq_begin + static_cast<int>(r / a.max_query_len);
  const int j = static_cast<int>(r % a.max_query_len);
  if (s >= a.seq_begin + a.num_seqs) return;
  const int q0 = __ldg(a.query_start_loc + s), L = __ldg(a.context_lens + s);
  const int qn = __ldg(a.query_start_loc + s + 1) - q0;
  if (j >= qn || q0 < 0 || static_cast<int64_t>(q0) + qn > a.num_tokens || L < 1 ||
      static_cast<int64_t>(L) > a.bt_stride * kBlock || qn > L || qn > a.max_query_len)
    return;
  const int64_t row = w * a.key_splits;
  float lse[kMaxKeySplits], v[kMaxKeySplits][PER], M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMaxKeySplits; ++i) {
    lse[i] = i < a.key_splits ? a.ws_lse[row + i] : -INFINITY;
    M = fmaxf(M, lse[i]);
    if (lse[i] != -INFINITY) {
      const float* src = a.ws_o + (row + i) * D + lane * PER;
      if constexpr (PER == 4) *reinterpret_cast<float4*>(v[i]) = *reinterpret_cast<const float4*>(src);
      else *reinterpret_cast<float2*>(v[i]) = *reinterpret_cast<const float2*>(src);
    }
  }
  float acc[PER] = {}, den = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxKeySplits; ++i)
    if (lse[i] != -INFINITY) {
      const float f = exp2f(lse[i] - M);
      den += f;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(f, v[i][e], acc[e]);
    }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int hq = static_cast<int>(w - r * a.num_q_heads);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                       (static_cast<int64_t>(q0 + j) * a.num_q_heads + hq) * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(out + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

template <int D>
cudaError_t launch_t(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     const CUtensorMap& omap, const PrefillArgs& a, cudaStream_t stream) {
  constexpr int smem = smem_bytes<D>();
  const bool parts = a.key_splits > 1;
  const bool lpt = a.longest_first && static_cast<int64_t>(a.num_seqs) * a.num_mtiles <= kLptUnits;
  auto kfn = parts ? pkv_prefill_int8_kernel<D, kKeyParts>
                   : (lpt ? pkv_prefill_int8_kernel<D, kLongestFirst> : pkv_prefill_int8_kernel<D, kPlain>);
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.num_mtiles, a.num_kv_heads, a.num_seqs * (parts ? a.key_splits : 1));
  PrefillArgs b = a;
  debug_wait_settings(&b.wait_limit_ns, &b.debug_stall);
  kfn<<<grid, kThreads, smem, stream>>>(qmap, kmap, vmap, omap, b);
  e = cudaGetLastError();
  if (e != cudaSuccess || !parts) return e;
  const int64_t warps = static_cast<int64_t>(a.num_seqs) * a.max_query_len * a.num_q_heads;
  pkv_prefill_merge_kernel<D><<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_int8(const CUtensorMap& qmap, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, const CUtensorMap& omap,
                                   const PrefillArgs& a, int head_size, cudaStream_t stream) {
  if (a.num_seqs == 0 || a.num_mtiles == 0) return cudaSuccess;
  return head_size == 128 ? launch_t<128>(qmap, kmap, vmap, omap, a, stream)
                          : launch_t<64>(qmap, kmap, vmap, omap, a, stream);
}

// Parts of the keys for a launch of `ctas` CTAs whose longest walks `tiles` key
// tiles: as many as leave each two tiles and have an SM each, the next power of
// two if that has them too (2 to 3 us shorter); none below six tiles, where the
// merge costs what the parts save.  64 tokens, 32 q / 8 kv heads, us in one
// part - in parts: 3 tiles 15.1 - 19.5 in 3, 4 tiles 17.1 - 16.3 in 4, 6 tiles
// 21.1 - 18.5 in 4 (21.7 in 3), 8 tiles 25.0 - 18.4 in 4 (22.2 in 2), 12 tiles
// 32.6 - 18.8 in 8 (22.0 in 6), 64 tiles 133 - 30.8 in 8.
int prefill_int8_key_splits(int64_t ctas, int tiles, int num_sms) {
  if (ctas <= 0 || tiles < 6) return 1;
  const int64_t most = std::min<int64_t>(num_sms / ctas, kMaxKeySplits);
  const int64_t n = std::max<int64_t>(std::min<int64_t>(most, tiles / 2), 1);
  int64_t p = 1;
  while (p < n) p *= 2;
  return static_cast<int>(p <= most ? p : n);
}

}  // namespace pkv
