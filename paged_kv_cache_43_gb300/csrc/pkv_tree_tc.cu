// pkv_tree_tc.cu -- attention of a tree of drafted tokens over bf16 and e4m3 caches, on
// tcgen05.
//
// Mathematics as in pkv_tree.cu.  A row is a (drafted token, q head) pair of one kv head;
// S = Q K^T and O += P V run on 128 rows x 64 keys, P = 2^(scale log2(e) s - m) rounded to
// bf16, as both operands of a product have one type (e4m3 caches: everything on fp16, to which
// codes widen exactly; K's descale joins the score scale, V's the output).  m is a reference, not the running maximum: it moves only
// when a step's weights sum to more than kTreeMost, so most steps need no pass for the maximum
// and no rescaling of O.  The denominator of bf16 sums the rounded weights, so the output
// is a convex combination of V rows.
//
// Work.  Few query rows share each key, so the keys' bytes are the bound (HBM) up to
// about 100 rows a kv head, the chain S - softmax - P V beyond.  All units (sequence, kv
// head) of the batch lie on one line, 64-key steps and a start each, which is cut into
// equal ranges, one a worker (its lengths are read on the device).  A worker is a CTA for
// each tile of 128 rows: they walk the same keys side by side, and find each other's in L2.
// A unit that lies in several ranges leaves partials, at most two a worker, which a second
// kernel merges; all others are written at once.  Two CTAs an SM (each 256 of the 512
// TMEM columns), so one's products and copies run under the other's softmax.  Warps:
//   0-3  softmax, a thread a row, and the rows out at the end of a unit
//   4, 5 start the TMA copies of K, of V (a box per cache block and 64 columns)
//   6    issues the products: S of the next 64 keys is formed while these are exponentiated
//        (S has two buffers, P lies over S)
//   7    finds the CTA's units and starts the copies of Q
//   8-11 (e4m3) widen codes, K's and V's in turn
// The copies of a unit's keys begin while the one before it is computed.
//
// What a key that a row does not see holds must not reach the row, although P = 0 there
// (0 x NaN): in the tiles with drafted keys the softmax warps zero V's rows behind the
// last key and its values that are not finite, and the rows that see those get them at
// the end.
//
// Measured (8 kv heads of 128): 8 sequences of 64 drafts over 2K to 8K keys, 32 q heads, 66 us,
// 3.0 TB/s of keys; 16 of 26 drafts over 16K to 32K keys, 64 q heads, 358 us, 4.4 TB/s (at 2070 MHz; 382 us
// where the load lasts and the power limit brings the clock to 1770 MHz); one of 300
// drafts over 16000 keys, 64 q heads, 165 us, 0.95 PFLOP/s.  A step takes 1.6 us a CTA, of
// which the tensor core works 0.34: the way from S over the softmax warps to P bounds it.
// e4m3, 128 sequences of 1 to 24 drafts over 64 to 8192 keys: 304 us, the same steps with half
// the bytes.
#include "pkv_tree_tc.cuh"

namespace pkv {

namespace {

constexpr int kKeys = kTreeStepKeys;            // keys of a step
constexpr int kStepBlocks = kKeys / kBlock;
constexpr int kRows = kTreeRows;
constexpr uint32_t kCols = 256;                 // TMEM columns of a CTA
// S of step h at 64 (h % 2), P over its first 32 columns; O at 128.
__device__ __forceinline__ uint32_t col_s(int h) { return 64u * (h & 1); }
constexpr uint32_t kColO = 128;

template <int D, bool FP8>
struct Lay {
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = kRows * 128;    // 64 columns: 128 rows x 128 B
  static constexpr int kQ = kHalves * kQHalf;
  static constexpr int kTHalf = kKeys * 128;
  static constexpr int kTile = kHalves * kTHalf;
  static constexpr int kCodes = kKeys * D;
  // Slots of K and as many of V.  e4m3: head_size 128 widens codes in place, in the first half
  // of the slot (its columns 0-63) where they landed; with 64, where a row's fp16 values lie over
  // other rows' codes, codes have a ring of their own.  (Of their own with 128, too, they left
  // room for one tile to be multiplied from: 128 sequences of 64 to 8192 keys 331 us.)
  static constexpr bool kInPlace = FP8 && D == 128;
  static constexpr int kSlots = FP8 && D == 64 ? 3 : 2 * 128 / D;
  static constexpr int kCodeSlots = FP8 && D == 64 ? 4 : 0;
  static constexpr int kLandSlots = kInPlace ? kSlots : kCodeSlots;
  static constexpr int kRing = 2 * kSlots * kTile, kCodeRing = 2 * kCodeSlots * kCodes;
  static constexpr int kStage = 4 * 32 * 128;   // rows on their way out: 32 x 32 fp32 a warp
};

template <int D, bool FP8>
struct Shared {
  using L = Lay<D, FP8>;
  uint64_t q_full, q_empty, q_conv, pv_done, o_done, fixed, drain;
  uint64_t s_full[2], p_full[2];
  uint64_t full[2][L::kSlots], empty[2][L::kSlots];                    // of K, of V
  uint64_t code_full[2][L::kLandSlots + 1], code_empty[2][L::kLandSlots + 1];   // e4m3: codes there
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Seg seg[kSegs];
  uint32_t tmem_base;
  int32_t abort;
  int32_t v_odd[2];   // by the segment's parity: its number + 1 if a drafted V value is not finite
};

// Two CTAs of 113 KB and the 1 KB that each costs are the SM's 228 KB.
template <int D, bool FP8>
constexpr int smem_bytes() {
  using L = Lay<D, FP8>;
  constexpr int need = L::kQ + L::kRing + L::kCodeRing + L::kStage + static_cast<int>(sizeof(Shared<D, FP8>));
  static_assert(need <= 113 * 1024, "two CTAs per SM");
  return need;
}

template <bool FP8>
constexpr int kThreads = FP8 ? 384 : 256;
// e4m3: launched with 80 registers a thread; the softmax warps take 128, the other two
// warpgroups keep 56.
constexpr int kRegsSoftmax = 128, kRegsOther = 56;
static_assert(128 * kRegsSoftmax + 256 * kRegsOther <= 384 * 80, "register split");

// Widens a tile's e4m3 codes (rows of D bytes, swizzled as they landed) into the fp16 tile
// layout; four warps, 16 rows each, read before they are written.  D = 128: 8 lanes, which a shared-memory access serves
// together, take 4 chunks of one half in two rows whose numbers differ in bits 0 and 2, so
// that reads and writes fall into different banks.
template <int D>
__device__ __forceinline__ void widen(const uint8_t* codes, uint8_t* tile, int w, int lane) {
  constexpr int kEach = D / 32;   // chunks of 16 codes of a lane
  const int c = D == 128 ? 4 * ((lane >> 3) & 1) + (lane & 3) : lane & 3;
  uint4 v[kEach];
  auto row = [&](int i) {
    return 16 * w + 8 * (D == 128 ? i >> 1 : i) +
           (D == 128 ? ((lane >> 4) ^ ((lane & 4) ? 5 : 0)) ^ (2 * (i & 1)) : lane >> 2);
  };
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = row(i);
    v[i] = *reinterpret_cast<const uint4*>(codes + swz8<D>(r, c));
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int r = row(i), j = 2 * (c & 3);
    uint8_t* to = tile + (c >> 2) * (kKeys * 128) + r * 128;
    const uint2 a = e4m3x4_to_f16x4(v[i].x), b = e4m3x4_to_f16x4(v[i].y);
    const uint2 d = e4m3x4_to_f16x4(v[i].z), e = e4m3x4_to_f16x4(v[i].w);
    *reinterpret_cast<uint4*>(to + ((j ^ (r & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint4*>(to + (((j + 1) ^ (r & 7)) << 4)) = make_uint4(d.x, d.y, e.x, e.y);
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads<FP8>, 2)
    pkv_tree_tc_kernel(const __grid_constant__ CUtensorMap qmap,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
  using L = Lay<D, FP8>;
  // (the merge, a programmatic dependent launch, waits for this grid's end itself)
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                            // [half][128 rows x 128 B]
  uint8_t* sKV = smem + L::kQ;                   // [K, V][slot][half][64 keys x 128 B]
  uint8_t* sCodes = sKV + L::kRing;              // [K, V][slot][64 keys x D]
  uint8_t* sStage = sCodes + L::kCodeRing;
  Shared<D, FP8>* sh = reinterpret_cast<Shared<D, FP8>*>(sStage + L::kStage);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int G = a.group, Hq = a.num_q_heads;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);

  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&qmap);
    prefetch_tensor_map(&kmap);
    prefetch_tensor_map(&vmap);
    mbar_init(bar(sh->q_full), 1);
    mbar_init(bar(sh->q_empty), 1);
    mbar_init(bar(sh->q_conv), 4);
    mbar_init(bar(sh->pv_done), 1);
    mbar_init(bar(sh->o_done), 1);
    mbar_init(bar(sh->fixed), 4);
    mbar_init(bar(sh->drain), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh->s_full[i]), 1);
      mbar_init(bar(sh->p_full[i]), 4);
      for (int j = 0; j < L::kSlots; ++j) {
        mbar_init(bar(sh->full[i][j]), FP8 ? 4 : 1);
        mbar_init(bar(sh->empty[i][j]), 1);
      }
      for (int j = 0; j < L::kLandSlots; ++j) {
        mbar_init(bar(sh->code_full[i][j]), 1);
        mbar_init(bar(sh->code_empty[i][j]), 4);
      }
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar(sh->seg_full[i]), 1);
      mbar_init(bar(sh->seg_empty[i]), FP8 ? 11 : 7);   // the warps that read it
    }
    sh->abort = 0;
    sh->v_odd[0] = sh->v_odd[1] = 0;
    fence_barrier_init();
  }
  if (warp == 7) tc::alloc(smem_u32(&sh->tmem_base), kCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
  volatile int32_t* abort = &sh->abort;
  const uint64_t wlim = wait_limit(a.wait_limit_ns);
  auto wait = [&](uint64_t& b, int use, int slots) {   // the phase of a slot's turn in the use-th round
    return quick_wait(smem_u32(&b), static_cast<uint32_t>(use / slots) & 1, abort, a.err, wlim);
  };
  // The CTA's i-th segment; false: there is none (or a wait gave up).
  auto take = [&](int i, Seg& g) {
    if (!wait(sh->seg_full[i % kSegs], i, kSegs)) return false;
    g = sh->seg[i % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(sh->seg_empty[i % kSegs]));
    return g.steps >= 0;
  };
  Seg g;

  if (warp >= 4) {
    if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 4 || warp == 5) {
      // ------------------------------------------------------------ copies of K, V
      const int is_v = warp - 4;
      constexpr bool kApart = FP8 && !L::kInPlace;   // codes have their own ring
      constexpr int kDepth = kApart ? L::kCodeSlots : L::kSlots;
      constexpr int kBytes = kApart ? L::kCodes : L::kTile;
      uint64_t* land = FP8 ? sh->code_full[is_v] : sh->full[is_v];
      uint64_t* empty = kApart ? sh->code_empty[is_v] : sh->empty[is_v];
      uint8_t* ring = (kApart ? sCodes : sKV) + is_v * kDepth * kBytes;
      const CUtensorMap* map = is_v ? &vmap : &kmap;
      // several row tiles read the same keys: then they stay in L2
      const uint64_t policy = a.cta_tiles > 1 ? policy_evict_normal() : policy_evict_first();
      // Test hook: the first K tile is withheld (no copy, no arrival).
      const bool withhold = a.debug_stall != 0 && !is_v;
      int n = 0;   // steps so far
      bool go = true;
      for (int si = 0; go && take(si, g); ++si) {
        const int32_t* bt = a.block_tables + g.s * a.bt_stride;
        const int b0 = g.step0 * kStepBlocks;
        const int b1 = min((g.L + kBlock - 1) / kBlock, b0 + g.steps * kStepBlocks);
        auto ids = [&](int k) {   // block ids of eight steps, a lane a block
          const int b = b0 + 32 * k + lane;
          return b < b1 ? __ldg(bt + b) : -1;
        };
        int cur = ids(0), next = ids(1);
        for (int h = 0; h < g.steps; ++h, ++n) {
          if (h > 0 && (h & 7) == 0) {
            cur = next;
            next = ids((h >> 3) + 1);
          }
          if (n >= kDepth && !wait(empty[n % kDepth], n - kDepth, kDepth)) {
            go = false;
            break;
          }
          if (withhold && n == 0) continue;
          const uint32_t dst = smem_u32(ring + n % kDepth * kBytes), full = bar(land[n % kDepth]);
          int id[kStepBlocks];
          bool ok[kStepBlocks];
          uint32_t bytes = 0;
#pragma unroll
          for (int b = 0; b < kStepBlocks; ++b) {
            id[b] = __shfl_sync(0xffffffffu, cur, kStepBlocks * (h & 7) + b);
            const bool in = b0 + h * kStepBlocks + b < b1;
            ok[b] = in && id[b] >= 0 && id[b] < a.num_blocks;
            if (!is_v && in && !ok[b] && lane == 0) raise_error(a.err, PKV_ERR_BLOCK_ID);
            bytes += ok[b] ? kBlock * D * (FP8 ? 1 : 2) : 0;
          }
          if (lane == 0) {
            if (bytes == 0) {
              mbar_arrive(full);
            } else {
              mbar_arrive_expect_tx(full, bytes);
#pragma unroll
              for (int b = 0; b < kStepBlocks; ++b) {
                if (!ok[b]) continue;
                if constexpr (FP8) {
                  tma_load_3d(dst + b * kBlock * D, map, full, 0, g.kvh, id[b] * kBlock, policy);
                } else {
#pragma unroll
                  for (int k = 0; k < L::kHalves; ++k)
                    tma_load_3d(dst + k * L::kTHalf + b * 2048, map, full, k * 64, g.kvh,
                                id[b] * kBlock, policy);
                }
              }
            }
          }
        }
      }
      // every copy has landed before the CTA's shared memory is given up
      for (int i = max(0, n - kDepth); i < n; ++i)
        if (lane == 0 && !(withhold && i == 0))
          (void)mbar_wait(bar(land[i % kDepth]), static_cast<uint32_t>(i / kDepth) & 1);
      __syncwarp();
    } else if (warp == 6) {
      // ------------------------------------------------------------ products
      constexpr uint32_t idS = FP8 ? tc::idesc_f16_f32(kRows, kKeys, 0, 0)
                                   : tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
      constexpr uint32_t idO = FP8 ? tc::idesc_f16_f32(kRows, D, 0, 1)
                                   : tc::idesc_bf16_f32(kRows, D, 0, 1);
      const uint64_t dq = tc::smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem_u32(sKV), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_u32(sKV) + L::kSlots * L::kTile, L::kTHalf, 1024);
      int base = 0;   // steps before this segment
      auto start_s = [&](int h) {   // S of the segment's step h
        const int n = base + h;
        if (!wait(sh->full[0][n % L::kSlots], n, L::kSlots)) return false;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint64_t db = dk + static_cast<uint64_t>((n % L::kSlots * L::kTile) >> 4);
          const uint32_t d = tmem + col_s(n);
          if constexpr (D == 128) {
            tc::mma_ss_x8<2, 4, 6, 1024, 1026, 1028, 1030, 2, 4, 6, 512, 514, 516, 518>(d, dq, db,
                                                                                      idS, 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_ss(d, dq + (kk * 32 >> 4), db + (kk * 32 >> 4), idS, kk > 0 ? 1u : 0u);
          }
          tc::commit(bar(sh->s_full[n & 1]));
          tc::commit(bar(sh->empty[0][n % L::kSlots]));
          if (h == g.steps - 1) tc::commit(bar(sh->q_empty));
        }
        __syncwarp();
        return true;
      };
      bool go = true;
      for (int si = 0; go && take(si, g); ++si) {
        go = wait(FP8 ? sh->q_conv : sh->q_full, si, 1) && start_s(0) && (g.steps < 2 || start_s(1));
        for (int h = 0; go && h < g.steps; ++h) {
          const int n = base + h;
          go = wait(sh->p_full[n & 1], n >> 1, 1) && wait(sh->full[1][n % L::kSlots], n, L::kSlots);
          if (!go) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint64_t db = dv + static_cast<uint64_t>((n % L::kSlots * L::kTile) >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
              tc::mma_ts(tmem + kColO, tmem + col_s(n) + 8 * kk, db + 128 * kk, idO,
                         h > 0 || kk > 0 ? 1u : 0u);
            tc::commit(bar(h == g.steps - 1 ? sh->o_done : sh->pv_done));
            tc::commit(bar(sh->empty[1][n % L::kSlots]));
          }
          __syncwarp();
          // (S over the columns that P was read from: products execute in their order)
          if (h + 2 < g.steps) go = start_s(h + 2);
        }
        base += g.steps;
      }
      if (tc::elect_one()) {   // every product completes before TMEM is freed
        tc::commit(bar(sh->drain));
        (void)mbar_wait(bar(sh->drain), 0);
      }
      __syncwarp();
    } else if (warp == 7) {
      // ------------------------------------------------------------ units, copies of Q
      const int tile_rows = a.tile_toks * G;
      int count = 0;         // segments so far
      tree_walk(a, kKeys, [&](const Seg& e) {
        if (count >= kSegs && !wait(sh->seg_empty[count % kSegs], count - kSegs, kSegs)) return false;
        if (lane == 0) {
          sh->seg[count % kSegs] = e;
          mbar_arrive(bar(sh->seg_full[count % kSegs]));
        }
        __syncwarp();
        if (count > 0 && !wait(sh->q_empty, count - 1, 1)) return false;
        if (lane == 0) {   // (rows behind the sequence's: other rows, or zeros; not used)
          mbar_arrive_expect_tx(bar(sh->q_full), L::kHalves * tile_rows * 128);
#pragma unroll
          for (int k = 0; k < L::kHalves; ++k)
            tma_load_3d(smem_u32(sQ + k * L::kQHalf), &qmap, bar(sh->q_full), k * 64, e.kvh * G,
                        e.q0 + e.row0 / G, policy_evict_normal());
        }
        ++count;
        return true;
      });
      if (count > 0 && lane == 0) (void)mbar_wait(bar(sh->q_full), (count - 1) & 1);   // (landed)
      __syncwarp();
      if (count < kSegs || wait(sh->seg_empty[count % kSegs], count - kSegs, kSegs)) {
        if (lane == 0) {
          sh->seg[count % kSegs].steps = -1;
          mbar_arrive(bar(sh->seg_full[count % kSegs]));
        }
      }
      __syncwarp();
    } else if constexpr (FP8) {
      // ------------------------------------------------------------ widening
      const int w = warp - 8;
      int base = 0;
      auto one = [&](int v, int n) {   // K's (0) or V's (1) tile of step n
        if (!wait(sh->code_full[v][n % L::kLandSlots], n, L::kLandSlots)) return false;
        uint8_t* tile = sKV + (v * L::kSlots + n % L::kSlots) * L::kTile;
        const uint8_t* codes = tile;
        if constexpr (!L::kInPlace) {
          codes = sCodes + (v * L::kCodeSlots + n % L::kCodeSlots) * L::kCodes;
          if (n >= L::kSlots && !wait(sh->empty[v][n % L::kSlots], n - L::kSlots, L::kSlots)) return false;
        }
        widen<D>(codes, tile, w, lane);
        fence_proxy_async();   // generic accesses, then the tensor core's reads and the next copy
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(sh->full[v][n % L::kSlots]));
          if (!L::kInPlace) mbar_arrive(bar(sh->code_empty[v][n % L::kLandSlots]));
        }
        return true;
      };
      bool go = true;
      for (int si = 0; go && take(si, g); ++si) {
        go = one(0, base);
        for (int h = 0; go && h < g.steps; ++h)   // (K a step ahead, as S is of P V)
          go = (h + 1 >= g.steps || one(0, base + h + 1)) && one(1, base + h);
        base += g.steps;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    tree_bad_sequences<D>(a, threadIdx.x, 128);
    const int row = warp * 32 + lane;            // tile row == TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    int base = 0, pv = 0;                        // steps, and products' pv_done, before this segment
    bool done = true;
    for (int si = 0; done && take(si, g); ++si) {
      const bool valid = row < g.rows, warp_valid = warp * 32 < g.rows;
      const TreeSeq q{g.q0, g.n, g.L, g.L - g.n, 0, false};
      // row r of the tile: its query row and head
      auto tok_of = [&](int r) { return g.q0 + (g.row0 + r) / G; };
      auto head_of = [&](int r) { return g.kvh * G + (g.row0 + r) % G; };
      const uint64_t* mask =
          a.tree_mask + static_cast<int64_t>(tok_of(valid ? row : g.rows - 1)) * a.mask_words;
      float sl2 = a.scale_log2, out_scale = 1.f;
      if constexpr (FP8) {   // this thread's row of Q to fp16, scaled by a power of two into its range
        const int64_t at = static_cast<int64_t>(g.s) * a.num_kv_heads + g.kvh;
        sl2 *= __ldg(a.k_descale + at);
        out_scale = __ldg(a.v_descale + at);
        if (!wait(sh->q_full, si, 1)) break;
        if (warp_valid) {
          uint8_t* qrow = sQ + row * 128;
          float amax = 0.f;
#pragma unroll
          for (int i = 0; i < L::kHalves * 8; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(qrow + (i >> 3) * L::kQHalf +
                                                            (((i & 7) ^ (row & 7)) << 4));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
          }
          const int ex = f16_fit_exponent(amax);
          const float down = pow2f(-ex);
          sl2 *= pow2f(ex);
#pragma unroll
          for (int i = 0; i < L::kHalves * 8; ++i) {
            uint4* p = reinterpret_cast<uint4*>(qrow + (i >> 3) * L::kQHalf + (((i & 7) ^ (row & 7)) << 4));
            const uint4 v = *p;
            *p = make_uint4(bf16x2_to_f16x2(v.x, down), bf16x2_to_f16x2(v.y, down),
                            bf16x2_to_f16x2(v.z, down), bf16x2_to_f16x2(v.w, down));
          }
          fence_proxy_async();   // generic writes, then the tensor core reads
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->q_conv));
      }
      float m = -INFINITY, l = 0.f;
      for (int h = 0; h < g.steps; ++h) {
        const int n = base + h;
        if (!wait(sh->s_full[n & 1], n >> 1, 1)) {
          done = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t tS = lanes + col_s(n);
        const int key0 = (g.step0 + h) * kKeys;
        const bool drafts = key0 + kKeys > q.first;   // keys that not every row sees, or none
        if (drafts) {
          // V's rows behind the last key become zero, and so do its drafted values that
          // are not finite.  (The wait for V is for its slot's next phase: P V of step n - 2 is
          // done, since S of this step was issued after it.)
          static_assert(L::kSlots >= 2, "phases of V's slots");
          if (!wait(sh->full[1][n % L::kSlots], n, L::kSlots)) {
            done = false;
            break;
          }
          constexpr int kEach = L::kHalves * 4;       // 16-byte chunks of a thread
          const int r = threadIdx.x >> 1, p = key0 + r;
          uint8_t* vrow = sKV + (L::kSlots + n % L::kSlots) * L::kTile + r * 128 +
                          (D == 128 ? (threadIdx.x & 1) * L::kTHalf : 0);
          auto chunk = [&](int i) {   // (in turns, so that 8 lanes' chunks lie in different banks)
            return reinterpret_cast<uint4*>(
                vrow + 16 * (D == 128 ? (i + r) & 7 : 4 * (threadIdx.x & 1) + ((i + r) & 3)));
          };
          if (p >= q.L) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) *chunk(i) = make_uint4(0, 0, 0, 0);
          } else if (p >= q.first) {
            uint32_t odd = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
              const uint4 v = *chunk(i);
              odd |= odd_halves<FP8>(v.x) | odd_halves<FP8>(v.y) | odd_halves<FP8>(v.z) | odd_halves<FP8>(v.w);
            }
            if (odd != 0) {
              sh->v_odd[si & 1] = si + 1;
#pragma unroll 1
              for (int i = 0; i < kEach; ++i) {
                const uint4 v = *chunk(i);
                *chunk(i) = make_uint4(even_value<FP8>(v.x), even_value<FP8>(v.y), even_value<FP8>(v.z),
                                       even_value<FP8>(v.w));
              }
            }
          }
          fence_proxy_async();   // generic writes, then the tensor core reads
        }
        if (warp_valid) {
          const uint64_t seen = drafts ? tree_bits(mask, q, key0) : ~0ull;
          float alpha = 1.f, ls;
          uint32_t pk[kKeys / 2];
          bool find = __any_sync(0xffffffffu, valid && m == -INFINITY);
#pragma unroll 1
          while (true) {
            if (find) {   // the largest visible score
              float top = -INFINITY;
#pragma unroll 1
              for (int c0 = 0; c0 < kKeys; c0 += 32) {
                uint32_t r[32];
                tc::ld32(tS + c0, r);
                tc::wait_ld();
                const uint32_t bits = static_cast<uint32_t>(seen >> c0);
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  top = fmaxf(top, (bits >> c & 1) ? __uint_as_float(r[c]) * sl2 : -INFINITY);
              }
              if (top > m) {
                alpha = m == -INFINITY ? 0.f : ex2(m - top);
                l *= alpha;
                m = top;
              }
            }
            const float neg_m = m == -INFINITY ? 0.f : -m;
            const uint64_t f2 = tc::pack_f32x2(sl2, sl2), a2 = tc::pack_f32x2(neg_m, neg_m);
            uint64_t acc = 0;
#pragma unroll
            for (int c0 = 0; c0 < kKeys; c0 += 32) {
              uint32_t r[32];
              tc::ld32(tS + c0, r);
              tc::wait_ld();
              const uint32_t bits = static_cast<uint32_t>(seen >> c0);
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                float y0, y1;
                tc::fma_f32x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]), f2, a2, y0, y1);
                if (drafts) {   // (warp-uniform)
                  y0 = (bits >> c & 1) ? y0 : -INFINITY;
                  y1 = (bits >> (c + 1) & 1) ? y1 : -INFINITY;
                }
                y0 = ex2(y0);
                y1 = ex2(y1);
                const uint32_t w = pack2<FP8>(y0, y1);
                pk[(c0 + c) / 2] = w;
                if constexpr (FP8) tc::add_f32x2(acc, y0, y1);
                else tc::add_f32x2(acc, bf16_lo(w), bf16_hi(w));
              }
            }
            ls = tc::sum_f32x2(acc);
            if (find || !__any_sync(0xffffffffu, valid && !(ls <= kTreeMost))) break;
            find = true;
          }
          if (h > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {   // rescale O
            // (P V of h - 1 is the last that was issued: that of h waits for this warp)
            if (!wait(sh->pv_done, pv + h - 1, 1)) {
              done = false;
              break;
            }
            tc::fence_after_sync();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t o[32];
              tc::ld32(lanes + kColO + c0, o);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tc::st32(lanes + kColO + c0, o);
            }
          }
          tc::st32(tS, pk);
          l += ls;
          tc::wait_st();
          tc::fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->p_full[n & 1]));
      }
      // ---- the rows out, 32 columns at a time through shared memory, 16-byte chunks of a row
      // swapped about so that neither a column nor a row of them falls into one bank
      if (lane == 0) mbar_arrive(bar(sh->fixed));   // (v_odd: every softmax warp's)
      done = done && wait(sh->o_done, si, 1) && wait(sh->fixed, si, 1);
      if (done && warp_valid) {
        tc::fence_after_sync();
        const bool odd = *reinterpret_cast<volatile int32_t*>(&sh->v_odd[si & 1]) == si + 1;
        const float inv = l == 0.f ? 0.f : out_scale / l;   // (a NaN stays)
        uint8_t* mine = sStage + warp * 32 * 128;
        const int count = min(g.rows - warp * 32, 32);
        const int64_t part = (static_cast<int64_t>(g.part) * a.cta_tiles + blockIdx.x % a.cta_tiles) * a.part_rows + warp * 32;
        // where this lane's row begins, in out or in the partials (rows behind the last: the last)
        const int mine_row = min(row, g.rows - 1);
        const int64_t at = (g.part < 0 ? static_cast<int64_t>(tok_of(mine_row)) * Hq + head_of(mine_row)
                                       : part + lane) * D;
        // (this lane's part of a row's 32 columns: 4 lanes a row of bf16, 8 of fp32)
        const int oc = g.part < 0 ? lane & 3 : lane & 7, orow = g.part < 0 ? lane >> 2 : lane >> 3;
        const int ostep = g.part < 0 ? 8 : 4;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tc::ld32(lanes + kColO + c0, o);
          tc::wait_ld();
          __syncwarp();   // (the columns before are read)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(mine + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                            __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
          __syncwarp();
#pragma unroll 2
          for (int r = orow; r < 32; r += ostep) {
            const uint8_t* src = mine + r * 128;
            const int64_t to = __shfl_sync(0xffffffffu, at, r) + c0;
            if (g.part < 0) {
              const float4 x = *reinterpret_cast<const float4*>(src + (((2 * oc) ^ (r & 7)) << 4));
              const float4 y = *reinterpret_cast<const float4*>(src + (((2 * oc + 1) ^ (r & 7)) << 4));
              if (r < count)
                *reinterpret_cast<uint4*>(out + to + 8 * oc) =
                    make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y),
                               pack_bf16(y.z, y.w));
            } else if (r < count) {
              *reinterpret_cast<float4*>(a.ws_o + to + 4 * oc) =
                  *reinterpret_cast<const float4*>(src + ((oc ^ (r & 7)) << 4));
            }
          }
        }
        if (odd) {
          __syncwarp();
#pragma unroll 1
          for (int r = 0; r < count; ++r) {
            const int64_t to = __shfl_sync(0xffffffffu, at, r);
#pragma unroll 1
            for (int d = lane; d < D; d += 32)
              add_odd_values<FP8, D>(a, g.s, g.kvh, q.first, g.step0 * kKeys,
                                     min(g.L, (g.step0 + g.steps) * kKeys),
                                     a.tree_mask + static_cast<int64_t>(tok_of(warp * 32 + r)) * a.mask_words,
                                     d, g.part < 0 ? nullptr : a.ws_o + to + d,
                                     g.part < 0 ? out + to + d : nullptr);
          }
        }
        if (g.part >= 0 && valid) a.ws_lse[part + lane] = l == 0.f ? -INFINITY : m + log2f(l);
      }
      base += g.steps;
      pv += g.steps - 1;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 7) {
    tc::fence_after_sync();
    tc::dealloc(tmem, kCols);
  }
}

// Merges the partials of the units that several workers computed: out = sum_i 2^(lse_i - M) O_i /
// sum_i 2^(lse_i - M).  The first worker of a unit holds its partial in the second of its
// two places, the others in their first.  A warp takes kMergeRows q heads of a query row, so that
// its way to the span (row, sequence, lengths: loads one after the other) is gone once for
// them, and their partials' loads overlap (8 sequences of 64 drafts, 32 q heads: 17 us with a
// warp a head).
constexpr int kMergeRows = 4;
template <int D>
__global__ void __launch_bounds__(128) pkv_tree_tc_merge_kernel(const TreeArgs a) {
  constexpr int PER = D / 32;
  constexpr int kEach = 32 / kMergeRows;   // partials looked up at a time
  // (a programmatic dependent launch: the partials are visible once this returns)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int chunks = (a.group + kMergeRows - 1) / kMergeRows;   // warps of a query row and kv head
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t t = w / (static_cast<int64_t>(a.num_kv_heads) * chunks);
  if (t >= a.num_tokens) return;
  const int in_row = static_cast<int>(w - t * a.num_kv_heads * chunks);
  const int kvh = in_row / chunks, g0 = (in_row - kvh * chunks) * kMergeRows;
  const int rows = min(a.group - g0, kMergeRows);
  TreeSeq q;
  const int s = tree_seq_of_row(a, static_cast<int>(t), q);
  if (s < 0) return;   // a row of no sequence, or of a bad one
  const int tile_rows = a.tile_toks * a.group;
  const int r = (static_cast<int>(t) - q.q0) * a.group + g0;   // (a token's rows are in one tile)
  const int tile = r / tile_rows, tg = tile / a.cta_tiles;
  const int2 span = a.span[(static_cast<int64_t>(s) * a.max_groups + tg) * a.num_kv_heads + kvh];
  // (one worker wrote the row itself; a span that there cannot be was not written, because a
  // wait gave up)
  if (span.y <= 1 || span.x < 0 || span.x >= a.workers || span.y > a.workers - span.x) return;
  auto place = [&](int i) {   // the first of the rows, in partial i
    return ((static_cast<int64_t>(span.x + i) * 2 + (i == 0 ? 1 : 0)) * a.cta_tiles +
            tile - tg * a.cta_tiles) * a.part_rows + r - tile * tile_rows;
  };
  // lane: row lane / kEach, partial lane % kEach of those looked up
  const int my_row = lane / kEach, my_part = lane % kEach;
  auto lse = [&](int i0) {
    return my_row < rows && i0 + my_part < span.y ? a.ws_lse[place(i0 + my_part) + my_row] : -INFINITY;
  };
  const float e0 = lse(0);
  float M = e0;
  bool nan = e0 != e0;
  for (int i0 = kEach; i0 < span.y; i0 += kEach) {
    const float e = lse(i0);
    M = fmaxf(M, e);
    nan = nan || e != e;
  }
#pragma unroll
  for (int off = kEach / 2; off > 0; off >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    nan = __shfl_xor_sync(0xffffffffu, nan ? 1 : 0, off) != 0 || nan;
  }
  if (nan) M = NAN;
  float acc[kMergeRows][PER] = {}, den = 0.f;
  for (int i0 = 0; i0 < span.y; i0 += kEach) {
    const float e = i0 == 0 ? e0 : lse(i0);
    // (below zero: a part that the row sees nothing of; one whose share is too small for fp32 still
    // counts, as what it holds may be infinite or NaN)
    const float f = e == -INFINITY ? -1.f : exp2f(e - M);
    den += e == -INFINITY ? 0.f : f;
#pragma unroll 2
    for (int p = 0; p < kEach; ++p) {
      if (i0 + p >= span.y) break;
      const float* o = a.ws_o + place(i0 + p) * D + lane * PER;
#pragma unroll
      for (int k = 0; k < kMergeRows; ++k) {
        const float wk = __shfl_sync(0xffffffffu, f, k * kEach + p);
        if (k < rows && !(wk < 0.f)) {   // (a NaN is a share)
          float v[PER];
          if constexpr (PER == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o + k * D);
          else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o + k * D);
#pragma unroll
          for (int x = 0; x < PER; ++x) acc[k][x] = fmaf(wk, v[x], acc[k][x]);
        }
      }
    }
  }
#pragma unroll
  for (int off = kEach / 2; off > 0; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
  const float inv = den == 0.f ? 0.f : 1.f / den;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                       (t * a.num_q_heads + kvh * a.group + g0) * D + lane * PER;
#pragma unroll
  for (int k = 0; k < kMergeRows; ++k) {
    const float ik = __shfl_sync(0xffffffffu, inv, k * kEach);
    if (k >= rows) break;
#pragma unroll
    for (int x = 0; x < PER; x += 2)
      *reinterpret_cast<__nv_bfloat162*>(out + k * D + x) =
          __floats2bfloat162_rn(acc[k][x] * ik, acc[k][x + 1] * ik);
  }
}

template <int D, bool FP8>
cudaError_t launch_t(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     const TreeArgs& a, cudaStream_t stream) {
  constexpr int smem = smem_bytes<D, FP8>();
  auto kfn = pkv_tree_tc_kernel<D, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kfn<<<static_cast<unsigned>(a.workers) * a.cta_tiles, kThreads<FP8>, smem, stream>>>(qmap, kmap, vmap, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const CUtensorMap& qmap, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, const TreeArgs& a, int head_size, bool fp8,
                           cudaStream_t stream) {
  TreeArgs b = a;
  debug_wait_settings(&b.wait_limit_ns, &b.debug_stall);
  cudaError_t e;
  if (a.keys_on_m)
    e = launch_tree_keys(qmap, kmap, vmap, b, fp8, stream);
  else if (fp8)
    e = head_size == 128 ? launch_t<128, true>(qmap, kmap, vmap, b, stream)
                         : launch_t<64, true>(qmap, kmap, vmap, b, stream);
  else
    e = head_size == 128 ? launch_t<128, false>(qmap, kmap, vmap, b, stream)
                         : launch_t<64, false>(qmap, kmap, vmap, b, stream);
  if (e != cudaSuccess || a.whole) return e;
  const int64_t warps = static_cast<int64_t>(a.num_tokens) * a.num_kv_heads *
                        ((a.group + kMergeRows - 1) / kMergeRows);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return head_size == 128 ? cudaLaunchKernelEx(&cfg, pkv_tree_tc_merge_kernel<128>, a)
                          : cudaLaunchKernelEx(&cfg, pkv_tree_tc_merge_kernel<64>, a);
}

}  // namespace pkv
