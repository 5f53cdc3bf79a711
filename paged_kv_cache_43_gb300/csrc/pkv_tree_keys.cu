// pkv_tree_keys.cu -- attention of a tree of drafted tokens on tcgen05 where a kv head has
// few query rows (at most 32), head_size 128.
//
// Mathematics as in pkv_tree_tc.cu, with keys instead of query rows on the products' M
// dimension: S^T = K Q^T (128 keys x N rows), O^T += V^T P^T (128 elements of the head x N).
// With query rows on M, a product costs what 128 rows cost, however few there are; here its
// cost is that of K's and V's way out of shared memory.
//
// A thread has a key: N scores in its TMEM lane.  The rows' references m lie in shared memory:
// the score of a unit's first key, and a row's maximum once a weight has passed kTreeMost
// (or if the first key is a draft, which not every row sees), which the four softmax warps
// agree on at a barrier every step; so most steps need no maximum over keys, which would go
// across lanes.  Denominators are sums a thread keeps for every row, added up at the end.  P^T
// goes through shared memory, a key's N weights in a row; O^T leaves as it lies, a lane an
// element of the head.
//
// Layout: one CTA an SM; the work's line, and what not-finite V values cost, as in
// pkv_tree_tc.cu.  Warps: 0-3 softmax; 4, 5 copies of K, V; 6 products; 7 units and Q; 8-11 the
// rows out (O^T has two buffers, so the next unit's products do not wait for it); 12-19
// (e4m3) widen codes.
//
// Bound by the keys' bytes (HBM): 64 sequences of 8 to 16 drafts over 128 to 4096 keys, 32 kv heads,
// 336 us, 6.2 TB/s, 0.92 of the copy rate (query rows on M: 374); e4m3 by its steps' chain (64
// sequences of 500 to 4000 keys, 8 kv heads, 16 rows 104 us, 2.6 TB/s, the shared-memory pipe 44 % and
// the issue slots 27 % busy; query rows on M: 165).
#include "pkv_tree_tc.cuh"

namespace pkv {

namespace {

constexpr int D = 128;
constexpr int kKeys = kTreeKeysStep;            // keys of a step
constexpr int kStepBlocks = kKeys / kBlock;
constexpr int kTHalf = kKeys * 128, kTile = 2 * kTHalf;
// Steps under way, with an S^T and a P^T each: a step's way from S^T over the softmax warps, P V and
// the next S^T into the same buffer takes 2.5 us, most of it the warps' waits for one another.
constexpr int kBufs = 3;
// TMEM: S^T of step h at 32 (h % 3), O^T of segment i at 128 + 32 (i % 2).
constexpr uint32_t kCols = 256;
__device__ __forceinline__ uint32_t col_s(int h) { return 32u * (h % kBufs); }
__device__ __forceinline__ uint32_t col_o(int i) { return 128u + 32u * (i & 1); }

// Slots of K and V tiles.  e4m3 codes land in the first half of a slot (its columns 0-63) and are
// widened in place: with rings of their own for the codes there was room for one tile of K to
// be multiplied from, and its way round (widen, product, widen) took 2 us a step.
constexpr int kKSlots = 2, kVSlots = 3;

template <bool FP8, int N>
struct Shared {
  uint64_t q_full, q_empty, q_conv, drain;
  uint64_t s_full[kBufs], p_full[kBufs];
  // of segment i: [i % 2]; its rows' sums and last product are there, its rows are out
  uint64_t sum_full[2], o_done[2], sum_empty[2];
  uint64_t k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots], v_empty[kVSlots];
  uint64_t k_land[kKSlots], v_land[kVSlots];   // e4m3: the codes are there
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Seg seg[kSegs];
  uint32_t tmem_base;
  int32_t abort;
  int32_t v_odd[2];              // a drafted V value of segment i is not finite: [i % 2]
  // (read and written 16 bytes at a time)
  alignas(16) uint32_t bits[4][N];   // of a step's keys 32 w + ..: which of them row c sees
  alignas(16) float scale[2][N];     // of segment i's rows: what scores are multiplied with (e4m3:
  alignas(16) float negm[2][N];      // Q's exponent is in it), and -m
  alignas(16) float alpha[N];        // what a step's new m makes of the sums so far, -1: no m yet
  float wide[2][4][N];               // a row's sum (of segment i), or maximum, over a warp's keys
  float inv[N];                      // what a row's O^T is multiplied with
  int64_t at[N];                     // where it goes: elements of out, or of the partials
};

template <bool FP8, int N>
constexpr int smem_bytes() {
  constexpr int need = 2 * N * 128 + kBufs * kKeys * 128 + (kKSlots + kVSlots) * kTile +
                       static_cast<int>(sizeof(Shared<FP8, N>)) + 1024;
  static_assert(need <= 227 * 1024 && N <= 32, "shared memory; a row's bit of 32");
  return need > 120 * 1024 ? need : 120 * 1024;   // (one CTA per SM)
}

template <bool FP8>
constexpr int kThreads = FP8 ? 640 : 384;
// Launched with 168 registers a thread (e4m3: 96), of which the other warpgroups hand some to
// the softmax warps.
constexpr int kRegsSoftmax = 240;
template <bool FP8>
constexpr int kRegsOther = FP8 ? 56 : 128;
static_assert(128 * kRegsSoftmax + 256 * kRegsOther<false> <= 384 * 168, "register split");
static_assert(128 * kRegsSoftmax + 512 * kRegsOther<true> <= 640 * 96, "register split");

// N TMEM columns of this thread's lane.
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Reduces M values a lane over the warp's lanes; a lane's result, that of the value whose number is
// returned, stays in v[0] (M = 16: two lanes have each).  A step halves what a lane holds: M - 1
// shuffles (and one) instead of 5 M.
template <int OFF, int N, int M, typename Op>
__device__ __forceinline__ int across(float (&v)[N], int lane, Op op) {   // (of the first M)
  if constexpr (OFF == 0) {
    return 0;
  } else if constexpr (M > 1) {
    constexpr int H = M / 2;
    const bool up = (lane & OFF) != 0;
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float keep = up ? v[H + i] : v[i], give = up ? v[i] : v[H + i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, OFF));
    }
    return (up ? H : 0) + across<OFF / 2, N, H>(v, lane, op);
  } else {
    v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], OFF));
    return across<OFF / 2, N, M>(v, lane, op);
  }
}

// Widens 16 rows (of batch b) of a tile's e4m3 codes in place into the fp16 tile layout (a row's
// codes lie where the first half of its fp16 values goes, and the warp reads all of its
// rows before it writes): 8 lanes, which a shared-memory access serves together, take 4 chunks of one half in two rows whose numbers
// differ in bits 0 and 2, so that reads and writes fall into different banks.
__device__ __forceinline__ void widen16(uint8_t* tile, int b, int lane) {
  const int c = 4 * ((lane >> 3) & 1) + (lane & 3), j = 2 * (c & 3);
  const int r0 = (lane >> 4) ^ ((lane & 4) ? 5 : 0);
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = *reinterpret_cast<const uint4*>(tile + swz8<D>(16 * b + 8 * (i >> 1) + (r0 ^ (2 * (i & 1))), c));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 16 * b + 8 * (i >> 1) + (r0 ^ (2 * (i & 1)));
    uint8_t* to = tile + (c >> 2) * kTHalf + r * 128;
    const uint2 x = e4m3x4_to_f16x4(v[i].x), y = e4m3x4_to_f16x4(v[i].y);
    const uint2 z = e4m3x4_to_f16x4(v[i].z), w = e4m3x4_to_f16x4(v[i].w);
    *reinterpret_cast<uint4*>(to + ((j ^ (r & 7)) << 4)) = make_uint4(x.x, x.y, y.x, y.y);
    *reinterpret_cast<uint4*>(to + (((j + 1) ^ (r & 7)) << 4)) = make_uint4(z.x, z.y, w.x, w.y);
  }
}

template <bool FP8, int N>
__global__ void __launch_bounds__(kThreads<FP8>, 1)
    pkv_tree_keys_kernel(const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
  using Sh = Shared<FP8, N>;
  // (the merge, a programmatic dependent launch, waits for this grid's end itself)
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;                                   // [slot][half][128 keys x 128 B]
  uint8_t* sV = sK + kKSlots * kTile;
  uint8_t* sP = sV + kVSlots * kTile;                   // [3][128 keys x 128 B]
  uint8_t* sQ = sP + kBufs * kKeys * 128;                   // [half][N rows x 128 B]
  Sh* sh = reinterpret_cast<Sh*>(sQ + 2 * N * 128);
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
    mbar_init(bar(sh->q_conv), 1);
    mbar_init(bar(sh->drain), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh->o_done[i]), 1);
      mbar_init(bar(sh->sum_full[i]), 4);
      mbar_init(bar(sh->sum_empty[i]), 4);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(bar(sh->s_full[i]), 1);
      mbar_init(bar(sh->p_full[i]), 4);
    }
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(bar(sh->k_full[i]), FP8 ? 8 : 1);
      mbar_init(bar(sh->k_empty[i]), 1);
      mbar_init(bar(sh->k_land[i]), 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(bar(sh->v_full[i]), FP8 ? 8 : 1);
      mbar_init(bar(sh->v_empty[i]), 1);
      mbar_init(bar(sh->v_land[i]), 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(bar(sh->seg_full[i]), 1);
      mbar_init(bar(sh->seg_empty[i]), FP8 ? 19 : 11);   // the warps that read it
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther<FP8>));
    if (warp == 4 || warp == 5) {
      // ------------------------------------------------------------ copies of K, V
      const bool is_v = warp == 5;
      const int depth = is_v ? kVSlots : kKSlots;
      uint64_t* land = FP8 ? (is_v ? sh->v_land : sh->k_land) : (is_v ? sh->v_full : sh->k_full);
      uint64_t* empty = is_v ? sh->v_empty : sh->k_empty;
      uint8_t* ring = is_v ? sV : sK;
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
        auto ids = [&](int k) {   // block ids of four steps, a lane a block
          const int b = b0 + 32 * k + lane;
          return b < b1 ? __ldg(bt + b) : -1;
        };
        int cur = ids(0), next = ids(1);
        for (int h = 0; h < g.steps; ++h, ++n) {
          if (h > 0 && (h & 3) == 0) {
            cur = next;
            next = ids((h >> 2) + 1);
          }
          if (n >= depth && !wait(empty[n % depth], n - depth, depth)) {
            go = false;
            break;
          }
          if (withhold && n == 0) continue;
          const uint32_t dst = smem_u32(ring + n % depth * kTile), full = bar(land[n % depth]);
          // blocks that there are, a bit each (bad ids are said once, and left out)
          const int blk = b0 + h * kStepBlocks + (lane & 7);
          const int id = __shfl_sync(0xffffffffu, cur, 8 * (h & 3) + (lane & 7));
          const bool in = blk < b1, ok = in && id >= 0 && id < a.num_blocks;
          if (!is_v && in && !ok && lane < 8) raise_error(a.err, PKV_ERR_BLOCK_ID);
          const uint32_t have = __ballot_sync(0xffffffffu, ok) & 0xffu;
          if (lane == 0) {
            if (have == 0) mbar_arrive(full);
            else mbar_arrive_expect_tx(full, __popc(have) * kBlock * D * (FP8 ? 1 : 2));
          }
          __syncwarp();
          if (lane < 8 && ok) {
            if constexpr (FP8) {
              tma_load_3d(dst + lane * kBlock * D, map, full, 0, g.kvh, id * kBlock, policy);
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                tma_load_3d(dst + k * kTHalf + lane * 2048, map, full, k * 64, g.kvh, id * kBlock,
                            policy);
            }
          }
          __syncwarp();
        }
      }
      // every copy has landed before the CTA's shared memory is given up
      for (int i = max(0, n - depth); i < n; ++i)
        if (lane == 0 && !(withhold && i == 0))
          (void)mbar_wait(bar(land[i % depth]), static_cast<uint32_t>(i / depth) & 1);
      __syncwarp();
    } else if (warp == 6) {
      // ------------------------------------------------------------ products
      constexpr uint32_t idS = FP8 ? tc::idesc_f16_f32(kKeys, N, 0, 0) : tc::idesc_bf16_f32(kKeys, N, 0, 0);
      constexpr uint32_t idO = FP8 ? tc::idesc_f16_f32(D, N, 1, 1) : tc::idesc_bf16_f32(D, N, 1, 1);
      const uint64_t dq = tc::smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_u32(sV), kTHalf, 1024);
      const uint64_t dp = tc::smem_desc_sw128(smem_u32(sP), 16, 1024);
      constexpr int QH = N * 8;   // from Q's first half to its second, in descriptor units
      int base = 0;   // steps before this segment
      auto start_s = [&](int h) {   // S^T of the segment's step h
        const int n = base + h;
        if (!wait(sh->k_full[n % kKSlots], n, kKSlots)) return false;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint64_t da = dk + static_cast<uint64_t>((n % kKSlots * kTile) >> 4);
          tc::mma_ss_x8<2, 4, 6, 1024, 1026, 1028, 1030, 2, 4, 6, QH, QH + 2, QH + 4, QH + 6>(
              tmem + col_s(n), da, dq, idS, 0u);
          tc::commit(bar(sh->s_full[n % kBufs]));
          tc::commit(bar(sh->k_empty[n % kKSlots]));
          if (h == g.steps - 1) tc::commit(bar(sh->q_empty));
        }
        __syncwarp();
        return true;
      };
      bool go = true;
      for (int si = 0; go && take(si, g); ++si) {
        go = wait(FP8 ? sh->q_conv : sh->q_full, si, 1);
        for (int h = 0; go && h < min(kBufs, g.steps); ++h) go = start_s(h);
        for (int h = 0; go && h < g.steps; ++h) {
          const int n = base + h;
          go = wait(sh->p_full[n % kBufs], n, kBufs) && wait(sh->v_full[n % kVSlots], n, kVSlots);
          // (O^T of the segment before the last is out)
          if (go && h == 0 && si >= 2) go = wait(sh->sum_empty[si & 1], (si >> 1) - 1, 1);
          if (!go) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint64_t da = dv + static_cast<uint64_t>((n % kVSlots * kTile) >> 4);
            const uint64_t db = dp + static_cast<uint64_t>((n % kBufs * kKeys * 128) >> 4);
            tc::mma_ss_x8<128, 256, 384, 512, 640, 768, 896, 128, 256, 384, 512, 640, 768, 896>(
                tmem + col_o(si), da, db, idO, h > 0 ? 1u : 0u);
            if (h == g.steps - 1) tc::commit(bar(sh->o_done[si & 1]));
            tc::commit(bar(sh->v_empty[n % kVSlots]));
          }
          __syncwarp();
          if (h + kBufs < g.steps) go = start_s(h + kBufs);
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
          mbar_arrive_expect_tx(bar(sh->q_full), 2 * tile_rows * 128);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            tma_load_3d(smem_u32(sQ + k * N * 128), &qmap, bar(sh->q_full), k * 64, e.kvh * G,
                        e.q0 + e.row0 / G, policy_evict_normal());
        }
        if constexpr (FP8) {   // Q to fp16, each row scaled by a power of two into its range
          const int i = count & 1;
          const float sl2 = a.scale_log2 *
              __ldg(a.k_descale + static_cast<int64_t>(e.s) * a.num_kv_heads + e.kvh);
          if ((count >= 2 && !wait(sh->sum_empty[i], (count >> 1) - 1, 1)) ||   // (scale is free)
              !wait(sh->q_full, count, 1))
            return false;
          const int c = lane & 15;   // 16 lanes a row, a 16-byte chunk each
#pragma unroll 4
          for (int r = lane >> 4; r < N; r += 2) {
            uint4* p = reinterpret_cast<uint4*>(sQ + (c >> 3) * N * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            const uint4 v = *p;
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
            for (int off = 8; off > 0; off >>= 1)
              amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const int ex = f16_fit_exponent(amax);
            const float down = pow2f(-ex);
            *p = make_uint4(bf16x2_to_f16x2(v.x, down), bf16x2_to_f16x2(v.y, down),
                            bf16x2_to_f16x2(v.z, down), bf16x2_to_f16x2(v.w, down));
            if (c == 0) sh->scale[i][r] = sl2 * pow2f(ex);
          }
          fence_proxy_async();   // generic writes, then the tensor core reads
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sh->q_conv));
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
    } else if (warp < 12) {
      // ------------------------------------------------------------ rows out
      const int key = threadIdx.x - 256;           // this thread's element of the head
      const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      auto all = [&](bool x) { return named_barrier_and(2, 128, x); };   // (as the softmax warps')
      for (int si = 0; all(take(si, g)); ++si) {
        const int i2 = si & 1;
        auto tok_of = [&](int r) { return g.q0 + (g.row0 + r) / G; };
        const float out_scale =
            FP8 ? __ldg(a.v_descale + static_cast<int64_t>(g.s) * a.num_kv_heads + g.kvh) : 1.f;
        if (!all(wait(sh->sum_full[i2], si >> 1, 1) && wait(sh->o_done[i2], si >> 1, 1))) break;
        tc::fence_after_sync();
        if (key < g.rows) {
          const float sum = (sh->wide[i2][0][key] + sh->wide[i2][1][key]) +
                            (sh->wide[i2][2][key] + sh->wide[i2][3][key]);
          sh->inv[key] = sum == 0.f ? 0.f : out_scale / sum;   // (a NaN stays)
          const int64_t part =
              (static_cast<int64_t>(g.part) * a.cta_tiles + blockIdx.x % a.cta_tiles) * a.part_rows + key;
          sh->at[key] = (g.part < 0 ? static_cast<int64_t>(tok_of(key)) * Hq + g.kvh * G + (g.row0 + key) % G
                                    : part) * D;
          if (g.part >= 0) a.ws_lse[part] = sum == 0.f ? -INFINITY : log2f(sum) - sh->negm[i2][key];
        }
        named_barrier(2, 128);
        const bool odd = *reinterpret_cast<volatile int32_t*>(&sh->v_odd[i2]) != 0;
#pragma unroll 1
        for (int c0 = 0; c0 < g.rows; c0 += 16) {
          uint32_t o[16];
          ld16(lanes + col_o(si) + c0, o);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sh->inv[c0 + i]);
          const int count = min(g.rows - c0, 16);
          if (g.part < 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < count) out[sh->at[c0 + i] + key] = __float2bfloat16(__uint_as_float(o[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < count) a.ws_o[sh->at[c0 + i] + key] = __uint_as_float(o[i]);
          }
        }
        if (odd)
#pragma unroll 1
          for (int r = 0; r < g.rows; ++r)
            add_odd_values<FP8, D>(a, g.s, g.kvh, g.L - g.n, g.step0 * kKeys,
                                   min(g.L, (g.step0 + g.steps) * kKeys),
                                   a.tree_mask + static_cast<int64_t>(tok_of(r)) * a.mask_words, key,
                                   g.part < 0 ? nullptr : a.ws_o + sh->at[r] + key,
                                   g.part < 0 ? out + sh->at[r] + key : nullptr);
        tc::fence_before_sync();
        named_barrier(2, 128);   // (inv, at and v_odd are read)
        if (key == 0) sh->v_odd[i2] = 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sh->sum_empty[i2]));
      }
    } else if constexpr (FP8) {
      // ------------------------------------------------------------ widening
      const int w = warp - 12;
      int base = 0;
      auto one = [&](uint64_t& land, uint64_t& full, uint8_t* tile, int n, int slots) {
        if (!wait(land, n, slots)) return false;
        widen16(tile, w, lane);
        fence_proxy_async();   // generic accesses, then the tensor core's reads and the next copy
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(full));
        return true;
      };
      auto one_k = [&](int n) {
        const int i = n % kKSlots;
        return one(sh->k_land[i], sh->k_full[i], sK + i * kTile, n, kKSlots);
      };
      auto one_v = [&](int n) {
        const int i = n % kVSlots;
        return one(sh->v_land[i], sh->v_full[i], sV + i * kTile, n, kVSlots);
      };
      bool go = true;
      for (int si = 0; go && take(si, g); ++si) {
        go = one_k(base);
        for (int h = 0; go && h < g.steps; ++h)   // (K a step ahead, as S is of P V)
          go = (h + 1 >= g.steps || one_k(base + h + 1)) && one_v(base + h);
        base += g.steps;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    tree_bad_sequences<D>(a, threadIdx.x, 128);
    const int key = threadIdx.x;                 // of a step's 128; also the element of the head
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // The four warps decide together, at barriers that each of them reaches the same number
    // of times whatever its own waits found: a wait that gave up ends all four.
    auto all = [&](bool x) { return named_barrier_and(1, 128, x); };
    int base = 0;                                // steps before this segment
    for (int si = 0; all(take(si, g)); ++si) {
      const TreeSeq q{g.q0, g.n, g.L, g.L - g.n, 0, false};
      const int i2 = si & 1;
      bool ok = true;   // this warp's waits went well
      if (si >= 2) ok = wait(sh->sum_empty[i2], (si >> 1) - 1, 1);   // (scale, negm and wide are free)
      float* const negm = sh->negm[i2];
      float* const scale = sh->scale[i2];
      uint64_t l[N / 2];   // sums of two rows each
#pragma unroll
      for (int c = 0; c < N / 2; ++c) l[c] = 0;
      // the mask bits of row threadIdx.x for the first step with drafts, under way early
      const int draft_step = max(q.first / kKeys - g.step0, 0);
      const uint64_t* mask = a.tree_mask +
          static_cast<int64_t>(g.q0 + (g.row0 + min(static_cast<int>(threadIdx.x), g.rows - 1)) / G) * a.mask_words;
      uint64_t bits_lo = 0, bits_hi = 0;
      auto look = [&](int h) {
        bits_lo = tree_bits(mask, q, (g.step0 + h) * kKeys);
        bits_hi = tree_bits(mask, q, (g.step0 + h) * kKeys + 64);
      };
      if (threadIdx.x < g.rows && draft_step < g.steps) look(draft_step);
      bool lacking = false;   // this thread's row (of its number) has no reference
      bool over = false;
      for (int h = 0; h < g.steps; ++h) {
        const int n = base + h;
        const uint32_t tS = lanes + col_s(n);
        const int key0 = (g.step0 + h) * kKeys, p = key0 + key;
        const bool drafts = key0 + kKeys > q.first;   // keys that not every row sees, or none
        if (drafts && threadIdx.x < g.rows) {   // (the last step's bits are read: its barriers)
          if (h != draft_step) look(h);
          sh->bits[0][threadIdx.x] = static_cast<uint32_t>(bits_lo);
          sh->bits[1][threadIdx.x] = static_cast<uint32_t>(bits_lo >> 32);
          sh->bits[2][threadIdx.x] = static_cast<uint32_t>(bits_hi);
          sh->bits[3][threadIdx.x] = static_cast<uint32_t>(bits_hi >> 32);
        }
        ok = ok && wait(sh->s_full[n % kBufs], n, kBufs);
        tc::fence_after_sync();
        // bit c: row c sees this thread's key
        uint32_t seen = ~0u;
        if (drafts) {
          // V's rows behind the last key become zero, and so do its drafted values that
          // are not finite.  (The wait for V is for its slot's next phase: P V of step n - 3 is
          // done, since S of this step was issued after it.)
          static_assert(kVSlots >= kBufs, "phases of V's slots");
          ok = ok && wait(sh->v_full[n % kVSlots], n, kVSlots);
          uint8_t* const vrow = sV + n % kVSlots * kTile + key * 128;
          auto chunk = [&](int i) {   // (in turns, so that 8 lanes' chunks lie in different banks)
            return reinterpret_cast<uint4*>(vrow + (i >> 3) * kTHalf + (((i + key) & 7) << 4));
          };
          if (ok && p >= q.L) {
#pragma unroll
            for (int i = 0; i < 16; ++i) *chunk(i) = make_uint4(0, 0, 0, 0);
          } else if (ok && p >= q.first) {
            uint32_t odd = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint4 v = *chunk(i);
              odd |= odd_halves<FP8>(v.x) | odd_halves<FP8>(v.y) | odd_halves<FP8>(v.z) | odd_halves<FP8>(v.w);
            }
            if (odd != 0) {
              sh->v_odd[i2] = 1;
#pragma unroll 1
              for (int i = 0; i < 16; ++i) {
                const uint4 v = *chunk(i);
                *chunk(i) = make_uint4(even_value<FP8>(v.x), even_value<FP8>(v.y), even_value<FP8>(v.z),
                                       even_value<FP8>(v.w));
              }
            }
          }
        }
        // The first key of a unit's first step, if all rows see it, gives the references.
        const bool given = h == 0 && key0 < q.first;
        if (!FP8 && h == 0 && ok && threadIdx.x < N) scale[threadIdx.x] = a.scale_log2;
        if (given && warp == 0 && ok) {
          float x[N];
#pragma unroll
          for (int c0 = 0; c0 < N; c0 += 16) ld16(tS + c0, reinterpret_cast<uint32_t*>(x) + c0);
          tc::wait_ld();
          if (lane == 0) {
#pragma unroll
            for (int c = 0; c < N; c += 4) {
              float4 f = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
              if constexpr (FP8) f = *reinterpret_cast<const float4*>(scale + c);
              auto m = [&](int i, float v) { return c + i < g.rows ? -v : -INFINITY; };
              *reinterpret_cast<float4*>(negm + c) = make_float4(
                  m(0, x[c] * f.x), m(1, x[c + 1] * f.y), m(2, x[c + 2] * f.z), m(3, x[c + 3] * f.w));
              *reinterpret_cast<float4*>(sh->alpha + c) = make_float4(1.f, 1.f, 1.f, 1.f);
            }
          }
        }
        if (given || drafts) named_barrier(1, 128);
        if (drafts) {
          seen = 0;
#pragma unroll
          for (int c = 0; c < N; c += 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(&sh->bits[warp][c]);
            const uint32_t four = (w.x >> lane & 1) | (w.y >> lane & 1) << 1 | (w.z >> lane & 1) << 2 |
                                  (w.w >> lane & 1) << 3;
            seen |= four << c;
          }
        }
        // ---- weights against the references that there are, N of this key, and the largest.  No
        // branch: the rows behind the tile's have a reference of infinity, their weights are 0.
        uint32_t w[N / 2];
        auto weigh = [&]() {
          float top = 0.f;
          const float sl2 = a.scale_log2;
          uint32_t all_r[N];   // (one wait: a load takes 0.2 us)
#pragma unroll
          for (int c0 = 0; c0 < N; c0 += 16) ld16(tS + c0, all_r + c0);
          tc::wait_ld();
#pragma unroll
          for (int c0 = 0; c0 < N; c0 += 16) {
            const uint32_t* r = all_r + c0;
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
              const ulonglong2 add = *reinterpret_cast<const ulonglong2*>(negm + c0 + c);
              ulonglong2 mul = make_ulonglong2(tc::pack_f32x2(sl2, sl2), tc::pack_f32x2(sl2, sl2));
              if constexpr (FP8) mul = *reinterpret_cast<const ulonglong2*>(scale + c0 + c);
              float y[4];
              tc::fma_f32x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]), mul.x, add.x, y[0], y[1]);
              tc::fma_f32x2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]), mul.y, add.y, y[2], y[3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = ex2(y[i]);
              top = tc::max3(top, y[0], y[1]);
              top = tc::max3(top, y[2], y[3]);
              w[(c0 + c) / 2] = pack2<FP8>(y[0], y[1]);
              w[(c0 + c) / 2 + 1] = pack2<FP8>(y[2], y[3]);
            }
          }
          if (drafts) {   // (what a key that a row does not see has weighed may raise top, no more)
#pragma unroll
            for (int c = 0; c < N / 2; ++c)
              w[c] &= ((seen >> (2 * c) & 1) ? 0xffffu : 0u) | ((seen >> (2 * c + 1) & 1) ? 0xffff0000u : 0u);
          }
          return top;
        };
        float top = 0.f;
        if (ok && (h > 0 || given)) top = weigh();
        if (!all(ok)) {   // (every warp leaves here, or none)
          over = true;
          break;
        }
        if (!all((h > 0 || given) && top <= kTreeMost && !lacking)) {
          // new references: each row's maximum over the step's keys
          float x[N];
#pragma unroll
          for (int c0 = 0; c0 < N; c0 += 16) ld16(tS + c0, reinterpret_cast<uint32_t*>(x) + c0);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < N; ++c) x[c] = (seen >> c & 1) ? x[c] * scale[c] : -INFINITY;
          const int at = across<16, N, N>(x, lane, [](float u, float v) { return fmaxf(u, v); });
          sh->wide[i2][warp][at] = x[0];
          named_barrier(1, 128);
          if (threadIdx.x < N) {
            const int c = threadIdx.x;
            const float x = fmaxf(fmaxf(sh->wide[i2][0][c], sh->wide[i2][1][c]),
                                  fmaxf(sh->wide[i2][2][c], sh->wide[i2][3][c]));
            // (h = 0: no reference yet; a row that has seen no key has 0, which its weights,
            // none, do not depend on)
            const float m = -negm[c];
            const bool first = h == 0 || sh->alpha[c] < 0.f;
            const bool none = first && x == -INFINITY;
            const bool grows = first ? !none : x > m;
            sh->alpha[c] = none ? -1.f : (first ? 0.f : (grows ? ex2(m - x) : 1.f));
            if (c >= g.rows) negm[c] = -INFINITY;
            else if (grows || h == 0) negm[c] = none ? 0.f : -x;
            lacking = none && c < g.rows;
          }
          named_barrier(1, 128);
          if (h > 0) {   // the sums so far, and O^T (once P V of the last step is done)
            ok = ok && wait(sh->v_empty[(n - 1) % kVSlots], n - 1, kVSlots);
            tc::fence_after_sync();
#pragma unroll 1
            for (int c0 = 0; ok && c0 < N; c0 += 16) {
              uint32_t o[16];
              ld16(lanes + col_o(si) + c0, o);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c)
                o[c] = __float_as_uint(__uint_as_float(o[c]) * fmaxf(sh->alpha[c0 + c], 0.f));
              st16(lanes + col_o(si) + c0, o);
            }
            tc::wait_st();
#pragma unroll
            for (int c = 0; c < N / 2; ++c) {
              const float2 v = *reinterpret_cast<const float2*>(&l[c]);
              l[c] = tc::pack_f32x2(v.x * fmaxf(sh->alpha[2 * c], 0.f), v.y * fmaxf(sh->alpha[2 * c + 1], 0.f));
            }
            named_barrier(1, 128);
            if (threadIdx.x < N && sh->alpha[threadIdx.x] >= 0.f) sh->alpha[threadIdx.x] = 1.f;
          }
          if (ok) (void)weigh();
        }
        // ---- to the sums (rounded, as they meet V: the output is a convex combination), and to
        // shared memory: 128 bytes for each key, N weights in them
        if (ok) {   // (else the next barrier ends it)
          uint8_t* prow = sP + n % kBufs * kKeys * 128 + key * 128;
#pragma unroll
          for (int c = 0; c < N / 2; ++c) tc::add_f32x2(l[c], lo2<FP8>(w[c]), hi2<FP8>(w[c]));
#pragma unroll
          for (int i = 0; i < N / 8; ++i)
            *reinterpret_cast<uint4*>(prow + ((i ^ (key & 7)) << 4)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          fence_proxy_async();   // generic writes, then the tensor core reads
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sh->p_full[n % kBufs]));
        }
      }
      if (over) break;
      // ---- denominators; the rows leave without these warps
      float sum[N];
#pragma unroll
      for (int c = 0; c < N / 2; ++c) {
        const float2 v = *reinterpret_cast<const float2*>(&l[c]);
        sum[2 * c] = v.x;
        sum[2 * c + 1] = v.y;
      }
      const int at = across<16, N, N>(sum, lane, [](float u, float v) { return u + v; });
      sh->wide[i2][warp][at] = sum[0];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh->sum_full[i2]));
      base += g.steps;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 7) {
    tc::fence_after_sync();
    tc::dealloc(tmem, kCols);
  }
}

template <bool FP8, int N>
cudaError_t launch_t(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     const TreeArgs& a, cudaStream_t stream) {
  constexpr int smem = smem_bytes<FP8, N>();
  auto kfn = pkv_tree_keys_kernel<FP8, N>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kfn<<<static_cast<unsigned>(a.workers) * a.cta_tiles, kThreads<FP8>, smem, stream>>>(qmap, kmap, vmap, a);
  return cudaGetLastError();
}

template <bool FP8>
cudaError_t launch_n(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                     const TreeArgs& a, cudaStream_t stream) {
  if (a.part_rows <= 16) return launch_t<FP8, 16>(qmap, kmap, vmap, a, stream);
  return launch_t<FP8, kTreeKeysRows>(qmap, kmap, vmap, a, stream);
}

}  // namespace

cudaError_t launch_tree_keys(const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const TreeArgs& a, bool fp8,
                             cudaStream_t stream) {
  return fp8 ? launch_n<true>(qmap, kmap, vmap, a, stream)
             : launch_n<false>(qmap, kmap, vmap, a, stream);
}

}  // namespace pkv
