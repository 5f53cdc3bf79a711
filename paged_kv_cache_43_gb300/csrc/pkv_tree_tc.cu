// pkv_tree_tc.cu -- attention of a tree of drafted tokens over bf16 and e4m3 caches, on
// tcgen05.
//
// Mathematics as in pkv_tree.cu.  A row is a (drafted token, q head) pair of one kv head;
// S = Q K^T and O += P V run on 128 rows x 64 keys, P = 2^(scale log2(e) s - m) rounded to
// bf16 (e4m3 caches: everything on fp16, to which codes widen exactly; K's descale joins the
// score scale, V's the output).  m is a reference, not the running maximum: it moves only
// when a step's weights sum to more than kMost, so most steps need no pass for the maximum
// and no rescaling of O.  The denominator of bf16 sums the rounded weights, so the output
// is a convex combination of V rows.
//
// Layout.  Few query rows share each key, so the keys' bytes are the bound (HBM) up to
// about 100 rows a kv head, the chain S - softmax - P V beyond.  Keys are cut into splits,
// one CTA each with one tile of 128 rows; two CTAs an SM (each 256 of the 512 TMEM columns),
// so one's products and copies run under the other's softmax.  Warps:
//   0-3  softmax, a thread a row; before that Q to shared memory, at the end the rows out
//   4, 5 start the TMA copies of K, of V (a box per cache block and 64 columns)
//   6    issues the products: S of the next 64 keys is formed while these are exponentiated
//        (S has two buffers, P lies over S)
//   7    tensor memory
//   8-11 (e4m3) widen K and V codes in place, two warps each
// What a key that a row does not see holds must not reach the row, although P = 0 there
// (0 x NaN): in the tiles with drafted keys the softmax warps zero V's rows behind the
// last key and its values that are not finite, and the rows that see those get them at
// the end.
#include <float.h>

#include "pkv_prefill_tc.cuh"
#include "pkv_tree.cuh"

namespace pkv {

namespace {

constexpr int kKeys = 64;                       // keys of a step
constexpr int kStepBlocks = kKeys / kBlock;
constexpr int kRows = 128;
constexpr uint32_t kCols = 256;                 // TMEM columns of a CTA
// S of step h at 64 (h % 2), P over its first 32 columns; O at 128.
__device__ __forceinline__ uint32_t col_s(int h) { return 64u * (h & 1); }
constexpr uint32_t kColO = 128;
// A step's weights may sum to this before the reference moves: bf16 weights and fp32 sums
// hold it easily; fp16 weights reach 65504.
template <bool FP8>
constexpr float kMost = FP8 ? 32768.f : 0x1p60f;

template <int D>
struct Lay {
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = kRows * 128;    // 64 columns: 128 rows x 128 B
  static constexpr int kQ = kHalves * kQHalf;
  static constexpr int kTHalf = kKeys * 128;
  static constexpr int kTile = kHalves * kTHalf;
  // K tiles are read once by S, V tiles wait for their softmax: one slot more
  static constexpr int kKSlots = 2 * 128 / D, kVSlots = 3 * 128 / D;
  static constexpr int kRingBytes = (kKSlots + kVSlots) * kTile;
};

template <int D>
struct Shared {
  uint64_t q_full, pv_done, o_done, drain;
  uint64_t s_full[2], p_full[2];
  uint64_t k_full[Lay<D>::kKSlots], k_empty[Lay<D>::kKSlots], k_land[Lay<D>::kKSlots];
  uint64_t v_full[Lay<D>::kVSlots], v_empty[Lay<D>::kVSlots], v_land[Lay<D>::kVSlots];
  uint32_t tmem_base;
  int32_t abort;
  int32_t v_odd;                                // a drafted V value is not finite
};

// Two CTAs of 113 KB and the 1 KB that each costs are the SM's 228 KB.
template <int D>
constexpr int smem_bytes() {
  constexpr int need = Lay<D>::kQ + Lay<D>::kRingBytes + static_cast<int>(sizeof(Shared<D>));
  static_assert(need <= 113 * 1024, "two CTAs per SM");
  static_assert(Lay<D>::kRingBytes >= kRows * D * 4, "the rows leave through the ring");
  return need;
}

template <bool FP8>
constexpr int kThreads = FP8 ? 384 : 256;
// e4m3: launched with 80 registers a thread; the softmax warps take 128, the other two
// warpgroups keep 56.
constexpr int kRegsSoftmax = 128, kRegsOther = 56;
static_assert(128 * kRegsSoftmax + 256 * kRegsOther <= 384 * 80, "register split");

__device__ __forceinline__ bool quick_wait(uint32_t bar, uint32_t parity, volatile int32_t* abort,
                                           int32_t* err, uint64_t limit_ns) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
         warp_wait(bar, parity, abort, err, limit_ns);
}

// Whether one of the 16-bit values in w has its exponent all ones.
template <bool FP8>
__device__ __forceinline__ bool odd_value(uint32_t w) {
  constexpr uint32_t e = FP8 ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}
template <bool FP8>
__device__ __forceinline__ uint32_t even_value(uint32_t w) {   // those values as zero
  constexpr uint32_t e = FP8 ? 0x7C00u : 0x7F80u;
  if ((w & e) == e) w &= 0xffff0000u;
  if ((w & (e << 16)) == (e << 16)) w &= 0xffffu;
  return w;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads<FP8>, 2)
    pkv_tree_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;                            // [half][128 rows x 128 B]
  uint8_t* sK = smem + L::kQ;                    // [slot][half][64 keys x 128 B]
  uint8_t* sV = sK + L::kKSlots * L::kTile;
  Shared<D>* sh = reinterpret_cast<Shared<D>*>(sK + L::kRingBytes);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&kmap);
    prefetch_tensor_map(&vmap);
  }
  const int s = blockIdx.z, split = blockIdx.x, G = a.group, Hq = a.num_q_heads;
  const int tile = blockIdx.y / a.num_kv_heads, kvh = blockIdx.y - tile * a.num_kv_heads;
  const TreeSeq q = tree_seq(a, s);
  if (q.err != 0 && split == 0 && blockIdx.y == 0 && threadIdx.x == 0) raise_error(a.err, q.err);
  const int row0 = tile * kRows, rows = min(q.n * G - row0, kRows);
  if (q.skip || rows <= 0) return;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  // row r of the tile: its query row and head
  auto tok_of = [&](int r) { return q.q0 + (row0 + r) / G; };
  auto head_of = [&](int r) { return kvh * G + (row0 + r) % G; };
  if (q.err != 0) {
    if (split == 0)
      for (int i = threadIdx.x; i < rows * D; i += blockDim.x)
        out[(static_cast<int64_t>(tok_of(i / D)) * Hq + head_of(i / D)) * D + i % D] =
            __float2bfloat16(0.f);
    return;
  }
  const int nsplit = tree_splits(a, q.L);
  if (split >= nsplit) return;
  const int key_begin = split * a.split_blocks * kBlock;
  const int key_end = min(q.L, key_begin + a.split_blocks * kBlock);
  const int N = (key_end - key_begin + kKeys - 1) / kKeys;   // steps
  const int b0 = key_begin / kBlock, b1 = (key_end + kBlock - 1) / kBlock;
  const int32_t* bt = a.block_tables + s * a.bt_stride;

  auto bar = [](uint64_t& b) { return smem_u32(&b); };
  if (threadIdx.x == 0) {
    mbar_init(bar(sh->q_full), 4);
    mbar_init(bar(sh->pv_done), 1);
    mbar_init(bar(sh->o_done), 1);
    mbar_init(bar(sh->drain), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sh->s_full[i]), 1);
      mbar_init(bar(sh->p_full[i]), 4);
    }
    for (int i = 0; i < L::kKSlots; ++i) {
      mbar_init(bar(sh->k_full[i]), FP8 && D == 128 ? 2 : 1);
      mbar_init(bar(sh->k_empty[i]), 1);
      mbar_init(bar(sh->k_land[i]), 1);
    }
    for (int i = 0; i < L::kVSlots; ++i) {
      mbar_init(bar(sh->v_full[i]), FP8 && D == 128 ? 2 : 1);
      mbar_init(bar(sh->v_empty[i]), 1);
      mbar_init(bar(sh->v_land[i]), 1);
    }
    sh->abort = 0;
    sh->v_odd = 0;
    fence_barrier_init();
  }
  if (warp == 7) tc::alloc(smem_u32(&sh->tmem_base), kCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem_base, 0);
  volatile int32_t* abort = &sh->abort;
  const uint64_t wlim = wait_limit(a.wait_limit_ns);
  auto wait = [&](uint64_t& b, int use, int slots) {   // the phase of a slot's `use`-th turn
    return quick_wait(smem_u32(&b), static_cast<uint32_t>(use / slots) & 1, abort, a.err, wlim);
  };

  if (warp >= 4) {
    if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 4 || warp == 5) {
      // ------------------------------------------------------------ copies
      const bool is_v = warp == 5;
      const int slots = is_v ? L::kVSlots : L::kKSlots;
      uint64_t* land = FP8 ? (is_v ? sh->v_land : sh->k_land) : (is_v ? sh->v_full : sh->k_full);
      uint64_t* empty = is_v ? sh->v_empty : sh->k_empty;
      uint8_t* ring = is_v ? sV : sK;
      // several row tiles read the same keys: then they stay in L2
      const uint64_t policy = q.n * G > kRows ? policy_evict_normal() : policy_evict_first();
      auto ids = [&](int g) {   // block ids of eight steps, a lane a block
        const int b = b0 + 32 * g + lane;
        return b < b1 ? __ldg(bt + b) : -1;
      };
      int cur = ids(0), next = ids(1);
      // Test hook: the first K tile is withheld (no copy, no arrival).
      const bool withhold = a.debug_stall != 0 && !is_v;
      int n = 0;
      for (; n < N; ++n) {
        if (n > 0 && (n & 7) == 0) {
          cur = next;
          next = ids((n >> 3) + 1);
        }
        if (n >= slots && !wait(empty[n % slots], n - slots, slots)) break;
        if (withhold && n == 0) continue;
        const uint32_t dst = smem_u32(ring + n % slots * L::kTile), full = bar(land[n % slots]);
        int id[kStepBlocks];
        bool ok[kStepBlocks];
        uint32_t bytes = 0;
#pragma unroll
        for (int b = 0; b < kStepBlocks; ++b) {
          id[b] = __shfl_sync(0xffffffffu, cur, kStepBlocks * (n & 7) + b);
          const bool in = b0 + n * kStepBlocks + b < b1;
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
                tma_load_3d(dst + b * kBlock * D, is_v ? &vmap : &kmap, full, 0, kvh,
                            id[b] * kBlock, policy);
              } else {
#pragma unroll
                for (int h = 0; h < L::kHalves; ++h)
                  tma_load_3d(dst + h * L::kTHalf + b * 2048, is_v ? &vmap : &kmap, full, h * 64,
                              kvh, id[b] * kBlock, policy);
              }
            }
          }
        }
      }
      // every copy has landed before the CTA's shared memory is given up
      for (int i = max(0, n - slots); i < n; ++i)
        if (lane == 0 && !(withhold && i == 0))
          (void)mbar_wait(bar(land[i % slots]), static_cast<uint32_t>(i / slots) & 1);
      __syncwarp();
    } else if (warp == 6) {
      // ------------------------------------------------------------ products
      constexpr uint32_t idS = FP8 ? tc::idesc_f16_f32(kRows, kKeys, 0, 0)
                                   : tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
      constexpr uint32_t idO = FP8 ? tc::idesc_f16_f32(kRows, D, 0, 1)
                                   : tc::idesc_bf16_f32(kRows, D, 0, 1);
      const uint64_t dq = tc::smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(smem_u32(sV), L::kTHalf, 1024);
      auto issue_s = [&](int h) {
        const uint64_t db = dk + static_cast<uint64_t>((h % L::kKSlots * L::kTile) >> 4);
        const uint32_t d = tmem + col_s(h);
        if constexpr (D == 128) {
          tc::mma_ss_x8<2, 4, 6, 1024, 1026, 1028, 1030, 2, 4, 6, 512, 514, 516, 518>(d, dq, db,
                                                                                    idS, 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_ss(d, dq + (kk * 32 >> 4), db + (kk * 32 >> 4), idS, kk > 0 ? 1u : 0u);
        }
        tc::commit(bar(sh->s_full[h & 1]));
        tc::commit(bar(sh->k_empty[h % L::kKSlots]));
      };
      auto issue_pv = [&](int h) {
        const uint64_t db = dv + static_cast<uint64_t>((h % L::kVSlots * L::kTile) >> 4);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc::mma_ts(tmem + kColO, tmem + col_s(h) + 8 * kk, db + 128 * kk, idO,
                     h > 0 || kk > 0 ? 1u : 0u);
        tc::commit(bar(h == N - 1 ? sh->o_done : sh->pv_done));
        tc::commit(bar(sh->v_empty[h % L::kVSlots]));
      };
      auto start_s = [&](int h) {
        if (!wait(sh->k_full[h % L::kKSlots], h, L::kKSlots)) return false;
        tc::fence_after_sync();
        if (tc::elect_one()) issue_s(h);
        __syncwarp();
        return true;
      };
      bool go = wait(sh->q_full, 0, 1) && start_s(0) && (N < 2 || start_s(1));
      for (int h = 0; go && h < N; ++h) {
        go = wait(sh->p_full[h & 1], h >> 1, 1) &&
             wait(sh->v_full[h % L::kVSlots], h, L::kVSlots);
        if (!go) break;
        tc::fence_after_sync();
        if (tc::elect_one()) issue_pv(h);
        __syncwarp();
        // (S over the columns that P was read from: products execute in their order)
        if (h + 2 < N) go = start_s(h + 2);
      }
      if (tc::elect_one()) {   // every product completes before TMEM is freed
        tc::commit(bar(sh->drain));
        (void)mbar_wait(bar(sh->drain), 0);
      }
      __syncwarp();
    } else if (FP8 && warp >= 8 && (D == 128 || warp == 8 || warp == 10)) {
      // ------------------------------------------------------------ widening
      // (D = 64: the widened rows lie over later rows' codes, so one warp takes a tile)
      const bool is_v = warp >= 10;
      const int slots = is_v ? L::kVSlots : L::kKSlots;
      for (int n = 0; n < N; ++n) {
        if (!wait((is_v ? sh->v_land : sh->k_land)[n % slots], n, slots)) break;
        uint8_t* t = (is_v ? sV : sK) + n % slots * L::kTile;
        if constexpr (D == 128) widen_tile_fp8<false, kKeys>(t, lane, (warp & 1) * 2, (warp & 1) * 2 + 2);
        else widen_tile_fp8_d64<false, kKeys>(t, lane);
        fence_proxy_async();   // generic writes, then the tensor core reads
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((is_v ? sh->v_full : sh->k_full)[n % slots]));
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int row = warp * 32 + lane;            // tile row == TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const bool valid = row < rows, warp_valid = warp * 32 < rows;
    float sl2 = fabsf(a.scale_log2), out_scale = 1.f;
    // ---- this warp's rows of Q to shared memory (a negative scale's sign goes with them)
    {
      constexpr int kChunks = D / 8, kPer = 32 / kChunks, kIters = 32 / kPer;
      const int c = lane % kChunks;
      uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
      if constexpr (FP8) {
        const int64_t at = static_cast<int64_t>(s) * a.num_kv_heads + kvh;
        const float kd = __ldg(a.k_descale + at);
        if (kd < 0.f) flip ^= 0x80008000u;
        sl2 *= fabsf(kd);
        out_scale = __ldg(a.v_descale + at);
      }
      int row_e = 0;
#pragma unroll
      for (int i0 = 0; i0 < kIters; i0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = warp * 32 + (i0 + i) * kPer + lane / kChunks;
          v[i] = make_uint4(0, 0, 0, 0);
          if (r < rows)
            v[i] = __ldg(reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(a.q) +
                (static_cast<int64_t>(tok_of(r)) * Hq + head_of(r)) * D + 8 * c));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = warp * 32 + (i0 + i) * kPer + lane / kChunks;
          uint32_t w[4] = {v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip};
          if constexpr (FP8) {   // to fp16, a row beyond its range scaled by a power of two
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
            for (int off = kChunks / 2; off > 0; off >>= 1)
              amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const int e = f16_fit_exponent(amax);
            const float down = pow2f(-e);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = bf16x2_to_f16x2(w[k], down);
            // lane j keeps the exponent of the warp's row j
            const int mine = __shfl_sync(0xffffffffu, e, lane % kPer * kChunks);
            if (lane / kPer == i0 + i) row_e = mine;
          }
          *reinterpret_cast<uint4*>(sQ + (c >> 3) * L::kQHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if constexpr (FP8) sl2 *= pow2f(row_e);
      fence_proxy_async();   // generic writes, then the tensor core reads
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sh->q_full));
    }
    sl2 = fmaxf(sl2, FLT_MIN);   // (above zero, so that a masked -inf stays what it is)
    const uint64_t* mask =
        a.tree_mask + static_cast<int64_t>(tok_of(valid ? row : rows - 1)) * a.mask_words;
    float m = -INFINITY, l = 0.f;
    bool done = true;
    for (int h = 0; h < N; ++h) {
      if (!wait(sh->s_full[h & 1], h >> 1, 1)) {
        done = false;
        break;
      }
      tc::fence_after_sync();
      const uint32_t tS = lanes + col_s(h);
      const int key0 = key_begin + h * kKeys;
      const bool drafts = key0 + kKeys > q.first;   // keys that not every row sees, or none
      if (drafts) {
        // V's rows behind the last key become zero, and so do its drafted values that
        // are not finite
        if (!wait(sh->v_full[h % L::kVSlots], h, L::kVSlots)) {
          done = false;
          break;
        }
        constexpr int kEach = L::kHalves * 4;       // 16-byte chunks of a thread
        const int r = threadIdx.x >> 1, p = key0 + r;
        uint8_t* vrow = sV + h % L::kVSlots * L::kTile + r * 128 +
                        (D == 128 ? (threadIdx.x & 1) * L::kTHalf : 0);
        if (p >= q.first) {
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            const int c = D == 128 ? (i + r) & 7 : (4 * (threadIdx.x & 1) + ((i + r) & 3));
            uint4* at = reinterpret_cast<uint4*>(vrow + 16 * c);
            if (p >= q.L) {
              *at = make_uint4(0, 0, 0, 0);
            } else {
              const uint4 v = *at;
              if (odd_value<FP8>(v.x) || odd_value<FP8>(v.y) || odd_value<FP8>(v.z) ||
                  odd_value<FP8>(v.w)) {
                *at = make_uint4(even_value<FP8>(v.x), even_value<FP8>(v.y), even_value<FP8>(v.z),
                                 even_value<FP8>(v.w));
                sh->v_odd = 1;
              }
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
#pragma unroll
            for (int c0 = 0; c0 < kKeys; c0 += 32) {
              uint32_t r[32];
              tc::ld32(tS + c0, r);
              tc::wait_ld();
              const uint32_t bits = static_cast<uint32_t>(seen >> c0);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                top = fmaxf(top, (bits >> c & 1) ? __uint_as_float(r[c]) : -INFINITY);
            }
            const float mt = top * sl2;
            if (mt > m) {
              alpha = m == -INFINITY ? 0.f : ex2(m - mt);
              l *= alpha;
              m = mt;
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
            if (drafts) {
              const uint32_t bits = static_cast<uint32_t>(seen >> c0);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(bits >> c & 1)) r[c] = 0xff800000u;   // -infinity
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              float y0, y1;
              tc::fma_f32x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]), f2, a2, y0, y1);
              y0 = ex2(y0);
              y1 = ex2(y1);
              const uint32_t w = pack2<FP8>(y0, y1);
              pk[(c0 + c) / 2] = w;
              if constexpr (FP8) tc::add_f32x2(acc, y0, y1);
              else tc::add_f32x2(acc, bf16_lo(w), bf16_hi(w));
            }
          }
          ls = tc::sum_f32x2(acc);
          if (find || !__any_sync(0xffffffffu, valid && !(ls <= kMost<FP8>))) break;
          find = true;
        }
        if (h > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {   // rescale O
          // (P V of h - 1 is the last that was issued: that of h waits for this warp)
          if (!quick_wait(bar(sh->pv_done), (h - 1) & 1, abort, a.err, wlim)) {
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
      if (lane == 0) mbar_arrive(bar(sh->p_full[h & 1]));
    }
    // ---- the rows out, through the ring (every tile has been read), 16-byte chunks of a
    // row swapped about so that neither a column nor a row of them falls into one bank
    const bool ok = done && quick_wait(bar(sh->o_done), 0, abort, a.err, wlim);
    named_barrier(1, 128);       // (v_odd: every softmax warp's)
    if (ok && warp_valid) {
      tc::fence_after_sync();
      const bool odd = *reinterpret_cast<volatile int32_t*>(&sh->v_odd) != 0;
      const float inv = l == 0.f ? 0.f : out_scale / l;   // (a NaN stays)
      uint8_t* mine = sK + warp * 32 * D * 4;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        tc::ld32(lanes + kColO + c0, o);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * inv);
        if (odd && valid) {   // V values that are not finite, of the drafts that this row sees
          for (int p = max(q.first, key_begin); p < key_end; ++p) {
            const int j = p - q.first, b = __ldg(bt + p / kBlock);
            if (!(__ldg(mask + (j >> 6)) >> (j & 63) & 1) || b < 0 || b >= a.num_blocks) continue;
            const int64_t at = ((static_cast<int64_t>(b) * kBlock + p % kBlock) * a.num_kv_heads + kvh) * D + c0;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              float v;
              if constexpr (FP8)
                v = f16_lo(e4m3x4_to_f16x4(static_cast<const uint8_t*>(a.v_cache)[at + c]).x);
              else
                v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.v_cache)[at + c]);
              if (!(fabsf(v) <= FLT_MAX)) o[c] = __float_as_uint(__uint_as_float(o[c]) + v);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(mine + lane * D * 4 + (((c0 / 4 + i) ^ (lane & 7)) << 4)) =
              make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
      }
      __syncwarp();
      const int count = min(rows - warp * 32, 32);
      if (nsplit == 1) {
        constexpr int kLanes = D / 8;              // lanes of a bf16 row
        const int c = lane % kLanes;
        for (int r = lane / kLanes; r < count; r += 32 / kLanes) {
          const uint8_t* src = mine + r * D * 4;
          const float4 x = *reinterpret_cast<const float4*>(src + (((2 * c) ^ (r & 7)) << 4));
          const float4 y = *reinterpret_cast<const float4*>(src + (((2 * c + 1) ^ (r & 7)) << 4));
          const int t = warp * 32 + r;
          *reinterpret_cast<uint4*>(out + (static_cast<int64_t>(tok_of(t)) * Hq + head_of(t)) * D + 8 * c) =
              make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y),
                         pack_bf16(y.z, y.w));
        }
      } else {
        constexpr int kLanes = D / 4;              // lanes of an fp32 row
        const int c = lane % kLanes;
        for (int r = lane / kLanes; r < count; r += 32 / kLanes) {
          const int t = warp * 32 + r;
          *reinterpret_cast<float4*>(a.ws_o + tree_partial(a, tok_of(t), head_of(t), split) * D + 4 * c) =
              *reinterpret_cast<const float4*>(mine + r * D * 4 + ((c ^ (r & 7)) << 4));
        }
        if (valid)
          a.ws_lse[tree_partial(a, tok_of(row), head_of(row), split)] =
              l == 0.f ? -INFINITY : m + log2f(l);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 7) {
    tc::fence_after_sync();
    tc::dealloc(tmem, kCols);
  }
}

template <int D, bool FP8>
cudaError_t launch_t(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeArgs& a,
                     cudaStream_t stream) {
  constexpr int smem = smem_bytes<D>();
  auto kfn = pkv_tree_tc_kernel<D, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  TreeArgs b = a;
  debug_wait_settings(&b.wait_limit_ns, &b.debug_stall);
  const int64_t tiles = (static_cast<int64_t>(a.max_query_len) * a.group + kRows - 1) / kRows;
  kfn<<<dim3(a.max_splits, static_cast<unsigned>(a.num_kv_heads * tiles), a.num_seqs),
        kThreads<FP8>, smem, stream>>>(kmap, vmap, b);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeArgs& a,
                           int head_size, bool fp8, cudaStream_t stream) {
  if (fp8) return head_size == 128 ? launch_t<128, true>(kmap, vmap, a, stream)
                                   : launch_t<64, true>(kmap, vmap, a, stream);
  return head_size == 128 ? launch_t<128, false>(kmap, vmap, a, stream)
                          : launch_t<64, false>(kmap, vmap, a, stream);
}

}  // namespace pkv
