// pkv_prefill_tc.cuh -- what the tcgen05 prefill kernels share: tile sizes, the
// ring of K/V tiles, bounded waits, widening of one-byte codes in place, and
// the longest-first choice of a CTA's work.
#pragma once

#include "pkv_common.cuh"
#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {

namespace {

constexpr int kTcRows = 128;      // UMMA M (rows of one query tile)
constexpr int kTcTiles = 2;       // query tiles per CTA
constexpr int kTcKeys = 128;      // keys per K/V tile
// One ring of K/V tile slots, filled in the order the products read them:
// K of key tile j is ring element 2j, V of key tile j element 2j + 1, element
// e in slot e % kRing.  (Separate K and V rings of 3 + 2 slots left V on the
// critical path: a V tile was issued only once the V two tiles back had been
// read, and its copy, ~1.5-2 us from L2, still in flight when P was ready.)
constexpr int kRing = 5;
__host__ __device__ constexpr int ring_slot(int e) { return e % kRing; }
__host__ __device__ constexpr uint32_t ring_phase(int e) {
  return static_cast<uint32_t>((e / kRing) & 1);
}
constexpr uint32_t kTmemCols = 512;
constexpr float kLazyRescale = 8.0f;  // log2 units: rescale O only past 2^8 growth

template <int D>
struct TcLayout {
  static constexpr int kHalves = D / 64;
  static constexpr int kQHalf = kTcRows * 128;       // 16 KB: 128 rows x 128 B
  static constexpr int kQTile = kHalves * kQHalf;
  static constexpr int kKvHalf = kTcKeys * 128;      // 16 KB: 128 keys x 128 B
  static constexpr int kTileBytes = kHalves * kKvHalf;  // one K (or V) tile
};

// Bounded wait that also gives up when another thread of the CTA has aborted.
// mbarrier.try_wait suspends the thread in hardware until the phase completes
// or a short time limit passes, so a waiting warp takes no issue slots from
// the softmax and MMA-issuing warps of its SM sub-partition.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity,
                                              volatile int32_t* abort, int32_t* err,
                                              uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort = 1;
      raise_error(err, PKV_ERR_TIMEOUT);
      return false;
    }
  }
}

// Warp-uniform version: lane 0 waits, the verdict is broadcast, and the other
// lanes then observe the (already completed) phase themselves.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int32_t* abort,
                                          int32_t* err, uint64_t limit_ns) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  if (lane == 0) ok = wait_or_abort(bar, parity, abort, err, limit_ns);
  ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  if (ok && lane != 0) ok = mbar_test(bar, parity);   // completed: observe it
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (K widened to code + 128 as fp16 subnormals, the 128 taken off the scores,
// would save two of the five operations for four codes, but ran slower: 819
// against 737 us for four 2048-token chunks over 2K to 8K keys.)
template <bool I8>
__device__ __forceinline__ uint2 codes_to_f16x4(uint32_t codes) {
  if constexpr (I8) return i8x4_to_f16x4(codes);
  else return e4m3x4_to_f16x4(codes);
}

// Widens one 128-key x 128 tile of e4m3 or int8 codes (128-byte swizzled rows at `tile`) in
// place into the fp16 tile layout (two 64-column halves, 16 KB apart,
// 128-byte swizzled); all 32 lanes of the calling warp.  A batch covers 16
// rows: a lane reads its 16-code chunk of 4 rows, and only after the warp has
// read the whole batch does it write the batch's fp16 chunks (those of half 0
// overwrite the same rows' codes); batches touch disjoint rows, so two warps
// may widen batches [b0, b1) of the same tile, and a batch is read while the
// one before it is converted.  8 lanes (which a shared-memory access serves
// together) take 4 chunks of one half in two rows whose numbers differ in bits
// 0 and 2: their reads and their writes fall into different banks.
template <bool I8>
__device__ __forceinline__ void widen_tile_fp8(uint8_t* tile, int lane, int b0, int b1) {
  const int c = 4 * ((lane >> 3) & 1) + (lane & 3);   // chunk: columns 16c .. 16c + 15
  const int j = 2 * (c & 3);        // its first 8-column chunk within the half
  const int r0 = (lane >> 4) ^ ((lane & 4) ? 5 : 0);
  uint8_t* half = tile + (c >> 2) * (kTcKeys * 128);
  uint4 codes[4], ahead[4];
  auto read = [&](int b, uint4 (&to)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * b + 8 * (i >> 1) + (r0 ^ (2 * (i & 1)));
      to[i] = *reinterpret_cast<const uint4*>(tile + r * 128 + ((c ^ (r & 7)) << 4));
    }
  };
  auto write = [&](int b, const uint4 (&from)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * b + 8 * (i >> 1) + (r0 ^ (2 * (i & 1)));
      const uint2 x = codes_to_f16x4<I8>(from[i].x), y = codes_to_f16x4<I8>(from[i].y);
      const uint2 z = codes_to_f16x4<I8>(from[i].z), w = codes_to_f16x4<I8>(from[i].w);
      *reinterpret_cast<uint4*>(half + r * 128 + ((j ^ (r & 7)) << 4)) =
          make_uint4(x.x, x.y, y.x, y.y);
      *reinterpret_cast<uint4*>(half + r * 128 + (((j + 1) ^ (r & 7)) << 4)) =
          make_uint4(z.x, z.y, w.x, w.y);
    }
  };
  read(b0, codes);
#pragma unroll 1
  for (int b = b0; b < b1; b += 2) {   // (an even number of batches)
    read(b + 1, ahead);
    __syncwarp();
    write(b, codes);
    if (b + 2 < b1) read(b + 2, codes);
    __syncwarp();
    write(b + 1, ahead);
  }
  __syncwarp();
}

// head_size 64: the tile's 128 code rows of 64 B (64-byte swizzle: chunk c of
// row r at r * 64 + ((c ^ (r / 2 % 4)) << 4)) land in its first 8 KB and
// widen into 128 fp16 rows of 128 B (128-byte swizzle).  Batch b (rows 16b ..
// 16b + 15) writes bytes [2048 b, 2048 b + 2048), the codes of batches 2b and
// 2b + 1; going from the last batch to the first, those were read earlier
// (or, for b = 0, by this batch before its writes).  A lane reads two 16-code
// chunks per batch.
template <bool I8>
__device__ __forceinline__ void widen_tile_fp8_d64(uint8_t* tile, int lane) {
  const int c = lane & 3;           // code chunk: columns 16c .. 16c + 15
  uint4 codes[2], ahead[2];
  auto read = [&](int b, uint4 (&to)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * b + 8 * i + (lane >> 2);
      to[i] = *reinterpret_cast<const uint4*>(tile + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
  };
  auto write = [&](int b, const uint4 (&from)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 16 * b + 8 * i + (lane >> 2);
      const uint2 x = codes_to_f16x4<I8>(from[i].x), y = codes_to_f16x4<I8>(from[i].y);
      const uint2 z = codes_to_f16x4<I8>(from[i].z), w = codes_to_f16x4<I8>(from[i].w);
      *reinterpret_cast<uint4*>(tile + r * 128 + (((2 * c) ^ (r & 7)) << 4)) =
          make_uint4(x.x, x.y, y.x, y.y);
      *reinterpret_cast<uint4*>(tile + r * 128 + (((2 * c + 1) ^ (r & 7)) << 4)) =
          make_uint4(z.x, z.y, w.x, w.y);
    }
  };
  constexpr int kBatches = kTcKeys / 16;
  read(kBatches - 1, codes);
#pragma unroll 1
  for (int b = kBatches - 1; b > 0; b -= 2) {   // (the next batch's codes are read first)
    read(b - 1, ahead);
    __syncwarp();
    write(b, codes);
    if (b > 1) read(b - 2, codes);
    __syncwarp();
    write(b - 1, ahead);
  }
  __syncwarp();
}

// Which (sequence, row-tile pair, kv head) this CTA computes.  The block
// scheduler starts CTAs in launch order, so with `longest_first` the grid is
// handed out longest first (list scheduling): the units (sequence, pair) are
// ranked by the number of 128-key tiles their rows see (a chunk's last
// pairs, and longer contexts, see more), ties by index, and the kv heads of a
// unit are consecutive CTAs.  Every CTA ranks the units itself (at most
// kLptUnits costs, in shared memory scratch that the K/V ring later reuses).
// Otherwise, or with more than kLptUnits units (many waves, little tail), the
// grid keeps its plain order (heaviest pair of each sequence first).
// Measured on GB300, the 4 x 512-token chunks of the mixed 32 q / 8 kv head
// batch alone: 104 -> 88 us longest first; beside that batch's decode launch
// the plain order is better (140 vs 144 us for both): its short CTAs end
// early and the decode CTAs, HBM-bound, run beside the long tensor-bound ones.
constexpr int kLptUnits = 128;

struct TcWork {
  int s, kvh, mtile;
};

__device__ __forceinline__ int tc_unit_cost(const PrefillArgs& a, int u, int toks) {
  const int s = a.seq_begin + u / a.num_mtiles;
  const int tok0 = (u % a.num_mtiles) * toks;
  const int L = __ldg(a.context_lens + s);
  const int q0 = __ldg(a.query_start_loc + s);
  const int qn = __ldg(a.query_start_loc + s + 1) - q0;
  if (qn <= 0 || tok0 >= qn || L < qn) return 0;   // nothing (or an error) to do
  const int pos_max = L - qn + min(tok0 + toks, qn) - 1;
  const int pos_min = L - qn + tok0;
  const int lo_min = max(a.window > 0 ? pos_min - a.window + 1 : 0, a.key_begin);
  const int j0 = lo_min > 0 ? lo_min / kTcKeys : 0;
  return (pos_max + kTcKeys) / kTcKeys - j0 + 1;   // key tiles + the CTA's own overhead
}

// Called by every thread of the CTA (it synchronises the CTA twice).
__device__ __forceinline__ TcWork pick_work(const PrefillArgs& a, int toks, int32_t* scratch) {
  const int nu = a.num_seqs * a.num_mtiles;
  if (nu > kLptUnits) {   // (the launcher does not choose this kernel then)
    return TcWork{a.seq_begin + static_cast<int>(blockIdx.z), static_cast<int>(blockIdx.y),
                  a.num_mtiles - 1 - static_cast<int>(blockIdx.x)};
  }
  const int b = static_cast<int>(blockIdx.x) +
                static_cast<int>(gridDim.x) * (static_cast<int>(blockIdx.y) +
                                               static_cast<int>(gridDim.y) *
                                                   static_cast<int>(blockIdx.z));
  const int r = b / a.num_kv_heads;   // this CTA's unit rank
  int32_t* cost = scratch;            // [nu]
  int32_t* pick = scratch + kLptUnits;
  for (int u = threadIdx.x; u < nu; u += blockDim.x) cost[u] = tc_unit_cost(a, u, toks);
  if (threadIdx.x == 0) *pick = 0;
  __syncthreads();
  for (int u = threadIdx.x; u < nu; u += blockDim.x) {
    const int c = cost[u];
    int rank = 0;
    for (int v = 0; v < nu; ++v) {
      const int cv = cost[v];
      rank += (cv > c || (cv == c && v < u)) ? 1 : 0;
    }
    if (rank == r) *pick = u;
  }
  fence_proxy_async();   // the ring's TMA writes later land on this scratch
  __syncthreads();
  const int u = *pick;
  return TcWork{a.seq_begin + u / a.num_mtiles, b % a.num_kv_heads, u % a.num_mtiles};
}

}  // namespace

}  // namespace pkv
