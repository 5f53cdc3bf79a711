// pkv_api.cu -- the C ABI of include/pkv.h: host-side argument checks, the
// split-K plan, TMA descriptor encoding and kernel dispatch.
//
// Nothing here allocates device memory or synchronises, except
// pkv_get_error(), which is documented as synchronising.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "pkv_common.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

// Per-device error word (PKV_ERR_* bits), OR-ed by the kernels.
__device__ int32_t g_error_word;

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int32_t* g_err_ptr[kMaxDevices] = {};
int g_num_sms[kMaxDevices] = {};

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Per device: the stream that a mixed batch's prefill launch (and a cascade
// call's shared-prefix launch) runs on while the decode launches run on the
// caller's stream, created once at the device's greatest priority (so that
// the block scheduler hands freed SMs to the tensor-core tiles first and the
// short decode CTAs fill their tail), and the events that fork it from the
// caller's stream and join it back.  `mu`
// keeps the record-wait-launch-record-wait sequence of one call from
// interleaving with another thread's.  side == nullptr: not available (the
// launches then stay on the caller's stream).
struct SideStream {
  std::mutex mu;
  cudaStream_t side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};
SideStream g_side[kMaxDevices];

// The CUDA error behind the most recent PKV_E_CUDA (process-wide).
std::atomic<int> g_last_cuda_error{0};

int cuda_fail(cudaError_t e) {
  g_last_cuda_error.store(static_cast<int>(e));
  return PKV_E_CUDA;
}

// Returns PKV_E_CUDA from the enclosing function when a CUDA call fails.
#define PKV_TRY(expr)                                   \
  do {                                                  \
    const cudaError_t e_ = (expr);                      \
    if (e_ != cudaSuccess) return cuda_fail(e_);        \
  } while (0)

void make_side_stream(SideStream* s) {
  int least = 0, greatest = 0;
  if (cudaDeviceGetStreamPriorityRange(&least, &greatest) != cudaSuccess) return;
  cudaStream_t st = nullptr;
  cudaEvent_t f = nullptr, j = nullptr;
  if (cudaStreamCreateWithPriority(&st, cudaStreamNonBlocking, greatest) == cudaSuccess &&
      cudaEventCreateWithFlags(&f, cudaEventDisableTiming) == cudaSuccess &&
      cudaEventCreateWithFlags(&j, cudaEventDisableTiming) == cudaSuccess) {
    s->side = st;
    s->fork = f;
    s->join = j;
    return;
  }
  if (j) cudaEventDestroy(j);
  if (f) cudaEventDestroy(f);
  if (st) cudaStreamDestroy(st);
  cudaGetLastError();
}

// Device-side address of the error word and the SM count, once per device
// (with the device's side stream).
int device_state(int32_t** err, int* num_sms, int* device = nullptr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PKV_E_CUDA;
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_err_ptr[dev] == nullptr) {
    void* p = nullptr;
    PKV_TRY(cudaGetSymbolAddress(&p, g_error_word));
    int sms = 0;
    PKV_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    make_side_stream(&g_side[dev]);
    g_err_ptr[dev] = static_cast<int32_t*>(p);
    g_num_sms[dev] = sms;
  }
  *err = g_err_ptr[dev];
  *num_sms = g_num_sms[dev];
  if (device) *device = dev;
  return PKV_OK;
}

// Whether work may be forked from `st` onto the side stream: the side stream
// is idle (not part of any capture), or it already belongs to the capture
// that `st` is in.  A side stream held by another thread's capture is left
// alone.
bool side_usable(cudaStream_t side, cudaStream_t st) {
  cudaStreamCaptureStatus ss = cudaStreamCaptureStatusNone, cs = cudaStreamCaptureStatusNone;
  unsigned long long sid = 0, cid = 0;
  if (cudaStreamGetCaptureInfo(side, &ss, &sid) != cudaSuccess ||
      cudaStreamGetCaptureInfo(st, &cs, &cid) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (ss == cudaStreamCaptureStatusNone) return cs != cudaStreamCaptureStatusInvalidated;
  return ss == cudaStreamCaptureStatusActive && cs == cudaStreamCaptureStatusActive && sid == cid;
}

// Fork-join around the device's side stream.  begin() makes the side stream
// wait for the work already on `st` and holds the side stream's lock;
// stream() is then where the forked launches go (the side stream, or `st`
// itself when the side stream is missing or held by another capture); join()
// makes `st` wait for them.  The destructor joins too (error paths), so a
// capture on `st` never ends with unjoined work.
class SideFork {
 public:
  SideFork(int dev, cudaStream_t st) : ss_(g_side[dev]), st_(st), pst_(st) {}
  SideFork(const SideFork&) = delete;
  SideFork& operator=(const SideFork&) = delete;
  ~SideFork() { (void)join(); }
  int begin() {
    if (ss_.side == nullptr) return PKV_OK;
    lock_ = std::unique_lock<std::mutex>(ss_.mu);
    if (!side_usable(ss_.side, st_)) return PKV_OK;
    PKV_TRY(cudaEventRecord(ss_.fork, st_));
    PKV_TRY(cudaStreamWaitEvent(ss_.side, ss_.fork, 0));
    pst_ = ss_.side;
    return PKV_OK;
  }
  cudaStream_t stream() const { return pst_; }
  int join() {
    if (pst_ == st_) return PKV_OK;
    pst_ = st_;
    cudaError_t e = cudaEventRecord(ss_.join, ss_.side);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(st_, ss_.join, 0);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e);
  }

 private:
  SideStream& ss_;
  cudaStream_t st_, pst_;
  std::unique_lock<std::mutex> lock_;
};

int encode_fn(PFN_cuTensorMapEncodeTiled_v12000* fn) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_encode == nullptr) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || f == nullptr)
      return PKV_E_CUDA;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  *fn = g_encode;
  return PKV_OK;
}

// TMA descriptor of one cache viewed as a 3-D tensor
// (head_size, num_kv_heads, num_blocks * 16).  bf16: a box of 64 columns x 1
// head x 16 rows (one cache block of one head, 128 bytes wide) with the
// 128-byte swizzle.  FP8 (e4m3 codes as bytes): a box of the whole head row x
// 1 head x 16 rows with the swizzle of the row's width (128 or 64 bytes), which
// keeps the kernels' per-lane fragment reads free of bank conflicts.
// The L2 fill size is capped at one head row (64, 128 or 256 bytes): a wider
// fill would pull the neighbouring kv head's row, which another CTA reads at
// some other time, and double the DRAM traffic of narrow rows.
int encode_cache_map(CUtensorMap* map, const void* base, const pkv_cache_desc& c) {
  PFN_cuTensorMapEncodeTiled_v12000 fn;
  if (int st = encode_fn(&fn)) return st;
  const bool fp8 = c.dtype == PKV_FP8_E4M3 || c.dtype == PKV_INT8;   // one-byte codes
  const cuuint64_t eb = fp8 ? 1 : 2;
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(c.head_size) * eb;
  const CUtensorMapL2promotion promo =
      row_bytes >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                       : (row_bytes >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                           : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_size),
                              static_cast<cuuint64_t>(c.num_kv_heads),
                              static_cast<cuuint64_t>(c.num_blocks) * c.block_size};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.head_size) * eb,
                                 static_cast<cuuint64_t>(c.num_kv_heads) * c.head_size * eb};
  const cuuint32_t box[3] = {fp8 ? static_cast<cuuint32_t>(c.head_size) : 64u, 1,
                             static_cast<cuuint32_t>(c.block_size)};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  (fp8 && row_bytes == 64) ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_128B,
                  promo,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_E_CUDA;
}

// TMA descriptor of an int8 cache for copies of one block of `heads` kv heads:
// the 3-D tensor (head_size, num_blocks * 16, num_kv_heads), the box a head
// row x 16 rows x `heads`, so that each head's rows land together, swizzled as
// above.
int encode_heads_map(CUtensorMap* map, const void* base, const pkv_cache_desc& c, int heads) {
  PFN_cuTensorMapEncodeTiled_v12000 fn;
  if (int st = encode_fn(&fn)) return st;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_size),
                              static_cast<cuuint64_t>(c.num_blocks) * c.block_size,
                              static_cast<cuuint64_t>(c.num_kv_heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.num_kv_heads) * c.head_size,
                                 static_cast<cuuint64_t>(c.head_size)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.head_size),
                             static_cast<cuuint32_t>(c.block_size), static_cast<cuuint32_t>(heads)};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  c.head_size == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  c.head_size == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_64B
                                    : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_E_CUDA;
}

// TMA descriptor of the bf16 query tensor [num_tokens, num_q_heads, D] viewed
// as (D, Hq, T) with a box of 64 columns x `group` heads x 128/group tokens:
// one box is the 128-row (token, head) tile of one kv head, 128 bytes wide
// (`toks` tokens instead, where it is given).
int encode_query_map(CUtensorMap* map, const void* q, int num_tokens, int num_q_heads,
                     int head_size, int group, int toks = 0) {
  PFN_cuTensorMapEncodeTiled_v12000 fn;
  if (int st = encode_fn(&fn)) return st;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_size),
                              static_cast<cuuint64_t>(num_q_heads),
                              static_cast<cuuint64_t>(num_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_size) * 2,
                                 static_cast<cuuint64_t>(num_q_heads) * head_size * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group),
                             static_cast<cuuint32_t>(toks > 0 ? toks : prefill_tc_tokens_per_tile(group))};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_E_CUDA;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_cache(const pkv_cache_desc* c) {
  if (c == nullptr) return PKV_E_NULL;
  if (c->dtype != PKV_F32 && c->dtype != PKV_BF16 && c->dtype != PKV_FP8_E4M3) return PKV_E_DTYPE;
  if (c->block_size != kBlock) return PKV_E_SHAPE;
  if (c->head_size != 64 && c->head_size != 128) return PKV_E_SHAPE;
  if (c->num_kv_heads < 1 || c->num_blocks < 0) return PKV_E_SHAPE;
  // TMA coordinates of cache rows are int32.
  if (static_cast<int64_t>(c->num_blocks) * c->block_size > INT32_MAX) return PKV_E_SHAPE;
  return PKV_OK;
}

// How the batch is cut: decode run, prefill rest, split-K chunk.
struct Plan {
  int num_decode = 0;     // sequences [0, num_decode) go to the decode kernel
  int split_blocks = 0;   // cache blocks per decode split
  int max_splits = 0;
  size_t ws_o_bytes = 0;  // fp32 partial outputs
  size_t ws_bytes = 0;    // total workspace
};

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int check_meta(const pkv_cache_desc* c, const pkv_attn_meta* m) {
  if (m == nullptr) return PKV_E_NULL;
  if (m->num_seqs < 0 || m->num_tokens < 0 || m->max_query_len < 0 || m->max_context_len < 0 ||
      m->block_table_stride < 1)
    return PKV_E_META;
  if (m->num_q_heads < 1 || m->num_q_heads % c->num_kv_heads != 0) return PKV_E_GQA;
  if (m->num_q_heads > 65535) return PKV_E_SHAPE;
  if (m->num_decode_seqs < -1 || m->num_decode_seqs > m->num_seqs) return PKV_E_META;
  if (m->sliding_window < 0) return PKV_E_META;
  if (m->kv_split_tokens != 0 &&
      (m->kv_split_tokens < 64 || m->kv_split_tokens > 2048 || m->kv_split_tokens % 64 != 0))
    return PKV_E_META;
  return PKV_OK;
}

// Cache blocks per decode split (CTA).  Measured on GB300 decode batches: 1024
// keys (512 KB of K+V per kv head at D=128) by default; 2048 for long contexts
// (>= 16K keys), which halves the split partials and the CTAs that find
// nothing to do; shorter chunks only while the batch would have fewer CTAs
// than SMs.  A CTA's fixed costs (barriers, Q, the first TMA round trip, its
// partial and the merge's read of it) outweigh more parallelism well before
// the GPU is full twice over: 2 sequences x 8 kv heads x 32K keys run in 51 us
// with 2048-key splits against 65 us with 512-key ones, 4 x 32 heads x 4K keys
// in 46 against 49 us, 8 x 8 kv heads x 2K keys in 23 against 25 us.
// `max_blocks`: blocks the longest row reads; `units`: (sequence, kv head,
// 8-head group) triples.
// Then the longest row's splits are evened out: their number is its blocks
// over that size rounded to nearest rather than up, each ceil(blocks / n)
// long and at most 128 (the kernel's 32 blocks per warp).  A 1024-key window
// spans 65 blocks: one split of 65, not 64 + 1, which would also cost a
// merge pass (measured with 1024-key windows: 146 -> 141 us on the
// 64 x 32-head batch, 112 -> 104 us on 256 x 8 kv heads, 27 -> 20 us on
// 16 x 8 kv heads).
int choose_split_blocks(int max_blocks, int64_t units, int num_sms, int kv_split_tokens) {
  if (kv_split_tokens > 0) return kv_split_tokens / kBlock;
  auto ctas = [&](int sb) { return units * ((max_blocks + sb - 1) / sb); };
  int split_blocks = 64;
  if (max_blocks * kBlock >= 16384 && ctas(128) >= num_sms) split_blocks = 128;
  while (split_blocks > 4 && ctas(split_blocks) < num_sms) split_blocks /= 2;
  if (max_blocks > 0) {
    constexpr int kMaxSplitBlocks = 128;
    int n = (max_blocks + split_blocks / 2) / split_blocks;
    n = std::max(n, (max_blocks + kMaxSplitBlocks - 1) / kMaxSplitBlocks);
    n = std::max(n, 1);
    split_blocks = (max_blocks + n - 1) / n;
  }
  return split_blocks;
}

int make_plan(const pkv_cache_desc* c, const pkv_attn_meta* m, int num_sms, Plan* p) {
  if (int st = check_cache(c)) return st;
  if (int st = check_meta(c, m)) return st;
  *p = Plan{};
  if (c->dtype == PKV_F32) return PKV_OK;  // one kernel, no workspace
  int nd = 0;
  if (m->max_query_len <= 1) nd = m->num_seqs;
  else if (m->num_decode_seqs >= 0) nd = m->num_decode_seqs;
  p->num_decode = nd;
  if (nd == 0) return PKV_OK;
  // Blocks a decode query may read: the whole context, or the window's span
  // (which can straddle one block boundary more than W / 16 blocks do).
  int max_blocks = (m->max_context_len + kBlock - 1) / kBlock;
  if (m->sliding_window > 0) {
    const int wb = (m->sliding_window + kBlock - 1) / kBlock + 1;
    if (wb < max_blocks) max_blocks = wb;
  }
  const int g_sub = (m->num_q_heads / c->num_kv_heads + 7) / 8;
  const int split_blocks = choose_split_blocks(
      max_blocks, static_cast<int64_t>(nd) * c->num_kv_heads * g_sub, num_sms, m->kv_split_tokens);
  p->split_blocks = split_blocks;
  p->max_splits = max_blocks > 0 ? (max_blocks + split_blocks - 1) / split_blocks : 1;
  if (p->max_splits > 1) {
    const size_t rows = static_cast<size_t>(nd) * m->num_q_heads * p->max_splits;
    p->ws_o_bytes = round_up(rows * c->head_size * sizeof(float), 256);
    p->ws_bytes = p->ws_o_bytes + round_up(rows * sizeof(float), 256);
  }
  return PKV_OK;
}

// Cascade attention over a decode batch whose sequences share their first
// P = common_prefix_blocks blocks: a prefix launch (every row against the
// shared keys, P blocks cut into prefix_splits chunks), a suffix launch (each
// row against its own keys after the prefix, the usual splits) and the
// combine, which merges prefix and suffix partials.  Workspace rows hold
// prefix_splits + suffix_max_splits partials.
struct CascadePlan {
  bool tc_prefix = false;    // shared keys on the tcgen05 kernel (G divides 128)
  int prefix_tiles = 0;      // tcgen05 prefix: 128-key tiles per CTA
  int prefix_mtiles = 0;     // tcgen05 prefix: query-row tiles
  int prefix_blocks = 0;
  int prefix_split_blocks = 0;
  int prefix_splits = 0;
  int num_decode = 0;        // leading decode sequences (one query row each)
  int rows = 0;              // query rows of the prefix launch (tokens)
  int col_groups = 0;        // 8-column groups of (sequence, q head in group) per kv head
  int split_blocks = 0;      // suffix split size
  int max_splits = 0;        // prefix_splits + the longest suffix's splits
  size_t ws_o_bytes = 0;
  size_t ws_bytes = 0;
};

int make_cascade_plan(const pkv_cache_desc* c, const pkv_attn_meta* m, int32_t prefix_blocks,
                      int num_sms, CascadePlan* p) {
  if (int st = check_cache(c)) return st;
  if (c->dtype != PKV_BF16 && c->dtype != PKV_FP8_E4M3) return PKV_E_DTYPE;
  if (int st = check_meta(c, m)) return st;
  // no window, and a prefix that every query follows; chunked-prefill rows
  // after num_decode_seqs decode sequences
  const bool chunks = m->max_query_len > 1;
  if (m->sliding_window != 0 || prefix_blocks < 1 || prefix_blocks > m->block_table_stride ||
      static_cast<int64_t>(prefix_blocks) * kBlock >= m->max_context_len ||
      (chunks && (m->num_decode_seqs < 0 || m->num_decode_seqs > m->num_seqs)))
    return PKV_E_META;
  *p = CascadePlan{};
  p->prefix_blocks = prefix_blocks;
  const int G = m->num_q_heads / c->num_kv_heads;
  // chunk rows: the shared keys and each chunk's own keys both on the tcgen05
  // kernel (group sizes dividing 128)
  if (chunks && !prefill_tc_supported(c->head_size, G)) return PKV_E_SHAPE;
  p->num_decode = chunks ? m->num_decode_seqs : m->num_seqs;
  p->rows = chunks ? m->num_tokens : m->num_seqs;
  p->col_groups = static_cast<int>((static_cast<int64_t>(m->num_seqs) * G + 7) / 8);
  // e4m3 caches: the shared keys only on the widening tcgen05 kernel
  if (c->dtype == PKV_FP8_E4M3 && !prefill_tc_supported(c->head_size, G)) return PKV_E_SHAPE;
  if (prefill_tc_supported(c->head_size, G)) {
    // tcgen05: all decode rows of a kv head in 128-row tiles, at least two
    // 128-key tiles per CTA, about half the SMs (their partials are merged)
    p->tc_prefix = true;
    const int per_cta = prefill_tc_tokens_per_cta(G);
    p->prefix_mtiles = (p->rows + per_cta - 1) / per_cta;
    const int ktiles = (prefix_blocks * kBlock + 127) / 128;
    const int64_t units = static_cast<int64_t>(p->prefix_mtiles) * c->num_kv_heads;
    int tiles = static_cast<int>((ktiles * units + num_sms / 2 - 1) / (num_sms / 2));
    tiles = tiles < 2 ? 2 : (tiles > ktiles ? ktiles : tiles);
    p->prefix_tiles = tiles;
    p->prefix_splits = (ktiles + tiles - 1) / tiles;
  } else {
    // mma.sync decode kernel over 8 (sequence, head) columns per CTA: 1024-key
    // chunks, shorter while the launch would not fill the GPU twice
    const int64_t prefix_units = static_cast<int64_t>(c->num_kv_heads) * p->col_groups;
    int psb = 64;
    while (psb > 4 && prefix_units * ((prefix_blocks + psb - 1) / psb) < 4LL * num_sms) psb /= 2;
    p->prefix_split_blocks = psb;
    p->prefix_splits = (prefix_blocks + psb - 1) / psb;
  }
  const int suffix_blocks = (m->max_context_len + kBlock - 1) / kBlock - prefix_blocks;
  const int g_sub = (G + 7) / 8;
  p->split_blocks = choose_split_blocks(
      suffix_blocks, static_cast<int64_t>(std::max(p->num_decode, 1)) * c->num_kv_heads * g_sub,
      num_sms, m->kv_split_tokens);
  // decode rows: the longest suffix's splits; chunk rows: one suffix partial
  p->max_splits = p->prefix_splits + (suffix_blocks + p->split_blocks - 1) / p->split_blocks;
  const size_t rows = static_cast<size_t>(p->rows) * m->num_q_heads * p->max_splits;
  p->ws_o_bytes = round_up(rows * c->head_size * sizeof(float), 256);
  p->ws_bytes = p->ws_o_bytes + round_up(rows * sizeof(float), 256);
  return PKV_OK;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

int attention_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, const int32_t* context_lens,
                   const int32_t* query_start_loc, float scale, const float* k_descale,
                   const float* v_descale, const pkv_cache_desc* cache,
                   const pkv_attn_meta* meta, void* workspace, size_t workspace_bytes,
                   void* stream);

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_write(const void* k, const void* v, const int64_t* slot_mapping,
                         int32_t num_tokens, void* k_cache, void* v_cache,
                         const pkv_cache_desc* cache, void* stream) {
  if (int st = check_cache(cache)) return st;
  if (cache->dtype == PKV_FP8_E4M3) return PKV_E_DTYPE;  // pkv_write_fp8
  if (num_tokens < 0) return PKV_E_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_E_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PKV_E_ALIGN;
  int32_t* err;
  int sms;
  if (int st = device_state(&err, &sms)) return st;
  const int ebytes = cache->dtype == PKV_BF16 ? 2 : 4;
  WriteArgs a{};
  a.k = k;
  a.v = v;
  a.slot_mapping = slot_mapping;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.err = err;
  a.num_slots = static_cast<int64_t>(cache->num_blocks) * cache->block_size;
  a.num_tokens = num_tokens;
  a.row_vecs = cache->num_kv_heads * cache->head_size * ebytes / 16;
  a.k_scale = a.v_scale = nullptr;
  a.head_size = cache->head_size;
  return launch_write(a, as_stream(stream), sms) == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}

extern "C" int pkv_write_fp8(const void* k, const void* v, const int64_t* slot_mapping,
                             int32_t num_tokens, void* k_cache, void* v_cache,
                             const float* k_scale, const float* v_scale,
                             const pkv_cache_desc* cache, void* stream) {
  if (int st = check_cache(cache)) return st;
  if (cache->dtype != PKV_FP8_E4M3) return PKV_E_DTYPE;
  if (num_tokens < 0) return PKV_E_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scale || !v_scale)
    return PKV_E_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
      (reinterpret_cast<uintptr_t>(k_scale) & 3u) || (reinterpret_cast<uintptr_t>(v_scale) & 3u))
    return PKV_E_ALIGN;
  int32_t* err;
  int sms;
  if (int st = device_state(&err, &sms)) return st;
  WriteArgs a{};
  a.k = k;
  a.v = v;
  a.slot_mapping = slot_mapping;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.err = err;
  a.num_slots = static_cast<int64_t>(cache->num_blocks) * cache->block_size;
  a.num_tokens = num_tokens;
  a.row_vecs = cache->num_kv_heads * cache->head_size / 16;  // 16 codes per vector
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.head_size = cache->head_size;
  return launch_write_fp8(a, as_stream(stream), sms) == cudaSuccess ? PKV_OK : PKV_E_CUDA;
}

extern "C" size_t pkv_attention_workspace_size(const pkv_cache_desc* cache,
                                               const pkv_attn_meta* meta) {
  int32_t* err;
  int sms;
  if (device_state(&err, &sms) != PKV_OK) return static_cast<size_t>(-1);
  Plan p;
  if (make_plan(cache, meta, sms, &p) != PKV_OK) return static_cast<size_t>(-1);
  return p.ws_bytes;
}

extern "C" int pkv_attention(void* out, const void* q, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens,
                             const int32_t* query_start_loc, float scale,
                             const pkv_cache_desc* cache, const pkv_attn_meta* meta,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (cache != nullptr && cache->dtype == PKV_FP8_E4M3) return PKV_E_DTYPE;  // pkv_attention_fp8
  return attention_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                        scale, nullptr, nullptr, cache, meta, workspace, workspace_bytes, stream);
}

extern "C" int pkv_attention_fp8(void* out, const void* q, const void* k_cache,
                                 const void* v_cache, const int32_t* block_tables,
                                 const int32_t* context_lens, const int32_t* query_start_loc,
                                 float scale, const float* k_descale, const float* v_descale,
                                 const pkv_cache_desc* cache, const pkv_attn_meta* meta,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  if (cache == nullptr) return PKV_E_NULL;
  if (cache->dtype != PKV_FP8_E4M3) return PKV_E_DTYPE;
  if (meta != nullptr && meta->num_seqs > 0 && meta->num_tokens > 0) {
    if (!k_descale || !v_descale) return PKV_E_NULL;
    if ((reinterpret_cast<uintptr_t>(k_descale) & 3u) ||
        (reinterpret_cast<uintptr_t>(v_descale) & 3u))
      return PKV_E_ALIGN;
  }
  return attention_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                        scale, k_descale, v_descale, cache, meta, workspace, workspace_bytes,
                        stream);
}

namespace pkv {
namespace {

int attention_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, const int32_t* context_lens,
                   const int32_t* query_start_loc, float scale, const float* k_descale,
                   const float* v_descale, const pkv_cache_desc* cache,
                   const pkv_attn_meta* meta, void* workspace, size_t workspace_bytes,
                   void* stream) {
  int32_t* err;
  int sms, dev;
  if (int st = device_state(&err, &sms, &dev)) return st;
  Plan p;
  if (int st = make_plan(cache, meta, sms, &p)) return st;
  if (meta->num_seqs == 0 || meta->num_tokens == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start_loc)
    return PKV_E_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(query_start_loc) & 3u))
    return PKV_E_ALIGN;
  if (p.ws_bytes > 0) {
    if (workspace == nullptr || workspace_bytes < p.ws_bytes) return PKV_E_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_E_ALIGN;
  }
  const cudaStream_t st = as_stream(stream);
  const float LOG2E = 1.4426950408889634f;

  if (cache->dtype == PKV_F32) {
    F32Args a{};
    a.out = static_cast<float*>(out);
    a.q = static_cast<const float*>(q);
    a.k_cache = static_cast<const float*>(k_cache);
    a.v_cache = static_cast<const float*>(v_cache);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start_loc = query_start_loc;
    a.err = err;
    a.bt_stride = meta->block_table_stride;
    a.num_seqs = meta->num_seqs;
    a.num_tokens = meta->num_tokens;
    a.num_q_heads = meta->num_q_heads;
    a.num_kv_heads = cache->num_kv_heads;
    a.head_size = cache->head_size;
    a.num_blocks = cache->num_blocks;
    a.window = meta->sliding_window;
    a.scale = scale;
    return launch_attention_f32(a, st) == cudaSuccess ? PKV_OK : PKV_E_CUDA;
  }

  if (cache->num_blocks == 0) return PKV_E_SHAPE;
  const bool fp8 = cache->dtype == PKV_FP8_E4M3;
  CUtensorMap kmap, vmap;
  if (int e = encode_cache_map(&kmap, k_cache, *cache)) return e;
  if (int e = encode_cache_map(&vmap, v_cache, *cache)) return e;
  const int G = meta->num_q_heads / cache->num_kv_heads;

  const int npf = meta->num_seqs - p.num_decode;
  auto decode_part = [&](cudaStream_t st) -> int {
    DecodeArgs d{};
    d.out = out;
    d.q = q;
    d.block_tables = block_tables;
    d.context_lens = context_lens;
    d.query_start_loc = query_start_loc;
    d.ws_o = p.ws_bytes ? static_cast<float*>(workspace) : nullptr;
    d.ws_lse = p.ws_bytes ? reinterpret_cast<float*>(static_cast<char*>(workspace) + p.ws_o_bytes)
                          : nullptr;
    d.err = err;
    d.bt_stride = meta->block_table_stride;
    d.num_seqs = p.num_decode;
    d.num_q_heads = meta->num_q_heads;
    d.num_kv_heads = cache->num_kv_heads;
    d.group = G;
    d.num_blocks = cache->num_blocks;
    d.split_blocks = p.split_blocks;
    d.max_splits = p.max_splits;
    d.num_tokens = meta->num_tokens;
    d.max_context_len = meta->max_context_len;
    d.window = meta->sliding_window;
    d.k_descale = k_descale;
    d.v_descale = v_descale;
    d.scale_log2 = scale * LOG2E;
    PKV_TRY(launch_decode_bf16(kmap, vmap, d, cache->head_size, fp8, st));
    PKV_TRY(launch_combine_bf16(d, cache->head_size, st, /*after_decode=*/true));
    return PKV_OK;
  };
  auto prefill_part = [&](cudaStream_t st) -> int {
    PrefillArgs f{};
    f.out = out;
    f.q = q;
    f.block_tables = block_tables;
    f.context_lens = context_lens;
    f.query_start_loc = query_start_loc;
    f.err = err;
    f.bt_stride = meta->block_table_stride;
    f.seq_begin = p.num_decode;
    f.num_seqs = npf;
    f.num_q_heads = meta->num_q_heads;
    f.num_kv_heads = cache->num_kv_heads;
    f.group = G;
    f.num_blocks = cache->num_blocks;
    f.num_tokens = meta->num_tokens;
    f.max_query_len = meta->max_query_len;
    f.window = meta->sliding_window;
    f.k_descale = k_descale;
    f.v_descale = v_descale;
    f.scale_log2 = scale * LOG2E;
    f.longest_first = p.num_decode == 0 ? 1 : 0;   // alone on the GPU, or beside decode
    if (prefill_tc_supported(cache->head_size, G)) {
      // tcgen05/TMEM kernel: two tiles of 128/G tokens x G heads per CTA.
      const int toks = prefill_tc_tokens_per_cta(G);
      f.num_mtiles = (meta->max_query_len + toks - 1) / toks;
      CUtensorMap qmap, omap;
      if (int e = encode_query_map(&qmap, q, meta->num_tokens, meta->num_q_heads,
                                   cache->head_size, G))
        return e;
      if (int e = encode_query_map(&omap, out, meta->num_tokens, meta->num_q_heads,
                                   cache->head_size, G))
        return e;
      PKV_TRY(launch_prefill_tc(qmap, kmap, vmap, omap, f, cache->head_size, fp8, st));
    } else {
      // group sizes that do not divide 128 rows: mma.sync kernel, 64 rows per
      // CTA.
      const int64_t rows = static_cast<int64_t>(meta->max_query_len) * G;
      f.num_mtiles = static_cast<int32_t>((rows + kPrefillRows - 1) / kPrefillRows);
      PKV_TRY(launch_prefill_bf16(kmap, vmap, f, cache->head_size, fp8, st));
    }
    return PKV_OK;
  };
  if (p.num_decode == 0) return prefill_part(st);
  if (npf == 0) return decode_part(st);
  // Decode and prefill rows in one batch: the prefill launch goes first, on
  // the device's high-priority side stream forked from the caller's stream,
  // and the decode launches follow on the caller's stream, so that the short
  // decode CTAs fill the SMs that the prefill's last wave leaves idle; the
  // side stream is joined back before the call returns.  (Measured on GB300,
  // the mixed 48-decode + 4 x 512-token-chunk batch of 32 q / 8 kv heads:
  // attention 170 us in one stream, 143 us forked.)
  SideFork fork(dev, st);
  if (int e = fork.begin()) return e;
  int rc = prefill_part(fork.stream());
  if (rc == PKV_OK) rc = decode_part(st);
  const int jr = fork.join();
  return rc != PKV_OK ? rc : jr;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_use_cascade(const pkv_attn_meta* meta, int32_t common_prefix_blocks) {
  // The gate the [book] gives for cascade attention: a common prefix of at
  // least 256 tokens, at least 8 requests, no sliding window.  Then, in place
  // of the pages' rough CTA/wave model, rules measured on GB300 (32 q / 8 kv
  // heads, head_size 128; the prefix launch on the side stream beside the
  // suffix launches):
  //  * decode rows (own keys U[128, 1024]): the plain call already meets
  //    repeated prefix reads in L2, so the cascade wins once the prefix is
  //    >= 512 tokens and the repeated prefix keys (sequences - 1) x prefix
  //    reach 16K (1.09x at 64 x 512, 1.17x at 16 x 2048, 1.19x at 8 x 8192,
  //    3.6x at 64 x 8192, 6.0x at 256 x 8192; 0.83-0.96x below, and at every
  //    256-token prefix);
  //  * with chunked-prefill rows: their prefix work is a dense contraction
  //    either way (the cascade saves K/V reads, not flops) and costs a second
  //    pass and a merge, so the cascade wins only for at most 512 chunk rows
  //    beside a prefix of >= 4096 tokens (1.14-1.22x with 0, 16 or 48 decode
  //    rows; 4 x 512 chunk rows: 0.58-0.93x at every prefix up to 4096).
  if (meta == nullptr) return 0;
  const int64_t p = static_cast<int64_t>(common_prefix_blocks) * kBlock;
  const bool pages_gate = p >= 256 && meta->num_seqs >= 8 && meta->sliding_window == 0;
  const bool chunks = meta->max_query_len > 1;
  if (!pages_gate || p >= meta->max_context_len) return 0;
  if (!chunks)
    return p >= 512 && (static_cast<int64_t>(meta->num_seqs) - 1) * p >= 16384 ? 1 : 0;
  if (meta->num_decode_seqs < 0 || meta->num_decode_seqs > meta->num_seqs) return 0;
  const int64_t chunk_rows = static_cast<int64_t>(meta->num_tokens) - meta->num_decode_seqs;
  return chunk_rows <= 512 && p >= 4096 ? 1 : 0;
}

extern "C" size_t pkv_attention_cascade_workspace_size(const pkv_cache_desc* cache,
                                                       const pkv_attn_meta* meta,
                                                       int32_t common_prefix_blocks) {
  int32_t* err;
  int sms;
  if (device_state(&err, &sms) != PKV_OK) return static_cast<size_t>(-1);
  CascadePlan p;
  if (make_cascade_plan(cache, meta, common_prefix_blocks, sms, &p) != PKV_OK)
    return static_cast<size_t>(-1);
  return p.ws_bytes;
}

namespace pkv {
namespace {

int cascade_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_tables, const int32_t* context_lens,
                 const int32_t* query_start_loc, float scale, int32_t common_prefix_blocks,
                 const float* k_descale, const float* v_descale, const pkv_cache_desc* cache,
                 const pkv_attn_meta* meta, void* workspace, size_t workspace_bytes,
                 void* stream);

}  // namespace
}  // namespace pkv

extern "C" int pkv_attention_cascade(void* out, const void* q, const void* k_cache,
                                     const void* v_cache, const int32_t* block_tables,
                                     const int32_t* context_lens, const int32_t* query_start_loc,
                                     float scale, int32_t common_prefix_blocks,
                                     const pkv_cache_desc* cache, const pkv_attn_meta* meta,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (cache != nullptr && cache->dtype == PKV_FP8_E4M3) return PKV_E_DTYPE;  // _fp8 variant
  return cascade_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                      scale, common_prefix_blocks, nullptr, nullptr, cache, meta, workspace,
                      workspace_bytes, stream);
}

extern "C" int pkv_attention_cascade_fp8(void* out, const void* q, const void* k_cache,
                                         const void* v_cache, const int32_t* block_tables,
                                         const int32_t* context_lens,
                                         const int32_t* query_start_loc, float scale,
                                         int32_t common_prefix_blocks, const float* k_descale,
                                         const float* v_descale, const pkv_cache_desc* cache,
                                         const pkv_attn_meta* meta, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  if (cache == nullptr) return PKV_E_NULL;
  if (cache->dtype != PKV_FP8_E4M3) return PKV_E_DTYPE;
  if (meta != nullptr && meta->num_seqs > 0 && meta->num_tokens > 0) {
    if (!k_descale || !v_descale) return PKV_E_NULL;
    if ((reinterpret_cast<uintptr_t>(k_descale) & 3u) ||
        (reinterpret_cast<uintptr_t>(v_descale) & 3u))
      return PKV_E_ALIGN;
  }
  return cascade_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                      scale, common_prefix_blocks, k_descale, v_descale, cache, meta, workspace,
                      workspace_bytes, stream);
}

namespace pkv {
namespace {

int cascade_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                 const int32_t* block_tables, const int32_t* context_lens,
                 const int32_t* query_start_loc, float scale, int32_t common_prefix_blocks,
                 const float* k_descale, const float* v_descale, const pkv_cache_desc* cache,
                 const pkv_attn_meta* meta, void* workspace, size_t workspace_bytes,
                 void* stream) {
  const bool fp8 = cache != nullptr && cache->dtype == PKV_FP8_E4M3;
  int32_t* err;
  int sms, dev;
  if (int st = device_state(&err, &sms, &dev)) return st;
  CascadePlan p;
  if (int st = make_cascade_plan(cache, meta, common_prefix_blocks, sms, &p)) return st;
  if (meta->num_seqs == 0 || meta->num_tokens == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start_loc)
    return PKV_E_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(query_start_loc) & 3u))
    return PKV_E_ALIGN;
  if (workspace == nullptr || workspace_bytes < p.ws_bytes) return PKV_E_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_E_ALIGN;
  if (cache->num_blocks == 0) return PKV_E_SHAPE;
  CUtensorMap kmap, vmap;
  if (int e = encode_cache_map(&kmap, k_cache, *cache)) return e;
  if (int e = encode_cache_map(&vmap, v_cache, *cache)) return e;
  const cudaStream_t st = as_stream(stream);
  DecodeArgs d{};
  d.out = out;
  d.q = q;
  d.block_tables = block_tables;
  d.context_lens = context_lens;
  d.query_start_loc = query_start_loc;
  d.ws_o = static_cast<float*>(workspace);
  d.ws_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.ws_o_bytes);
  d.err = err;
  d.bt_stride = meta->block_table_stride;
  d.num_seqs = meta->num_seqs;
  d.num_q_heads = meta->num_q_heads;
  d.num_kv_heads = cache->num_kv_heads;
  d.group = meta->num_q_heads / cache->num_kv_heads;
  d.num_blocks = cache->num_blocks;
  d.max_splits = p.max_splits;
  d.num_tokens = meta->num_tokens;
  d.max_context_len = meta->max_context_len;
  d.scale_log2 = scale * 1.4426950408889634f;
  d.k_descale = k_descale;
  d.v_descale = v_descale;
  d.force_partial = 1;
  d.prefix_splits = p.prefix_splits;
  // The prefix and suffix launches write disjoint split slots and meet only
  // in the merge: the prefix goes on the side stream (high priority; the
  // tcgen05 prefix grid is sized to about half the SMs) and the suffix on
  // the caller's stream beside it, joined before the merge.
  SideFork fork(dev, st);
  if (int e = fork.begin()) return e;
  const cudaStream_t pst = fork.stream();
  // prefix: every row against the shared keys, through sequence 0's table
  if (p.tc_prefix) {
    PrefillArgs f{};
    f.out = out;
    f.q = q;
    f.block_tables = block_tables;
    f.context_lens = context_lens;
    f.query_start_loc = query_start_loc;
    f.err = err;
    f.bt_stride = meta->block_table_stride;
    f.num_seqs = p.rows;              // the prefix launch's rows: query tokens
    f.casc_seqs = meta->num_seqs;
    f.num_q_heads = meta->num_q_heads;
    f.num_kv_heads = cache->num_kv_heads;
    f.group = d.group;
    f.num_blocks = cache->num_blocks;
    f.num_mtiles = p.prefix_mtiles;
    f.num_tokens = meta->num_tokens;
    f.max_query_len = 1;
    f.scale_log2 = d.scale_log2;
    f.cascade_prefix = 1;
    f.prefix_len = p.prefix_blocks * kBlock;
    f.prefix_tiles = p.prefix_tiles;
    f.max_splits = p.max_splits;
    f.ws_o = d.ws_o;
    f.ws_lse = d.ws_lse;
    f.k_descale = k_descale;
    f.v_descale = v_descale;
    CUtensorMap qmap;
    if (int e = encode_query_map(&qmap, q, meta->num_tokens, meta->num_q_heads,
                                 cache->head_size, d.group))
      return e;
    PKV_TRY(launch_prefill_tc(qmap, kmap, vmap, qmap, f, cache->head_size, fp8, pst));  // (no output map: workspace rows)
  } else {
    DecodeArgs pa = d;
    pa.split_blocks = p.prefix_split_blocks;
    pa.prefix_len = p.prefix_blocks * kBlock;
    pa.prefix_col_groups = p.col_groups;
    PKV_TRY(launch_cascade_prefix_bf16(kmap, vmap, pa, cache->head_size, pst));
  }
  // suffix: each row against its own keys after the prefix (decode rows on
  // the split-K decode kernel, chunk rows causally on the tcgen05 kernel);
  // then the merges
  DecodeArgs sa = d;
  sa.num_seqs = p.num_decode;
  sa.split_blocks = p.split_blocks;
  sa.key_begin_blocks = p.prefix_blocks;
  sa.split_base = p.prefix_splits;
  PKV_TRY(launch_decode_bf16(kmap, vmap, sa, cache->head_size, fp8, st));
  const int npf = meta->num_seqs - p.num_decode;
  if (npf > 0) {
    PrefillArgs f{};
    f.out = out;
    f.q = q;
    f.block_tables = block_tables;
    f.context_lens = context_lens;
    f.query_start_loc = query_start_loc;
    f.err = err;
    f.bt_stride = meta->block_table_stride;
    f.seq_begin = p.num_decode;
    f.num_seqs = npf;
    f.num_q_heads = meta->num_q_heads;
    f.num_kv_heads = cache->num_kv_heads;
    f.group = d.group;
    f.num_blocks = cache->num_blocks;
    f.num_tokens = meta->num_tokens;
    f.max_query_len = meta->max_query_len;
    f.k_descale = k_descale;
    f.v_descale = v_descale;
    f.scale_log2 = d.scale_log2;
    const int toks = prefill_tc_tokens_per_cta(d.group);
    f.num_mtiles = (meta->max_query_len + toks - 1) / toks;
    f.key_begin = p.prefix_blocks * kBlock;
    f.split_base = p.prefix_splits;
    f.max_splits = p.max_splits;
    f.ws_o = d.ws_o;
    f.ws_lse = d.ws_lse;
    CUtensorMap qmap;
    if (int e = encode_query_map(&qmap, q, meta->num_tokens, meta->num_q_heads,
                                 cache->head_size, d.group))
      return e;
    PKV_TRY(launch_prefill_tc(qmap, kmap, vmap, qmap, f, cache->head_size, fp8, st));  // (workspace rows)
  }
  if (int e = fork.join()) return e;
  PKV_TRY(launch_combine_bf16(sa, cache->head_size, st));
  if (npf > 0) {
    // chunk rows are the query tokens after the decode rows
    DecodeArgs mr = sa;
    mr.merge_rows_begin = p.num_decode;
    mr.merge_rows_end = meta->num_tokens;
    mr.num_seqs = meta->num_tokens - p.num_decode;
    mr.casc_seqs = meta->num_seqs;
    PKV_TRY(launch_combine_bf16(mr, cache->head_size, st));
  }
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

namespace pkv {
namespace {
// Test hook (pkv_debug_wait_test): 0 = off.
std::atomic<uint64_t> g_debug_wait_limit_ns{0};
std::atomic<int32_t> g_debug_stall{0};
constexpr uint64_t kDebugWaitLimitNs = 20000;   // 20 us
}  // namespace

void debug_wait_settings(uint64_t* limit_ns, int32_t* stall) {
  *limit_ns = g_debug_wait_limit_ns.load(std::memory_order_relaxed);
  *stall = g_debug_stall.load(std::memory_order_relaxed);
}
}  // namespace pkv

extern "C" int pkv_debug_wait_test(int enable) {
  pkv::g_debug_wait_limit_ns.store(enable ? pkv::kDebugWaitLimitNs : 0);
  pkv::g_debug_stall.store(enable ? 1 : 0);
  return PKV_OK;
}

// ------------------------------------------------------------- int8 caches

namespace pkv {
namespace {

int check_cache_int8(const pkv_cache_desc* c) {
  if (c == nullptr) return PKV_E_NULL;
  if (c->dtype != PKV_INT8) return PKV_E_DTYPE;
  pkv_cache_desc as_bytes = *c;
  as_bytes.dtype = PKV_FP8_E4M3;   // the same limits as the other one-byte cache
  return check_cache(&as_bytes);
}

// How an int8 batch's decode sequences are cut.  Two kernels:
//  * the split kernel (pkv_decode.cu) with the e4m3 plan: a CTA per (split of a
//    sequence, kv head), merged in the CTA;
//  * teams (pkv_decode_int8.cu): the sequences' blocks on one line in equal
//    ranges, a team of warps reading 4 or 8 heads (or groups of 8 q heads) in one
//    copy.
// Teams where they have 4 warps or more and a range gets 32 blocks or more, by
// max_context_len.  Measured, split against teams, us (q / kv heads, head_size
// 128): 32 / 8, 16 sequences of 8K to 16K keys 85 - 78, 64 of 64 to 8192 102 - 94,
// 512 of 64 to 512 71 - 63; 32 / 32, 128 of 1K to 3K 328 - 306; 128 / 8, 128 of 1K to
// 3K 183 - 136; below the rule 32 / 8, 8 of 2000 15 - 25, 128 of 100 to 1000 36 - 38;
// teams of one warp (10 / 5), 16 of 8K to 16K 58 - 62.
constexpr int kTeamRangeBlocks = 32;

// Up to kDecodeCluster splits of a row are a thread-block cluster, which merges its
// partials itself: no merge launch, no workspace to ask for (the host's side of a
// call 19.7 - 10.2 us).  Contexts of up to kOneSplitBlocks take one split, of up to
// kSmallClusterBlocks at most 8, of up to kClusterBlocks at most 16; longer ones
// the general rule's splits, a workspace and a merge launch where they are more.
// Measured, us on the device, workspace - 8 - 16 (32 / 8 heads of 128): 1 sequence
// of 100 keys 7.2 - 5.9 - 6.5 (one split 5.2), of 500 7.8 - 5.6 - 6.0 (one 9.8), of
// 1000 8.6 - 6.5 - 7.2, of 2000 11.9 - 8.2 - 7.9, of 4000 13.2 - 10.8 - 9.7, of 8000
// 15.0 - 16.6 - 13.2, of 16000 19.6 - 26 - 20.4; 4 of 1000 10.2 - 7.9 - 8.3; 8 of 6000
// 25.6 - 23.3 - 23.6.
// Only where the GPU holds all the launch's CTAs at a time: past that a cluster waits
// for room for all of it.  Workspace - clusters: 32 sequences of 1K to 3K keys, 32 / 8
// heads of 128 (768 CTAs) 37.5 - 47, of 64 27.3 - 32.6; 16 of 8K to 16K, 10 / 5 (1280 CTAs)
// 58 - 73; below 32 of 1K to 3K, 10 / 5, 30.0 - 27.7.
constexpr int kDecodeCtasPerSm = 4;
constexpr int kOneSplitBlocks = 8;
constexpr int kSmallClusterBlocks = 96;
constexpr int kClusterBlocks = 1024;

struct Int8Plan {
  Plan split;              // num_decode, and the split kernel's cut
  bool teams = false;
  bool cluster = false;    // the split kernel's CTAs of a row merge among themselves
  int col_groups = 1;      // groups of 8 q heads per kv head
  int team_heads = 1, team_warps = 1;
  int teams_per_range = 1;
  int num_ranges = 1;      // ranges that give every resident team one
  int max_ranges = 1;      // that there can be: the workspace has two slots for each
  size_t ws_o_bytes = 0, ws_lse_bytes = 0;
  size_t decode_bytes = 0;   // workspace of the decode kernel taken
  // prefill: parts of the keys, and their workspace behind the decode's
  int key_splits = 1;
  size_t pf_o_bytes = 0;
  size_t ws_bytes = 0;
};

// A batch's meta with its bounds no looser than they have to be (and far from
// the ends of 32 bits): no context is longer than its table row holds, no
// sequence has more rows than the batch, and a window of 2^30 keys hides none.
pkv_attn_meta int8_meta(const pkv_attn_meta& m) {
  pkv_attn_meta t = m;
  t.max_context_len = static_cast<int32_t>(std::min<int64_t>(
      {m.max_context_len, static_cast<int64_t>(m.block_table_stride) * kBlock, 1 << 30}));
  if (t.sliding_window >= 1 << 30) t.sliding_window = 0;
  t.max_query_len = std::min(m.max_query_len, m.num_tokens);
  return t;
}

int make_int8_decode_plan(const pkv_cache_desc* c, const pkv_attn_meta* m, int num_sms,
                          Int8Plan* p) {
  *p = Int8Plan{};
  pkv_cache_desc as_bytes = *c;
  as_bytes.dtype = PKV_FP8_E4M3;
  if (int st = make_plan(&as_bytes, m, num_sms, &p->split)) return st;
  const int split_span = p->split.split_blocks * p->split.max_splits;
  if (m->kv_split_tokens == 0 && p->split.max_splits > 1 && split_span <= kOneSplitBlocks) {
    p->split.split_blocks = split_span;
    p->split.max_splits = 1;
  }
  const int most = split_span <= kSmallClusterBlocks ? kDecodeCluster / 2 : kDecodeCluster;
  // (splits that the caller asked for go through the workspace, and so do those
  // beside chunk rows, whose CTAs rarely leave a cluster its SMs at one time: 16 rows
  // of 1K to 8K keys and 2 x 1024 tokens 156 us, 179 with clusters)
  const bool may = m->kv_split_tokens == 0 && p->split.num_decode == m->num_seqs;
  int blocks_each = p->split.split_blocks, splits = p->split.max_splits;
  if (splits > most && split_span <= kClusterBlocks) {
    blocks_each = (split_span + most - 1) / most;
    splits = (split_span + blocks_each - 1) / blocks_each;
  }
  const int64_t rows = static_cast<int64_t>(p->split.num_decode) * c->num_kv_heads *
                       ((m->num_q_heads / c->num_kv_heads + 7) / 8);
  p->cluster = may && splits > 1 && splits <= kDecodeCluster &&
               rows * splits <= static_cast<int64_t>(kDecodeCtasPerSm) * num_sms;
  if (p->cluster) {
    p->split.split_blocks = blocks_each;
    p->split.max_splits = splits;
  }
  if (p->cluster || p->split.max_splits <= 1) p->split.ws_o_bytes = p->split.ws_bytes = 0;
  p->decode_bytes = p->split.ws_bytes;
  const int nd = p->split.num_decode;
  if (nd == 0) return PKV_OK;
  p->col_groups = (m->num_q_heads / c->num_kv_heads + 7) / 8;
  // a team: kv heads side by side, read in one copy (the largest power of two
  // that divides their number), times the groups of 8 q heads that share them
  int cols = 1;
  while (2 * cols <= std::min(p->col_groups, kDecInt8Warps)) cols *= 2;
  while (2 * p->team_heads * cols <= kDecInt8Warps && c->num_kv_heads % (2 * p->team_heads) == 0)
    p->team_heads *= 2;
  p->team_warps = p->team_heads * cols;
  p->teams_per_range = c->num_kv_heads / p->team_heads * ((p->col_groups + cols - 1) / cols);
  p->num_ranges = std::max(
      num_sms * kDecInt8CtasPerSm * (kDecInt8Warps / p->team_warps) / p->teams_per_range, 1);
  int64_t longest = (static_cast<int64_t>(m->max_context_len) + kBlock - 1) / kBlock;
  if (m->sliding_window > 0)   // W keys span at most (W + 14) / 16 + 1 blocks
    longest = std::min(longest, (static_cast<int64_t>(m->sliding_window) + 14) / kBlock + 1);
  const int64_t blocks = longest * nd;
  if (nd <= 65535 && (p->team_warps < 4 ||   // (the split kernel's grid.z: sequences)
                      blocks < static_cast<int64_t>(kTeamRangeBlocks) * p->num_ranges))
    return PKV_OK;
  const int64_t line = blocks + static_cast<int64_t>(kSeqCost) * nd;
  const int64_t ranges =
      m->kv_split_tokens > 0
          ? (line + m->kv_split_tokens / kBlock - 1) / (m->kv_split_tokens / kBlock)
          : std::min<int64_t>(p->num_ranges, (line + kMinRangeBlocks - 1) / kMinRangeBlocks);
  // (counts that the kernel holds in 32 bits)
  if (ranges * p->teams_per_range > INT32_MAX / 2 || line / p->num_ranges > INT32_MAX / 2)
    return nd <= 65535 ? PKV_OK : PKV_E_SHAPE;
  p->teams = true;
  p->max_ranges = static_cast<int>(std::max<int64_t>(ranges, 1));
  p->decode_bytes = 0;
  if (p->max_ranges > 1) {
    const size_t rows = 2 * static_cast<size_t>(p->max_ranges) * m->num_q_heads;
    p->ws_o_bytes = round_up(rows * c->head_size * sizeof(float), 256);
    p->ws_lse_bytes = round_up(rows * sizeof(float), 256);
    p->decode_bytes = p->ws_o_bytes + p->ws_lse_bytes +
                      round_up(static_cast<size_t>(nd) * sizeof(int2), 256);
  }
  return PKV_OK;
}

int make_int8_plan(const pkv_cache_desc* c, const pkv_attn_meta* m, int num_sms, Int8Plan* p) {
  if (int st = make_int8_decode_plan(c, m, num_sms, p)) return st;
  const int npf = m->num_seqs - p->split.num_decode;
  const int G = m->num_q_heads / c->num_kv_heads;
  if (npf > 65535 && G <= 128) return PKV_E_SHAPE;   // (the prefill kernel's grid.z)
  if (npf > 0 && G <= 128) {
    // keys a CTA's rows see at most: the context, or the window before each of them
    int64_t keys = m->max_context_len;
    const int toks = prefill_tc_tokens_per_cta(G);
    if (m->sliding_window > 0) keys = std::min<int64_t>(keys, int64_t{m->sliding_window} + toks);
    const int64_t ctas = static_cast<int64_t>(npf) * ((m->max_query_len + toks - 1) / toks) *
                         c->num_kv_heads;
    p->key_splits = prefill_int8_key_splits(ctas, static_cast<int>((keys + 127) / 128), num_sms);
    if (p->key_splits > 1) {
      // (max_query_len rows a sequence: few CTAs, few rows)
      const size_t rows = static_cast<size_t>(npf) * m->max_query_len * m->num_q_heads * p->key_splits;
      p->pf_o_bytes = round_up(rows * c->head_size * sizeof(float), 256);
      p->ws_bytes = p->pf_o_bytes + round_up(rows * sizeof(float), 256);
    }
  }
  p->ws_bytes += p->decode_bytes;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_write_int8(const void* k, const void* v, const int32_t* block_tables,
                              const int32_t* context_lens, const int32_t* query_start_loc,
                              void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                              const pkv_cache_desc* cache, const pkv_attn_meta* meta,
                              void* stream) {
  if (int st = check_cache_int8(cache)) return st;
  if (int st = check_meta(cache, meta)) return st;
  if (meta->num_seqs == 0 || meta->num_tokens == 0) return PKV_OK;
  if (!k || !v || !block_tables || !context_lens || !query_start_loc || !k_cache || !v_cache ||
      !k_scales || !v_scales)
    return PKV_E_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(query_start_loc) ||
      !aligned4(k_scales) || !aligned4(v_scales))
    return PKV_E_ALIGN;
  WriteInt8Args a{};
  a.k = k;
  a.v = v;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start_loc = query_start_loc;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.bt_stride = meta->block_table_stride;
  a.num_seqs = meta->num_seqs;
  a.num_tokens = meta->num_tokens;
  a.num_kv_heads = cache->num_kv_heads;
  a.head_size = cache->head_size;
  a.num_blocks = cache->num_blocks;
  a.max_query_len = meta->max_query_len;
  // one row a sequence: its one block; else rows / 16 + 2 a sequence
  a.num_units = meta->max_query_len == 1
                    ? meta->num_seqs
                    : meta->num_tokens / kBlock + 2 * static_cast<int64_t>(meta->num_seqs) + 1;
  if (a.num_units * cache->num_kv_heads > INT32_MAX) return PKV_E_SHAPE;   // (the grid)
  int sms;
  if (int st = device_state(&a.err, &sms)) return st;
  PKV_TRY(launch_write_int8(a, as_stream(stream)));
  return PKV_OK;
}

extern "C" size_t pkv_attention_int8_workspace_size(const pkv_cache_desc* cache,
                                                    const pkv_attn_meta* meta) {
  if (check_cache_int8(cache) != PKV_OK || check_meta(cache, meta) != PKV_OK)
    return static_cast<size_t>(-1);
  int32_t* err;
  int sms;
  Int8Plan p;
  const pkv_attn_meta tight = int8_meta(*meta);
  if (device_state(&err, &sms) != PKV_OK || make_int8_plan(cache, &tight, sms, &p) != PKV_OK)
    return static_cast<size_t>(-1);
  return p.ws_bytes;
}

extern "C" int pkv_attention_int8(void* out, const void* q, const void* k_cache,
                                  const void* v_cache, const int32_t* block_tables,
                                  const int32_t* context_lens, const int32_t* query_start_loc,
                                  float scale, const float* k_scales, const float* v_scales,
                                  const pkv_cache_desc* cache, const pkv_attn_meta* given,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_cache_int8(cache)) return st;
  if (int st = check_meta(cache, given)) return st;
  const pkv_attn_meta tight = int8_meta(*given);
  const pkv_attn_meta* meta = &tight;
  if (meta->num_seqs == 0 || meta->num_tokens == 0) return PKV_OK;
  if (cache->num_blocks == 0) return PKV_E_SHAPE;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start_loc ||
      !k_scales || !v_scales)
    return PKV_E_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(query_start_loc) ||
      !aligned4(k_scales) || !aligned4(v_scales))
    return PKV_E_ALIGN;
  int32_t* err;
  int sms, dev;
  if (int st = device_state(&err, &sms, &dev)) return st;
  Int8Plan p;
  if (int st = make_int8_plan(cache, meta, sms, &p)) return st;
  if (p.ws_bytes > 0) {
    if (workspace == nullptr || workspace_bytes < p.ws_bytes) return PKV_E_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_E_ALIGN;
  }
  const cudaStream_t st = as_stream(stream);
  const float scale_log2 = scale * 1.4426950408889634f;
  const int G = meta->num_q_heads / cache->num_kv_heads;
  const int nd = p.split.num_decode, npf = meta->num_seqs - nd;
  CUtensorMap kmap, vmap;   // one head's block a copy: the split and the prefill kernels
  if (!p.teams || npf > 0) {
    if (int e = encode_cache_map(&kmap, k_cache, *cache)) return e;
    if (int e = encode_cache_map(&vmap, v_cache, *cache)) return e;
  }
  auto team_part = [&](cudaStream_t st) -> int {
    CUtensorMap khmap, vhmap;
    if (int e = encode_heads_map(&khmap, k_cache, *cache, p.team_heads)) return e;
    if (int e = encode_heads_map(&vhmap, v_cache, *cache, p.team_heads)) return e;
    TeamDecodeArgs d{};
    d.out = out;
    d.q = q;
    d.k_scales = k_scales;
    d.v_scales = v_scales;
    d.block_tables = block_tables;
    d.context_lens = context_lens;
    d.query_start_loc = query_start_loc;
    if (p.decode_bytes > 0) {
      char* ws = static_cast<char*>(workspace);
      d.ws_o = reinterpret_cast<float*>(ws);
      d.ws_lse = reinterpret_cast<float*>(ws + p.ws_o_bytes);
      d.span = reinterpret_cast<int2*>(ws + p.ws_o_bytes + p.ws_lse_bytes);
    }
    d.err = err;
    d.bt_stride = meta->block_table_stride;
    d.num_seqs = nd;
    d.num_tokens = meta->num_tokens;
    d.num_q_heads = meta->num_q_heads;
    d.num_kv_heads = cache->num_kv_heads;
    d.group = G;
    d.col_groups = p.col_groups;
    d.num_blocks = cache->num_blocks;
    d.max_context_len = meta->max_context_len;
    d.window = meta->sliding_window;
    d.range_blocks = meta->kv_split_tokens / kBlock;
    d.num_ranges = p.num_ranges;
    d.max_ranges = p.max_ranges;
    d.team_warps = p.team_warps;
    d.team_heads = p.team_heads;
    d.teams_per_range = p.teams_per_range;
    const int cta_teams = kDecInt8Warps / p.team_warps;
    d.grid = static_cast<uint32_t>((static_cast<int64_t>(p.max_ranges) * p.teams_per_range +
                                    cta_teams - 1) / cta_teams);
    d.scale_log2 = scale_log2;
    PKV_TRY(launch_team_decode(khmap, vhmap, d, cache->head_size, p.max_ranges > 1, st));
    return PKV_OK;
  };
  auto decode_part = [&](cudaStream_t st) -> int {
    if (p.teams) return team_part(st);
    DecodeArgs d{};
    d.out = out;
    d.q = q;
    d.block_tables = block_tables;
    d.context_lens = context_lens;
    d.query_start_loc = query_start_loc;
    d.ws_o = p.decode_bytes ? static_cast<float*>(workspace) : nullptr;
    d.ws_lse = p.decode_bytes ? reinterpret_cast<float*>(static_cast<char*>(workspace) + p.split.ws_o_bytes)
                          : nullptr;
    d.err = err;
    d.bt_stride = meta->block_table_stride;
    d.num_seqs = nd;
    d.num_q_heads = meta->num_q_heads;
    d.num_kv_heads = cache->num_kv_heads;
    d.group = G;
    d.num_blocks = cache->num_blocks;
    d.split_blocks = p.split.split_blocks;
    d.max_splits = p.split.max_splits;
    d.num_tokens = meta->num_tokens;
    d.max_context_len = meta->max_context_len;
    d.window = meta->sliding_window;
    d.k_scales = k_scales;
    d.v_scales = v_scales;
    d.scale_log2 = scale_log2;
    d.cluster = p.cluster;
    PKV_TRY(launch_decode_int8(kmap, vmap, d, cache->head_size, st));
    if (!p.cluster) PKV_TRY(launch_combine_bf16(d, cache->head_size, st, /*after_decode=*/true));
    return PKV_OK;
  };
  auto prefill_part = [&](cudaStream_t st) -> int {
    if (G > 128) {   // more q heads on a kv head than a query tile has rows
      AttnInt8Args a{};
      a.out = out;
      a.q = q;
      a.k_cache = k_cache;
      a.v_cache = v_cache;
      a.k_scales = k_scales;
      a.v_scales = v_scales;
      a.block_tables = block_tables;
      a.context_lens = context_lens;
      a.query_start_loc = query_start_loc;
      a.err = err;
      a.bt_stride = meta->block_table_stride;
      a.seq_begin = nd;
      a.num_seqs = meta->num_seqs;
      a.num_tokens = meta->num_tokens;
      a.num_q_heads = meta->num_q_heads;
      a.num_kv_heads = cache->num_kv_heads;
      a.num_blocks = cache->num_blocks;
      a.max_query_len = meta->max_query_len;
      a.window = meta->sliding_window;
      a.scale_log2 = scale_log2;
      PKV_TRY(launch_attention_int8(a, cache->head_size, st));
      return PKV_OK;
    }
    PrefillArgs f{};
    f.out = out;
    f.q = q;
    f.block_tables = block_tables;
    f.context_lens = context_lens;
    f.query_start_loc = query_start_loc;
    f.err = err;
    f.bt_stride = meta->block_table_stride;
    f.seq_begin = nd;
    f.num_seqs = npf;
    f.num_q_heads = meta->num_q_heads;
    f.num_kv_heads = cache->num_kv_heads;
    f.group = G;
    f.num_blocks = cache->num_blocks;
    f.num_tokens = meta->num_tokens;
    f.max_query_len = meta->max_query_len;
    f.window = meta->sliding_window;
    f.k_scales = k_scales;
    f.v_scales = v_scales;
    f.scale_log2 = scale_log2;
    f.key_splits = p.key_splits;
    if (p.key_splits > 1) {
      char* ws = static_cast<char*>(workspace) + p.decode_bytes;
      f.ws_o = reinterpret_cast<float*>(ws);
      f.ws_lse = reinterpret_cast<float*>(ws + p.pf_o_bytes);
    }
    const int toks = prefill_tc_tokens_per_cta(G);
    f.num_mtiles = (meta->max_query_len + toks - 1) / toks;
    // Longest first where the CTAs are more than the SMs, beside decode rows too
    // (plain - longest first: 4 x 2048 tokens 577 - 562 us, 48 decode rows and 4 x
    // 512 127 - 124, 16 and 2 x 1024 165 - 156); else the ranking costs 0.8 us.
    f.longest_first = static_cast<int64_t>(npf) * f.num_mtiles * cache->num_kv_heads > sms;
    CUtensorMap qmap, omap;
    if (int e = encode_query_map(&qmap, q, meta->num_tokens, meta->num_q_heads, cache->head_size, G))
      return e;
    if (int e =
            encode_query_map(&omap, out, meta->num_tokens, meta->num_q_heads, cache->head_size, G))
      return e;
    PKV_TRY(launch_prefill_int8(qmap, kmap, vmap, omap, f, cache->head_size, st));
    return PKV_OK;
  };
  if (nd == 0) return prefill_part(st);
  if (npf == 0) return decode_part(st);
  // decode and prefill rows in one batch: as pkv_attention
  SideFork fork(dev, st);
  if (int e = fork.begin()) return e;
  int rc = prefill_part(fork.stream());
  if (rc == PKV_OK) rc = decode_part(st);
  const int jr = fork.join();
  return rc != PKV_OK ? rc : jr;
}

// -------------------------------------------------------------- page copies

namespace pkv {
namespace {

// The blocks that the pairs of one launch read and write: open addressing
// over a table four times the pairs a launch holds.
class PairSet {
 public:
  // Whether (from, to) may join the launch: `from` is not written in it, `to`
  // neither read nor written.
  bool independent(int from, int to) const {
    return (flags(from) & kWritten) == 0 && flags(to) == 0;
  }
  void add(int from, int to) {
    mark(from, kRead);
    mark(to, kWritten);
  }
  void clear() { std::fill(flag_, flag_ + kSlots, uint8_t{0}); }

 private:
  static constexpr int kLog2Slots = 11, kSlots = 1 << kLog2Slots;
  static_assert(kSlots >= 4 * kCopyPairs, "at most half full");
  static constexpr uint8_t kRead = 1, kWritten = 2;
  int find(int block) const {
    unsigned i = (static_cast<uint32_t>(block) * 2654435769u) >> (32 - kLog2Slots);
    while (flag_[i] != 0 && key_[i] != block) i = (i + 1) % kSlots;
    return static_cast<int>(i);
  }
  uint8_t flags(int block) const { return flag_[find(block)]; }
  void mark(int block, uint8_t f) {
    const int i = find(block);
    key_[i] = block;
    flag_[i] |= f;
  }
  int32_t key_[kSlots];
  uint8_t flag_[kSlots] = {};
};

}  // namespace
}  // namespace pkv

extern "C" int pkv_copy_blocks(void* const* buffers, const int64_t* page_bytes,
                               int32_t num_buffers, int32_t num_blocks, const int32_t* pairs,
                               int32_t num_pairs, void* stream) {
  if (num_buffers < 0 || num_blocks < 0 || num_pairs < 0) return PKV_E_SHAPE;
  if (num_buffers == 0 || num_pairs == 0) return PKV_OK;
  if (!buffers || !page_bytes || !pairs) return PKV_E_NULL;
  for (int i = 0; i < num_buffers; ++i) {
    if (!buffers[i]) return PKV_E_NULL;
    if (page_bytes[i] < 1 || page_bytes[i] > (int64_t{1} << 30)) return PKV_E_SHAPE;
    if (!aligned4(buffers[i]) || page_bytes[i] % 4 != 0) return PKV_E_ALIGN;
  }
  for (int64_t i = 0; i < 2 * static_cast<int64_t>(num_pairs); ++i)
    if (pairs[i] < 0 || pairs[i] >= num_blocks) return PKV_E_SHAPE;
  int32_t* err;
  int sms;
  if (int st = device_state(&err, &sms)) return st;
  const cudaStream_t st = as_stream(stream);
  CopyArgs a;
  PairSet set;
  a.num_pairs = 0;
  auto flush = [&]() -> int {
    for (int b0 = 0; b0 < num_buffers; b0 += kCopyBuffers) {
      a.num_buffers = std::min(kCopyBuffers, num_buffers - b0);
      uint32_t units = 0;
      for (int i = 0; i < a.num_buffers; ++i) {
        CopyBuffer& b = a.buffers[i];
        b.base = buffers[b0 + i];
        b.page_bytes = page_bytes[b0 + i];
        b.unit_begin = units;
        if (b.page_bytes > kCopyUnit / 2) {
          b.split = static_cast<int32_t>((b.page_bytes + kCopyUnit - 1) / kCopyUnit);
          units += static_cast<uint32_t>(a.num_pairs) * b.split;
        } else {
          const int per = static_cast<int>(kCopyUnit / b.page_bytes);
          b.split = -per;
          units += (a.num_pairs + per - 1) / per;
        }
      }
      PKV_TRY(launch_copy_blocks(a, units, st));
    }
    a.num_pairs = 0;
    set.clear();
    return PKV_OK;
  };
  for (int i = 0; i < num_pairs; ++i) {
    const int from = pairs[2 * i], to = pairs[2 * i + 1];
    if (from == to) continue;
    if (a.num_pairs == kCopyPairs || !set.independent(from, to))
      if (int e = flush()) return e;
    a.pairs[a.num_pairs++] = make_int2(from, to);
    set.add(from, to);
  }
  return a.num_pairs > 0 ? flush() : PKV_OK;
}

// ------------------------------------- steps with drafted tokens: rotation and write

namespace pkv {
namespace {

int check_rope(const pkv_rope_desc* d) {
  if (d == nullptr) return PKV_E_NULL;
  if (d->dtype != PKV_BF16 && d->dtype != PKV_F32) return PKV_E_DTYPE;
  if (d->head_size != 64 && d->head_size != 128) return PKV_E_SHAPE;
  if (d->num_tokens < 0 || d->num_q_heads < 1 || d->num_kv_heads < 1 ||
      static_cast<int64_t>(d->num_q_heads) + 2 * static_cast<int64_t>(d->num_kv_heads) > 65535 ||
      d->rot_dim < 0 || d->rot_dim > d->head_size || d->rot_dim % 2 != 0 || d->max_position < 0)
    return PKV_E_SHAPE;
  return PKV_OK;
}

// Rows of `heads` heads, `stride` elements from one token to the next: rows apart, each
// begins on 16 bytes.
int check_rows(const void* p, int64_t stride, int heads, const pkv_rope_desc& d) {
  if (p == nullptr) return PKV_E_NULL;
  const int64_t e = d.dtype == PKV_F32 ? 4 : 2;
  if (stride < static_cast<int64_t>(heads) * d.head_size || stride > INT64_MAX / 16) return PKV_E_SHAPE;
  return aligned16(p) && stride * e % 16 == 0 ? PKV_OK : PKV_E_ALIGN;
}

// What the three calls share; v, slots and the caches are null for rows alone.
int rope_impl(void* q_out, void* k_out, const void* q, const void* k, const void* v,
              const int64_t* positions, const float* cos_sin, const void* q_weight,
              const void* k_weight, const int64_t* slot_mapping, void* k_cache, void* v_cache,
              const float* k_scale, const float* v_scale, const pkv_rope_desc* rope,
              const pkv_cache_desc* cache, void* stream) {
  if (int st = check_rope(rope)) return st;
  const pkv_rope_desc& d = *rope;
  if (cache != nullptr && (cache->num_kv_heads != d.num_kv_heads || cache->head_size != d.head_size))
    return PKV_E_SHAPE;
  if (d.num_tokens == 0) return PKV_OK;
  if (!positions || (!cos_sin && d.rot_dim > 0)) return PKV_E_NULL;
  if (int st = check_rows(q, d.q_stride, d.num_q_heads, d)) return st;
  if (int st = check_rows(k, d.k_stride, d.num_kv_heads, d)) return st;
  if (int st = check_rows(q_out, d.q_out_stride, d.num_q_heads, d)) return st;
  if (cache != nullptr) {
    if (int st = check_rows(v, d.v_stride, d.num_kv_heads, d)) return st;
    if (!slot_mapping || !k_cache || !v_cache) return PKV_E_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_E_ALIGN;
  } else if (int st = check_rows(k_out, d.k_out_stride, d.num_kv_heads, d)) {
    return st;
  }
  if ((reinterpret_cast<uintptr_t>(positions) & 7u) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
      !aligned16(cos_sin) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned4(k_scale) ||
      !aligned4(v_scale))
    return PKV_E_ALIGN;
  RopeArgs a{};
  int sms;
  if (int st = device_state(&a.err, &sms)) return st;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.slot_mapping = slot_mapping;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  if (cache != nullptr) a.num_slots = static_cast<int64_t>(cache->num_blocks) * cache->block_size;
  a.q_stride = d.q_stride;
  a.k_stride = d.k_stride;
  a.v_stride = d.v_stride;
  a.q_out_stride = d.q_out_stride;
  a.k_out_stride = d.k_out_stride;
  a.num_tokens = d.num_tokens;
  a.num_q_heads = d.num_q_heads;
  a.num_kv_heads = d.num_kv_heads;
  a.max_position = d.max_position;
  a.rot_dim = d.rot_dim;
  a.interleaved = d.interleaved != 0;
  a.eps = d.eps;
  PKV_TRY(launch_rope(a, d.head_size, d.dtype == PKV_F32, k_scale != nullptr, sms,
                      as_stream(stream)));
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_rope_write(void* q_out, const void* q, const void* k, const void* v,
                              const int64_t* positions, const float* cos_sin,
                              const void* q_weight, const void* k_weight,
                              const int64_t* slot_mapping, void* k_cache, void* v_cache,
                              const pkv_rope_desc* rope, const pkv_cache_desc* cache,
                              void* stream) {
  if (int st = check_cache(cache)) return st;
  if (rope == nullptr) return PKV_E_NULL;
  if (cache->dtype != rope->dtype) return PKV_E_DTYPE;   // (e4m3: pkv_rope_write_fp8)
  return rope_impl(q_out, nullptr, q, k, v, positions, cos_sin, q_weight, k_weight, slot_mapping,
                   k_cache, v_cache, nullptr, nullptr, rope, cache, stream);
}

extern "C" int pkv_rope_write_fp8(void* q_out, const void* q, const void* k, const void* v,
                                  const int64_t* positions, const float* cos_sin,
                                  const void* q_weight, const void* k_weight,
                                  const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                  const float* k_scale, const float* v_scale,
                                  const pkv_rope_desc* rope, const pkv_cache_desc* cache,
                                  void* stream) {
  if (int st = check_cache(cache)) return st;
  if (rope == nullptr || !k_scale || !v_scale) return PKV_E_NULL;
  if (cache->dtype != PKV_FP8_E4M3 || rope->dtype != PKV_BF16) return PKV_E_DTYPE;
  return rope_impl(q_out, nullptr, q, k, v, positions, cos_sin, q_weight, k_weight, slot_mapping,
                   k_cache, v_cache, k_scale, v_scale, rope, cache, stream);
}

extern "C" int pkv_rope(void* q_out, void* k_out, const void* q, const void* k,
                        const int64_t* positions, const float* cos_sin, const void* q_weight,
                        const void* k_weight, const pkv_rope_desc* rope, void* stream) {
  return rope_impl(q_out, k_out, q, k, nullptr, positions, cos_sin, q_weight, k_weight, nullptr,
                   nullptr, nullptr, nullptr, nullptr, rope, nullptr, stream);
}

// ------------------------------------- attention of a tree of drafted tokens

namespace pkv {
namespace {

struct TreePlan {
  // fp32
  int split_blocks = 0;
  int max_splits = 0;
  // tcgen05
  bool keys_on_m = false;
  int tile_toks = 0, part_rows = 0, cta_tiles = 0, max_groups = 0, workers = 0;
  bool whole = false;
  int64_t range = 0;
  size_t ws_o_bytes = 0, ws_lse_bytes = 0;
  size_t ws_bytes = 0;
};

// Tiles of 32 (row, q head) pairs of one kv head, for the longest sequence.
int64_t tree_tiles(const pkv_cache_desc& c, const pkv_attn_meta& m) {
  return (static_cast<int64_t>(m.max_query_len) * (m.num_q_heads / c.num_kv_heads) + 31) / 32;
}

int check_tree(const pkv_cache_desc* c, const pkv_attn_meta* m) {
  if (int st = check_cache(c)) return st;
  if (int st = check_meta(c, m)) return st;
  if (m->sliding_window != 0) return PKV_E_META;
  if (m->num_seqs > 65535 || tree_tiles(*c, *m) * c->num_kv_heads > 65535)   // (the grid)
    return PKV_E_SHAPE;
  if (c->dtype != PKV_F32 && m->num_q_heads / c->num_kv_heads > kTreeRows) return PKV_E_SHAPE;
  return PKV_OK;
}

void make_tree_plan(const pkv_cache_desc* c, const pkv_attn_meta* m, int num_sms, TreePlan* p) {
  *p = TreePlan{};
  if (c->dtype == PKV_F32) {
    const int64_t blocks = std::max<int64_t>((static_cast<int64_t>(m->max_context_len) + kBlock - 1) / kBlock, 1);
    const int64_t units = std::max<int64_t>(m->num_seqs * tree_tiles(*c, *m) * c->num_kv_heads, 1);
    int64_t sb = m->kv_split_tokens / kBlock;
    if (sb == 0) {
      sb = 64;
      while (sb > 4 && units * ((blocks + sb - 1) / sb) < 2 * num_sms) sb /= 2;
    }
    p->split_blocks = static_cast<int>(sb);
    p->max_splits = static_cast<int>((blocks + sb - 1) / sb);
    if (p->max_splits > 1) {
      const size_t n = static_cast<size_t>(m->num_tokens) * m->num_q_heads * p->max_splits;
      p->ws_o_bytes = round_up(n * c->head_size * sizeof(float), 256);
      p->ws_lse_bytes = round_up(n * sizeof(float), 256);
      p->ws_bytes = p->ws_o_bytes + p->ws_lse_bytes;
    }
    return;
  }
  // Keys on M: at most 32 rows a kv head and head_size 128 (64 sequences of 500 to 4000 keys, 8 kv
  // heads, us, rows on M / keys on M: bf16 4 rows 98 / 97, 32 rows 108 / 100, 64 rows 107 / 167;
  // e4m3 159 / 106, 167 / 137, 160 / 234).
  const int group = m->num_q_heads / c->num_kv_heads;
  const int64_t most_rows = static_cast<int64_t>(m->max_query_len) * group;
  p->keys_on_m = c->head_size == 128 && most_rows <= kTreeKeysRows;
  const int step_keys = p->keys_on_m ? kTreeKeysStep : kTreeStepKeys;
  const int tile_rows = p->keys_on_m ? kTreeKeysRows : kTreeRows;
  p->tile_toks = std::max(std::min(m->max_query_len, tile_rows / group), 1);
  p->part_rows = p->keys_on_m ? p->tile_toks * group : kTreeRows;
  const int tiles = std::max((m->max_query_len + p->tile_toks - 1) / p->tile_toks, 1);
  // A worker is as many CTAs as there are row tiles: they share the keys' way through L2 (16
  // sequences of 16K to 32K keys with 2 tiles: 356 us, with a CTA a worker 456).  Of more than
  // 8 tiles it takes 2 to 8 at a time, the most that leave the fewest places of the last group
  // empty (sequences of 8000 to 16000 keys, us: 9 tiles 3 at a time 89, 4 106; 19 tiles 5 at a time 165, 4 163,
  // 2 167; 4 sequences of 38 tiles 2 at a time 585, 4 634).  One at a time would lose
  // where there are few sequences (9 tiles 112, 19 tiles 196) and gain where there are many (16 of 4000
  // keys, 19 tiles, 636 for 673).
  // The longest tree makes the worker for all: of sequences with fewer tiles its other CTAs do nothing
  // (100 sequences of 1 to 8 drafts x 4 heads over 500 to 4000 keys beside one of 8 drafts 154 us, of
  // 64, two tiles, 231, of 256, eight tiles, 760).
  constexpr int kMaxTiles = 8;
  p->cta_tiles = std::min(tiles, kMaxTiles);
  auto padded = [&](int c) { return (tiles + c - 1) / c * c; };
  if (tiles > kMaxTiles)
    for (int c = kMaxTiles - 1; c >= 2; --c)
      if (padded(c) < padded(p->cta_tiles)) p->cta_tiles = c;
  p->max_groups = (tiles + p->cta_tiles - 1) / p->cta_tiles;
  const int ctas_per_sm = p->keys_on_m ? 1 : 2;
  const int64_t most = std::max(num_sms * ctas_per_sm / p->cta_tiles, 1);
  const int64_t units = std::max<int64_t>(static_cast<int64_t>(m->num_seqs) * p->max_groups * c->num_kv_heads, 1);
  const int64_t steps = (static_cast<int64_t>(m->max_context_len) + step_keys - 1) / step_keys;
  // Contexts of up to 1024 keys are not cut: no partials, no second kernel (200 sequences of 100
  // to 600 keys with 64 rows a kv head 124 us, cut 177; 16 of 1000 keys 24.8, cut 30.8).  One
  // sequence of 1000 keys is faster cut on the device (22.4, cut 19.9), but not as a plain
  // call, which then has a workspace to get and a second launch (22.6, cut 27.3).
  const int64_t kWholeSteps = p->keys_on_m ? 8 : 16;
  if (m->kv_split_tokens > 0) {
    p->range = std::max(m->kv_split_tokens / step_keys, 1);
    p->workers = static_cast<int>(std::min<int64_t>((units * (steps + kTreeStart) + p->range - 1) / p->range, INT32_MAX / 16));
    p->range = std::max(p->range, (units * (steps + kTreeStart) + p->workers - 1) / p->workers);
  } else if (steps <= kWholeSteps) {
    p->whole = true;
    p->workers = static_cast<int>(std::min(units, most));
    return;
  } else {
    p->workers = static_cast<int>(std::max<int64_t>(std::min(most, units * (steps + kTreeStart) / kTreeMinRange), 1));
  }
  const size_t rows = static_cast<size_t>(p->workers) * 2 * p->cta_tiles * p->part_rows;
  p->ws_o_bytes = round_up(rows * c->head_size * sizeof(float), 256);
  p->ws_lse_bytes = round_up(rows * sizeof(float), 256);
  p->ws_bytes = p->ws_o_bytes + p->ws_lse_bytes + round_up(static_cast<size_t>(units) * sizeof(int2), 256);
}

int tree_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
              const int32_t* block_tables, const int32_t* context_lens,
              const int32_t* query_start_loc, const int64_t* tree_mask, float scale,
              const float* k_descale, const float* v_descale, const pkv_cache_desc* cache,
              const pkv_attn_meta* meta, void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_tree(cache, meta)) return st;
  if (meta->num_seqs == 0 || meta->num_tokens == 0 || meta->max_query_len == 0) return PKV_OK;
  if (cache->num_blocks == 0) return PKV_E_SHAPE;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start_loc ||
      !tree_mask)
    return PKV_E_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(query_start_loc) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return PKV_E_ALIGN;
  int32_t* err;
  int sms;
  if (int st = device_state(&err, &sms)) return st;
  TreePlan p;
  make_tree_plan(cache, meta, sms, &p);
  if (p.ws_bytes > 0) {
    if (workspace == nullptr || workspace_bytes < p.ws_bytes) return PKV_E_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PKV_E_ALIGN;
  }
  TreeArgs a{};
  a.out = out;
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start_loc = query_start_loc;
  a.tree_mask = reinterpret_cast<const uint64_t*>(tree_mask);
  a.k_descale = k_descale;
  a.v_descale = v_descale;
  if (p.ws_bytes > 0) {
    char* ws = static_cast<char*>(workspace);
    a.ws_o = reinterpret_cast<float*>(ws);
    a.ws_lse = reinterpret_cast<float*>(ws + p.ws_o_bytes);
    a.span = reinterpret_cast<int2*>(ws + p.ws_o_bytes + p.ws_lse_bytes);
  }
  a.err = err;
  a.bt_stride = meta->block_table_stride;
  a.num_seqs = meta->num_seqs;
  a.num_tokens = meta->num_tokens;
  a.num_q_heads = meta->num_q_heads;
  a.num_kv_heads = cache->num_kv_heads;
  a.group = meta->num_q_heads / cache->num_kv_heads;
  a.num_blocks = cache->num_blocks;
  a.max_query_len = meta->max_query_len;
  a.max_context_len = meta->max_context_len;
  a.mask_words = (meta->max_query_len + 63) / 64;
  a.split_blocks = p.split_blocks;
  a.max_splits = p.max_splits;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.keys_on_m = p.keys_on_m;
  a.part_rows = p.part_rows;
  a.tile_toks = p.tile_toks;
  a.cta_tiles = p.cta_tiles;
  a.max_groups = p.max_groups;
  a.workers = p.workers;
  a.whole = p.whole;
  a.range = p.range;
  const cudaStream_t st = as_stream(stream);
  if (cache->dtype == PKV_F32) {
    PKV_TRY(launch_tree_f32(a, cache->head_size, st));
    return PKV_OK;
  }
  CUtensorMap qmap, kmap, vmap;
  if (int e = encode_query_map(&qmap, q, meta->num_tokens, meta->num_q_heads, cache->head_size,
                               a.group, a.tile_toks))
    return e;
  if (int e = encode_cache_map(&kmap, k_cache, *cache)) return e;
  if (int e = encode_cache_map(&vmap, v_cache, *cache)) return e;
  PKV_TRY(launch_tree_tc(qmap, kmap, vmap, a, cache->head_size, cache->dtype == PKV_FP8_E4M3, st));
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_attention_tree_workspace_size(const pkv_cache_desc* cache,
                                                    const pkv_attn_meta* meta) {
  int32_t* err;
  int sms;
  if (check_tree(cache, meta) != PKV_OK || device_state(&err, &sms) != PKV_OK)
    return static_cast<size_t>(-1);
  TreePlan p;
  make_tree_plan(cache, meta, sms, &p);
  return p.ws_bytes;
}

extern "C" int pkv_attention_tree(void* out, const void* q, const void* k_cache,
                                  const void* v_cache, const int32_t* block_tables,
                                  const int32_t* context_lens, const int32_t* query_start_loc,
                                  const int64_t* tree_mask, float scale,
                                  const pkv_cache_desc* cache, const pkv_attn_meta* meta,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (cache != nullptr && cache->dtype == PKV_FP8_E4M3) return PKV_E_DTYPE;  // pkv_attention_tree_fp8
  return tree_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                   tree_mask, scale, nullptr, nullptr, cache, meta, workspace, workspace_bytes,
                   stream);
}

extern "C" int pkv_attention_tree_fp8(void* out, const void* q, const void* k_cache,
                                      const void* v_cache, const int32_t* block_tables,
                                      const int32_t* context_lens,
                                      const int32_t* query_start_loc, const int64_t* tree_mask,
                                      float scale, const float* k_descale,
                                      const float* v_descale, const pkv_cache_desc* cache,
                                      const pkv_attn_meta* meta, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (cache == nullptr) return PKV_E_NULL;
  if (cache->dtype != PKV_FP8_E4M3) return PKV_E_DTYPE;
  if (meta != nullptr && meta->num_seqs > 0 && meta->num_tokens > 0) {
    if (!k_descale || !v_descale) return PKV_E_NULL;
    if (!aligned4(k_descale) || !aligned4(v_descale)) return PKV_E_ALIGN;
  }
  return tree_impl(out, q, k_cache, v_cache, block_tables, context_lens, query_start_loc,
                   tree_mask, scale, k_descale, v_descale, cache, meta, workspace,
                   workspace_bytes, stream);
}

// ------------------------------------- the rows of accepted drafts

extern "C" int pkv_accept_drafts(void* const* buffers, const int64_t* row_bytes,
                                 int32_t num_buffers, int32_t num_blocks,
                                 const int32_t* block_tables, int32_t block_table_stride,
                                 const int32_t* context_lens, const int32_t* query_start_loc,
                                 int32_t num_seqs, const int32_t* accepted,
                                 const int32_t* num_accepted, int32_t max_accepted,
                                 int32_t* new_context_lens, void* stream) {
  if (num_buffers < 0 || num_blocks < 0 || num_seqs < 0 || max_accepted < 0) return PKV_E_SHAPE;
  if (block_table_stride < 1) return PKV_E_META;
  if (static_cast<int64_t>(num_blocks) * kBlock > INT32_MAX) return PKV_E_SHAPE;
  if (num_seqs == 0) return PKV_OK;
  if (!block_tables || !context_lens || !query_start_loc || !num_accepted ||
      (!accepted && max_accepted > 0) || (num_buffers > 0 && (!buffers || !row_bytes)))
    return PKV_E_NULL;
  for (int i = 0; i < num_buffers; ++i) {
    if (!buffers[i]) return PKV_E_NULL;
    if (row_bytes[i] < 1 || row_bytes[i] > (int64_t{1} << 26)) return PKV_E_SHAPE;
    if (!aligned4(buffers[i]) || row_bytes[i] % 4 != 0) return PKV_E_ALIGN;
  }
  if (!aligned4(block_tables) || !aligned4(context_lens) || !aligned4(query_start_loc) ||
      !aligned4(accepted) || !aligned4(num_accepted) || !aligned4(new_context_lens))
    return PKV_E_ALIGN;
  // (every CTA of a sequence reads all of these, so its new length goes elsewhere)
  auto over_new = [&](const int32_t* p, int64_t n) {
    const uintptr_t in = reinterpret_cast<uintptr_t>(p), to = reinterpret_cast<uintptr_t>(new_context_lens);
    return to < in + n * sizeof(int32_t) && in < to + num_seqs * sizeof(int32_t);
  };
  if (new_context_lens != nullptr &&
      (over_new(context_lens, num_seqs) || over_new(num_accepted, num_seqs) ||
       over_new(query_start_loc, static_cast<int64_t>(num_seqs) + 1) ||
       over_new(accepted, static_cast<int64_t>(num_seqs) * max_accepted) ||
       over_new(block_tables, static_cast<int64_t>(num_seqs) * block_table_stride)))
    return PKV_E_META;
  AcceptArgs a{};
  int sms;
  if (int st = device_state(&a.err, &sms)) return st;
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.query_start_loc = query_start_loc;
  a.accepted = accepted;
  a.num_accepted = num_accepted;
  a.new_lens = new_context_lens;
  a.bt_stride = block_table_stride;
  a.num_blocks = num_blocks;
  a.num_seqs = num_seqs;
  a.max_accepted = max_accepted;
  // (without buffers, one launch for the new lengths)
  for (int b0 = 0; b0 == 0 || b0 < num_buffers; b0 += kAcceptBuffers) {
    a.num_buffers = std::min(kAcceptBuffers, num_buffers - b0);
    for (int i = 0; i < a.num_buffers; ++i) a.buffers[i] = {buffers[b0 + i], row_bytes[b0 + i]};
    a.report = b0 == 0;
    PKV_TRY(launch_accept(a, as_stream(stream)));
  }
  return PKV_OK;
}

extern "C" int pkv_get_error(int32_t* error_bits, int clear) {
  if (error_bits == nullptr) return PKV_E_NULL;
  int32_t* err;
  int sms;
  if (int st = device_state(&err, &sms)) return st;
  PKV_TRY(cudaDeviceSynchronize());
  PKV_TRY(cudaMemcpy(error_bits, err, sizeof(int32_t), cudaMemcpyDeviceToHost));
  if (clear) {
    PKV_TRY(cudaMemset(err, 0, sizeof(int32_t)));
    PKV_TRY(cudaDeviceSynchronize());
  }
  return PKV_OK;
}

extern "C" int pkv_last_cuda_error(void) { return g_last_cuda_error.load(); }

extern "C" const char* pkv_last_cuda_error_string(void) {
  return cudaGetErrorString(static_cast<cudaError_t>(g_last_cuda_error.load()));
}

extern "C" const char* pkv_status_string(int status) {
  switch (status) {
    case PKV_OK: return "ok";
    case PKV_E_NULL: return "a required pointer is NULL";
    case PKV_E_DTYPE:
      return "dtype not supported by this call (PKV_F32/PKV_BF16: pkv_write, pkv_attention; "
             "PKV_FP8_E4M3: pkv_write_fp8, pkv_attention_fp8; "
             "PKV_INT8: pkv_write_int8, pkv_attention_int8)";
    case PKV_E_SHAPE: return "unsupported or out-of-range shape (block_size 16, head_size 64/128)";
    case PKV_E_GQA: return "num_q_heads is not a multiple of num_kv_heads";
    case PKV_E_WORKSPACE: return "workspace missing or smaller than pkv_attention_workspace_size";
    case PKV_E_ALIGN: return "pointer not aligned (16 B tensors, 4 B int32 metadata, 256 B workspace)";
    case PKV_E_CUDA: return "CUDA launch or driver call failed";
    case PKV_E_META: return "inconsistent pkv_attn_meta";
    default: return "unknown status";
  }
}
