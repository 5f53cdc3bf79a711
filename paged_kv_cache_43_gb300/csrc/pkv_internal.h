// pkv_internal.h -- argument blocks and launchers shared between the C-ABI
// front end (pkv_api.cu) and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"

namespace pkv {

// Keys per cache block; the only block size the kernels take.
constexpr int kBlock = 16;

struct WriteArgs {
  const void* k;
  const void* v;
  const int64_t* slot_mapping;
  void* k_cache;
  void* v_cache;
  int32_t* err;
  int64_t num_slots;    // num_blocks * block_size
  int32_t num_tokens;
  int32_t row_vecs;     // 16-byte vectors per token row (num_kv_heads*head_size*bytes/16)
  // FP8 cache: per-kv-head quantisation scales (null otherwise)
  const float* k_scale;
  const float* v_scale;
  int32_t head_size;
};

// Split-K decode over sequences [0, num_seqs) (each with one query row).
struct DecodeArgs {
  void* out;                     // bf16 [T, Hq, D]
  const void* q;                 // bf16 [T, Hq, D]
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  float* ws_o;                   // [num_seqs, Hq, max_splits, D] fp32 (split > 1 only)
  float* ws_lse;                 // [num_seqs, Hq, max_splits]   log2-domain
  int32_t* err;
  int64_t bt_stride;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;                 // num_q_heads / num_kv_heads
  int32_t num_blocks;
  int32_t split_blocks;          // cache blocks per split
  int32_t max_splits;
  int32_t num_tokens;            // rows of q/out: query_start_loc must stay inside
  int32_t max_context_len;       // bound the split buffer was sized for
  int32_t window;                // sliding window (keys per query), 0 = none
  const float* k_descale;        // FP8 cache: [num_seqs_total, Hkv] (null otherwise)
  const float* v_descale;
  float scale_log2;              // scale * log2(e)
  // Cascade attention (all zero otherwise).
  int32_t key_begin_blocks;      // suffix launch: a sequence's keys start at this block
  int32_t split_base;            // first workspace split slot this launch writes
  int32_t force_partial;         // write partials even when a row has one split
  int32_t prefix_splits;         // combine: leading split slots that hold prefix partials
  int32_t prefix_len;            // prefix launch: the shared keys [0, prefix_len)
  int32_t prefix_col_groups;     // prefix launch: 8-column groups per kv head
  // Combine over token rows [merge_rows_begin, merge_rows_end) (> begin: the
  // cascade merge of chunked-prefill rows, each with prefix_splits prefix
  // partials and one suffix partial); 0, 0 otherwise.
  int32_t merge_rows_begin;
  int32_t merge_rows_end;
  int32_t casc_seqs;             // sequences of the batch (rows mode: row -> sequence)
  // Test hook (pkv_debug_wait_test): main-loop wait limit (0 = the default)
  // and, when set, warp 0 of every CTA withholds its first block load so
  // that its wait runs out.
  uint64_t wait_limit_ns;
  int32_t debug_stall;
  // Int8 cache: block scales [num_blocks, Hkv] (null otherwise); cluster != 0:
  // the max_splits (<= kDecodeCluster) CTAs of a row are a cluster that merges
  // its partials itself
  const float* k_scales;
  const float* v_scales;
  int32_t cluster;
};
constexpr int kDecodeCluster = 16;   // (more than 8: where the GPU allows it, as this one does)

// Varlen causal attention over sequences [seq_begin, seq_begin + num_seqs).
struct PrefillArgs {
  void* out;
  const void* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  int32_t* err;
  int64_t bt_stride;
  int32_t seq_begin;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t num_blocks;
  int32_t num_mtiles;            // grid.x: row tiles of the longest sequence
  int32_t num_tokens;
  int32_t max_query_len;
  int32_t window;                // sliding window (keys per query), 0 = none
  const float* k_descale;        // FP8 cache: [num_seqs_total, Hkv] (null otherwise)
  const float* v_descale;
  float scale_log2;
  // tcgen05 kernel: hand the CTAs out longest first (a launch that has the
  // GPU to itself); 0 keeps the plain order, whose short CTAs finish early
  // and leave SMs to a decode launch running beside it.
  int32_t longest_first;
  // Cascade prefix launch of the tcgen05 kernel (cascade_prefix = 1): the
  // decode rows 0 .. num_seqs - 1 (row t = sequence t) against the shared keys
  // [0, prefix_len) of block-table row 0, prefix_tiles 128-key tiles per CTA
  // (grid.z = prefix split); normalised fp32 partials and log2-sum-exps go to
  // ws_o / ws_lse at split slot blockIdx.z of rows [seq, q head, max_splits].
  int32_t cascade_prefix;
  int32_t prefix_len;
  int32_t prefix_tiles;
  int32_t max_splits;
  float* ws_o;
  float* ws_lse;
  // Cascade prefix launch: the batch's sequences (query_start_loc has
  // casc_seqs + 1 entries), to find each row's sequence for its descales.
  int32_t casc_seqs;
  // Cascade suffix launch of the tcgen05 kernel (key_begin > 0): every row
  // sees only keys >= key_begin (the shared prefix is the prefix launch's),
  // and writes its normalised fp32 partial and log2-sum-exp to ws_o / ws_lse
  // at split slot split_base of rows [token, q head, max_splits].
  int32_t key_begin;
  int32_t split_base;
  // Test hook (pkv_debug_wait_test), tcgen05 kernel: main-loop wait limit (0
  // = the default) and, when set, the K producer withholds the CTA's first K
  // tile so that the waits for it run out.
  uint64_t wait_limit_ns;
  int32_t debug_stall;
  // Int8 cache: block scales [num_blocks, Hkv] (null otherwise), and the parts
  // each row's keys are cut into (> 1: partials to ws_o [sequence, row, q head,
  // key_splits, D] and ws_lse, then a merge)
  const float* k_scales;
  const float* v_scales;
  int32_t key_splits;
};

// Settings of the test hook, applied to the decode and tcgen05 prefill
// launches made after pkv_debug_wait_test (pkv_api.cu).
void debug_wait_settings(uint64_t* limit_ns, int32_t* stall);

// fp32 I/O: one CTA per (query row, q head), every sequence.
struct F32Args {
  float* out;
  const float* q;
  const float* k_cache;
  const float* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  int32_t* err;
  int64_t bt_stride;
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_size;
  int32_t num_blocks;
  int32_t window;                // sliding window (keys per query), 0 = none
  float scale;
};

// ---- int8 caches (one fp32 scale per block and kv head)

struct WriteInt8Args {
  const void* k;                 // bf16 [T, Hkv, D]
  const void* v;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  void* k_cache;
  void* v_cache;
  float* k_scales;               // [num_blocks, Hkv]
  float* v_scales;
  int32_t* err;
  int64_t bt_stride;
  int64_t num_units;             // touched blocks at most (one unit each)
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_kv_heads;
  int32_t head_size;
  int32_t num_blocks;
  int32_t max_query_len;
};

struct AttnInt8Args {
  void* out;                     // bf16 [T, Hq, D]
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  int32_t* err;
  int64_t bt_stride;
  int32_t seq_begin;             // sequences [seq_begin, num_seqs)
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t num_blocks;
  int32_t max_query_len;
  int32_t window;
  float scale_log2;
};

// Decode over sequences [0, num_seqs) of an int8 cache by teams of warps
// (pkv_decode_int8.cu): large batches.
constexpr int kDecInt8Warps = 8;       // of a CTA
constexpr int kDecInt8CtasPerSm = 2;   // resident CTAs per SM
// Blocks of a range at least: below this a CTA's start and its partial cost
// more than the keys it reads.
constexpr int kMinRangeBlocks = 16;
// What a sequence counts on the line of blocks before its own: its query, the
// first copies' latency, its output (256 sequences of 64 to 8192 keys, 8 kv
// heads: 146 us with 0, 139 with 2, 138 with 4).
constexpr int kSeqCost = 4;
struct TeamDecodeArgs {
  void* out;                     // bf16 [T, Hq, D]
  const void* q;
  const float* k_scales;
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  float* ws_o;                   // [2 max_ranges, Hq, D] partial outputs
  float* ws_lse;                 // [2 max_ranges, Hq], log2 domain
  int2* span;                    // [num_seqs]: first range, ranges (null: one range)
  int32_t* err;
  int64_t bt_stride;
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t col_groups;            // groups of 8 q heads per kv head
  int32_t num_blocks;
  int32_t max_context_len;
  int32_t window;
  int32_t range_blocks;          // blocks of a range (0: an equal share)
  int32_t num_ranges;            // ranges that give every resident team one
  int32_t team_warps;            // 1, 2, 4 or 8 warps that walk a range together:
  int32_t team_heads;            // this many kv heads (dividing num_kv_heads) x groups of 8 q heads
  int32_t teams_per_range;
  int32_t max_ranges;            // ranges the workspace holds
  uint32_t grid;
  float scale_log2;
  uint64_t wait_limit_ns;        // test hook, as DecodeArgs
  int32_t debug_stall;
};

// ---- page copies
constexpr int kCopyPairs = 512;
constexpr int kCopyBuffers = 64;
constexpr int kCopyUnit = 16384;   // bytes a CTA copies

struct CopyBuffer {
  void* base;
  int64_t page_bytes;
  uint32_t unit_begin;       // first CTA of this buffer
  int32_t split;             // > 0: units a page is cut into; < 0: -(small pages in a unit)
};
struct CopyArgs {
  CopyBuffer buffers[kCopyBuffers];
  int2 pairs[kCopyPairs];    // (from, to): no block is read and written, or written twice
  int32_t num_buffers;
  int32_t num_pairs;
};

// ---- norms, rotation and write in one pass
struct RopeArgs {
  void* q_out;                   // [T, Hq, D] rows, q_out_stride elements apart (as all below)
  void* k_out;                   // rows only (no slot_mapping), else null
  const void* q;
  const void* k;
  const void* v;                 // null: rows only
  const int64_t* positions;
  const float* cos_sin;          // [max_position, rot_dim]: cosines, then sines
  const void* q_weight;          // [D], null: no norm
  const void* k_weight;
  const int64_t* slot_mapping;   // null: rows only
  void* k_cache;
  void* v_cache;
  const float* k_scale;          // e4m3: per kv head (null otherwise)
  const float* v_scale;
  int32_t* err;
  int64_t num_slots;
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t max_position;
  int32_t rot_dim;
  int32_t interleaved;
  int32_t groups_per_token;      // set by the launch
  float eps;
};
cudaError_t launch_rope(const RopeArgs& a, int head_size, bool f32, bool fp8, int num_sms,
                        cudaStream_t stream);

// ---- attention of a tree of drafted tokens
struct TreeArgs {
  void* out;                     // [T, Hq, D]
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  const uint64_t* tree_mask;     // [T, mask_words]
  const float* k_descale;        // e4m3: [num_seqs, Hkv] (null otherwise)
  const float* v_descale;
  float* ws_o;                   // fp32 kernel: [T, Hq, max_splits, D] (max_splits > 1 only);
                                 // tcgen05: [workers, 2, cta_tiles, part_rows, D]
  float* ws_lse;                 // the same without D, log2 domain
  int32_t* err;
  int64_t bt_stride;
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  int32_t num_blocks;
  int32_t max_query_len;
  int32_t max_context_len;
  int32_t mask_words;
  int32_t split_blocks;          // fp32 kernel: cache blocks per split (a multiple of 4)
  int32_t max_splits;
  float scale_log2;
  // The tcgen05 kernels.
  int32_t keys_on_m;             // pkv_tree_keys.cu, else pkv_tree_tc.cu
  int32_t part_rows;             // (row, q head) pairs that a tile has at most
  int32_t tile_toks;             // query rows of a tile
  int32_t cta_tiles;             // CTAs of a worker: row tiles of a unit, side by side
  int32_t max_groups;            // groups of that many tiles, for the longest sequence
  int32_t workers;
  int32_t whole;                 // units are not cut: no workspace, no merge
  int64_t range;                 // steps of a worker, 0: equal shares (of kTreeMinRange or more)
  int2* span;                    // [num_seqs, max_groups, Hkv]: a unit's first worker, workers
  uint64_t wait_limit_ns;        // test hook, as DecodeArgs
  int32_t debug_stall;
};
constexpr int kTreeRows = 128, kTreeStepKeys = 64;         // pkv_tree_tc.cu
// Steps that a unit counts on the line of work for its start and end (64 sequences of 128 to 4096
// keys, 32 kv heads: 369 us with 1, 365 with 2, 347 with 4).
constexpr int kTreeStart = 4;
// Steps that a worker has at least where the work is cut into equal parts (one sequence of 1500
// keys, 8 kv heads, 64 rows, us: with 1 32.6, 2 23.4, 4 21.1, 6 22.9, 16 29.2).
constexpr int kTreeMinRange = 4;
constexpr int kTreeKeysRows = 32, kTreeKeysStep = 128;     // pkv_tree_keys.cu
// Tiles of at most kTreeKeysRows rows, head_size 128 (called by launch_tree_tc).
cudaError_t launch_tree_keys(const CUtensorMap& qmap, const CUtensorMap& kmap,
                             const CUtensorMap& vmap, const TreeArgs& a, bool fp8,
                             cudaStream_t stream);
// qmap: the queries in boxes of 64 columns x group heads x tile_toks rows.
cudaError_t launch_tree_tc(const CUtensorMap& qmap, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, const TreeArgs& a, int head_size, bool fp8,
                           cudaStream_t stream);
cudaError_t launch_tree_f32(const TreeArgs& a, int head_size, cudaStream_t stream);

// ---- the rows of accepted drafts
constexpr int kAcceptBuffers = 64;
struct AcceptBuffer {
  void* base;                    // [num_blocks, 16, row_bytes]
  int64_t row_bytes;
};
struct AcceptArgs {
  AcceptBuffer buffers[kAcceptBuffers];
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start_loc;
  const int32_t* accepted;       // [num_seqs, max_accepted]
  const int32_t* num_accepted;   // [num_seqs]
  int32_t* new_lens;             // [num_seqs] or null
  int32_t* err;
  int64_t bt_stride;
  int32_t num_buffers;
  int32_t num_blocks;
  int32_t num_seqs;
  int32_t max_accepted;
  int32_t report;                // this launch raises errors and writes new_lens
};
cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t stream);

cudaError_t launch_write(const WriteArgs& a, cudaStream_t stream, int num_sms);
cudaError_t launch_write_int8(const WriteInt8Args& a, cudaStream_t stream);
cudaError_t launch_attention_int8(const AttnInt8Args& a, int head_size, cudaStream_t stream);
cudaError_t launch_team_decode(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const TeamDecodeArgs& a, int head_size, bool merge,
                               cudaStream_t stream);
// The decode kernel over int8 caches with block scales (a.k_scales, a.v_scales).
cudaError_t launch_decode_int8(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const DecodeArgs& a, int head_size, cudaStream_t stream);
cudaError_t launch_copy_blocks(const CopyArgs& a, unsigned units, cudaStream_t stream);
cudaError_t launch_write_fp8(const WriteArgs& a, cudaStream_t stream, int num_sms);
// fp8 = true: the caches hold e4m3 codes (the maps are uint8, unswizzled).
cudaError_t launch_decode_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const DecodeArgs& a, int head_size, bool fp8,
                               cudaStream_t stream);
// after_decode: launched right after launch_decode_bf16 on the same stream
// (a programmatic dependent launch; false when other work sits between them).
cudaError_t launch_combine_bf16(const DecodeArgs& a, int head_size, cudaStream_t stream,
                                bool after_decode = false);
// Cascade prefix launch: every decode row of the batch (all sequences, all q
// heads) against the shared prefix keys, read once per 8 columns; partials to
// split slots [0, prefix_splits).
cudaError_t launch_cascade_prefix_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                       const DecodeArgs& a, int head_size, cudaStream_t stream);
cudaError_t launch_prefill_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                const PrefillArgs& a, int head_size, bool fp8,
                                cudaStream_t stream);
cudaError_t launch_attention_f32(const F32Args& a, cudaStream_t stream);

// tcgen05 prefill: query tiles of 128 rows = (128 / group) tokens x group heads,
// two tiles per CTA.
bool prefill_tc_supported(int head_size, int group);
int prefill_tc_tokens_per_tile(int group);
int prefill_tc_tokens_per_cta(int group);
// fp8 = true: e4m3 caches, widened to fp16 in shared memory.
// omap: the output tensor viewed like qmap (full query tiles of a plain
// launch leave through it; cascade launches write the workspace instead).
cudaError_t launch_prefill_tc(const CUtensorMap& qmap, const CUtensorMap& kmap,
                              const CUtensorMap& vmap, const CUtensorMap& omap,
                              const PrefillArgs& a, int head_size, bool fp8,
                              cudaStream_t stream);

// Int8 caches with block scales (a.k_scales, a.v_scales; pkv_prefill_int8.cu); any
// group of at most 128.
int prefill_int8_key_splits(int64_t ctas, int tiles, int num_sms);
cudaError_t launch_prefill_int8(const CUtensorMap& qmap, const CUtensorMap& kmap,
                                   const CUtensorMap& vmap, const CUtensorMap& omap,
                                   const PrefillArgs& a, int head_size, cudaStream_t stream);

// Rows of the prefill kernel's query tile (grid.x covers ceil(q_len*G / this)).
constexpr int kPrefillRows = 64;

}  // namespace pkv
