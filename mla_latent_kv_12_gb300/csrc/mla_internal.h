// Internal declarations shared by the host API and the kernel launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mla.h"

namespace mla {

// Per-thread detail of the last error (set by the host API).
void set_error_detail(const char* fmt, ...);

constexpr int kMaxRotaryDims = 256;

struct RopeParams {
  const void* in;
  void* out;
  int64_t rows, tokens, inner, width;
  int64_t in_stride[3];
  int64_t out_stride[3];
  int32_t rotary_dims;
  const int32_t* row_offsets;
  int64_t position_offset;
  float inv_freq[kMaxRotaryDims / 2];
};
cudaError_t launch_rope(const RopeParams& p, int dtype, cudaStream_t stream);

// Geometry of a decode call (all strides in elements).
struct DecodeGeometry {
  const void* q;
  int64_t q_row_stride, q_head_stride;
  const void* latent;
  int64_t latent_row_stride, latent_batch_stride;
  const void* rope;
  int64_t rope_row_stride, rope_batch_stride;
  const int32_t* kv_start;
  const int32_t* kv_len;
  int32_t batch, s_q, heads, rank, rope_dim;
  int64_t t_max;
  const int32_t* sel;
  const int32_t* sel_count;
  int32_t k_max;
  float scale_log2;  // softmax_scale * log2(e)
  void* ctx_out;
  int64_t ctx_row_stride, ctx_head_stride;
  float* lse_out;
  int32_t* device_status;
  // 8-bit cache (null codes: `latent` is read): e4m3 codes with byte strides,
  // and one exponent byte per 2^block_shift buffer rows.
  const uint8_t* codes;
  int64_t codes_row_stride, codes_batch_stride;
  const uint8_t* scales;
  int64_t scales_batch_stride;
  int32_t block_shift;
  // Paged cache (null table: windows): pages of page_size rows; no kv_start, no batch strides.
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width, page_size, num_pages;
  int64_t latent_page_stride, rope_page_stride;
  const int32_t* counts;      // [batch] new tokens of each row (null: s_q)
  const uint64_t* tree;       // [n_q][tree_words] ancestor masks (null: tokens in a row)
  int32_t tree_words;
};

// CUDA-core decode of the f32 path (any shape; f32 q and cache).
size_t simt_decode_workspace(const DecodeGeometry& g, int* splits_out);
cudaError_t launch_simt_decode(const DecodeGeometry& g, int dtype, int out_dtype, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream);

// Tensor-core decode (bf16, heads 64 or 128, rank 512, rope 64).  With a tail, the
// split combine is fused with the W_UV projection (bf16 context in
// g.ctx_out, n_q <= 64, v_dim 128) and `tail->out` receives [n_q, H*v].
struct DecodeTail {
  const void* w;  // kv_b_proj [heads*(nope+v_dim), rank] bf16
  void* out;
  int64_t out_row_stride;
  int out_dtype;
  int32_t heads, nope, v_dim, rank;
};
size_t tc_decode_workspace(int32_t n_q);
size_t tc_paged_workspace(int32_t n_q);   // of the same kernels over pages
cudaError_t launch_tc_decode(const DecodeGeometry& g, int out_dtype, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream, const DecodeTail* tail = nullptr);

// The same over a paged cache whose pages are a multiple of 8 rows (no selection); launch_tc_decode
// serves the others, row by row.
cudaError_t launch_tc_paged(const DecodeGeometry& g, int out_dtype, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream);

struct AbsorbParams {
  const void* q_nope;
  int64_t q_row_stride, q_head_stride;
  const void* w;
  void* out;
  int64_t out_row_stride, out_head_stride;
  int32_t n_q, heads, nope, v_dim, rank;
};
// RoPE of the query's rope part folded into the tensor-core absorb launch
// (bf16, 64 rotary dims = the whole rope part): q_rope[n, h, 0:64] enters
// pair-interleaved and leaves rotated at q_out[n, h, out_col : out_col+64].
// Position of query row n = b*s_q + i is offset_b + i.
struct AbsorbRope {
  const void* q_rope;
  int64_t row_stride, head_stride;
  int32_t s_q;
  const int32_t* row_offsets;  // device [batch] or NULL
  int64_t position_offset;     // used when row_offsets is NULL
  int32_t out_col;
  float inv_freq[32];
};
// The page's f32 roundings of the inverse frequencies:
// invf_j = f32(pow(f32 theta, f32(f32(-2j) / d))).
void rope_inverse_frequencies(float theta, int rotary_dims, float* inv_freq);

cudaError_t launch_simt_absorb(const AbsorbParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_tc_absorb(const AbsorbParams& p, cudaStream_t stream, const AbsorbRope* rope = nullptr);
// CUDA-core matrix-vector absorb for 1..4 query rows (bf16, rank 512, nope 128).
bool gemv_absorb_serves(const AbsorbParams& p);
cudaError_t launch_gemv_absorb(const AbsorbParams& p, cudaStream_t stream, const AbsorbRope* rope = nullptr);

struct ProjectParams {
  const void* ctx;
  int64_t ctx_row_stride, ctx_head_stride;
  const void* w;
  void* out;
  int64_t out_row_stride;
  int32_t n_q, heads, nope, v_dim, rank;
};
cudaError_t launch_simt_project(const ProjectParams& p, int dtype, int out_dtype,
                                cudaStream_t stream);
cudaError_t launch_tc_project(const ProjectParams& p, int out_dtype, cudaStream_t stream);

cudaError_t launch_gather(const DecodeGeometry& g, int dtype, void* out, cudaStream_t stream);

// Append of S new tokens per batch row (RMSNorm of the latent, RoPE of the key).
constexpr int kMaxAppendRank = 1024;
struct AppendParams {
  const void* latent_raw;
  int64_t lr_row_stride, lr_tok_stride;
  const void* rope_raw;
  int64_t rr_row_stride, rr_tok_stride;
  const void* weight;
  float eps;
  const int32_t* row_offsets;
  void* cache_latent;
  int64_t cl_row_stride, cl_batch_stride;
  void* cache_rope;
  int64_t cr_row_stride, cr_batch_stride;
  const int32_t* kv_start;
  const int32_t* kv_len;
  int32_t* kv_len_out;
  int32_t batch, s_new, rank, rope_dim;
  int64_t t_max;
  int32_t* status;
  float inv_freq[kMaxRotaryDims / 2];
};
cudaError_t launch_append(const AppendParams& p, int in_dtype, int cache_dtype, cudaStream_t stream);

// Writing and reading an 8-bit latent cache (append, quantise, dequantise).
struct EncodeParams {
  const void* latent_raw;   // append: new tokens; quantise: the latent buffer
  int64_t lr_row_stride, lr_tok_stride;
  const void* rope_raw;
  int64_t rr_row_stride, rr_tok_stride;
  const void* weight;
  float eps;
  const int32_t* row_offsets;
  uint8_t* codes;
  int64_t codes_row_stride, codes_batch_stride;
  uint8_t* scales;
  int64_t scales_batch_stride;
  int32_t block_shift;
  void* rope;
  int64_t rope_row_stride, rope_batch_stride;
  void* latent_out;         // dequantise
  int64_t lo_row_stride, lo_batch_stride;
  const int32_t* kv_start;
  const int32_t* kv_len;
  int32_t* kv_len_out;
  int32_t batch, s_new, rank, rope_dim;
  int64_t t_max;
  int32_t* status;
  int32_t tile_rows, lengths_here;   // set by the launcher
  float inv_freq[kMaxRotaryDims / 2];
};
cudaError_t launch_append_q8(const EncodeParams& p, int in_dtype, int rope_dtype, bool vec, cudaStream_t stream);
cudaError_t launch_quantize(const EncodeParams& p, int dtype, bool vec, cudaStream_t stream);
cudaError_t launch_dequantize(const EncodeParams& p, int dtype, bool vec, cudaStream_t stream);

// Attention weight of every cached key, accumulated over heads and query tokens.
struct KeyWeightParams {
  DecodeGeometry g;         // q, cache, windows (ctx_out, lse_out and the selection unused)
  const float* lse;
  float* weights;
  int64_t weights_batch_stride;
  float decay;
  int32_t n_new;
};
cudaError_t launch_simt_key_weights(const KeyWeightParams& p, cudaStream_t stream);
cudaError_t launch_tc_key_weights(const KeyWeightParams& p, cudaStream_t stream);

// Eviction: the kept positions of each row, and the in-place compaction.
struct EvictParams {
  const float* weights;
  int64_t weights_batch_stride;
  const int32_t* kv_start;
  const int32_t* kv_len;
  int64_t t_max;
  int32_t batch, n_keep, n_sink, n_recent;
  int32_t* kept;
  int64_t kept_stride;
  int32_t* counts;
  int32_t* kv_len_out;
  int32_t* status;
};
cudaError_t launch_evict_plan(const EvictParams& p, cudaStream_t stream);
constexpr int kMaxStateArrays = 8;
struct CompactArray {
  uint8_t* data;
  int64_t row_bytes_stride, batch_bytes_stride;
  int32_t row_bytes;
  int32_t unit;             // bytes moved together: 16, 8, 4, 2 or 1
};
struct CompactParams {
  CompactArray a[kMaxStateArrays];
  int32_t n_arrays;
  const int32_t* kv_start;
  const int32_t* kept;
  int64_t kept_stride;
  const int32_t* counts;
  int32_t n_keep, batch;
  int64_t t_max;
  int32_t* status;
};
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);

// Writing a paged cache: append, tree plan, commit of an accepted path.
struct AppendPagedParams {
  const void* latent_raw;
  int64_t lr_row_stride, lr_tok_stride;
  const void* rope_raw;
  int64_t rr_row_stride, rr_tok_stride;
  const void* weight;
  float eps;
  const int32_t* positions;   // [batch][s_new] (null: the token's key index)
  void* latent;
  int64_t l_row_stride, l_page_stride;
  void* rope;
  int64_t r_row_stride, r_page_stride;
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width, page_size, num_pages;
  const int32_t* kv_len;
  const int32_t* counts;
  int32_t* kv_len_out;
  int32_t batch, s_new, rank, rope_dim;
  int32_t* status;
  int32_t lengths_here;       // set by the launcher: the kernel writes kv_len_out (2: which is kv_len)
  float inv_freq[kMaxRotaryDims / 2];
};
// vec: rank a multiple of 8, latents and the norm weight in rows of whole 16 bytes.
cudaError_t launch_append_paged(AppendPagedParams p, int in_dtype, int cache_dtype, bool vec, cudaStream_t stream);

constexpr int kMaxTreeNodes = 1024;
struct TreePlanParams {
  const int32_t* parents;
  int64_t parents_stride;
  const int32_t* kv_len;
  const int32_t* counts;
  int32_t* positions;
  uint64_t* mask;
  int32_t batch, n_nodes;
  int32_t* status;
};
cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream);

constexpr int kMaxCommitArrays = 256;
struct CommitArray {
  uint8_t* data;
  int64_t row_bytes_stride, page_bytes_stride;
  int32_t row_bytes;
  int32_t unit;               // bytes moved together: 16, 8, 4, 2 or 1
};
struct CommitParams {
  CommitArray a[kMaxCommitArrays];
  int32_t n_arrays;
  const int32_t* table;
  int64_t table_stride;
  int32_t table_width, page_size, num_pages;
  const int32_t* kv_len;
  const int32_t* path;
  int64_t path_stride;
  const int32_t* counts;
  int32_t path_width;
  int32_t* kv_len_out;
  int32_t batch;
  int32_t* status;
  int32_t lengths_here;
};
cudaError_t launch_commit_paged(CommitParams& p, cudaStream_t stream);

// Deterministic top-k selection of positions from per-row f32 scores.
struct SelectParams {
  const float* scores;
  int64_t row_stride;
  const int32_t* lengths;
  int32_t n_rows, top_k;
  int32_t* selected;
  int64_t out_stride;
  int32_t* counts;
  int32_t* status;
};
cudaError_t launch_select_topk(const SelectParams& p, cudaStream_t stream);

// Row gather of a right-aligned cache state array (rollback, filter, merge):
// dst[i, c] = c < zero_below[i] ? 0 : src[src_row[i], (c + shift[i]) mod src_width].
// Sizes and strides in bytes.
struct ShiftRowsParams {
  const void* src;
  int64_t src_col_bytes, src_batch_bytes;
  int32_t src_batch, src_width;
  void* dst;
  int64_t dst_col_bytes, dst_batch_bytes;
  int32_t dst_width, n_rows;
  int64_t row_bytes;
  const int32_t* src_row;     // NULL: row i
  const int32_t* shift;       // NULL: 0
  const int32_t* zero_below;  // NULL: 0
  int32_t* status;
  int32_t units_per_col, cols_per_cta;  // set by the launcher
};
cudaError_t launch_shift_rows(const ShiftRowsParams& p, int vec_bytes, cudaStream_t stream);
cudaError_t launch_rollback_lengths(const int32_t* before, const int32_t* keep, const int32_t* kv_len,
                                    int32_t* kv_len_out, int32_t batch, int32_t* status, cudaStream_t stream);

// Reconstruction of per-head keys and values from latent rows (prefill).
struct ReconstructParams {
  const void* latent;
  int64_t latent_row_stride, n_rows;
  const void* kv_b_proj;
  int32_t heads, nope, v_dim, rank;
  void* k_nope;
  int64_t k_row_stride, k_head_stride;
  void* v;
  int64_t v_row_stride, v_head_stride;
  int32_t* status;
};
cudaError_t launch_tc_reconstruct(const ReconstructParams& p, cudaStream_t stream);

// Causal prefill attention over materialised per-head keys / values.
struct PrefillParams {
  const void* q_nope;
  int64_t qn_row_stride, qn_head_stride;
  const void* q_rope;
  int64_t qr_row_stride, qr_head_stride;
  const void* k_nope;
  int64_t k_row_stride, k_head_stride;
  const void* v;
  int64_t v_row_stride, v_head_stride;
  const void* rope;
  int64_t rope_row_stride;
  const int32_t* kv_start;
  const int32_t* kv_len;
  int64_t t_max;
  int32_t packed;
  int32_t batch, s_q, heads, nope, rope_dim, v_dim;
  float softmax_scale;
  void* out;
  int64_t out_row_stride;
  int32_t out_dtype;
  float* lse;
  int32_t* status;
};
cudaError_t launch_tc_prefill(const PrefillParams& p, cudaStream_t stream);

// Failure-detection self-test (a bounded wait on a barrier that never completes).
cudaError_t launch_bounded_wait(long long limit_cycles, int32_t* status, long long* waited, cudaStream_t stream);

// Number of SMs of the current device (cached per device).
int device_sm_count();

}  // namespace mla
