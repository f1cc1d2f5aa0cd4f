// Parameters of the 8-bit cache, attention-weight and eviction kernels (not part of the C ABI).
#pragma once

#include "common.cuh"

namespace pkv {

struct AppendQ8Params {
  const void* k_new;           // [num_new, H_kv, d], bf16 or f32
  const void* v_new;
  const int32_t* cu_new;       // [num_seqs + 1]
  const int32_t* start_pos;    // [num_seqs]
  const int32_t* block_table;  // [num_seqs, max_pages]
  void* k_pages;               // [P, ps, H_kv, d] codes
  void* v_pages;
  float* k_scales;             // [P, ps / block, H_kv]
  float* v_scales;
  unsigned int* err;
  int num_seqs, num_new, max_pages, num_pages, page_size, page_shift, block_shift, H_kv;
  int cache_dtype, rows_f32;
};

struct CopyPagesQ8Params {
  uint8_t* k_pages;
  uint8_t* v_pages;
  float* k_scales;
  float* v_scales;
  const int32_t* src;
  const int32_t* dst;
  unsigned int* err;
  int n, num_pages;
  size_t page_bytes;           // codes of a page
  int page_scales;             // scales of a page
};

struct CacheAttnParams {
  const __nv_bfloat16* q;      // [S, H, q_len, d]
  const void* k_pages;         // [P, ps, H_kv, d]
  const void* v_pages;
  const float* k_scales;       // [P, ps / block, H_kv]; null for a bf16 cache
  const float* v_scales;
  const int32_t* block_table;  // [S, max_pages]
  const int32_t* seq_lens;     // [S]
  __nv_bfloat16* out;          // [S, H, q_len, d]
  float* weights;              // [S, H_kv, weights_stride] or null
  float* ws_o;                 // [S, H, max_splits, d]
  float2* ws_ml;               // [S, H, max_splits]: max in log2 units, sum
  float* logits;               // [S, H_kv, logit_tokens, H / H_kv]: scores in log2 units
  float* neg_lse;              // [S, H, lse_stride]: minus log2 of each row's sum, -infinity past q_len
  unsigned int* err;
  int num_seqs, q_len, H, H_kv, page_size, page_shift, block_shift, num_pages, max_pages, max_seq_len;
  int split_tokens, max_splits, weights_stride, logit_tokens, lse_stride;
  int merge_ctas, merge_warps, token_lanes, range_tokens;   // set by the launcher
  int cache_dtype, causal;
  float scale_log2;            // scale * log2(e)
};

struct EvictParams {
  void* k_pages;               // [P, ps, H_kv, d]
  void* v_pages;
  float* k_scales;             // [P, ps / block, H_kv]; null for a bf16 or f32 cache
  float* v_scales;
  const float* weights;        // [S, H_kv, weights_stride]
  float* weights_out;
  const int32_t* block_table;  // [S, max_pages]
  const int32_t* dst_table;
  const int32_t* seq_lens;     // [S]
  int32_t* new_lens;
  int32_t* kept;               // [S, H_kv, budget]
  float2* row_scale;           // [S, H_kv, budget]: old (k, v) scale of every kept row
  float2* block_scale;         // [S, H_kv, max_blocks]: new (k, v) scale of every block
  unsigned int* err;
  int num_seqs, H_kv, num_pages, page_size, page_shift, block_shift, max_pages, max_seq_len;
  int budget, recent, weights_stride, row_bytes, slice_bytes, max_blocks, cache_dtype;   // slice_bytes: set by the launcher
};

// Split plan of single-token attention: tokens a split, splits of the longest sequence.
void cache_decode_plan(int num_seqs, int H, int H_kv, int max_seq_len, int page_size, int* split_tokens,
                       int* max_splits);

cudaError_t launch_append_q8(const AppendQ8Params& p, cudaStream_t stream);
cudaError_t launch_copy_pages_q8(const CopyPagesQ8Params& p, cudaStream_t stream);
cudaError_t launch_cache_decode(const CacheAttnParams& p, cudaStream_t stream);
cudaError_t launch_prompt_weights(const CacheAttnParams& p, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);

}  // namespace pkv
