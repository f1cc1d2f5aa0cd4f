// C ABI of the 8-bit cache, of attention weights and of eviction: host-side
// validation, planning and dispatch.  Nothing here allocates device memory or
// synchronises.
#include <cmath>

#include "cache_attn.cuh"

namespace {

bool aligned(const void* p, unsigned a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }
bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
int log2i(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

bool is_q8(int dtype) { return dtype == PKV_I8 || dtype == PKV_E4M3; }
bool good_page(int page_size) { return pow2(page_size) && page_size >= 16 && page_size <= 256; }
bool good_block(int block, int page_size) { return pow2(block) && block >= 16 && block <= page_size; }

// Workspace of attention over the cache, one after the other and 256-byte aligned:
// partial outputs, (max, sum) pairs, scores, row sums.
struct Workspace {
  size_t o = 0, ml = 0, logits = 0, lse = 0;
  size_t total() const { return up256(o) + up256(ml) + up256(logits) + up256(lse); }
};

// Rows of the log2-sums a (sequence, head) has: whole tiles of the weights kernel.
size_t lse_rows(int q_len) { return ((size_t)q_len + 127) / 128 * 128; }

// Whether a call's query rows go through the split kernel as so many heads (each
// 16 rows of a kv head read its keys again, but the keys are split over CTAs) or
// through the prefill kernel (whose tile of 128 rows of one head costs the same
// however few are filled, and which walks all keys in one CTA).  Per 128 keys and
// kv head the first takes about 2400 cycles of an SM for each 16 rows, the second
// about 3000 for each head: even at some 16 rows a head, and at more where the
// prefill's CTAs do not fill the 148 SMs.
bool few_rows(int num_seqs, int q_len, int H, int H_kv, int max_seq_len, bool weights) {
  if (q_len == 1) return true;
  if ((long long)(H / H_kv) * q_len > 256 || (long long)H * q_len > 65535) return false;
  // the scores of every row go through memory
  if (weights && (long long)num_seqs * H * q_len * max_seq_len > (1LL << 27)) return false;
  return q_len <= 16 || ((long long)q_len * num_seqs * H <= 16LL * 148 && max_seq_len >= 2048);
}

Workspace attn_workspace(int num_seqs, int q_len, int H, int H_kv, int max_seq_len, int page_size, bool weights) {
  Workspace w;
  if (few_rows(num_seqs, q_len, H, H_kv, max_seq_len, weights)) {
    const int rows = H * q_len;
    int split = 0, nsplit = 0;
    pkv::cache_decode_plan(num_seqs, rows, H_kv, max_seq_len, page_size, &split, &nsplit);
    const size_t per = (size_t)num_seqs * rows * nsplit;
    if (nsplit > 1) w.o = per * 128 * sizeof(float);
    if (nsplit > 1 || weights) w.ml = per * sizeof(float2);
    if (weights) w.logits = (size_t)num_seqs * rows * max_seq_len * sizeof(float);
  } else if (weights) {
    w.lse = (size_t)num_seqs * H * lse_rows(q_len) * sizeof(float);
  }
  return w;
}

bool good_sizes(int num_seqs, int q_len, int H, int H_kv, int max_seq_len, int page_size) {
  return num_seqs >= 1 && q_len >= 1 && H >= 1 && H_kv >= 1 && H % H_kv == 0 && max_seq_len >= q_len &&
         good_page(page_size);
}

int run_attn(const void* q, const void* k_pages, const void* v_pages, const void* k_scales, const void* v_scales,
             const int32_t* block_table, const int32_t* seq_lens, int page_size, int block_tokens, int num_seqs,
             int q_len, int H, int H_kv, int d, int num_pages, int max_pages_per_seq, int max_seq_len, int causal,
             float scale, int cache_dtype, void* out, float* weights, int weights_stride, void* workspace,
             size_t workspace_bytes, void* stream) {
  const bool q8 = is_q8(cache_dtype);
  if (!aligned(q, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return PKV_ERR_INVALID_ARG;
  if (q8 && (!aligned(k_scales, 4) || !aligned(v_scales, 4))) return PKV_ERR_INVALID_ARG;
  if (!good_sizes(num_seqs, q_len, H, H_kv, max_seq_len, page_size) || num_pages < 1 || max_pages_per_seq < 1 ||
      (causal != 0 && causal != 1) || !std::isfinite(scale) || scale <= 0.f)
    return PKV_ERR_INVALID_ARG;
  if (q8 && !good_block(block_tokens, page_size)) return PKV_ERR_INVALID_ARG;
  if ((long long)max_pages_per_seq * page_size < max_seq_len) return PKV_ERR_INVALID_ARG;
  if (weights && weights_stride < max_seq_len) return PKV_ERR_INVALID_ARG;
  if (d != 128 || num_seqs > 65535 || H > 65535 || (long long)num_pages * page_size > (1LL << 31))
    return PKV_ERR_UNSUPPORTED;
  if (weights && H / H_kv > 256) return PKV_ERR_UNSUPPORTED;
  // a grid's second axis: 128-key tiles of the prompt's weights
  if (weights && !few_rows(num_seqs, q_len, H, H_kv, max_seq_len, true) && max_seq_len > 65535 * 128)
    return PKV_ERR_UNSUPPORTED;
  const Workspace w = attn_workspace(num_seqs, q_len, H, H_kv, max_seq_len, page_size, weights != nullptr);
  if (w.total() > 0 && (!aligned(workspace, 256) || workspace_bytes < w.total())) return PKV_ERR_WORKSPACE;
  if (weights && !few_rows(num_seqs, q_len, H, H_kv, max_seq_len, true)) {    // q is read again once out is written
    const uintptr_t a = reinterpret_cast<uintptr_t>(q), b = reinterpret_cast<uintptr_t>(out);
    const uintptr_t bytes = (uintptr_t)num_seqs * H * q_len * d * sizeof(__nv_bfloat16);
    if (a < b + bytes && b < a + bytes) return PKV_ERR_INVALID_ARG;
  }

  pkv::CacheAttnParams p{};
  if (int r = pkv::device_error_word(&p.err)) return r;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_pages = k_pages, p.v_pages = v_pages;
  if (q8) p.k_scales = static_cast<const float*>(k_scales), p.v_scales = static_cast<const float*>(v_scales);
  p.block_table = block_table, p.seq_lens = seq_lens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.weights = weights, p.weights_stride = weights_stride;
  char* ws = static_cast<char*>(workspace);
  auto take = [&](size_t n) -> void* {
    if (!n) return nullptr;
    void* at = ws;
    ws += up256(n);
    return at;
  };
  p.ws_o = static_cast<float*>(take(w.o));
  p.ws_ml = static_cast<float2*>(take(w.ml));
  p.logits = static_cast<float*>(take(w.logits));
  p.neg_lse = static_cast<float*>(take(w.lse));
  p.num_seqs = num_seqs, p.q_len = q_len, p.H = H, p.H_kv = H_kv;
  p.page_size = page_size, p.page_shift = log2i(page_size), p.block_shift = q8 ? log2i(block_tokens) : 0;
  p.num_pages = num_pages, p.max_pages = max_pages_per_seq, p.max_seq_len = max_seq_len;
  p.logit_tokens = max_seq_len;
  p.cache_dtype = cache_dtype, p.causal = causal;
  p.scale_log2 = scale * pkv::kLog2e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few_rows(num_seqs, q_len, H, H_kv, max_seq_len, weights != nullptr)) {
    p.H = H * q_len;
    pkv::cache_decode_plan(num_seqs, p.H, H_kv, max_seq_len, page_size, &p.split_tokens, &p.max_splits);
    return pkv::cuda_status(pkv::launch_cache_decode(p, st));
  }
  pkv::PrefillParams f{};
  f.Q = q, f.K = k_pages, f.V = v_pages, f.O = out;
  f.block_table = block_table, f.seq_lens = seq_lens;
  f.err = p.err;
  f.B = num_seqs, f.H = H, f.H_kv = H_kv, f.q_len = q_len, f.d = d;
  f.paged = 1, f.page_size = page_size, f.page_shift = p.page_shift;
  f.num_pages = num_pages, f.max_pages = max_pages_per_seq, f.max_seq_len = max_seq_len;
  f.causal = causal, f.scale_log2 = p.scale_log2;
  if (q8) f.cache_dtype = cache_dtype, f.block_shift = p.block_shift, f.k_scales = p.k_scales, f.v_scales = p.v_scales;
  p.lse_stride = (int)lse_rows(q_len);
  f.neg_lse = p.neg_lse, f.lse_stride = p.lse_stride;
  const cudaError_t e = pkv::launch_prefill_bf16(f, st);
  if (e != cudaSuccess || !weights) return pkv::cuda_status(e);
  return pkv::cuda_status(pkv::launch_prompt_weights(p, st));
}

}  // namespace

extern "C" {

int paged_kv_append_q8(const void* k_new, const void* v_new, const int32_t* cu_new, const int32_t* start_pos,
                       const int32_t* block_table, int max_pages_per_seq, int num_seqs, int num_new, void* k_pages,
                       void* v_pages, void* k_scales, void* v_scales, int num_pages, int page_size,
                       int block_tokens, int H_kv, int d, int dtype, int cache_dtype, void* stream) {
  if (num_new < 0 || num_seqs < 1 || max_pages_per_seq < 1 || num_pages < 1 || H_kv < 1 || !good_page(page_size) ||
      !good_block(block_tokens, page_size) || (dtype != PKV_BF16 && dtype != PKV_F32) || !is_q8(cache_dtype))
    return PKV_ERR_INVALID_ARG;
  if (d != 128) return PKV_ERR_UNSUPPORTED;
  if (num_new == 0) return PKV_OK;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(k_scales, 4) || !aligned(v_scales, 4) || !aligned(cu_new, 4) || !aligned(start_pos, 4) ||
      !aligned(block_table, 4))
    return PKV_ERR_INVALID_ARG;
  if ((long long)num_pages * page_size > (1LL << 31)) return PKV_ERR_UNSUPPORTED;
  pkv::AppendQ8Params p{};
  if (int r = pkv::device_error_word(&p.err)) return r;
  p.k_new = k_new, p.v_new = v_new, p.cu_new = cu_new, p.start_pos = start_pos, p.block_table = block_table;
  p.k_pages = k_pages, p.v_pages = v_pages;
  p.k_scales = static_cast<float*>(k_scales), p.v_scales = static_cast<float*>(v_scales);
  p.num_seqs = num_seqs, p.num_new = num_new, p.max_pages = max_pages_per_seq, p.num_pages = num_pages;
  p.page_size = page_size, p.page_shift = log2i(page_size), p.block_shift = log2i(block_tokens), p.H_kv = H_kv;
  p.cache_dtype = cache_dtype, p.rows_f32 = dtype == PKV_F32;
  return pkv::cuda_status(pkv::launch_append_q8(p, static_cast<cudaStream_t>(stream)));
}

int paged_kv_copy_pages_q8(void* k_pages, void* v_pages, void* k_scales, void* v_scales, const int32_t* src,
                           const int32_t* dst, int n, int num_pages, int page_size, int block_tokens, int H_kv,
                           int d, int cache_dtype, void* stream) {
  if (n < 0 || num_pages < 1 || H_kv < 1 || !good_page(page_size) || !good_block(block_tokens, page_size) ||
      !is_q8(cache_dtype))
    return PKV_ERR_INVALID_ARG;
  if (d != 128) return PKV_ERR_UNSUPPORTED;
  if (n == 0) return PKV_OK;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_scales, 4) || !aligned(v_scales, 4) ||
      !aligned(src, 4) || !aligned(dst, 4))
    return PKV_ERR_INVALID_ARG;
  if ((long long)num_pages * page_size > (1LL << 31)) return PKV_ERR_UNSUPPORTED;
  pkv::CopyPagesQ8Params p{};
  if (int r = pkv::device_error_word(&p.err)) return r;
  p.k_pages = static_cast<uint8_t*>(k_pages), p.v_pages = static_cast<uint8_t*>(v_pages);
  p.k_scales = static_cast<float*>(k_scales), p.v_scales = static_cast<float*>(v_scales);
  p.src = src, p.dst = dst, p.n = n, p.num_pages = num_pages;
  p.page_bytes = (size_t)page_size * H_kv * d;
  p.page_scales = page_size / block_tokens * H_kv;
  return pkv::cuda_status(pkv::launch_copy_pages_q8(p, static_cast<cudaStream_t>(stream)));
}

size_t paged_attn_q8_workspace_size(int num_seqs, int q_len, int H, int H_kv, int max_seq_len, int page_size) {
  if (!good_sizes(num_seqs, q_len, H, H_kv, max_seq_len, page_size)) return 0;
  return attn_workspace(num_seqs, q_len, H, H_kv, max_seq_len, page_size, false).total();
}

int paged_attn_q8(const void* q, const void* k_pages, const void* v_pages, const void* k_scales,
                  const void* v_scales, const int32_t* block_table, const int32_t* seq_lens, int page_size,
                  int block_tokens, int num_seqs, int q_len, int H, int H_kv, int d, int num_pages,
                  int max_pages_per_seq, int max_seq_len, int causal, float scale, int cache_dtype, void* out,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!is_q8(cache_dtype)) return PKV_ERR_INVALID_ARG;
  return run_attn(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, page_size, block_tokens, num_seqs,
                  q_len, H, H_kv, d, num_pages, max_pages_per_seq, max_seq_len, causal, scale, cache_dtype, out,
                  nullptr, 0, workspace, workspace_bytes, stream);
}

size_t paged_attn_weights_workspace_size(int num_seqs, int q_len, int H, int H_kv, int max_seq_len, int page_size) {
  if (!good_sizes(num_seqs, q_len, H, H_kv, max_seq_len, page_size)) return 0;
  return attn_workspace(num_seqs, q_len, H, H_kv, max_seq_len, page_size, true).total();
}

int paged_attn_weights(const void* q, const void* k_pages, const void* v_pages, const void* k_scales,
                       const void* v_scales, const int32_t* block_table, const int32_t* seq_lens, int page_size,
                       int block_tokens, int num_seqs, int q_len, int H, int H_kv, int d, int num_pages,
                       int max_pages_per_seq, int max_seq_len, int causal, float scale, int cache_dtype, void* out,
                       void* weights, int weights_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (!is_q8(cache_dtype) && cache_dtype != PKV_BF16)
    return cache_dtype == PKV_F32 ? PKV_ERR_UNSUPPORTED : PKV_ERR_INVALID_ARG;
  if (!aligned(weights, 4)) return PKV_ERR_INVALID_ARG;
  return run_attn(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, page_size, block_tokens, num_seqs,
                  q_len, H, H_kv, d, num_pages, max_pages_per_seq, max_seq_len, causal, scale, cache_dtype, out,
                  static_cast<float*>(weights), weights_stride, workspace, workspace_bytes, stream);
}

size_t paged_kv_evict_workspace_size(int num_seqs, int H_kv, int budget, int block_tokens, int cache_dtype) {
  if (num_seqs < 1 || H_kv < 1 || budget < 1 || !is_q8(cache_dtype) || !good_block(block_tokens, 256)) return 0;
  const size_t pairs = (size_t)num_seqs * H_kv;
  const size_t blocks = ((size_t)budget + block_tokens - 1) / block_tokens;
  return up256(pairs * budget * sizeof(float2)) + up256(pairs * blocks * sizeof(float2));
}

int paged_kv_evict(void* k_pages, void* v_pages, void* k_scales, void* v_scales, const void* weights,
                   void* weights_out, int weights_stride, const int32_t* block_table, const int32_t* dst_table,
                   const int32_t* seq_lens, int32_t* new_lens, int32_t* kept, int budget, int recent, int num_seqs,
                   int H_kv, int d, int num_pages, int page_size, int block_tokens, int max_pages_per_seq,
                   int max_seq_len, int cache_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const bool q8 = is_q8(cache_dtype);
  if (!q8 && cache_dtype != PKV_BF16 && cache_dtype != PKV_F32) return PKV_ERR_INVALID_ARG;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(weights, 4) || !aligned(weights_out, 4) ||
      !aligned(block_table, 4) || !aligned(dst_table, 4) || !aligned(seq_lens, 4) || !aligned(new_lens, 4) ||
      !aligned(kept, 4) || new_lens == seq_lens)
    return PKV_ERR_INVALID_ARG;
  if (q8 && (!aligned(k_scales, 4) || !aligned(v_scales, 4) || !good_block(block_tokens, page_size)))
    return PKV_ERR_INVALID_ARG;
  if (budget < 1 || recent < 0 || recent > budget || num_seqs < 1 || H_kv < 1 || num_pages < 1 ||
      !good_page(page_size) || max_pages_per_seq < 1 || max_seq_len < 1 || weights_stride < max_seq_len ||
      (long long)max_pages_per_seq * page_size < max_seq_len)
    return PKV_ERR_INVALID_ARG;
  if (q8 ? d != 128 : (d != 64 && d != 128)) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || H_kv > 65535 || budget > (1 << 30) || (long long)num_pages * page_size > (1LL << 31))
    return PKV_ERR_UNSUPPORTED;
  const size_t need = paged_kv_evict_workspace_size(num_seqs, H_kv, budget, block_tokens, cache_dtype);
  if (need > 0 && (!aligned(workspace, 256) || workspace_bytes < need)) return PKV_ERR_WORKSPACE;
  pkv::EvictParams p{};
  if (int r = pkv::device_error_word(&p.err)) return r;
  p.k_pages = k_pages, p.v_pages = v_pages;
  if (q8) {
    p.k_scales = static_cast<float*>(k_scales), p.v_scales = static_cast<float*>(v_scales);
    p.block_shift = log2i(block_tokens);
    p.max_blocks = (int)(((long long)budget + block_tokens - 1) / block_tokens);
    p.row_scale = static_cast<float2*>(workspace);
    p.block_scale = reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                              up256((size_t)num_seqs * H_kv * budget * sizeof(float2)));
  }
  p.weights = static_cast<const float*>(weights), p.weights_out = static_cast<float*>(weights_out);
  p.weights_stride = weights_stride;
  p.block_table = block_table, p.dst_table = dst_table, p.seq_lens = seq_lens, p.new_lens = new_lens, p.kept = kept;
  p.num_seqs = num_seqs, p.H_kv = H_kv, p.num_pages = num_pages;
  p.page_size = page_size, p.page_shift = log2i(page_size);
  p.max_pages = max_pages_per_seq, p.max_seq_len = max_seq_len;
  p.budget = budget, p.recent = recent;
  p.row_bytes = d * (q8 ? 1 : cache_dtype == PKV_BF16 ? 2 : 4);
  p.cache_dtype = cache_dtype;
  return pkv::cuda_status(pkv::launch_evict(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
