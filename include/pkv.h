/*
 * pkv.h - exact attention over contiguous and paged K/V on B200 (sm_100a).
 *
 * A small C ABI: plain pointers and sizes, no C++ or framework types.
 *
 * What is computed, for every (batch or sequence, query head, query row):
 *
 *     O = softmax(Q K^T * scale) V
 *
 * exactly as defined in "Flash Attention: Fast, Memory-Efficient Attention for
 * LLMs", section "Standard Attention: The Memory Problem" (S = QK^T,
 * P = softmax(S), O = PV), but computed the way its section "The Algorithm"
 * describes: K/V are streamed in tiles, a running row maximum and running row
 * sum rescale an on-chip output accumulator, and S and P never reach global
 * memory.  Paged K/V are read in place through each sequence's block table
 * ("What is Paged FlashAttention?", sections "How does it work?" and
 * "Practical example"): token t of sequence s lives in physical page
 * block_table[s][t / page_size] at offset t % page_size, with no gather into a
 * contiguous copy first.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Pointers named as device pointers must point to memory of the current CUDA
 *   device; the caller owns all memory.  Q/K/V/O, pages, tables and the
 *   workspace must be 16-byte aligned.  The library allocates nothing, frees
 *   nothing and never synchronises: all work is enqueued on `stream`
 *   (a cudaStream_t; NULL = the legacy default stream).
 * - Every function returns a pkv_status.  Argument errors are found on the
 *   host, before anything is launched, and nothing is launched then.  Launch
 *   failures return PKV_ERR_CUDA.  Errors that only the device can see
 *   (a page id outside [0, num_pages), a sequence length outside its table,
 *   a pipeline wait that ran out) never fault: the kernel skips the access,
 *   records a bit in a library-wide device error word and carries on;
 *   pkv_last_device_error() reads and clears it.  A page outside the pool is
 *   never read and its keys are left out of the softmax (decode and prefill
 *   alike), so that sequence gets attention over its other keys; a length
 *   outside its table is clamped into range.
 * - Masking: query row i (0-based, of q_len rows) may see key j (of kv_len keys)
 *   iff j <= i + (kv_len - q_len) when causal, every j < kv_len otherwise.
 *   With q_len == kv_len that is the lower triangle; with q_len == 1 (decode)
 *   every key is visible.
 * - Element types: PKV_BF16 (bfloat16 in and out, float32 accumulation, P
 *   rounded to bf16 before the PV product on the tensor-core path) and
 *   PKV_F32 (float32 in and out, float32 FMA throughout).
 * - Head dimension d: 128 for PKV_BF16; 64 or 128 for PKV_F32.
 * - Device reset: the library looks up, once per device, the device addresses
 *   of its own static arrays (the device error word; the scratch of
 *   paged_decode_noalloc) and keeps them for the life of the process.  A
 *   cudaDeviceReset, or anything else that destroys and re-creates a device's
 *   primary context, leaves those addresses stale: do not call the library on
 *   a device after resetting it in the same process.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,   /* a pointer, size, alignment or value is invalid */
  PKV_ERR_UNSUPPORTED = 2,   /* valid, but this build has no kernel for it (e.g. d = 96) */
  PKV_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
  PKV_ERR_TIMEOUT = 4,       /* device: a pipeline wait gave up (pkv_last_device_error) */
  PKV_ERR_BAD_TABLE = 5,     /* device: a page id or sequence length was out of range */
  PKV_ERR_WORKSPACE = 6,     /* workspace missing or smaller than paged_attn_workspace_size() */
  PKV_ERR_OUT_OF_PAGES = 7   /* allocator: not enough free pages (nothing was changed) */
} pkv_status;

typedef enum { PKV_F32 = 0, PKV_BF16 = 1, PKV_I8 = 2, PKV_E4M3 = 3 } pkv_dtype;

/* Device error bits, as returned in *bits by pkv_last_device_error(). */
#define PKV_DEVERR_BAD_PAGE 0x1u   /* block_table entry outside [0, num_pages): its keys left out */
#define PKV_DEVERR_BAD_LEN 0x2u    /* seq_len outside [q_len, min(max_seq_len, pages*page_size)] */
#define PKV_DEVERR_TIMEOUT 0x4u    /* a bounded mbarrier wait ran out; the tile was abandoned */

/*
 * attn_prefill - attention over contiguous Q, K, V.
 *
 * Defines: "Flash Attention: Fast, Memory-Efficient Attention for LLMs",
 * sections "Standard Attention" (the operation) and "The Algorithm" (tiling
 * with online softmax; causal tiles past the diagonal are skipped, as its
 * "Flash Attention 2" section describes).
 *
 * Q, K, V, O : device pointers, [B, H, N, d] row-major (d contiguous), element
 *              type `dtype`.  O is written, nothing else is.
 * B, H, N, d : batch, heads, sequence length (queries = keys = N), head dim.
 *              B, H, N >= 1.
 * causal     : 0 or 1 (lower-triangular mask).
 * scale      : multiplier of QK^T, usually 1/sqrt(d); must be finite and > 0.
 * dtype      : PKV_BF16 (tcgen05 tensor-core kernel) or PKV_F32 (FMA kernel).
 * stream     : cudaStream_t the work is enqueued on.
 */
PKV_API int attn_prefill(const void* Q, const void* K, const void* V, void* O,
                 int B, int H, int N, int d, int causal, float scale,
                 int dtype, void* stream);

/*
 * pkv_test_prefill_stalled - test hook for the failure path; not for use in
 * production.
 *
 * The pages have no counterpart: it exists so that tests can make the bf16
 * prefill's bounded pipeline waits run out without faulting or hanging a GPU.
 * It runs what attn_prefill runs for dtype PKV_BF16 (same arguments, same
 * checks), except that every pipeline wait gives up after wait_limit_us
 * microseconds and the loader of each CTA's first work item never issues the
 * K load of K/V tile `stall_tile` (0-based).  Every CTA whose first item has
 * more than stall_tile K/V tiles then records PKV_DEVERR_TIMEOUT, stops,
 * drains the loads and MMAs it issued, frees its tensor memory and exits;
 * the output is undefined.  pkv_last_device_error() then returns
 * PKV_ERR_TIMEOUT, and later calls run normally.
 *
 * stall_tile    : >= 0.
 * wait_limit_us : in [1, 10^7].
 */
PKV_API int pkv_test_prefill_stalled(const void* Q, const void* K, const void* V, void* O,
                                     int B, int H, int N, int d, int causal, float scale,
                                     int stall_tile, int wait_limit_us, void* stream);

/*
 * attn_prefill_fp8qk - attention with e4m3 (FP8) Q and K, bf16 V and output.
 *
 * Defines: "Flash Attention: Fast, Memory-Efficient Attention for LLMs",
 * section "Flash Attention 3" (FP8 tensor cores for the QK^T product).  What
 * is computed, exactly as attn_prefill does it otherwise:
 *
 *     O = softmax((q_descale * Q8) (k_descale * K8)^T * scale) V
 *
 * where Q8, K8 hold e4m3 codes (1 sign, 4 exponent bits with bias 7, 3
 * mantissa bits; no infinities) and the descales are the per-tensor factors
 * the caller quantized with.  S = Q K^T runs on tcgen05 kind::f8f6f4; P and V
 * stay bf16 for the PV product.
 *
 * Q8, K8 : device, [B, H, N, d] e4m3 bytes.   V, O : device, [B, H, N, d] bf16.
 * d      : 128.  scale, q_descale, k_descale: finite and > 0.
 */
PKV_API int attn_prefill_fp8qk(const void* Q8, const void* K8, const void* V, void* O,
                               int B, int H, int N, int d, int causal, float scale,
                               float q_descale, float k_descale, void* stream);

/*
 * paged_attn_workspace_size - bytes of scratch paged_attn needs.
 *
 * Decode (q_len == 1) splits each sequence's keys into fixed-size chunks that
 * run in parallel and are merged with a log-sum-exp combine; the partial
 * (O, max, sum) of every chunk lives in this workspace.  The size depends only
 * on these arguments (same arguments, same plan).  Returns 0 when one chunk
 * per sequence suffices (no workspace needed), and 0 for invalid arguments.
 */
PKV_API size_t paged_attn_workspace_size(int num_seqs, int H, int d, int max_seq_len, int page_size);

/*
 * paged_attn - attention of new query tokens against a paged K/V cache.
 *
 * Defines: "What is Paged FlashAttention?", sections "How does it work?"
 * (locate pages through the block table, load K/V tiles, online softmax,
 * accumulate without a full-cache gather) and "Practical example" (logical
 * page t / page_size, offset t % page_size, physical page
 * block_table[logical]).  Pages follow "FlashAttention and PagedAttention:
 * Two Fixes for Two Different Bottlenecks", section "PagedAttention ... How
 * it works": fixed-size blocks, a per-sequence block table, blocks may be
 * shared by several sequences (pages are only read here).
 *
 * q           : device, [num_seqs, H, q_len, d]; the q_len newest tokens of each
 *               sequence (their K/V are already in the cache).
 * k_pages,
 * v_pages     : device, [num_pages, page_size, H_kv, d].
 * block_table : device int32, [num_seqs, max_pages_per_seq]; entries past
 *               ceil(seq_lens[s] / page_size) are never read (pad with -1).
 * seq_lens    : device int32, [num_seqs]; kv length of each sequence, the q_len
 *               new tokens included.  Must satisfy
 *               q_len <= seq_lens[s] <= min(max_seq_len, max_pages_per_seq * page_size).
 * page_size   : tokens per page, a power of two in [16, 256].
 * q_len       : 1 = decode (split-K kernel); > 1 = paged prefill (tensor-core
 *               kernel for PKV_BF16, FMA kernel for PKV_F32).
 * H, H_kv     : query heads and kv heads; H % H_kv == 0 (query head h reads
 *               kv head h / (H / H_kv)).
 * num_pages   : pages in the pool (page ids must be < num_pages).
 * max_seq_len : host-known upper bound of seq_lens (plans the split-K grid).
 * out         : device, [num_seqs, H, q_len, d], element type `dtype`.
 * workspace   : device scratch of >= paged_attn_workspace_size(num_seqs, H, d,
 *               max_seq_len, page_size) bytes, 256-byte aligned (NULL if that
 *               size is 0).  Its contents need no initialisation and are
 *               garbage afterwards.  Two calls in flight at once need two
 *               workspaces.
 *
 * Launches (all on `stream`): q_len == 1 enqueues the split kernel and, when
 * some sequence spans more than one split, a merge kernel after it.  With
 * H > H_kv the merge is a programmatic dependent launch: it may be scheduled
 * while the split kernel drains, and it waits on the device for that kernel's
 * results, so stream order is kept (also under stream capture).
 */
PKV_API int paged_attn(const void* q, const void* k_pages, const void* v_pages,
               const int32_t* block_table, const int32_t* seq_lens,
               int page_size, int num_seqs, int q_len, int H, int H_kv, int d,
               int num_pages, int max_pages_per_seq, int max_seq_len,
               int causal, float scale, int dtype,
               void* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * paged_decode_noalloc - paged decode that allocates nothing and needs no
 * workspace argument.
 *
 * The pages have no counterpart for this entry point; it exists for callers
 * that cannot allocate device memory where they call attention: a plugin
 * invoked from another runtime's enqueue hook that offers no allocator, a
 * latency-critical loop in which cudaMalloc/cudaFree would synchronise the
 * device, or a process whose device memory a pool has reserved in full.
 *
 * It computes what paged_attn computes for q_len == 1 and PKV_BF16 (decode:
 * every cached key is visible), with the same kernels and split plan, and the
 * same meaning, layout and validation of the arguments paged_attn shares with
 * it (d must be 128).  The split partials live in a static device array of
 * PKV_NOALLOC_SCRATCH_BYTES inside the library: every GPU that loads the
 * library holds that memory until the process exits.
 *
 * - Limit: when paged_attn_workspace_size(num_seqs, H, d, max_seq_len,
 *   page_size) exceeds PKV_NOALLOC_SCRATCH_BYTES the call returns
 *   PKV_ERR_WORKSPACE and launches nothing.
 * - Set-up: the first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current) and caches it for the
 *   life of the process (so not across a device reset, see above); make that
 *   first call before any stream capture.
 * - Sharing: all calls on a device use the same array, which keeps the last
 *   call's contents.  No part of it needs to start at zero (a call writes every
 *   partial it reads), but calls whose kernels overlap on the GPU (other
 *   streams, other host threads) race on it: serialise them.
 */
#define PKV_NOALLOC_SCRATCH_BYTES (64u << 20)
PKV_API int paged_decode_noalloc(const void* q, const void* k_pages, const void* v_pages,
                                 const int32_t* block_table, const int32_t* seq_lens,
                                 int page_size, int num_seqs, int H, int H_kv, int d,
                                 int num_pages, int max_pages_per_seq, int max_seq_len,
                                 float scale, void* out, void* stream);

/* ------------------------------------------------------------------------ */
/* The write side of the paged cache.                                       */
/* ------------------------------------------------------------------------ */

/*
 * paged_kv_append - write new tokens' K and V rows into their pages.
 *
 * Defines: "Flash Attention: Fast, Memory-Efficient Attention for LLMs",
 * section "KV Cache" (each decode step appends the new K_t, V_t; prefill
 * stores the K/V of every prompt token), with the address of token position
 * pos of sequence s given by "What is Paged FlashAttention?", "Practical
 * example": page block_table[s][pos / page_size], offset pos % page_size.
 *
 * k_new, v_new : device, [num_new, H_kv, d]: rows of all sequences' new tokens,
 *                sequence by sequence.
 * cu_new       : device int32 [num_seqs + 1], non-decreasing, cu_new[0] = 0,
 *                cu_new[num_seqs] = num_new: sequence s owns rows
 *                [cu_new[s], cu_new[s+1]).
 * start_pos    : device int32 [num_seqs]: position of sequence s's first new
 *                token (its length before the append).
 * block_table  : device int32 [num_seqs, max_pages_per_seq]; the pages covering
 *                the new positions must already be allocated (pkv_alloc_reserve).
 * k_pages,
 * v_pages      : device, [num_pages, page_size, H_kv, d], written in place.
 * dtype        : PKV_BF16 or PKV_F32; d is 64 or 128.
 * A row whose page id is outside [0, num_pages) or whose position is past the
 * table is skipped and flagged (PKV_DEVERR_BAD_PAGE / PKV_DEVERR_BAD_LEN).
 * Rows must not target the same slot twice in one call.
 * Returns PKV_OK without reading any pointer or launching when num_new == 0;
 * PKV_ERR_INVALID_ARG for a negative num_new, num_seqs, max_pages_per_seq,
 * num_pages or H_kv below 1, a page_size that is not a power of two in
 * [16, 256], an unknown dtype, or a null or misaligned pointer (16 bytes for
 * row data, 4 for the int32 arrays); PKV_ERR_UNSUPPORTED for d other than 64
 * or 128, or a pool of more than 2^31 token rows.
 */
PKV_API int paged_kv_append(const void* k_new, const void* v_new, const int32_t* cu_new,
                            const int32_t* start_pos, const int32_t* block_table,
                            int max_pages_per_seq, int num_seqs, int num_new, void* k_pages,
                            void* v_pages, int num_pages, int page_size, int H_kv, int d,
                            int dtype, void* stream);

/*
 * paged_kv_copy_pages - copy whole pages (K and V): page src[i] -> page dst[i].
 *
 * Defines the copy half of copy-on-write ("FlashAttention and PagedAttention:
 * Two Fixes for Two Different Bottlenecks", section "PagedAttention ... How it
 * works": sequences share prefix blocks and copy only when they diverge).
 * src, dst : device int32 [n]; ids in [0, num_pages) (others are skipped and
 *            flagged); a dst must not also be a src in the same call.
 * Returns PKV_OK without reading any pointer or launching when n == 0;
 * PKV_ERR_INVALID_ARG for a negative n, num_pages or H_kv below 1, a page_size
 * that is not a power of two in [16, 256], an unknown dtype, or a null or
 * misaligned pointer (16 bytes for the pools, 4 for src and dst);
 * PKV_ERR_UNSUPPORTED for d other than 64 or 128.
 */
PKV_API int paged_kv_copy_pages(void* k_pages, void* v_pages, const int32_t* src,
                                const int32_t* dst, int n, int num_pages, int page_size,
                                int H_kv, int d, int dtype, void* stream);

/* ------------------------------------------------------------------------ */
/* The 8-bit cache.                                                         */
/* ------------------------------------------------------------------------ */

/*
 * Pages hold codes, k_pages and v_pages [num_pages, page_size, H_kv, d] bytes,
 * and every block of block_tokens tokens of a page has one float32 scale for
 * each kv head, k_scales and v_scales [num_pages, page_size / block_tokens, H_kv]:
 *
 *     K[token t][head h][c] = code[t][h][c] * k_scales[page][offset / block_tokens][h]
 *
 * cache_dtype  : PKV_I8 (two's complement codes -127 .. 127) or PKV_E4M3 (1 sign,
 *                4 exponent bits with bias 7, 3 mantissa bits, largest 448).
 * block_tokens : a power of two in [16, page_size].
 * d            : 128.
 */

/*
 * paged_kv_append_q8 - quantise new tokens' K and V rows into their pages.
 *
 * For each block of a page that the call writes into, and each kv head, K and V
 * apart, with amax the largest magnitude among the call's new rows of the block:
 *
 *     s_new          = max(s_old, amax / qmax, 2^-126)    qmax = 127 or 448
 *     code(new row)  = nearest(x / s_new)
 *     code(old row)  = nearest(code * s_old / s_new)      where s_new > s_old
 *
 * nearest() rounds the exact quotient, ties to even.  s_old is 0 where the call
 * writes the block's first token (a reused page needs no clearing), else the
 * block's scale so far, and its old rows are those before the call's first.  So
 * no value is ever clipped, and codes change only where a scale grows.  A block
 * that takes in a NaN or an infinity gets scale NaN, with codes 0 for the call's
 * rows (older rows keep theirs, which stand for NaN now as well), and stays NaN
 * until its first token is written anew: rows that see the block get NaN from
 * attention over it, others do not.  The weights that a row gives (below) become
 * NaN with a block of K, and do not depend on V.
 *
 * k_new, v_new, cu_new, start_pos, block_table, num_new, num_seqs and the pool's
 * sizes mean what they mean in paged_kv_append.  dtype is the new rows' type,
 * PKV_BF16 or PKV_F32.  Rows of two sequences must not fall into one block in
 * one call.  Rows whose page is outside the pool or past the table are skipped
 * and flagged.  Returns PKV_OK without reading any pointer when num_new == 0.
 */
PKV_API int paged_kv_append_q8(const void* k_new, const void* v_new, const int32_t* cu_new,
                               const int32_t* start_pos, const int32_t* block_table,
                               int max_pages_per_seq, int num_seqs, int num_new, void* k_pages,
                               void* v_pages, void* k_scales, void* v_scales, int num_pages,
                               int page_size, int block_tokens, int H_kv, int d, int dtype,
                               int cache_dtype, void* stream);

/*
 * paged_kv_copy_pages_q8 - copy whole pages (codes and scales, K and V): page
 * src[i] -> page dst[i], as paged_kv_copy_pages does for the other caches.
 */
PKV_API int paged_kv_copy_pages_q8(void* k_pages, void* v_pages, void* k_scales, void* v_scales,
                                   const int32_t* src, const int32_t* dst, int n, int num_pages,
                                   int page_size, int block_tokens, int H_kv, int d,
                                   int cache_dtype, void* stream);

/*
 * paged_attn_q8 - attention of new query tokens against an 8-bit paged cache.
 *
 * What paged_attn computes with K and V the values the codes stand for; q and
 * out are PKV_BF16.  Arguments that both have mean the same (the page table, the
 * lengths, q_len == 1 for decode, causal, the rules for bad pages and lengths).
 * A few query rows (what a verifying step has: q_len up to 16, and more where
 * that leaves most of the GPU idle) run on the split kernel of the single-token
 * case, more of them on the prefill kernel; the choice depends on the sizes alone.
 * Rounding: scores and sums are float32 and out is rounded once; P is rounded for
 * the product with V: by the split kernel to f16, or over a bf16 cache to two bf16
 * parts (off by at most 2^-11 of sum P |V|), by the prefill kernel, with its value
 * scale, to bf16 (2^-8 of it, as in paged_attn).
 * workspace : device scratch of >= paged_attn_q8_workspace_size() bytes, 256-byte
 *             aligned (NULL if that size is 0), one for each call in flight.
 * Codes of live tokens are finite: an e4m3 NaN code (0x7f, 0xff) never comes from
 * paged_kv_append_q8, and what attention makes of one is not defined.
 */
PKV_API size_t paged_attn_q8_workspace_size(int num_seqs, int q_len, int H, int H_kv,
                                            int max_seq_len, int page_size);
PKV_API int paged_attn_q8(const void* q, const void* k_pages, const void* v_pages,
                          const void* k_scales, const void* v_scales, const int32_t* block_table,
                          const int32_t* seq_lens, int page_size, int block_tokens, int num_seqs,
                          int q_len, int H, int H_kv, int d, int num_pages, int max_pages_per_seq,
                          int max_seq_len, int causal, float scale, int cache_dtype, void* out,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Attention weights, and eviction by them.                                 */
/* ------------------------------------------------------------------------ */

/*
 * paged_attn_weights - attention that also accumulates how much weight each
 * key received.
 *
 * out is what paged_attn (cache_dtype PKV_BF16) or paged_attn_q8 (PKV_I8,
 * PKV_E4M3) computes, and for every sequence s, kv head k and visible key j
 *
 *     weights[s][k][j] += sum over the query heads h of k, and the q_len rows i,
 *                         of P[s][h][i][j],   P = softmax(Q K^T * scale)
 *
 * in float32.  Keys of a page outside the pool get nothing, and entries from a
 * sequence's length on are neither read nor written.  The sums have a fixed
 * order: the same call gives the same bits.
 *
 * k_scales, v_scales, block_tokens : as in paged_attn_q8; not looked at when
 *             cache_dtype is PKV_BF16.
 * weights   : device float32 [num_seqs, H_kv, weights_stride], added to.  Two calls
 *             in flight must not share it.
 * weights_stride : >= max_seq_len.
 * workspace : >= paged_attn_weights_workspace_size() bytes, 256-byte aligned.  With a
 *             few rows it holds their scores, 4 num_seqs H q_len max_seq_len bytes:
 *             a batch with one long sequence is better cut into two calls.
 * Where the prefill kernel takes the rows, out must not overlap q (PKV_ERR_INVALID_ARG):
 * q is read again for the weights once out is written.
 * H / H_kv is at most 256, and max_seq_len at most 8388480 where the prefill kernel
 * takes the rows.  A PKV_F32 cache is PKV_ERR_UNSUPPORTED.
 */
PKV_API size_t paged_attn_weights_workspace_size(int num_seqs, int q_len, int H, int H_kv,
                                                 int max_seq_len, int page_size);
PKV_API int paged_attn_weights(const void* q, const void* k_pages, const void* v_pages,
                               const void* k_scales, const void* v_scales,
                               const int32_t* block_table, const int32_t* seq_lens, int page_size,
                               int block_tokens, int num_seqs, int q_len, int H, int H_kv, int d,
                               int num_pages, int max_pages_per_seq, int max_seq_len, int causal,
                               float scale, int cache_dtype, void* out, void* weights,
                               int weights_stride, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * paged_kv_evict - shorten every sequence to `budget` tokens.
 *
 * A sequence of L tokens keeps m = min(L, budget).  Each kv head keeps, of its
 * own, the last min(recent, L) tokens and, of the others, the ones with the
 * largest weights (equal weights: the lowest index; a NaN counts as smaller
 * than any number).  Kept tokens keep their order and become tokens 0 .. m - 1
 * through dst_table.  Heads of one sequence may keep different tokens: what is
 * stored at a token's slot of head h belongs to token kept[s][h][slot].
 *
 * weights     : device float32 [num_seqs, H_kv, weights_stride], as
 *               paged_attn_weights accumulates them.
 * weights_out : the kept tokens' weights go to entries 0 .. m - 1 and zero to
 *               m .. L - 1; the rest is left alone.  May be `weights` itself.
 * block_table : where the tokens are; dst_table: where they go, same shape.  A
 *               page of dst_table is either the one that block_table has at
 *               that place (compaction in place; the two tables may be the same
 *               array) or a page that no sequence of the call reads or writes
 *               otherwise.  A page that several sequences of the call read is
 *               a destination of none (pkv_alloc_compact sees to all this).
 * seq_lens    : lengths before; new_lens: lengths after (another array).
 * kept        : device int32 [num_seqs, H_kv, budget]: the kept tokens' old
 *               indices, ascending, -1 from m on.
 * budget      : in [1, 2^30]; recent: in [0, budget].
 * cache_dtype : PKV_BF16 or PKV_F32 (d 64 or 128; k_scales, v_scales and
 *               block_tokens are not looked at), PKV_I8 or PKV_E4M3 (d 128).
 *               An 8-bit block's new scale is the largest of its rows' scales,
 *               and a row of another scale gets nearest(code * s_old / s_new);
 *               a NaN scale makes the block NaN with codes 0.  Scales are >= 0 or
 *               NaN; a zero scale (rows of zeros) moves like any other.
 * workspace   : >= paged_kv_evict_workspace_size() bytes, 256-byte aligned (NULL
 *               if that size is 0), one for each call in flight.
 * An 8-bit row loses precision each time that it joins a block of a larger
 * scale s_new: at most half a step, s_new / 2 for int8 and the larger of 2^-4 of
 * the value and 2^-10 s_new for e4m3.  A block's scale is inherited, so it does not
 * shrink when the row that set it has gone: one eviction of many tokens costs
 * less than one at every step (int8, 16-token blocks, normal rows, budget 256, one
 * token a step, simulated: a row's mean error 0.8% of its norm at first, 1.3% after
 * 64 steps, 1.5% after 256; rows of very different sizes lose more).
 * A token whose page is outside the pool is not moved, and a length outside its
 * table is clamped; both are flagged.
 */
PKV_API size_t paged_kv_evict_workspace_size(int num_seqs, int H_kv, int budget, int block_tokens,
                                             int cache_dtype);
PKV_API int paged_kv_evict(void* k_pages, void* v_pages, void* k_scales, void* v_scales,
                           const void* weights, void* weights_out, int weights_stride,
                           const int32_t* block_table, const int32_t* dst_table,
                           const int32_t* seq_lens, int32_t* new_lens, int32_t* kept, int budget,
                           int recent, int num_seqs, int H_kv, int d, int num_pages,
                           int page_size, int block_tokens, int max_pages_per_seq,
                           int max_seq_len, int cache_dtype, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * pkv_alloc_* - host page allocator (bookkeeping only; host memory).
 *
 * Defines: "FlashAttention and PagedAttention: Two Fixes for Two Different
 * Bottlenecks", section "PagedAttention ... How it works" (fixed-size blocks,
 * per-sequence block table, allocation on demand, shared prefixes with
 * copy-on-write) and "Flash Attention: Fast, Memory-Efficient Attention for
 * LLMs", section "PagedAttention (vLLM)" (pages of finished sequences are
 * freed and reused).  Policy: the smallest free page id is handed out first;
 * pages carry reference counts; only a shared, partially filled last page is
 * ever copied, just before the sequence writes into it.  Not thread-safe.
 *
 * pkv_alloc_create    : pool of num_pages pages of page_size tokens; tables
 *                       hold at most max_pages_per_seq pages.  NULL on error.
 * pkv_alloc_add_seq   : register an empty sequence under seq_id.
 * pkv_alloc_reserve   : grow seq_id by n_tokens.  *start_pos gets the position
 *                       of its first new token.  If its partially filled last
 *                       page is shared, that page is replaced by a fresh one
 *                       and the copy the caller must run first (with
 *                       paged_kv_copy_pages) is returned in *cow_src ->
 *                       *cow_dst with *n_cow = 1 (else *n_cow = 0).
 *                       PKV_ERR_OUT_OF_PAGES leaves everything unchanged.
 * pkv_alloc_fork      : child_id shares all of parent_id's pages (same length).
 * pkv_alloc_compact   : make the n listed sequences (each once) new_lens[i]
 *                       tokens long (0 <= new_lens[i] <= their length), as
 *                       paged_kv_evict leaves them: of the pages a sequence
 *                       still needs, those that others share are replaced by
 *                       fresh ones, and the pages past them are given up.  The
 *                       tables before the call are paged_kv_evict's block_table,
 *                       those after it its dst_table; pages given up must not be
 *                       written before that call has run (later calls on its
 *                       stream are late enough).  List all sequences of one
 *                       paged_kv_evict call in one call.  PKV_ERR_OUT_OF_PAGES
 *                       leaves everything unchanged.
 * pkv_alloc_free_seq  : drop seq_id; pages nobody else holds return to the pool.
 * pkv_alloc_seq_len   : current length of seq_id.
 * pkv_alloc_block_table: host arrays table [n][max_pages_per_seq] (-1 padded)
 *                       and seq_lens [n] for the n listed sequences.
 * pkv_alloc_num_free  : free pages (-1 for NULL).
 * pkv_alloc_page_refs : reference count of a page (-1 if out of range).
 */
typedef struct pkv_allocator pkv_allocator;
PKV_API pkv_allocator* pkv_alloc_create(int num_pages, int page_size, int max_pages_per_seq);
PKV_API void pkv_alloc_destroy(pkv_allocator* a);
PKV_API int pkv_alloc_add_seq(pkv_allocator* a, int seq_id);
PKV_API int pkv_alloc_reserve(pkv_allocator* a, int seq_id, int n_tokens, int32_t* start_pos,
                              int32_t* cow_src, int32_t* cow_dst, int* n_cow);
PKV_API int pkv_alloc_fork(pkv_allocator* a, int parent_id, int child_id);
PKV_API int pkv_alloc_compact(pkv_allocator* a, const int* seq_ids, int n, const int* new_lens);
PKV_API int pkv_alloc_free_seq(pkv_allocator* a, int seq_id);
PKV_API int pkv_alloc_seq_len(const pkv_allocator* a, int seq_id, int* len);
PKV_API int pkv_alloc_block_table(const pkv_allocator* a, const int* seq_ids, int n,
                                  int32_t* table, int32_t* seq_lens);
PKV_API int pkv_alloc_num_free(const pkv_allocator* a);
PKV_API int pkv_alloc_page_refs(const pkv_allocator* a, int page);

/*
 * pkv_resolve - host-side page-table address resolution (for tests and tools).
 *
 * Defines: "What is Paged FlashAttention?", section "Practical example".
 * block_table_row : host int32 array of n_entries page ids.
 * token           : 0-based token index; must be < n_entries * page_size.
 * phys, offset    : host outputs: block_table_row[token / page_size] and
 *                   token % page_size.  (page_size 256, row [5,1,9], token 300
 *                   -> phys 1, offset 44.)
 */
PKV_API int pkv_resolve(const int32_t* block_table_row, int n_entries, int page_size,
                int token, int32_t* phys, int32_t* offset);

/*
 * pkv_last_device_error - read and clear the device error word.
 *
 * Synchronises `stream`, then returns PKV_ERR_TIMEOUT if a wait gave up,
 * PKV_ERR_BAD_TABLE if a page id or length was out of range, PKV_OK otherwise.
 * `bits` (host, may be NULL) receives the raw PKV_DEVERR_* bits.  The word is
 * per device and shared by every call on it.
 */
PKV_API int pkv_last_device_error(void* stream, unsigned int* bits);

/* pkv_status_string - static, NUL-terminated description of a status code. */
PKV_API const char* pkv_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
