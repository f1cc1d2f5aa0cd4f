// The write side of the 8-bit paged cache: new tokens' K/V rows quantised into
// their pages, and whole pages copied with their scales (copy-on-write).
//
// Each block of `block_tokens` tokens of a page has one scale per kv head.  A
// call that writes rows of a block takes the largest magnitude `amax` of those
// rows and sets
//
//     s_new = max(s_old, amax / qmax, 2^-126)      (s_old = 0 where the call
//                                                   writes the block's token 0)
//     code(new rows)  = RNE(x / s_new)
//     code(old rows)  = RNE(code * s_old / s_new)  where s_new > s_old
//
// so a block never clips.  (s_new NaN: codes 0 for the new rows, the old ones stay.)  Quotients are rounded exactly (q8.cuh): the result
// does not depend on how a prompt was cut into calls other than through the
// definition above.
//
// One CTA per (block of the call, a few of the 2 H_kv (head, K or V) pairs): a warp
// takes 16 of a pair's rows, so a 16-token block has 8 pairs a CTA and a 128-token
// block one; a 256-token block has one as well, 32 rows a warp.  Lane i holds elements 4i .. 4i+3 of a row, so a row of new values is
// one 256-byte load and its codes one 128-byte store.  The rows are read twice,
// the second time from L1, four at a time: with 16 in registers the rounding is 16
// copies of its code, which cost a decode step's single row 2 us of instruction
// fetches (6.2 against 4.2 us) and gained a prompt nothing.  What bounds a prompt
// is the rounding's instructions, some 31 a code on 67% of the issue slots (78 us for
// 30027 rows of 8 heads); the floor of 2 bytes read and 1 written per element is
// 28 us.
#include "cache_attn.cuh"
#include "q8.cuh"

namespace pkv {
namespace {

constexpr int D = 128;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWarpRows = 16;        // rows of a block that a warp takes (of 256 tokens: 32)
constexpr int kBatch = 4;            // rows it loads at once

// Four consecutive elements of a new row as stored (bf16 or f32).
template <typename T> struct Row4;
template <> struct Row4<__nv_bfloat16> {
  uint2 w;
  PKV_DEVINLINE void load(const void* base, size_t row, int lane) {
    w = *reinterpret_cast<const uint2*>(static_cast<const char*>(base) + (row * 32 + lane) * 8);
  }
  // magnitudes compare as integers; NaN and infinity are the largest
  PKV_DEVINLINE uint32_t amax() const {
    const uint32_t m = __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
  }
  PKV_DEVINLINE float at(int i) const {
    const uint32_t v = i < 2 ? w.x : w.y;
    return (i & 1) ? bf16hi(v) : bf16lo(v);
  }
};
template <> struct Row4<float> {
  uint4 w;
  PKV_DEVINLINE void load(const void* base, size_t row, int lane) {
    w = *reinterpret_cast<const uint4*>(static_cast<const char*>(base) + (row * 32 + lane) * 16);
  }
  PKV_DEVINLINE uint32_t amax() const {
    return max(max(w.x & 0x7fffffffu, w.y & 0x7fffffffu), max(w.z & 0x7fffffffu, w.w & 0x7fffffffu));
  }
  PKV_DEVINLINE float at(int i) const {
    return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w);
  }
};

// Item i of the grid -> (sequence, block of the sequence).  Sequence s owns the
// items from cu_new[s] / block + 2 s on, which leaves room for every block its
// rows can touch: n rows touch at most floor(n / block) + 2 blocks.
template <int kCache, typename T>
__global__ void __launch_bounds__(kThreads, 4) append_q8_kernel(const AppendQ8Params p) {
  __shared__ int s_row0, s_rows, s_off, s_dst, s_taken;
  __shared__ uint32_t s_max[kWarps];
  if (threadIdx.x == 0) s_rows = s_taken = 0;
  __syncthreads();
  // The thread whose sequence has this item looks the block up: a search by one
  // thread would be a chain of dependent loads.
  const int item = blockIdx.x;
  for (int s = threadIdx.x; s < p.num_seqs; s += kThreads) {
    const int c0 = p.cu_new[s], c1 = p.cu_new[s + 1];
    if (item < (c0 >> p.block_shift) + 2 * s || item >= (c1 >> p.block_shift) + 2 * s + 2) continue;
    // One sequence has the item if cu_new never falls; if it does, the first to get
    // here keeps what the others would otherwise overwrite part by part.
    if (atomicExch(&s_taken, 1)) break;
    const int n = c1 - c0;
    const int start = p.start_pos[s];
    const int k = item - ((c0 >> p.block_shift) + 2 * s);        // k-th block of this sequence's rows
    const int bt = 1 << p.block_shift;
    int rows = 0, row0 = 0, off = 0, dst = -1;
    if (n > 0 && c0 >= 0 && c0 + n <= p.num_new) {
      if (start < 0) {
        if (k == 0) flag_error(p.err, PKV_DEVERR_BAD_LEN);
      } else {
        const long long pos = max((long long)start, (((long long)start >> p.block_shift) + k) << p.block_shift);
        const long long end = min((long long)start + n, ((pos >> p.block_shift) + 1) << p.block_shift);
        if (pos < end) {
          rows = (int)(end - pos);
          row0 = c0 + (int)(pos - start);
          off = (int)(pos & (bt - 1));
          const long long lp = pos >> p.page_shift;
          if (lp >= p.max_pages) {
            flag_error(p.err, PKV_DEVERR_BAD_LEN);
          } else {
            const int phys = p.block_table[(size_t)s * p.max_pages + lp];
            if (phys < 0 || phys >= p.num_pages)
              flag_error(p.err, PKV_DEVERR_BAD_PAGE);
            else                                                   // block index in the pool
              dst = (phys << (p.page_shift - p.block_shift)) +
                    (int)((pos & (p.page_size - 1)) >> p.block_shift);
          }
        }
      }
    }
    s_row0 = row0, s_off = off, s_dst = dst;
    s_rows = dst < 0 ? 0 : rows;
  }
  __syncthreads();
  const int rows = s_rows;
  if (rows == 0) return;
  const int row0 = s_row0, off = s_off, dst = s_dst;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bt = 1 << p.block_shift;
  const int parts = min(kWarps, bt / kWarpRows);                       // warps a pair
  const int pair = blockIdx.y * (kWarps / parts) + warp / parts;
  const int part = warp % parts;
  const bool live = pair < 2 * p.H_kv;
  {
    const int h = live ? pair >> 1 : 0;
    const void* src = (pair & 1) ? p.v_new : p.k_new;
    uint8_t* pages = static_cast<uint8_t*>((pair & 1) ? p.v_pages : p.k_pages);
    float* scale = ((pair & 1) ? p.v_scales : p.k_scales) + (size_t)dst * p.H_kv + h;
    const size_t src_row = (size_t)row0 * p.H_kv + h;
    uint32_t* code = reinterpret_cast<uint32_t*>(pages + (((size_t)dst << p.block_shift) * p.H_kv + h) * D) + lane;
    const size_t code_stride = (size_t)p.H_kv * D / 4;              // words between tokens

    uint32_t m = 0;
    Row4<T> x[kBatch];
    auto load = [&](int r0) {                                       // rows r0, r0 + parts, ...: all before any is used
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (r0 + i * parts < rows) x[i].load(src, src_row + (size_t)(r0 + i * parts) * p.H_kv, lane);
    };
    if (live) {
#pragma unroll 1
      for (int r0 = part; r0 < rows; r0 += kBatch * parts) {
        load(r0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (r0 + i * parts < rows) m = max(m, x[i].amax());
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (parts > 1) {
      if (lane == 0) s_max[warp] = m;
    }
    const float was = live && off > 0 ? *scale : 0.f;
    __syncthreads();                                                // the maxima are there, the old scale is read
    if (!live) return;
    if (parts > 1)
      for (int i = 0; i < parts; ++i) m = max(m, s_max[warp - part + i]);
    const float old = was;
    const bool broken = m >= 0x7f800000u || isnan(old);             // NaN or infinity: the block reads NaN
    const float s = broken ? __uint_as_float(0x7fffffffu)
                           : fmaxf(fmaxf(old, __fdiv_rn(__uint_as_float(m), code_max<kCache>())), kMinScale);
    if (lane == 0 && part == 0) *scale = s;
    if (off > 0 && s > old) {
      const float ratio = __fdiv_rn(old, s);
#pragma unroll 4
      for (int r = part; r < off; r += parts)
        code[r * code_stride] = requantize4<kCache>(code[r * code_stride], ratio, old, s);
    }
    const float lift = s < kTinyScale ? kTinyLift : 1.f;
    const float den = s * lift, inv = __fdiv_rn(1.f, den);
    auto store = [&](int r, const Row4<T>& y) {
      float v[4], q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = y.at(i) * lift;
        q[i] = v[i] * inv;
      }
      const uint32_t w = codes_of4<kCache>(q, [&](int i, float h) { return fmaf(-h, den, v[i]); });
      code[(size_t)(off + r) * code_stride] = broken ? 0u : w;
    };
#pragma unroll 1
    for (int r0 = part; r0 < rows; r0 += kBatch * parts) {
      load(r0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (r0 + i * parts < rows) store(r0 + i * parts, x[i]);
    }
  }
}

// grid = (pairs, chunks of a page): codes in 16-byte vectors, then the scales.
__global__ void __launch_bounds__(kThreads) copy_pages_q8_kernel(const CopyPagesQ8Params p) {
  const int src = p.src[blockIdx.x], dst = p.dst[blockIdx.x];
  if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.num_pages) {
    if (blockIdx.y == 0 && threadIdx.x == 0) flag_error(p.err, PKV_DEVERR_BAD_PAGE);
    return;
  }
  const size_t vec = p.page_bytes / 16;
  const uint4* ks = reinterpret_cast<const uint4*>(p.k_pages + (size_t)src * p.page_bytes);
  const uint4* vs = reinterpret_cast<const uint4*>(p.v_pages + (size_t)src * p.page_bytes);
  uint4* kd = reinterpret_cast<uint4*>(p.k_pages + (size_t)dst * p.page_bytes);
  uint4* vd = reinterpret_cast<uint4*>(p.v_pages + (size_t)dst * p.page_bytes);
  for (size_t v = (size_t)blockIdx.y * kThreads + threadIdx.x; v < vec; v += (size_t)gridDim.y * kThreads) {
    kd[v] = ks[v];
    vd[v] = vs[v];
  }
  if (blockIdx.y == 0)
    for (int i = threadIdx.x; i < p.page_scales; i += kThreads) {
      p.k_scales[(size_t)dst * p.page_scales + i] = p.k_scales[(size_t)src * p.page_scales + i];
      p.v_scales[(size_t)dst * p.page_scales + i] = p.v_scales[(size_t)src * p.page_scales + i];
    }
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Params& p, cudaStream_t stream) {
  const long long items = ((long long)p.num_new >> p.block_shift) + 2LL * p.num_seqs;
  if (items > 0x7fffffffLL) return cudaErrorNotSupported;
  const int parts = (1 << p.block_shift) / kWarpRows < kWarps ? (1 << p.block_shift) / kWarpRows : kWarps;
  const int pairs = kWarps / parts;                                // (head, K or V) pairs a CTA
  const long long groups = (2LL * p.H_kv + pairs - 1) / pairs;
  if (groups > 65535) return cudaErrorNotSupported;
  const dim3 grid((unsigned)items, (unsigned)groups);
  if (p.cache_dtype == PKV_I8) {
    if (p.rows_f32) append_q8_kernel<PKV_I8, float><<<grid, kThreads, 0, stream>>>(p);
    else append_q8_kernel<PKV_I8, __nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (p.rows_f32) append_q8_kernel<PKV_E4M3, float><<<grid, kThreads, 0, stream>>>(p);
    else append_q8_kernel<PKV_E4M3, __nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_copy_pages_q8(const CopyPagesQ8Params& p, cudaStream_t stream) {
  const size_t vec = p.page_bytes / 16;
  unsigned chunks = (unsigned)((vec + kThreads * 4 - 1) / (kThreads * 4));     // 16 KB per CTA and matrix
  chunks = chunks < 1 ? 1 : (chunks > 65535 ? 65535 : chunks);
  copy_pages_q8_kernel<<<dim3(p.n, chunks), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pkv
