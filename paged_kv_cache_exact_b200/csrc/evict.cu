// Eviction by accumulated attention weight.
//
// Sequence s holds L tokens and keeps m = min(L, budget).  For each kv head the
// last min(recent, L) tokens stay, and of the others the m - min(recent, m)
// with the largest accumulated weight (equal weights: the lowest index; a NaN
// counts as the smallest).  The kept tokens keep their order and become tokens
// 0 .. m - 1.
//
// Two kernels:
//
// * select_kernel, one CTA per (sequence, kv head): a radix selection of the
//   threshold weight over the L - recent candidates (an order-preserving map of
//   float32 to integers, 8 bits a pass), then one ordered sweep that writes the
//   kept indices and compacts the weights.  For an 8-bit cache it also takes
//   every kept row's old scale and gives each destination block the largest of
//   its rows' scales, before any row moves.
// * move_kernel, one CTA per (sequence, kv head, K or V, slice of a row):
//   gathers the kept rows into their new places.  A kept token never moves to a
//   higher index, so a CTA that reads a chunk of rows, waits for all its
//   threads and writes them, chunk by chunk in ascending order, may compact in
//   place: what it overwrites it has already read, and another CTA never
//   touches its slice of the rows.
#include "cache_attn.cuh"
#include "q8.cuh"

namespace pkv {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;
constexpr int kSliceBytes = 32;                                   // two 16-byte loads
constexpr int kMoveRows = kMoveThreads / 2 * kMoveUnroll;         // rows a chunk

// float32 -> uint32 with the same order (-0 and +0 equal, NaN lowest).
PKV_DEVINLINE uint32_t order_key(float f) {
  if (isnan(f)) return 0u;
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

PKV_DEVINLINE int clamped_len(const EvictParams& p, int s) {
  const int cap = min(p.max_seq_len, p.max_pages * p.page_size);
  return max(0, min(p.seq_lens[s], cap));
}

// the physical row of token t of sequence s, or -1 where the table has no page for it
PKV_DEVINLINE long long token_row(const EvictParams& p, const int32_t* table, int s, int t) {
  const int phys = table[(size_t)s * p.max_pages + (t >> p.page_shift)];
  if (phys < 0 || phys >= p.num_pages) {
    flag_error(p.err, PKV_DEVERR_BAD_PAGE);
    return -1;
  }
  return ((long long)phys << p.page_shift) + (t & (p.page_size - 1));
}

// NaN wins over every number.
PKV_DEVINLINE float max_nan(float a, float b) { return isnan(a) ? a : isnan(b) ? b : fmaxf(a, b); }

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictParams p) {
  __shared__ unsigned int hist[256];
  __shared__ unsigned int s_prefix;
  __shared__ int s_need;
  __shared__ unsigned int warp_sum[kSelectWarps];
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = clamped_len(p, s);
  if (h == 0 && tid == 0) {
    if (L != p.seq_lens[s]) flag_error(p.err, PKV_DEVERR_BAD_LEN);
    p.new_lens[s] = min(L, p.budget);
  }
  const size_t sh = (size_t)s * p.H_kv + h;
  const float* w = p.weights + sh * p.weights_stride;
  float* wo = p.weights_out + sh * p.weights_stride;
  int* kept = p.kept + sh * p.budget;
  const int m = min(L, p.budget);
  const int old = m < L ? L - p.recent : 0;         // tokens that compete; none if all stay
  const int pick = m < L ? p.budget - p.recent : 0;

  // threshold key: fewer than `pick` keys are larger, at least `pick` are larger or equal
  uint32_t prefix = 0;
  int need = pick;
  if (pick > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : (0xffffffffu << (shift + 8));
      for (int t = tid; t < old; t += kSelectThreads) {
        const uint32_t k = order_key(w[t]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int left = need, b = 255;
        while (b > 0 && (int)hist[b] < left) left -= hist[b--];
        s_prefix = prefix | ((uint32_t)b << shift);
        s_need = left;
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
  }

  // ordered sweep
  int base_gt = 0, base_eq = 0;
  for (int t0 = 0; t0 < L; t0 += kSelectThreads) {
    const int t = t0 + tid;
    bool gt = false, eq = false;
    float x = 0.f;
    if (t < L) {
      x = w[t];
      const uint32_t k = order_key(x);
      gt = t >= old || (pick > 0 && k > prefix);
      eq = !gt && pick > 0 && k == prefix;
    }
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) warp_sum[warp] = (__popc(be) << 16) | __popc(bg);
    __syncthreads();
    uint32_t before = 0, total = 0;
    for (int i = 0; i < kSelectWarps; ++i) {
      const uint32_t v = warp_sum[i];
      if (i < warp) before += v;
      total += v;
    }
    const uint32_t lt = (1u << lane) - 1u;
    const int n_gt = base_gt + (before & 0xffff) + __popc(bg & lt);
    const int n_eq = base_eq + (before >> 16) + __popc(be & lt);
    if (gt || (eq && n_eq < need)) {
      const int j = n_gt + min(n_eq, need);
      kept[j] = t;
      wo[j] = x;
    }
    base_gt += total & 0xffff;
    base_eq += total >> 16;
    __syncthreads();
  }
  for (int t = m + tid; t < L; t += kSelectThreads) wo[t] = 0.f;
  for (int j = m + tid; j < p.budget; j += kSelectThreads) kept[j] = -1;
  if (!p.k_scales) return;

  // 8-bit: old scales of the kept rows, then the scales of the destination blocks
  float2* row_scale = p.row_scale + sh * p.budget;
  __syncthreads();
  for (int j = tid; j < m; j += kSelectThreads) {
    const int t = kept[j];
    float2 v = make_float2(0.f, 0.f);
    const long long r = token_row(p, p.block_table, s, t);
    if (r >= 0) {
      const size_t i = (size_t)(r >> p.block_shift) * p.H_kv + h;
      v = make_float2(p.k_scales[i], p.v_scales[i]);
    }
    row_scale[j] = v;
  }
  __syncthreads();
  const int bt = 1 << p.block_shift;
  const int blocks = (m + bt - 1) >> p.block_shift;
  for (int b = warp; b < blocks; b += kSelectWarps) {
    float k = 0.f, v = 0.f;
    for (int j = (b << p.block_shift) + lane; j < min(m, (b + 1) << p.block_shift); j += 32) {
      const float2 r = row_scale[j];
      k = max_nan(k, r.x);
      v = max_nan(v, r.y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      k = max_nan(k, __shfl_xor_sync(0xffffffffu, k, o));
      v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    if (lane == 0) {
      p.block_scale[sh * p.max_blocks + b] = make_float2(k, v);
      const long long r = token_row(p, p.dst_table, s, b << p.block_shift);
      if (r >= 0 && k != 0.f) {
        const size_t i = (size_t)(r >> p.block_shift) * p.H_kv + h;
        p.k_scales[i] = k;
        p.v_scales[i] = v;
      }
    }
  }
}

template <int kCache>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p) {
  const int slices = p.row_bytes / kSliceBytes;
  const bool is_v = (int)blockIdx.x >= slices;
  const int slice = blockIdx.x - (is_v ? slices : 0);
  const int h = blockIdx.y, s = blockIdx.z;
  const int m = min(clamped_len(p, s), p.budget);
  const size_t sh = (size_t)s * p.H_kv + h;
  const int* kept = p.kept + sh * p.budget;
  uint8_t* pages = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + (size_t)h * p.row_bytes +
                   slice * kSliceBytes + (threadIdx.x & 1) * 16;
  const size_t stride = (size_t)p.H_kv * p.row_bytes;
  for (int j0 = 0; j0 < m; j0 += kMoveRows) {
    uint4 x[kMoveUnroll];
    long long from[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = j0 + u * (kMoveThreads / 2) + (threadIdx.x >> 1);
      from[u] = -1;
      if (j < m) from[u] = token_row(p, p.block_table, s, kept[j]);
      if (from[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(pages + from[u] * stride);
    }
    __syncthreads();                                               // every row of the chunk is read
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = j0 + u * (kMoveThreads / 2) + (threadIdx.x >> 1);
      if (from[u] < 0) continue;
      const long long to = token_row(p, p.dst_table, s, j);
      if (to < 0) continue;
      if (kCache == PKV_I8 || kCache == PKV_E4M3) {
        const float2 rs = p.row_scale[sh * p.budget + j];
        const float2 bs = p.block_scale[sh * p.max_blocks + (j >> p.block_shift)];
        const float a = is_v ? rs.y : rs.x, b = is_v ? bs.y : bs.x;
        if (isnan(b)) {
          x[u] = make_uint4(0u, 0u, 0u, 0u);
        } else if (a != b) {
          const float ratio = __fdiv_rn(a, b);
          x[u].x = requantize4<kCache>(x[u].x, ratio, a, b);
          x[u].y = requantize4<kCache>(x[u].y, ratio, a, b);
          x[u].z = requantize4<kCache>(x[u].z, ratio, a, b);
          x[u].w = requantize4<kCache>(x[u].w, ratio, a, b);
        } else if (to == from[u]) {
          continue;
        }
      } else if (to == from[u]) {
        continue;
      }
      *reinterpret_cast<uint4*>(pages + to * stride) = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  select_kernel<<<dim3(p.H_kv, p.num_seqs), kSelectThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(2 * p.row_bytes / kSliceBytes, p.H_kv, p.num_seqs);
  if (p.cache_dtype == PKV_I8) move_kernel<PKV_I8><<<grid, kMoveThreads, 0, stream>>>(p);
  else if (p.cache_dtype == PKV_E4M3) move_kernel<PKV_E4M3><<<grid, kMoveThreads, 0, stream>>>(p);
  else move_kernel<PKV_BF16><<<grid, kMoveThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pkv
