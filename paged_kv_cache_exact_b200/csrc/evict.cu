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
// * select_kernel, one CTA per (sequence, kv head).  A thread holds its tokens'
//   weights in registers as integers of the same order (32768 tokens a CTA;
//   longer rows are read again).  The threshold is found four bits at a time from
//   the highest bit in which keys differ: a thread counts its keys into 16
//   eight-bit counters in registers, then one warp and one block reduction.
//   (Counting into shared memory puts nearly all keys into a few bins, as weights
//   crowd near zero, and the atomics serialise; a bit at a time takes a barrier a
//   bit.)  One scan over all warps' counts gives every kept token its place.  For an 8-bit cache the
//   CTA also takes every kept row's old scale and gives each destination block the
//   largest of its rows' scales, before any row moves.
// * move_kernel, one CTA per (sequence, kv head, K or V, slice of a row):
//   gathers the kept rows into their new places.  A kept token never moves to a
//   higher index, so a CTA that reads a chunk of rows, waits for all its
//   threads and writes them, chunk by chunk in ascending order, may compact in
//   place: what it overwrites it has already read, and another CTA never
//   touches its slice of the rows.  The next chunk's addresses are fetched while
//   this one's rows are on their way.
#include "cache_attn.cuh"
#include "q8.cuh"

namespace pkv {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256;
// rows a thread has in flight: what fits 64 registers (four CTAs an SM)
template <int kCache> constexpr int move_unroll() { return kCache == PKV_BF16 ? 8 : 4; }

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

// kKeys: tokens a thread holds.
template <int kKeys>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictParams p) {
  __shared__ int part[16][kSelectWarps + 1];                     // every warp's counts of the 16 digits
  __shared__ int s_digit, s_need;
  __shared__ uint32_t s_lo[kSelectWarps], s_hi[kSelectWarps];
  __shared__ uint32_t counts[kKeys * kSelectWarps];              // (equal << 16) | larger, then their prefix sums
  __shared__ uint32_t row_total[32];
  static_assert(kSelectWarps == 32 && kKeys <= 32, "one warp sums the warps' counts");
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
  constexpr int kSegment = kKeys * kSelectThreads;  // tokens in registers at a time
  const int segments = (L + kSegment - 1) / kSegment;

  uint32_t key[kKeys];                              // of token t0 + i * 1024 + tid
  auto load = [&](int seg) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int t = seg * kSegment + i * kSelectThreads + tid;
      key[i] = t < L ? order_key(w[t]) : 0u;
    }
  };
  load(0);

  // threshold key: fewer than `pick` keys are larger, at least `pick` are larger or equal
  uint32_t threshold = 0xffffffffu;
  int need = 0;                                     // how many equal to it stay
  if (pick > 0) {
    uint32_t lo = 0xffffffffu, hi = 0u;
    for (int seg = 0; seg < segments; ++seg) {
      if (seg > 0) load(seg);
#pragma unroll
      for (int i = 0; i < kKeys; ++i)
        if (seg * kSegment + i * kSelectThreads + tid < old) {
          lo = min(lo, key[i]);
          hi = max(hi, key[i]);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) s_lo[warp] = lo, s_hi[warp] = hi;
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, s_lo[lane]);
    hi = __reduce_max_sync(0xffffffffu, s_hi[lane]);
    // The threshold is the `need`-th largest of the keys that agree with `threshold`
    // above bit `shift`; keys larger than those are counted out of `need` already.
    need = pick;
    const int bits = lo == hi ? 0 : 32 - __clz(lo ^ hi);
    int shift = (bits + 3) / 4 * 4;
    threshold = shift == 32 ? 0u : hi >> shift << shift;
    while (shift > 0) {
      shift -= 4;
      unsigned long long c0 = 0, c1 = 0;            // counts of digits 0 .. 7 and 8 .. 15, a byte each
      int count = 0;                                // lane 2d (and 2d + 1): the warp's count of digit d
      for (int seg = 0; seg < segments; ++seg) {
        if (segments > 1) load(seg);
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
          const uint32_t d = (key[i] ^ threshold) >> shift;          // threshold has zeros from bit shift + 3 down
          const unsigned long long one = 1ull << ((d & 7u) * 8u);
          const bool in = seg * kSegment + i * kSelectThreads + tid < old;
          if (in && d < 8u) c0 += one;
          if (in && (d & ~7u) == 8u) c1 += one;
        }
        // Over the warp, halving the counts a lane holds with the lanes that share
        // them (16-bit counts, two a word: 32 keys * 32 lanes fit; REDUX takes
        // longer than these nine shuffles).
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t two = (uint32_t)((j < 4 ? c0 : c1) >> (16 * (j & 3)));
          v[j] = (two & 0xffu) | ((two & 0xff00u) << 8);
        }
        c0 = c1 = 0;
#pragma unroll
        for (int o = 16, n = 4; n >= 1; o >>= 1, n >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int j = 0; j < n; ++j) {
            const uint32_t send = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        // lanes 4j .. 4j + 3 hold digits 2j and 2j + 1
        count += (lane & 2) ? v[0] >> 16 : v[0] & 0xffffu;
      }
      if ((lane & 1) == 0) part[lane >> 1][warp] = count;
      __syncthreads();
      if (warp == 0) {
        // lane 2d + e sums half the warps' counts of digit d, then the counts of larger digits
        int n = 0;
#pragma unroll
        for (int i = 0; i < kSelectWarps / 2; ++i) n += part[lane >> 1][(lane & 1) * (kSelectWarps / 2) + i];
        n += __shfl_xor_sync(0xffffffffu, n, 1);
        int from = n;                               // digit d and larger
#pragma unroll
        for (int o = 2; o < 32; o <<= 1) {
          const int u = __shfl_down_sync(0xffffffffu, from, o);
          if (lane + o < 32) from += u;
        }
        const uint32_t enough = __ballot_sync(0xffffffffu, from >= need);
        const int top = 31 - __clz(enough);         // the largest digit with `need` keys from it on (0 has them)
        if (lane == top) {
          s_digit = lane >> 1;
          s_need = need - (from - n);
        }
      }
      __syncthreads();
      const int digit = s_digit;
      need = s_need;
      threshold |= (uint32_t)digit << shift;
    }
  }

  // ordered sweep, a segment at a time
  int base_gt = 0, base_eq = 0;
  for (int seg = 0; seg < segments; ++seg) {
    if (segments > 1) load(seg);
    const int t0 = seg * kSegment;
    uint32_t gt_mask = 0, eq_mask = 0;              // bit i: this thread's token i
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int t = t0 + i * kSelectThreads + tid;
      const bool gt = t < L && (t >= old || (pick > 0 && key[i] > threshold));
      const bool eq = t < old && pick > 0 && key[i] == threshold;
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      gt_mask |= (uint32_t)gt << i;
      eq_mask |= (uint32_t)eq << i;
      if (lane == 0) counts[i * kSelectWarps + warp] = (__popc(be) << 16) | __popc(bg);
    }
    float x[kKeys];                                 // the weights themselves, before any is overwritten
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      x[i] = ((gt_mask | eq_mask) >> i) & 1u ? w[t0 + i * kSelectThreads + tid] : 0.f;
    __syncthreads();
    auto scan = [&](uint32_t v) {                   // inclusive, over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      return v;
    };
    if (warp < kKeys) {                             // warp i: the counts of row i before each warp
      const uint32_t v = counts[warp * kSelectWarps + lane], sum = scan(v);
      counts[warp * kSelectWarps + lane] = sum - v;
      if (lane == 31) row_total[warp] = sum;
    }
    __syncthreads();
    const uint32_t total = lane < kKeys ? row_total[lane] : 0u, row_sum = scan(total);
    const uint32_t lt = (1u << lane) - 1u;
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const bool gt = (gt_mask >> i) & 1u, eq = (eq_mask >> i) & 1u;
      const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
      const uint32_t before = counts[i * kSelectWarps + warp] + __shfl_sync(0xffffffffu, row_sum - total, i);
      if (!(bg | be)) continue;                     // warp-uniform
      const int n_gt = base_gt + (int)(before & 0xffff) + __popc(bg & lt);
      const int n_eq = base_eq + (int)(before >> 16) + __popc(be & lt);
      if (gt || (eq && n_eq < need)) {
        const int j = n_gt + min(n_eq, need);
        kept[j] = t0 + i * kSelectThreads + tid;
        wo[j] = x[i];                               // j <= t: in place, read already
      }
    }
    const uint32_t all = __shfl_sync(0xffffffffu, row_sum, 31);
    base_gt += all & 0xffff;
    base_eq += all >> 16;
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
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const EvictParams p) {
  constexpr int kMoveUnroll = move_unroll<kCache>();
  const int slices = p.row_bytes / p.slice_bytes;
  const bool is_v = (int)blockIdx.x >= slices;
  const int slice = blockIdx.x - (is_v ? slices : 0);
  const int h = blockIdx.y, s = blockIdx.z;
  const int m = min(clamped_len(p, s), p.budget);
  const size_t sh = (size_t)s * p.H_kv + h;
  const int* kept = p.kept + sh * p.budget;
  const int per_row = p.slice_bytes / 16;                          // threads a row
  const int rows = kMoveThreads / per_row;                         // rows a step; a chunk is kMoveUnroll steps
  const int mine = threadIdx.x / per_row;
  uint8_t* pages = static_cast<uint8_t*>(is_v ? p.v_pages : p.k_pages) + (size_t)h * p.row_bytes +
                   slice * p.slice_bytes + threadIdx.x % per_row * 16;
  const size_t stride = (size_t)p.H_kv * p.row_bytes;
  int from[kMoveUnroll];                                           // physical rows; a pool has at most 2^31
  auto find = [&](int j0) {
    int t[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = j0 + u * rows + mine;
      t[u] = j < m ? kept[j] : -1;
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) from[u] = t[u] >= 0 ? (int)token_row(p, p.block_table, s, t[u]) : -1;
  };
  find(0);
  for (int j0 = 0; j0 < m; j0 += kMoveUnroll * rows) {
    uint4 x[kMoveUnroll];
    int was[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      was[u] = from[u];
      if (was[u] >= 0) x[u] = *reinterpret_cast<const uint4*>(pages + was[u] * stride);
    }
    int to[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = j0 + u * rows + mine;
      to[u] = was[u] >= 0 ? (int)token_row(p, p.dst_table, s, j) : -1;
    }
    find(j0 + kMoveUnroll * rows);
    __syncthreads();                                               // every row of the chunk is read
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = j0 + u * rows + mine;
      if (to[u] < 0) continue;
      bool changed = to[u] != was[u];
      if (kCache == PKV_I8 || kCache == PKV_E4M3) {
        const float2 rs = p.row_scale[sh * p.budget + j];
        const float2 bs = p.block_scale[sh * p.max_blocks + (j >> p.block_shift)];
        const float a = is_v ? rs.y : rs.x, b = is_v ? bs.y : bs.x;
        if (isnan(b)) {
          x[u] = make_uint4(0u, 0u, 0u, 0u);
          changed = true;
        } else if (a != b) {
          const float ratio = __fdiv_rn(a, b);
          x[u].x = requantize4<kCache>(x[u].x, ratio, a, b);
          x[u].y = requantize4<kCache>(x[u].y, ratio, a, b);
          x[u].z = requantize4<kCache>(x[u].z, ratio, a, b);
          x[u].w = requantize4<kCache>(x[u].w, ratio, a, b);
          changed = true;
        }
      }
      if (changed) *reinterpret_cast<uint4*>(pages + to[u] * stride) = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  const dim3 rows(p.H_kv, p.num_seqs);
  // registers for the longest sequence's weights: 4, 16 or 32 a thread
  if (p.max_seq_len <= 4 * kSelectThreads) select_kernel<4><<<rows, kSelectThreads, 0, stream>>>(p);
  else if (p.max_seq_len <= 16 * kSelectThreads) select_kernel<16><<<rows, kSelectThreads, 0, stream>>>(p);
  else select_kernel<32><<<rows, kSelectThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // Wide slices make whole 128-byte requests; narrow ones make more CTAs of few
  // (sequence, head) pairs.  Halve while there are fewer than 4 CTAs per SM.
  EvictParams q = p;
  q.slice_bytes = p.row_bytes < 128 ? p.row_bytes : 128;
  while (q.slice_bytes > 32 && 2LL * p.row_bytes / q.slice_bytes * p.H_kv * p.num_seqs < 148LL * 4) q.slice_bytes /= 2;
  const dim3 grid(2 * p.row_bytes / q.slice_bytes, p.H_kv, p.num_seqs);
  if (p.cache_dtype == PKV_I8) move_kernel<PKV_I8><<<grid, kMoveThreads, 0, stream>>>(q);
  else if (p.cache_dtype == PKV_E4M3) move_kernel<PKV_E4M3><<<grid, kMoveThreads, 0, stream>>>(q);
  else move_kernel<PKV_BF16><<<grid, kMoveThreads, 0, stream>>>(q);
  return cudaGetLastError();
}

}  // namespace pkv
