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
// * select_kernel, one CTA per (sequence, kv head).  The weights, as integers of
//   the same order, pass through shared memory so that a thread holds a run of
//   consecutive tokens in registers (32768 tokens a CTA; longer rows are read
//   again, 32768 at a time).  The threshold is found eight bits at a time from the
//   highest bit in which keys differ: a histogram in shared memory and a scan of
//   its 256 bins, ending early where a digit's keys are all wanted.  With runs of
//   tokens a thread's kept ones are consecutive in the result, so one scan over
//   the threads' counts places them; they are written to shared memory and copied
//   out whole.  For an 8-bit cache the CTA also takes every kept row's old scale
//   and gives each destination block the largest of its rows' scales, before any
//   row moves.
// * move_kernel, one CTA per (sequence, kv head, K or V, slice of a row), and one
//   for the weights: gathers the kept rows into their new places.  A kept token never moves to a
//   higher index, so a CTA that reads a chunk of rows, waits for all its
//   threads and writes them, chunk by chunk in ascending order, may compact in
//   place: what it overwrites it has already read, and another CTA never
//   touches its slice of the rows.  The next chunk's addresses are fetched while
//   this one's rows are on their way.
#include <mutex>

#include "cache_attn.cuh"
#include "q8.cuh"

namespace pkv {
namespace {

// rows a thread has in flight: what fits 64 registers (four CTAs an SM)
template <int kCache> constexpr int move_unroll() { return kCache == PKV_BF16 ? 6 : 4; }

// float32 -> uint32 with the same order (-0 and +0 equal, NaN lowest).
PKV_DEVINLINE uint32_t order_key(float f) {
  if (isnan(f)) return 0u;
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

PKV_DEVINLINE int clamped_len(const EvictParams& p, int s) {
  const int cap = p.max_seq_len;                   // the table holds at least as many tokens (checked by the host)
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

// Shared-memory word of a segment's token: a word of padding every 32 keeps the
// reads of runs of 4, 16 and 32 tokens a thread free of bank conflicts.
PKV_DEVINLINE int padded(int i) { return i + (i >> 5); }

PKV_DEVINLINE uint32_t warp_scan(uint32_t v, int lane) {           // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// kKeys: tokens a thread holds; kSelectThreads: threads of the CTA.
template <int kKeys, int kSelectThreads>
__global__ void __launch_bounds__(kSelectThreads, 1024 / kSelectThreads) select_kernel(const EvictParams p) {
  constexpr int kSelectWarps = kSelectThreads / 32;
  extern __shared__ uint32_t words[];               // a segment's keys, then its kept tokens
  __shared__ __align__(16) int hist[256];
  __shared__ uint32_t s_lo[kSelectWarps], s_hi[kSelectWarps], s_count[kSelectWarps];
  __shared__ int s_digit, s_need, s_here;
  asm volatile("griddepcontrol.launch_dependents;");              // the move kernel may be scheduled
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = clamped_len(p, s);
  if (h == 0 && tid == 0) {
    if (L != p.seq_lens[s]) flag_error(p.err, PKV_DEVERR_BAD_LEN);
    p.new_lens[s] = min(L, p.budget);
  }
  const size_t sh = (size_t)s * p.H_kv + h;
  const float* w = p.weights + sh * p.weights_stride;
  int* kept = p.kept + sh * p.budget;
  const int m = min(L, p.budget);
  const int old = m < L ? L - p.recent : 0;         // tokens that compete; none if all stay
  const int pick = m < L ? p.budget - p.recent : 0;
  constexpr int kSegment = kKeys * kSelectThreads;  // tokens in registers at a time
  const int segments = (L + kSegment - 1) / kSegment;

  uint32_t key[kKeys];                              // of tokens seg * kSegment + tid * kKeys + i
  auto load = [&](int seg) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int at = i * kSelectThreads + tid;
      if (seg * kSegment + at < L) words[padded(at)] = order_key(w[seg * kSegment + at]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kKeys; ++i) key[i] = words[padded(tid * kKeys + i)];     // past L: not looked at
    __syncthreads();
  };
  if (segments <= 1) load(0);

  // threshold key: fewer than `pick` keys are larger, at least `pick` are larger or equal
  uint32_t threshold = 0xffffffffu;
  int need = 0;                                     // how many that equal it stay
  if (pick > 0) {
    // f(key) for every competing token, one segment from registers, more from memory
    auto each = [&](auto f) {
      if (segments <= 1) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          if (tid * kKeys + i < old) f(key[i]);
      } else {
        for (int t = tid; t < old; t += kSelectThreads) f(order_key(w[t]));
      }
    };
    uint32_t lo = 0xffffffffu, hi = 0u;
    each([&](uint32_t k) {
      lo = min(lo, k);
      hi = max(hi, k);
    });
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) s_lo[warp] = lo, s_hi[warp] = hi;
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, s_lo[lane % kSelectWarps]);
    hi = __reduce_max_sync(0xffffffffu, s_hi[lane % kSelectWarps]);
    // The threshold is the `need`-th largest of the keys that agree with `threshold`
    // from bit `shift` on; keys larger than those are counted out of `need` already.
    need = pick;
    int shift = lo == hi ? 0 : 32 - __clz(lo ^ hi);
    threshold = shift == 32 ? 0u : hi >> shift << shift;
    while (shift > 0) {
      const int bits = min(shift, 8);
      shift -= bits;
      for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      each([&](uint32_t k) {
        const uint32_t d = (k ^ threshold) >> shift;                 // threshold has zeros in this digit and below
        if (d < 256u && (bits == 8 || d < (1u << bits))) atomicAdd(&hist[d], 1);   // an integer sum: any order
      });
      __syncthreads();
      if (warp == 0) {                              // lane l: bins 255 - 8 l and the seven below, from the top
        const int4 a = *reinterpret_cast<const int4*>(&hist[248 - 8 * lane]);
        const int4 b = *reinterpret_cast<const int4*>(&hist[252 - 8 * lane]);
        const int n[8] = {b.w, b.z, b.y, b.x, a.w, a.z, a.y, a.x};
        int sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += n[i];
        int above = (int)warp_scan((uint32_t)sum, lane) - sum;       // keys in larger bins than this lane's
        if (above < need && above + sum >= need) {
          int digit = 255 - 8 * lane, here = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (here == 0) {
              if (above + n[i] >= need) here = n[i], digit -= i;
              else above += n[i];
            }
          s_digit = digit;
          s_need = need - above;
          s_here = here;
        }
      }
      __syncthreads();
      threshold |= (uint32_t)s_digit << shift;
      need = s_need;
      if (s_here == need) {                         // every key from this digit on is wanted: keys with it are
        need = L;                                   // >= threshold, whose lower bits are zero
        break;
      }
    }
  }

  // ordered sweep, a segment at a time
  int base_gt = 0, base_eq = 0;
  for (int seg = 0; seg < segments; ++seg) {
    if (segments > 1) load(seg);
    const int t0 = seg * kSegment + tid * kKeys;
    uint32_t n = 0;                                 // (equal << 16) | larger: a segment has at most 32768 of each
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int t = t0 + i;
      const bool gt = t < L && (t >= old || key[i] > threshold);
      const bool eq = t < old && key[i] == threshold;
      n += (gt ? 1u : 0u) + (eq ? 0x10000u : 0u);
    }
    const uint32_t in_warp = warp_scan(n, lane);
    if (lane == 31) s_count[warp] = in_warp;
    __syncthreads();
    const uint32_t warps = warp_scan(lane < kSelectWarps ? s_count[lane] : 0u, lane);
    const uint32_t total = __shfl_sync(0xffffffffu, warps, 31);
    const uint32_t before = (warp ? __shfl_sync(0xffffffffu, warps, warp - 1) : 0u) + in_warp - n;
    const int first = base_gt + min(base_eq, need);                 // where this segment's kept tokens start
    int n_gt = base_gt + (int)(before & 0xffffu), n_eq = base_eq + (int)(before >> 16);
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int t = t0 + i;
      const bool gt = t < L && (t >= old || key[i] > threshold);
      const bool eq = t < old && key[i] == threshold;
      if (gt || (eq && n_eq < need)) words[n_gt + min(n_eq, need) - first] = t;
      n_gt += gt;
      n_eq += eq;
    }
    base_gt += total & 0xffffu;
    base_eq += total >> 16;
    __syncthreads();
    const int last = base_gt + min(base_eq, need);
    for (int j = first + tid; j < last; j += kSelectThreads) kept[j] = (int)words[j - first];
    __syncthreads();
  }
  for (int j = m + tid; j < p.budget; j += kSelectThreads) kept[j] = -1;
  if (!p.k_scales) return;

  // 8-bit: old scales of the kept rows, then the scales of the destination blocks
  float2* row_scale = p.row_scale + sh * p.budget;
  __syncthreads();
  for (int j = tid; j < m; j += kSelectThreads) {
    const int t = kept[j];
    float2 v = make_float2(-1.f, -1.f);             // a row that is not moved has no say
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
    float k = -1.f, v = -1.f;
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
      if (r >= 0 && k != -1.f) {                    // some row is moved
        const size_t i = (size_t)(r >> p.block_shift) * p.H_kv + h;
        p.k_scales[i] = k;
        p.v_scales[i] = v;
      }
    }
  }
}

// The weights of one (sequence, head), by the same rule as its rows.
template <int kMoveThreads>
PKV_DEVINLINE void move_weights(const EvictParams& p) {
  constexpr int kUnroll = 8;
  const int h = blockIdx.y, s = blockIdx.z;
  const int L = clamped_len(p, s), m = min(L, p.budget);
  const size_t sh = (size_t)s * p.H_kv + h;
  const int* kept = p.kept + sh * p.budget;
  const float* w = p.weights + sh * p.weights_stride;
  float* wo = p.weights_out + sh * p.weights_stride;
  for (int j0 = 0; j0 < m; j0 += kMoveThreads * kUnroll) {
    float x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u * kMoveThreads + threadIdx.x;
      x[u] = j < m ? w[kept[j]] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int j = j0 + u * kMoveThreads + threadIdx.x;
      if (j < m) wo[j] = x[u];
    }
  }
  for (int t = m + threadIdx.x; t < L; t += kMoveThreads) wo[t] = 0.f;
}

template <int kCache, int kMoveThreads>
__global__ void __launch_bounds__(kMoveThreads, 1024 / kMoveThreads) move_kernel(const EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");              // the kept tokens and the scales are there
  constexpr int kMoveUnroll = move_unroll<kCache>();
  const int slices = p.row_bytes / p.slice_bytes;
  if ((int)blockIdx.x == 2 * slices) {
    move_weights<kMoveThreads>(p);
    return;
  }
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

// At most 64 registers: an SM holds four CTAs of 256 threads or eight of 128.  The
// wide ones have more rows in flight where all CTAs run at once; beyond that the
// narrow ones waste less of the last turn (1280 CTAs, 32 sequences x 8 heads: 105 us
// wide, 100 narrow; 576 CTAs, 8 long sequences: 68 us wide, 94 narrow).
template <int kCache>
cudaError_t launch_move(const EvictParams& p, dim3 grid, cudaStream_t stream) {
  // Few CTAs are launched as a programmatic dependent of the selection, scheduled
  // while that drains (one short sequence 12.4 -> 10.3 us).  More than an SM each
  // would pile up on the SMs that are free first (32 sequences 119 -> 127 us).
  const long long ctas = (long long)grid.x * grid.y * grid.z;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas <= 148 ? 1 : 0;
  const bool wide = ctas <= 148LL * 4;
  cfg.blockDim = dim3(wide ? 256 : 128);
  return wide ? cudaLaunchKernelEx(&cfg, move_kernel<kCache, 256>, p)
              : cudaLaunchKernelEx(&cfg, move_kernel<kCache, 128>, p);
}

template <int kKeys, int kSelectThreads>
cudaError_t launch_select(const EvictParams& p, dim3 grid, cudaStream_t stream) {
  // The shared-memory limit is an attribute per device; host threads may get
  // here at once, so the once-per-device record is kept under a lock.
  constexpr int kSmem = (kKeys * kSelectThreads + kKeys * kSelectThreads / 32) * 4;
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute((select_kernel<kKeys, kSelectThreads>), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  select_kernel<kKeys, kSelectThreads><<<grid, kSelectThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  const dim3 rows(p.H_kv, p.num_seqs);
  // Registers for the longest sequence's weights, and no more threads than that
  // takes: barriers are cheaper and more CTAs fit an SM.
  cudaError_t e = p.max_seq_len <= 1024    ? launch_select<4, 256>(p, rows, stream)
                  : p.max_seq_len <= 4096  ? launch_select<16, 256>(p, rows, stream)
                  : p.max_seq_len <= 8192  ? launch_select<16, 512>(p, rows, stream)
                  : p.max_seq_len <= 16384 ? launch_select<16, 1024>(p, rows, stream)
                                           : launch_select<32, 1024>(p, rows, stream);
  if (e != cudaSuccess) return e;
  // Wide slices make whole 128-byte requests; narrow ones make more CTAs of few
  // (sequence, head) pairs.  Halve while there are fewer than 4 CTAs per SM.
  EvictParams q = p;
  q.slice_bytes = p.row_bytes < 128 ? p.row_bytes : 128;
  while (q.slice_bytes > 32 && 2LL * p.row_bytes / q.slice_bytes * p.H_kv * p.num_seqs < 148LL * 4) q.slice_bytes /= 2;
  const dim3 grid(2 * p.row_bytes / q.slice_bytes + 1, p.H_kv, p.num_seqs);      // + the weights
  if (p.cache_dtype == PKV_I8) return launch_move<PKV_I8>(q, grid, stream);
  if (p.cache_dtype == PKV_E4M3) return launch_move<PKV_E4M3>(q, grid, stream);
  return launch_move<PKV_BF16>(q, grid, stream);
}

}  // namespace pkv
