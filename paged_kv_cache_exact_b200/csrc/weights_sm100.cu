// Attention weights of many query rows: for every visible key, the softmax
// weights of a call's query rows summed over the rows and over the query heads
// of the key's kv head.
//
//     W[s, kvh, j] += sum_h sum_i 2^(c q_hi . k_j - lse_hi),   c = scale * log2(e)
//
// The rows' log2-sums lse come from the prefill kernel, so this is one more
// Q K^T and one exponential per visible pair.  The product is taken transposed,
// S^T = K Q^T: a CTA owns 128 keys (the M rows, one TMEM lane and one thread of
// each epilogue warpgroup per key), keeps them in shared memory and streams every
// Q tile that sees them, so a key's sum is a sum along a thread's own registers:
// no reduction between threads, no atomics, and a fixed order.
//
// Bound: 128 x 128 exponentials take 1024 cycles of an SM's MUFU, the tile's MMA
// half of that, so the MMA and the loads hide behind the exponentials.  Warp 0
// streams Q tiles and their lse by TMA (4 stages), warp 1 issues the MMAs into 4
// TMEM buffers, and three epilogue warpgroups take the tiles in turn; a warp loads
// the next quarter of its tile from TMEM while it sums this one, and a quarter of
// the exponentials is computed on the FMA pipe, which is idle otherwise.  A tile
// takes some 1375 cycles now, with the MUFU 56% and the issue slots 44% busy: what is
// left is latency between the epilogue's warps.  With the
// attention before it, 32 heads of 4096 causal rows: two groups 315 us, four 288,
// the first keys of every head first 241, then three groups with the loads ahead
// 239 and with the FMA pipe's share 231.
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "cache_attn.cuh"
#include "q8.cuh"
#include "sm100_ptx.cuh"

namespace pkv {
namespace {

using namespace sm100;

constexpr int D = 128;
constexpr int BK = 128;                 // keys per CTA
constexpr int BQ = 128;                 // query rows per tile
constexpr int kStages = 4;              // Q ring depth
constexpr int kBufs = 4;                // S^T buffers in TMEM
constexpr int kEpiGroups = 3;           // epilogue warpgroups
constexpr int kEpiWarps = 4 * kEpiGroups;
constexpr int kThreads = (kEpiWarps + 4) * 32;
constexpr int kTileBytes = BQ * D * 2;  // 32 KB
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kLseBytes = BQ * 4;
constexpr uint64_t kWaitNs = 2000000000ull;

constexpr int kOffK = 0;
constexpr int kOffQ = kOffK + kTileBytes;
constexpr int kOffLse = kOffQ + kStages * kTileBytes;
constexpr int kOffBar = kOffLse + kStages * kLseBytes;
enum Bar { kBarQFull = 0, kBarQEmpty = kBarQFull + kStages, kBarSFull = kBarQEmpty + kStages,
           kBarSEmpty = kBarSFull + kBufs, kBarDrain = kBarSEmpty + kBufs, kNumBars };
constexpr int kOffTmem = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmem + 4;
constexpr int kOffSum = (kOffAbort + 4 + 15) & ~15;               // float[kEpiGroups - 1][BK]: the other groups' sums
constexpr int kSmemBytes = kOffSum + (kEpiGroups - 1) * BK * 4 + 1024;
constexpr uint32_t kIdesc = make_idesc_bf16(BK, BQ, false);       // K (K-major) x Q (K-major)

PKV_DEVINLINE void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

PKV_DEVINLINE float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// acc += 2^x for a pair: x = n + f with n the nearest integer, 2^f by the degree-5
// polynomial that interpolates it at the Chebyshev nodes of [-1/2, 1/2] (relative
// error 2.2e-7 in float32), 2^n by its exponent bits.  Below 2^-126 it gives 2^-126,
// which is nothing to a sum of weights; NaN stays NaN.
PKV_DEVINLINE uint64_t exp2_pair_add(uint64_t x2, uint64_t acc) {
  float a, b;
  unf2(x2, a, b);
  x2 = f2(max_nan(a, -126.f), max_nan(b, -126.f));
  const uint64_t t = add2(x2, f2(12582912.f, 12582912.f));         // 1.5 * 2^23 + n
  const uint64_t f = sub2(x2, sub2(t, f2(12582912.f, 12582912.f)));
  uint64_t y = f2(0x1.5f0890p-10f, 0x1.5f0890p-10f);
  y = fma2(y, f, f2(0x1.3d1070p-7f, 0x1.3d1070p-7f));
  y = fma2(y, f, f2(0x1.c6af6cp-5f, 0x1.c6af6cp-5f));
  y = fma2(y, f, f2(0x1.ebf906p-3f, 0x1.ebf906p-3f));
  y = fma2(y, f, f2(0x1.62e430p-1f, 0x1.62e430p-1f));
  y = fma2(y, f, f2(0x1.000002p+0f, 0x1.000002p+0f));
  float ta, tb;
  unf2(t, ta, tb);                                                 // n in the low bits, which shift to the exponent
  const uint64_t scale = f2(__uint_as_float((__float_as_uint(ta) << 23) + 0x3f800000u),
                            __uint_as_float((__float_as_uint(tb) << 23) + 0x3f800000u));
  return fma2(y, scale, acc);
}

// 16 consecutive head dims of a cached row as bf16 (two 16-byte chunks).
template <int kCache>
PKV_DEVINLINE void load_row16(const char* row, int c, uint4& a, uint4& b) {
  if (kCache == PKV_BF16) {
    a = *reinterpret_cast<const uint4*>(row + c * 32);
    b = *reinterpret_cast<const uint4*>(row + c * 32 + 16);
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(row + c * 16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {                                  // codes are exact in bf16
      float v[4];
      values_of4<kCache>(w[i], v);
      o[2 * i] = pack_bf16x2(v[0], v[1]);
      o[2 * i + 1] = pack_bf16x2(v[2], v[3]);
    }
    a = make_uint4(o[0], o[1], o[2], o[3]);
    b = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <int kCache>
__global__ void __launch_bounds__(kThreads, 1)
prompt_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const CacheAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kOffBar + 8 * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the first keys of every head first: causal rows see them most
  const int s = blockIdx.z, kvh = blockIdx.x;
  const int k0 = blockIdx.y * BK;
  const int group = p.H / p.H_kv;
  const int cap = p.max_seq_len;                   // the table holds at least as many tokens (checked by the host)
  const int kv_len = max(0, min(p.seq_lens[s], cap));              // the prefill kernel flags a bad length
  if (k0 >= kv_len) return;
  const int off = kv_len - p.q_len;
  const int n_q = (p.q_len + BQ - 1) / BQ;
  // first Q tile with a row that sees key k0 (causal: rows i >= j - off)
  const int first_q = p.causal ? max(0, k0 - off) / BQ : 0;
  const int per_head = n_q - first_q;
  const int n_tiles = per_head * group;                            // >= group: the last row sees every key

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t cnt = 1;
      if (i >= kBarQEmpty && i < kBarQEmpty + kStages) cnt = 1 + 128;      // MMA done, lse read
      if (i >= kBarSEmpty && i < kBarSEmpty + kBufs) cnt = 128;
      mbar_init(bar(i), cnt);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + kOffTmem, 512);
    tmem_relinquish();
  }
  // This CTA's keys, into the 128-byte-swizzled layout of a TMA tile; rows past
  // the sequence and rows of bad pages are zero.
  bool key_ok = false;                                             // epilogue threads: my key counts
  float key_scale = 1.f;
  if (warp >= 4) {
    const int t = threadIdx.x - 128;
    for (int i = t; i < BK * 8; i += kEpiWarps * 32) {
      const int r = i >> 3, c = i & 7;
      const int tok = k0 + r;
      uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
      if (tok < kv_len) {
        const int phys = p.block_table[(size_t)s * p.max_pages + (tok >> p.page_shift)];
        if (phys >= 0 && phys < p.num_pages) {
          const size_t row = ((size_t)phys << p.page_shift) + (tok & (p.page_size - 1));
          constexpr int kRow = D * (kCache == PKV_BF16 ? 2 : 1);
          load_row16<kCache>(static_cast<const char*>(p.k_pages) + (row * p.H_kv + kvh) * kRow, c, a, b);
        }
      }
      uint8_t* at = smem + kOffK + (c >> 2) * kHalfBytes + r * 128;
      const int c0 = 2 * (c & 3);
      *reinterpret_cast<uint4*>(at + ((c0 ^ (r & 7)) << 4)) = a;
      *reinterpret_cast<uint4*>(at + (((c0 + 1) ^ (r & 7)) << 4)) = b;
    }
    fence_proxy_async_smem();
    const int tok = k0 + (t & 127);
    if (tok < kv_len) {
      const int phys = p.block_table[(size_t)s * p.max_pages + (tok >> p.page_shift)];
      key_ok = phys >= 0 && phys < p.num_pages;
      if (kCache != PKV_BF16 && key_ok) {
        const size_t row = ((size_t)phys << p.page_shift) + (tok & (p.page_size - 1));
        key_scale = p.k_scales[(row >> p.block_shift) * p.H_kv + kvh];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);

  auto wait = [&](int b, uint32_t parity) -> bool {
    if (mbar_try_wait(bar(b), parity)) return true;
    if (*abort_flag) return false;
    if (!mbar_wait_abortable(bar(b), parity, kWaitNs, abort_flag)) {
      if (!*abort_flag) {
        *abort_flag = 1;
        flag_error(p.err, PKV_DEVERR_TIMEOUT);
      }
      return false;
    }
    return true;
  };
  auto wwait = [&](int b, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(b, parity)); };

  float sum = 0.f;
  if (warp == 0) {
    // ------------------------------------------------------------- loader --
    if (lane == 0) prefetch_tmap(&tmQ);
    int landed = -1;                                               // last tile whose load was issued
    bool ok = true;
    for (int n = 0; n < n_tiles && ok; ++n) {
      const int st = n % kStages;
      ok = wwait(kBarQEmpty + st, ((n / kStages) & 1) ^ 1);
      if (!ok) break;
      if (lane == 0) {
        const int h = kvh * group + n / per_head;
        const int q0 = (first_q + n % per_head) * BQ;
        const uint32_t full = bar(kBarQFull + st);
        mbar_arrive_expect_tx(full, kTileBytes + kLseBytes);
        for (int c = 0; c < 2; ++c)
          tma_load_3d(sbase + kOffQ + st * kTileBytes + c * kHalfBytes, &tmQ, c * 64, q0, s * p.H + h, full);
        bulk_load(sbase + kOffLse + st * kLseBytes, p.neg_lse + ((size_t)s * p.H + h) * p.lse_stride + q0, kLseBytes, full);
      }
      __syncwarp();
      landed = n;
    }
    if (!ok)                                                       // drain the loads in flight
      for (int n = max(0, landed - kStages + 1); n <= landed; ++n)
        mbar_wait_bounded(bar(kBarQFull + n % kStages), (n / kStages) & 1, kWaitNs);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA --
    const bool leader = elect_one();
    const uint64_t dk = make_sdesc(sbase + kOffK, 16, 1024);
    bool ok = true;
    for (int n = 0; n < n_tiles && ok; ++n) {
      const int st = n % kStages, buf = n % kBufs;
      ok = wwait(kBarQFull + st, (n / kStages) & 1) && wwait(kBarSEmpty + buf, ((n / kBufs) & 1) ^ 1);
      if (!ok) break;
      tc_fence_after();
      if (leader) {
        const uint64_t dq = make_sdesc(sbase + kOffQ + st * kTileBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t koff = ((kk / 4) * kHalfBytes + (kk % 4) * 32) >> 4;
          mma_ss(tmem + 128 * buf, dk + koff, dq + koff, kIdesc, kk > 0);
        }
        mma_commit(bar(kBarSFull + buf));
        mma_commit(bar(kBarQEmpty + st));
      }
      __syncwarp();
    }
    if (!ok) {
      if (leader) mma_commit(bar(kBarDrain));
      __syncwarp();
      mbar_wait_bounded(bar(kBarDrain), 0, kWaitNs);
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- epilogue --
    const int wg = (warp - 4) >> 2;                                // takes tiles wg, wg + kEpiGroups, ...
    const int r = threadIdx.x & 127;                               // my key = my TMEM lane
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c = p.scale_log2 * key_scale;
    const uint64_t c2 = f2(c, c);
    bool ok = true;
    for (int n = wg; n < n_tiles && ok; n += kEpiGroups) {
      const int st = n % kStages, buf = n % kBufs;
      ok = wwait(kBarSFull + buf, (n / kBufs) & 1) && wwait(kBarQFull + st, (n / kStages) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tS = tmem + lane_addr + 128 * buf;
      // columns (query rows) of this tile that see my key
      const int q0 = (first_q + n % per_head) * BQ;
      const int first_col = p.causal ? k0 + r - off - q0 : 0;
      const int end_col = p.q_len - q0;
      const float4* lse = reinterpret_cast<const float4*>(smem + kOffLse + st * kLseBytes);
      uint64_t acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = f2(0.f, 0.f);
      auto tile = [&](auto edge) {
        uint32_t xs[2][32];
        tmem_ld32(tS, xs[0]);
        tmem_wait_ld();
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t (&x)[32] = xs[ch & 1];
          if (ch < 3) tmem_ld32(tS + 32 * (ch + 1), xs[(ch + 1) & 1]);         // lands while this quarter is summed
          if (!decltype(edge)::value || 32 * ch < end_col) {       // else: no row in this quarter
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 e = lse[8 * ch + i];                      // minus lse
              const uint64_t y0 =
                  fma2(f2(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1])), c2, f2(e.x, e.y));
              const uint64_t y1 =
                  fma2(f2(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])), c2, f2(e.z, e.w));
              if ((i == 1 || i == 5) && !decltype(edge)::value) {
                acc[2 * (i & 1)] = exp2_pair_add(y0, acc[2 * (i & 1)]);
                acc[2 * (i & 1) + 1] = exp2_pair_add(y1, acc[2 * (i & 1) + 1]);
                continue;
              }
              float v[4];
              unf2(y0, v[0], v[1]);
              unf2(y1, v[2], v[3]);
              if (decltype(edge)::value) {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                  if (32 * ch + 4 * i + b < first_col || 32 * ch + 4 * i + b >= end_col) v[b] = -INFINITY;
              }
              acc[2 * (i & 1)] = add2(acc[2 * (i & 1)], f2(ex2(v[0]), ex2(v[1])));
              acc[2 * (i & 1) + 1] = add2(acc[2 * (i & 1) + 1], f2(ex2(v[2]), ex2(v[3])));
            }
          }
          if (ch < 3) tmem_wait_ld();
          if (ch == 2) {                                           // all of the tile is in registers
            tc_fence_before();
            mbar_arrive(bar(kBarSEmpty + buf));
          }
        }
      };
      // The diagonal, and a last tile that is not full: its rows past q_len are zeros,
      // which an infinite key would turn into NaN.  Warp-uniform.
      if ((p.causal && k0 + BK - 1 - off > q0) || end_col < BQ) tile(std::true_type{});
      else tile(std::false_type{});
      mbar_arrive(bar(kBarQEmpty + st));                           // lse read
      float lo, hi;
      unf2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), lo, hi);
      sum += lo + hi;
    }
    tmem_wait_ld();
    if (wg > 0) reinterpret_cast<float*>(smem + kOffSum)[(wg - 1) * BK + r] = sum;
  }
  tc_fence_before();
  __syncthreads();
  if (warp >= 4 && warp < 8 && key_ok && !*abort_flag) {
    const int r = threadIdx.x & 127;
#pragma unroll
    for (int i = 0; i + 1 < kEpiGroups; ++i) sum += reinterpret_cast<const float*>(smem + kOffSum)[i * BK + r];
    p.weights[((size_t)s * p.H_kv + kvh) * p.weights_stride + k0 + r] += sum;
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn get_encode() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  return fn;
}

template <int kCache>
cudaError_t launch_weights(const CUtensorMap& tq, const CacheAttnParams& p, cudaStream_t stream) {
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(prompt_weights_kernel<kCache>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  const long long key_tiles = ((long long)p.max_seq_len + BK - 1) / BK;      // at most 65535: checked by the host
  const dim3 grid(p.H_kv, (unsigned)key_tiles, p.num_seqs);
  prompt_weights_kernel<kCache><<<grid, kThreads, kSmemBytes, stream>>>(tq, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_weights(const CacheAttnParams& p, cudaStream_t stream) {
  EncodeFn enc = get_encode();
  if (!enc) return cudaErrorInvalidValue;
  CUtensorMap tq;
  const cuuint64_t dims[3] = {D, (cuuint64_t)p.q_len, (cuuint64_t)p.num_seqs * p.H};
  const cuuint64_t strides[2] = {D * 2, (cuuint64_t)D * 2 * p.q_len};
  const cuuint32_t box[3] = {64, BQ, 1}, one[3] = {1, 1, 1};
  if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.q), dims, strides, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (p.cache_dtype == PKV_I8) return launch_weights<PKV_I8>(tq, p, stream);
  if (p.cache_dtype == PKV_E4M3) return launch_weights<PKV_E4M3>(tq, p, stream);
  return launch_weights<PKV_BF16>(tq, p, stream);
}

}  // namespace pkv
