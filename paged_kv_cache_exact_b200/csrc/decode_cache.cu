// Attention of single tokens, or of a few, over a cache held in 8 bits, and the
// same (over an 8-bit or a bf16 cache) that also adds every key's softmax weight
// to an accumulator.  Several query tokens are taken as more heads: the rows
// [H, q_len] of a sequence lie one after the other, and row (h, i) differs from a
// head of its own only in the last key it sees.
//
// What bounds it is reading the cache: 256 bytes (8-bit) or 512 bytes (bf16)
// per token and kv head, plus 8 bytes of scales per block.  So every K/V row
// is read once for all query heads of its kv head.  Each of a CTA's four warps
// takes chunks of 16 tokens of its own (two at a time of an 8-bit cache) through a
// two-step cp.async ring: 8 KB a warp (96 KB an SM of three CTAs, 64 KB of two where
// a kv head has more than 8 rows) are on their way while as much is worked on, and no
// barrier joins the warps before the end.
//
// Products.  With up to 8 query heads per kv head (16 in two tiles) scores and
// outputs are small matrix products, written transposed so that the long axis
// is M: S^T = K Q^T (M = 16 tokens, N = 8 heads, 8 steps over the head dim) and
// O^T = V^T P^T (M = 16 head dims, 8 tiles, N = 8 heads, one step of 16 tokens),
// both mma.sync m16n8k16; tcgen05's smallest tile (M = 64 in TMEM) would be
// three quarters padding, and the tensor pipe is far from the bound here.
// The index that a product sums over may be permuted freely and so may the rows
// of O^T, which is what lets each lane read 16 consecutive bytes of a row from the
// ring:
//   K: lane (g, t) = (lane / 4, lane % 4) reads rows g and g + 8;
//   V: lane (g, t) reads rows 2t, 2t+1, 2t+8, 2t+9 at bytes 16 g, and pairs of
//      rows are interleaved in registers (prmt), which transposes V.
// S^T comes out with a token per row and lane group, P^T goes in with a head
// per column: one movmatrix transposes each 8 x 8 block.
//
// Numbers.  Codes of both formats are exact in f16, so products run on f16
// codes: q is scaled by a power of two per head so that its largest element
// lies in [2^14, 2^15) (f16 keeps 11 bits, bf16 has 8: exact but for elements
// below 2^-24 of the largest, whose error is under 2^-39 of it).  P is rounded to
// f16, lifted by 2^7 against the reference maximum so that weights down to 2^-21
// of the largest keep all 11 bits and those below 2^-32 of it vanish.  A bf16 cache runs on bf16
// products with P in two bf16 parts (16 bits: one part alone would be off by up to
// 2^-8 where a few keys share the weight, and the pipe has room).  Scales are applied
// in float32: ks to the score, vs to each chunk's P V product (a chunk of 16
// tokens lies in one block).  Sums and maxima are float32; the reference
// maximum moves only when a score passes it by 2^8 (O and l share it: exact).
//
// Weights need the row's final maximum and sum, so the scores (float32, base-2
// units) go to the workspace and a second kernel turns them into weights once
// the splits are merged: each (sequence, kv head, token) has its own lanes, so
// there are no atomics and the sums have one order.
#include <mutex>

#include "cache_attn.cuh"
#include "cp_async.cuh"
#include "q8.cuh"
#include "sm100_ptx.cuh"

namespace pkv {
namespace {

using sm100::f2;
using sm100::fma2;
using sm100::unf2;

constexpr int D = 128;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSplitPages = 256;               // table entries staged per CTA (16-token pages)
constexpr int kMaxSplitTokens = 4096;
constexpr int kOneSplit = 512;
constexpr int kMaxSplits = 1024;

// d[16x8] += a[16x16] * b[16x8], f32 accumulation
template <bool kF16>
PKV_DEVINLINE void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                            uint32_t b0, uint32_t b1) {
  if (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

PKV_DEVINLINE uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

PKV_DEVINLINE uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Codes 0,1 (lo) and 2,3 (hi) of a word as f16 pairs.
template <int kCache>
PKV_DEVINLINE void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kCache == PKV_I8) {
    // code + 128 in the mantissa of 1024 + u, then minus 1152: both exact
    const uint32_t u = w ^ 0x80808080u;
    lo = __byte_perm(u, 0x64646464u, 0x4140);
    hi = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  }
}

// Where a 16-byte piece of a row lies in shared memory: pieces are permuted so
// that the eight lanes of a fragment read meet eight different bank groups, K's
// (two rows, four pieces) and V's (four rows, two pieces).
PKV_DEVINLINE int k_swizzle(int row) { return (row & 1) << 2; }
PKV_DEVINLINE int v_swizzle(int row) { return row & 6; }

template <int kCache>
struct Layout {
  static constexpr bool kBf16 = kCache == PKV_BF16;
  static constexpr int kRowBytes = D * (kBf16 ? 2 : 1);
  static constexpr int kVec = kBf16 ? 8 : 4;                // 16-byte pieces per lane, chunk and matrix
  static constexpr int kRowLanes = kRowBytes / 16;          // lanes that copy a row
  static constexpr int kUnroll = kBf16 ? 1 : 2;             // chunks a warp works on at once
  static constexpr int kStages = 2;                         // ring depth, in steps of kUnroll chunks
  static constexpr int kChunkBytes = 2 * kVec * 32 * 16;    // K, then V: 4 or 8 KB
  static constexpr int kStageBytes = kUnroll * kChunkBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr float kLift = kBf16 ? 0.f : 7.f;
};

// kOne: one query head per kv head; a lane then works on column 2 t4 alone (the
// real one is column 0, of lanes t4 = 0).
template <int kCache, int NT, bool kWeights, bool kOne>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
cache_decode_kernel(const CacheAttnParams p) {
  using Lay = Layout<kCache>;
  constexpr bool kBf16 = Lay::kBf16;
  constexpr int kHeads = 8 * NT;
  constexpr int U = Lay::kUnroll;
  constexpr int J = kOne ? 1 : 2;                            // columns of a lane
  extern __shared__ __align__(16) uint8_t ring[];            // [warp][stage][chunk][K, V][row]
  __shared__ int s_pages[kMaxSplitPages];
  __shared__ __align__(8) float s_scale[kWarps][Lay::kStages][U][2];      // (ks, vs) of the chunks in the ring
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  asm volatile("griddepcontrol.launch_dependents;");

  const int split = blockIdx.y, s = blockIdx.z;
  const int group = p.H / p.H_kv;
  const int n_hg = (group + kHeads - 1) / kHeads;
  const int kvh = blockIdx.x / n_hg;
  const int hg0 = (blockIdx.x % n_hg) * kHeads;             // first head within the group
  const int h0 = kvh * group + hg0;
  const int nh = min(kHeads, group - hg0);
  const int q_len = p.q_len;                                 // p.H counts rows: heads times q_len
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;

  // The split's table entries are fetched along with the length: what lies past the
  // sequence is not looked at.
  const int t_begin = split * p.split_tokens;
  const int lp0 = t_begin >> p.page_shift;
  const int n_lp = min(p.max_pages - lp0, (p.split_tokens + p.page_size - 1) >> p.page_shift);
  int mine_lp[kMaxSplitPages / kThreads];
#pragma unroll
  for (int i = 0; i < kMaxSplitPages / kThreads; ++i)
    mine_lp[i] = tid + i * kThreads < n_lp ? p.block_table[(size_t)s * p.max_pages + lp0 + tid + i * kThreads] : -1;
  int L = p.seq_lens[s];
  const int cap = p.max_seq_len;                   // the table holds at least as many tokens (checked by the host)
  if (L < q_len || L > cap) {
    if (split == 0 && blockIdx.x == 0 && tid == 0) flag_error(p.err, PKV_DEVERR_BAD_LEN);
    L = max(0, min(L, cap));
  }
  if (L <= 0) {
    if (split == 0)
      for (int i = tid; i < nh * D; i += kThreads)
        p.out[((size_t)s * p.H + h0) * D + i] = __float2bfloat16_rn(0.f);
    return;
  }
  if (t_begin >= L) return;
  const int t_end = min(L, t_begin + p.split_tokens);
  const int nsplit = (L + p.split_tokens - 1) / p.split_tokens;
  const int lp1 = (t_end - 1) >> p.page_shift;
#pragma unroll
  for (int i = 0; i < kMaxSplitPages / kThreads; ++i) {
    int phys = mine_lp[i];
    if (tid + i * kThreads > lp1 - lp0) break;
    if (phys < 0 || phys >= p.num_pages) {
      flag_error(p.err, PKV_DEVERR_BAD_PAGE);
      phys = -1;
    }
    s_pages[tid + i * kThreads] = phys;
  }

  // Q^T as the B operand: column n = g is head g, and each lane holds the head
  // dims that its K loads bring (see the loads below).
  uint32_t qb[NT][D / 16][2];
  float hm[NT][2];                                           // score multiplier of heads 2 t4, 2 t4 + 1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const bool live = 8 * nt + g < nh;
    const char* qrow = reinterpret_cast<const char*>(p.q + ((size_t)s * p.H + h0 + (live ? 8 * nt + g : 0)) * D);
    if (kBf16) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {                          // d = 32 c + 8 t4 + 0 .. 7
        const uint4 x = *reinterpret_cast<const uint4*>(qrow + 64 * c + 16 * t4);
        qb[nt][2 * c][0] = live ? x.x : 0u;
        qb[nt][2 * c][1] = live ? x.y : 0u;
        qb[nt][2 * c + 1][0] = live ? x.z : 0u;
        qb[nt][2 * c + 1][1] = live ? x.w : 0u;
      }
      hm[nt][0] = hm[nt][1] = p.scale_log2;
    } else {
      uint4 x[4];
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {                          // d = 64 c + 16 t4 + 0 .. 15
        x[2 * c] = *reinterpret_cast<const uint4*>(qrow + 128 * c + 32 * t4);
        x[2 * c + 1] = *reinterpret_cast<const uint4*>(qrow + 128 * c + 32 * t4 + 16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the head's largest element is in [2^e, 2^(e+1)): multiply by 2^(14 - e)
      const int e = max((int)(top >> 7) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + max(14 - e, -126)) << 23);
      const float down = __uint_as_float((uint32_t)(127 + min(e - 14, 126)) << 23);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int w = 0; w < 4; ++w) {                        // step 4 c + w: d = 64 c + 16 t4 + 4 w + 0 .. 3
          const uint4 y = x[2 * c + (w >> 1)];
          const uint32_t lo = (w & 1) ? y.z : y.x, hi = (w & 1) ? y.w : y.y;
          qb[nt][4 * c + w][0] = live ? pack_f16x2(bf16lo(lo) * up, bf16hi(lo) * up) : 0u;
          qb[nt][4 * c + w][1] = live ? pack_f16x2(bf16lo(hi) * up, bf16hi(hi) * up) : 0u;
        }
      hm[nt][0] = p.scale_log2 * __shfl_sync(0xffffffffu, down, 8 * t4);
      hm[nt][1] = p.scale_log2 * __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
    }
  }
  __syncthreads();                                           // s_pages ready

  const int stride = p.H_kv * Lay::kRowBytes;                // bytes between tokens of a page
  // this lane's 16 bytes of a row in a copy
  const char* kbase = static_cast<const char*>(p.k_pages) + (size_t)kvh * Lay::kRowBytes + 16 * (lane % Lay::kRowLanes);
  const char* vbase = static_cast<const char*>(p.v_pages) + (size_t)kvh * Lay::kRowBytes + 16 * (lane % Lay::kRowLanes);
  const int pmask = p.page_size - 1;
  const int n_chunks = (t_end - t_begin + 15) >> 4;

  auto chunk_row = [&](int c, bool& ok) -> size_t {          // first physical row of chunk c
    const int tok = t_begin + 16 * c;
    const int phys = c < n_chunks ? s_pages[(tok >> p.page_shift) - lp0] : -1;
    ok = phys >= 0;
    return ((size_t)(ok ? phys : 0) << p.page_shift) + (tok & pmask);
  };
  // Copy chunk c into the ring (zeros for a chunk that is not there, a bad page,
  // and V rows past the sequence, which may hold NaN).  Consecutive lanes take
  // consecutive bytes of a row: eight lanes make one 128-byte request, where a
  // fragment's own order (four rows per eight lanes) would make four.
  const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + warp * Lay::kStages * Lay::kStageBytes;
  constexpr int kRowsAtOnce = 32 / Lay::kRowLanes;
  // With weights the cache's lines are the first to leave L2, so that more of the
  // scores are still there for the next kernel (from a cold L2, 64 sequences of 512
  // to 8192 tokens, 64/8 heads, bf16: 229 -> 225 us; 8 of 2000 to 30001, 32/8, e4m3:
  // 90 -> 84).  Scores that are the last to leave gained 64/8 heads 4 us more and
  // cost 64/2 heads 5.
  const uint64_t policy = kWeights ? l2_evict_first() : 0;
  auto prefetch = [&](int c, uint32_t dst) {
    bool ok;
    const size_t row = chunk_row(c, ok);
    const int left = t_end - t_begin - 16 * c;               // rows of the chunk within the sequence
    const char* k0 = kbase + row * stride;
    const char* v0 = vbase + row * stride;
#pragma unroll
    for (int i = 0; i < Lay::kVec; ++i) {
      const int r = lane / Lay::kRowLanes + kRowsAtOnce * i, ch = lane % Lay::kRowLanes;
      const uint32_t dk = dst + r * Lay::kRowBytes + ((ch ^ k_swizzle(r)) << 4);
      const uint32_t dv = dst + Lay::kChunkBytes / 2 + r * Lay::kRowBytes + ((ch ^ v_swizzle(r)) << 4);
      if (kWeights) {
        cp_async16(dk, k0 + r * stride, ok, policy);
        cp_async16(dv, v0 + r * stride, ok && r < left, policy);
      } else {
        cp_async16(dk, k0 + r * stride, ok);
        cp_async16(dv, v0 + r * stride, ok && r < left);
      }
    }
  };
  auto prefetch_step = [&](int c, int st) {                  // chunks c, c + kWarps, ...
#pragma unroll
    for (int u = 0; u < U; ++u) prefetch(c + u * kWarps, mine + st * Lay::kStageBytes + u * Lay::kChunkBytes);
    if (!kBf16 && lane < 2 * U) {                            // a lane a scale: K's and V's of each chunk
      bool ok;
      const size_t at = (chunk_row(c + (lane >> 1) * kWarps, ok) >> p.block_shift) * p.H_kv + kvh;
      float* to = &s_scale[warp][st][lane >> 1][lane & 1];
      if (ok) cp_async4(static_cast<uint32_t>(__cvta_generic_to_shared(to)), ((lane & 1) ? p.v_scales : p.k_scales) + at);
      else *to = 1.f;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < Lay::kStages - 1; ++i) prefetch_step(warp + i * kWarps * U, i);

  int end[NT][2];                                            // keys before it are seen by column 2 t4 + j
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = (hg0 + 8 * nt + 2 * t4 + j) % q_len;
      end[nt][j] = p.causal ? min(t_end, L - q_len + row + 1) : t_end;
    }

  float o[NT][8][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
  }

  int st = 0;
  for (int c = warp; c < n_chunks; c += kWarps * U) {
    __syncwarp();                                            // every lane has read the stage that is refilled now
    prefetch_step(c + (Lay::kStages - 1) * kWarps * U, st == 0 ? Lay::kStages - 1 : st - 1);
    cp_async_wait<Lay::kStages - 1>();
    __syncwarp();                                            // every lane's copies have landed
    const uint8_t* stage = ring + (warp * Lay::kStages + st) * Lay::kStageBytes;
    const int now = st;
    st = st == Lay::kStages - 1 ? 0 : st + 1;
    // K: rows g and g + 8, 16-byte pieces t4, t4 + 4, ...; V: piece g (and g + 8)
    // of rows 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
    uint4 kx[U][Lay::kVec], vx[U][Lay::kVec];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t* kc = stage + u * Lay::kChunkBytes;
      const uint8_t* vc = kc + Lay::kChunkBytes / 2;
#pragma unroll
      for (int i = 0; i < Lay::kVec / 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = g + 8 * e;
          kx[u][e * (Lay::kVec / 2) + i] =
              *reinterpret_cast<const uint4*>(kc + r * Lay::kRowBytes + (((4 * i + t4) ^ k_swizzle(r)) << 4));
        }
#pragma unroll
      for (int i = 0; i < Lay::kVec; ++i) {
        const int r = 2 * t4 + (i & 1) + 8 * ((i >> 1) & 1);
        vx[u][i] = *reinterpret_cast<const uint4*>(vc + r * Lay::kRowBytes + (((g + 8 * (i >> 2)) ^ v_swizzle(r)) << 4));
      }
    }
    int tok[U];
    bool page_ok[U];
    float2 scales[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int cu = c + u * kWarps;
      tok[u] = t_begin + 16 * cu;
      page_ok[u] = cu < n_chunks && s_pages[(tok[u] >> p.page_shift) - lp0] >= 0;
      scales[u] = kBf16 ? make_float2(1.f, 1.f) : *reinterpret_cast<const float2*>(s_scale[warp][now][u]);
      // A NaN value scale makes the output of every row that sees the block NaN.  Said
      // to O here, it reaches neither the other rows (P = 0 times NaN) nor the weights.
      if (!kBf16 && isnan(scales[u].y)) {                    // the same on every lane
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < J; ++j)
            if (tok[u] < end[nt][j]) {
#pragma unroll
              for (int i = 0; i < 8; ++i) o[nt][i][j] = o[nt][i][2 + j] = scales[u].y;
            }
        scales[u].y = 1.f;
      }
    }
    // S^T = K Q^T, in two chains of four steps
    float sc[U][NT][4], sd[U][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][nt][e] = sd[u][nt][e] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t* kw = reinterpret_cast<const uint32_t*>(kx[u]);
        uint32_t a0, a1, a2, a3;
        if (kBf16) {
          a0 = kw[2 * i], a2 = kw[2 * i + 1];
          a1 = kw[16 + 2 * i], a3 = kw[16 + 2 * i + 1];
        } else {
          codes_to_f16<kCache>(kw[i], a0, a2);
          codes_to_f16<kCache>(kw[8 + i], a1, a3);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816<!kBf16>((i & 1) ? sd[u][nt] : sc[u][nt], a0, a1, a2, a3, qb[nt][i][0], qb[nt][i][1]);
      }

    // scores of tokens g, g + 8 and heads 2 t4, 2 t4 + 1 in base-2 units
    bool passed = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float (&x)[4] = sc[u][nt];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float f = hm[nt][j] * scales[u].x;
          const int left = page_ok[u] ? end[nt][j] - tok[u] : 0;         // visible tokens of the chunk
          x[j] = g < left ? (x[j] + sd[u][nt][j]) * f : -INFINITY;
          x[2 + j] = g + 8 < left ? (x[2 + j] + sd[u][nt][2 + j]) * f : -INFINITY;
          passed = passed || fmaxf(x[j], x[2 + j]) > m[nt][j] + (Lay::kLift + 8.f);
        }
      }
      if (kWeights) {
        // [S, H_kv, tokens, group]; tokens past the sequence are not written
        float* lg = p.logits + (((size_t)s * p.H_kv + kvh) * p.logit_tokens + tok[u] + g) * group + hg0 + 2 * t4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool in = tok[u] + g + 8 * e < t_end;
            float* at = lg + (size_t)(8 * e) * group + 8 * nt;
            if ((group & 1) == 0) {
              if (in && 8 * nt + 2 * t4 < nh)
                *reinterpret_cast<float2*>(at) = make_float2(sc[u][nt][2 * e], sc[u][nt][2 * e + 1]);
            } else {
              if (in && 8 * nt + 2 * t4 < nh) at[0] = sc[u][nt][2 * e];
              if (in && 8 * nt + 2 * t4 + 1 < nh) at[1] = sc[u][nt][2 * e + 1];
            }
          }
      }
    }
    if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          float mx = fmaxf(sc[0][nt][j], sc[0][nt][2 + j]);
#pragma unroll
          for (int u = 1; u < U; ++u) mx = fmaxf(mx, fmaxf(sc[u][nt][j], sc[u][nt][2 + j]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (mx > m[nt][j] + (Lay::kLift + 8.f)) {
            const float mn = mx - Lay::kLift;
            const float a = ex2(m[nt][j] - mn);              // from -inf: 0
            m[nt][j] = mn;
            l[nt][j] *= a;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[nt][i][j] *= a;
              o[nt][i][2 + j] *= a;
            }
          }
        }
    }
    // P^T as the B operand: column n = head, rows = the chunk's tokens
    uint32_t pb[U][NT][2], plo[kBf16 ? NT : 1][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float pr[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float ref = m[nt][j] == -INFINITY ? 0.f : m[nt][j];
          pr[j] = ex2(sc[u][nt][j] - ref);
          pr[2 + j] = ex2(sc[u][nt][2 + j] - ref);
          l[nt][j] += pr[j] + pr[2 + j];
        }
        if (kBf16) {                                         // what bf16 leaves of P goes in a second product
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t hi = pack_bf16x2(pr[2 * e], pr[2 * e + 1]);
            pb[u][nt][e] = transpose8x8(hi);
            plo[kBf16 ? nt : 0][e] =
                transpose8x8(pack_bf16x2(pr[2 * e] - bf16lo(hi), pr[2 * e + 1] - bf16hi(hi)));
          }
        } else {
          pb[u][nt][0] = transpose8x8(pack_f16x2(pr[0], pr[1]));
          pb[u][nt][1] = transpose8x8(pack_f16x2(pr[2], pr[3]));
        }
      }
    }
    // O^T += vs V^T P^T
    if (kBf16) {
      const uint32_t* vw = reinterpret_cast<const uint32_t*>(vx[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {                          // word i of rows 2t, 2t+1, 2t+8, 2t+9
        const int b0 = (i >> 2) * 16 + (i & 3);
        const uint32_t r0 = vw[b0], r1 = vw[b0 + 4], r2 = vw[b0 + 8], r3 = vw[b0 + 12];
        const uint32_t a0 = __byte_perm(r0, r1, 0x5410), a1 = __byte_perm(r0, r1, 0x7632);
        const uint32_t a2 = __byte_perm(r2, r3, 0x5410), a3 = __byte_perm(r2, r3, 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816<false>(o[nt][i], a0, a1, a2, a3, pb[0][nt][0], pb[0][nt][1]);
          mma16816<false>(o[nt][i], a0, a1, a2, a3, plo[nt][0], plo[nt][1]);
        }
      }
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // bytes 4w .. 4w+3 of rows (2t, 2t+1) and (2t+8, 2t+9), interleaved by row
          const uint32_t* vw = reinterpret_cast<const uint32_t*>(vx[u]);
          const float vs = scales[u].y;
          uint32_t a[4], b[4];
          codes_to_f16<kCache>(__byte_perm(vw[w], vw[4 + w], 0x5140), a[0], a[1]);
          codes_to_f16<kCache>(__byte_perm(vw[w], vw[4 + w], 0x7362), a[2], a[3]);
          codes_to_f16<kCache>(__byte_perm(vw[8 + w], vw[12 + w], 0x5140), b[0], b[1]);
          codes_to_f16<kCache>(__byte_perm(vw[8 + w], vw[12 + w], 0x7362), b[2], b[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {                    // tile 2w + e: head dims 16 g + 4w + 2e, + 1
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<true>(acc, a[2 * e], a[2 * e + 1], b[2 * e], b[2 * e + 1], pb[u][nt][0], pb[u][nt][1]);
#pragma unroll
              if (kOne) {
                float (&oo)[4] = o[nt][2 * w + e];
                unf2(fma2(f2(vs, vs), f2(acc[0], acc[2]), f2(oo[0], oo[2])), oo[0], oo[2]);
              } else {
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                  float* oo = &o[nt][2 * w + e][q];
                  unf2(fma2(f2(vs, vs), f2(acc[q], acc[q + 1]), f2(oo[0], oo[1])), oo[0], oo[1]);
                }
              }
            }
        }
    }
  }
  cp_async_wait<0>();
  __syncthreads();                                           // the rings become the merge buffer

  // merge the warps
  float (*s_o)[kHeads][D] = reinterpret_cast<float (*)[kHeads][D]>(ring);
  static_assert(kWarps * kHeads * D * 4 <= Lay::kRingBytes, "merge buffer");
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float v = l[nt][j];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      const int head = 8 * nt + 2 * t4 + j;
      if (g == 0) {
        s_m[warp][head] = m[nt][j];
        s_l[warp][head] = v;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = 2 * i;                                 // of this lane's 16 head dims
        const int d = kBf16 ? (e >> 3) * 64 + 8 * g + (e & 7) : 16 * g + e;
        *reinterpret_cast<float2*>(&s_o[warp][head][d]) = make_float2(o[nt][i][j], o[nt][i][2 + j]);
      }
    }
  __syncthreads();
  for (int i = tid; i < nh * D; i += kThreads) {
    const int r = i / D, col = i % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][r]);
    float acc = 0.f, lsum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float wt = s_m[w][r] == -INFINITY && M == -INFINITY ? 1.f : ex2(s_m[w][r] - M);
      acc = fmaf(wt, s_o[w][r][col], acc);
      lsum = fmaf(wt, s_l[w][r], lsum);
    }
    const size_t sh = (size_t)s * p.H + h0 + r;
    if (nsplit == 1)
      p.out[sh * D + col] = __float2bfloat16_rn(lsum == 0.f ? 0.f : acc / lsum);
    else
      p.ws_o[(sh * p.max_splits + split) * D + col] = acc;
    if (col == 0 && (kWeights || nsplit > 1)) p.ws_ml[sh * p.max_splits + split] = make_float2(M, lsum);
  }
}

// (max, sum) of all splits of one (sequence, head), by a whole warp.
PKV_DEVINLINE void merge_ml(const float2* ml, int nsplit, int lane, float& M, float& lsum) {
  M = -INFINITY;
  for (int j = lane; j < nsplit; j += 32) M = fmaxf(M, ml[j].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  lsum = 0.f;
  for (int j = lane; j < nsplit; j += 32) {
    const float2 v = ml[j];
    lsum = fmaf(v.x == -INFINITY && M == -INFINITY ? 1.f : ex2(v.x - M), v.y, lsum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
}

// Splits -> output: p.merge_warps warps per (sequence, head) take its splits in
// turn (one warp walks 30 splits in 8 dependent rounds of loads); lane i owns head
// dims 4i .. 4i+3.
constexpr int kMergeWarps = 8;
PKV_DEVINLINE void merge_rows(const CacheAttnParams& p, int cta) {
  __shared__ float4 s_acc[kMergeWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mw = p.merge_warps, part = warp % mw;
  const long long sh = (long long)cta * (kMergeWarps / mw) + warp / mw;
  const int cap = p.max_seq_len;                   // the table holds at least as many tokens (checked by the host)
  const bool row = sh < (long long)p.num_seqs * p.H;
  const int L = row ? max(0, min(p.seq_lens[sh / p.H], cap)) : 0;
  const int nsplit = (L + p.split_tokens - 1) / p.split_tokens;
  const bool live = nsplit > 1;                     // one split: written by the split kernel
  float M = -INFINITY, lsum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    const float2* ml = p.ws_ml + sh * p.max_splits;
    merge_ml(ml, nsplit, lane, M, lsum);
    const float4* po = reinterpret_cast<const float4*>(p.ws_o + sh * p.max_splits * D) + lane;
#pragma unroll 4
    for (int j = part; j < nsplit; j += mw) {
      const float mj = ml[j].x;
      const float w = mj == -INFINITY && M == -INFINITY ? 1.f : ex2(mj - M);
      const float4 x = po[(size_t)j * (D / 4)];
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
    }
  }
  s_acc[warp][lane] = acc;
  __syncthreads();
  if (!live || part) return;
  for (int i = 1; i < mw; ++i) {
    const float4 x = s_acc[warp + i][lane];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  const bool none = lsum == 0.f;
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(p.out + sh * D) + 2 * lane;
  out[0] = __floats2bfloat162_rn(none ? 0.f : acc.x / lsum, none ? 0.f : acc.y / lsum);
  out[1] = __floats2bfloat162_rn(none ? 0.f : acc.z / lsum, none ? 0.f : acc.w / lsum);
}

constexpr int kWeightThreads = 256;
constexpr int kMaxGroup = 256;                    // query rows per kv head

// Groups of 4 and 8 rows: a thread a token, four tokens' scores and weights in
// flight (e4m3, 8 kv heads; 8 sequences of 2000 to 30001 tokens, 4 rows: 87 us
// with one token a thread at a time, 82 so; 64 of 512 to 8192, 8 rows: 151 -> 148).
template <int kVec>
PKV_DEVINLINE void thread_weights(const float* lg, const float* s_lse, float* w, int t0, int t_end) {
  constexpr int kTokens = 4;
  float4 e[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) e[i] = reinterpret_cast<const float4*>(s_lse)[i];
  const float4* x = reinterpret_cast<const float4*>(lg);
  for (int t1 = t0 + threadIdx.x; t1 < t_end; t1 += kTokens * kWeightThreads) {
    float4 v[kTokens][kVec];
    float old[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      const int t = t1 + u * kWeightThreads;
      if (t < t_end) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[u][i] = x[(size_t)t * kVec + i];
        old[u] = w[t];
      }
    }
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      const int t = t1 + u * kWeightThreads;
      if (t < t_end) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          sum += (ex2(v[u][i].x - e[i].x) + ex2(v[u][i].y - e[i].y)) +
                 (ex2(v[u][i].z - e[i].z) + ex2(v[u][i].w - e[i].w));
        w[t] = old[u] + sum;
      }
    }
  }
}

// Scores -> weights, for a range of a sequence's tokens and a kv head.  p.token_lanes
// lanes share a token's scores (32 of them where a kv head has that many rows) and
// their sums are added up in one order; a token's weight is the sum over the
// group's rows of 2^(x - lse).
PKV_DEVINLINE void range_weights(const CacheAttnParams& p, int range, int kvh, int s) {
  __shared__ __align__(16) float s_lse[kMaxGroup];
  const int cap = p.max_seq_len;                   // the table holds at least as many tokens (checked by the host)
  const int L = max(0, min(p.seq_lens[s], cap));
  const int t0 = range * p.range_tokens;
  if (t0 >= L) return;
  const int group = p.H / p.H_kv;
  const int nsplit = (L + p.split_tokens - 1) / p.split_tokens;
  const float2* ml = p.ws_ml + ((size_t)s * p.H + kvh * group) * p.max_splits;
  // no visible key: every score is -inf, and 2^(-inf - 0) = 0
  bool broken = false;                            // this thread's row saw a NaN
  if (group <= kWeightThreads / 32) {             // a warp a row
    const int h = threadIdx.x >> 5;
    if (h < group) {
      float M, lsum;
      merge_ml(ml + (size_t)h * p.max_splits, nsplit, threadIdx.x & 31, M, lsum);
      if ((threadIdx.x & 31) == 0) s_lse[h] = lsum == 0.f ? 0.f : M + log2f(lsum);
      broken = isnan(lsum);
    }
  } else if (threadIdx.x < group) {               // a thread a row
    const float2* row = ml + (size_t)threadIdx.x * p.max_splits;
    float M = -INFINITY, lsum = 0.f;
#pragma unroll 8
    for (int j = 0; j < nsplit; ++j) M = fmaxf(M, row[j].x);
#pragma unroll 8
    for (int j = 0; j < nsplit; ++j) {
      const float2 v = row[j];
      lsum = fmaf(v.x == -INFINITY && M == -INFINITY ? 1.f : ex2(v.x - M), v.y, lsum);
    }
    s_lse[threadIdx.x] = lsum == 0.f ? 0.f : M + log2f(lsum);
    broken = isnan(lsum);
  }
  const bool some_broken = __syncthreads_or(broken);
  const size_t sk = (size_t)s * p.H_kv + kvh;
  const float* lg = p.logits + sk * p.logit_tokens * group;
  float* w = p.weights + sk * p.weights_stride;
  const int t_end = min(L, t0 + p.range_tokens);
  if (some_broken) {
    // A NaN row gives NaN to the keys that it sees, and nothing to the others, whose
    // score of -inf minus NaN would be NaN too: what a key is seen by is looked up.
    for (int t = t0 + threadIdx.x; t < t_end; t += kWeightThreads) {
      const int phys = p.block_table[(size_t)s * p.max_pages + (t >> p.page_shift)];
      if (phys < 0 || phys >= p.num_pages) continue;
      float sum = 0.f;
      for (int h = 0; h < group; ++h)
        if (!p.causal || t <= L - p.q_len + h % p.q_len) sum += ex2(lg[(size_t)t * group + h] - s_lse[h]);
      w[t] += sum;
    }
    return;
  }
  if (group == 8) return thread_weights<2>(lg, s_lse, w, t0, t_end);
  if (group == 4) return thread_weights<1>(lg, s_lse, w, t0, t_end);
  const int lanes = p.token_lanes, mine = threadIdx.x % lanes;
  for (int t1 = t0; t1 < t_end; t1 += kWeightThreads / lanes) {              // a warp's trip count is uniform
    const int t = t1 + threadIdx.x / lanes;
    float sum = 0.f;
    if (t < t_end) {
      const float* x = lg + (size_t)t * group;
      if ((group & 3) == 0) {
#pragma unroll 2
        for (int h = 4 * mine; h < group; h += 4 * lanes) {
          const float4 v = *reinterpret_cast<const float4*>(x + h);
          const float4 e = *reinterpret_cast<const float4*>(s_lse + h);
          sum += (ex2(v.x - e.x) + ex2(v.y - e.y)) + (ex2(v.z - e.z) + ex2(v.w - e.w));
        }
      } else {
        for (int h = mine; h < group; h += lanes) sum += ex2(x[h] - s_lse[h]);
      }
    }
    for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (t < t_end && mine == 0) w[t] += sum;
  }
}

// What follows the split kernel, in one launch: the first p.merge_ctas CTAs merge
// splits; the others take the weights' ranges.
static_assert(kMergeWarps * 32 == kWeightThreads, "one block size");
__global__ void __launch_bounds__(kWeightThreads) cache_finish_kernel(const CacheAttnParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x < p.merge_ctas) {
    merge_rows(p, blockIdx.x);
    return;
  }
  const int ranges = (p.max_seq_len + p.range_tokens - 1) / p.range_tokens;
  const int i = blockIdx.x - p.merge_ctas;
  const int pair = i / ranges;
  range_weights(p, i - pair * ranges, pair % p.H_kv, pair / p.H_kv);
}

template <int kCache, int NT, bool kWeights, bool kOne>
cudaError_t launch_split(const CacheAttnParams& p, dim3 grid, cudaStream_t stream) {
  // The shared-memory limit is an attribute per device; host threads may get
  // here at once, so the once-per-device record is kept under a lock.
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(cache_decode_kernel<kCache, NT, kWeights, kOne>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<kCache>::kRingBytes);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  cache_decode_kernel<kCache, NT, kWeights, kOne><<<grid, kThreads, Layout<kCache>::kRingBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int kCache, bool kWeights>
cudaError_t launch_decode(const CacheAttnParams& p, cudaStream_t stream) {
  const int group = p.H / p.H_kv;
  const int heads = group > 8 ? 16 : 8;
  const dim3 grid(p.H_kv * ((group + heads - 1) / heads), p.max_splits, p.num_seqs);
  if (group > 8) return launch_split<kCache, 2, kWeights, false>(p, grid, stream);
  return group > 1 ? launch_split<kCache, 1, kWeights, false>(p, grid, stream)
                   : launch_split<kCache, 1, kWeights, true>(p, grid, stream);
}

// The kernel after the split kernel, as its programmatic dependent: it may be
// scheduled while the split kernel drains and waits for its results itself.
template <typename Kernel>
cudaError_t launch_after(Kernel kernel, dim3 grid, int threads, const CacheAttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

void cache_decode_plan(int num_seqs, int H, int H_kv, int max_seq_len, int page_size, int* split_tokens,
                       int* max_splits) {
  const int group = H / H_kv;
  const int heads = group > 8 ? 16 : 8;
  const long long pairs = (long long)num_seqs * H_kv * ((group + heads - 1) / heads);
  // At least what the four warps work on at once: two chunks of 16 tokens each.
  const int unit = 128 < page_size ? page_size : 128;
  int st = unit;
  // Short contexts: one split, as the merge's launch costs more than the splits
  // save (one sequence of 437 tokens, 8 kv heads: 10.4 us in 7 splits, 8.3 in one).
  if (max_seq_len <= kOneSplit) st = kOneSplit;
  // Little work: as many splits as run at once, three CTAs an SM (one sequence of
  // 32000 tokens, 8 kv heads: 41 us in 128-token splits, four turns and a half; 23 in one).
  const long long turn = (pairs * max_seq_len + 148 * 3 - 1) / (148 * 3);
  if (st < turn && turn <= 1024) st = (int)((turn + unit - 1) / unit * unit);
  // Double while at least 8 CTAs per SM remain.  A split writes (and the merge
  // reads) 512 bytes per query head: with few heads that is little, and shorter
  // splits balance ragged lengths better (64 sequences x 32 heads, int8: 441 us at
  // 1024 tokens, 455 at 4096; 16 long ones x 8 heads a kv head: 141 and 137 us).
  const int most = group >= 4 ? kMaxSplitTokens : 1024;
  while (turn > 1024 && st < most && pairs * ((max_seq_len + 2LL * st - 1) / (2LL * st)) >= 148LL * 8) st *= 2;
  while (((long long)max_seq_len + st - 1) / st > kMaxSplits && st < kMaxSplitTokens) st *= 2;
  *split_tokens = st;
  *max_splits = (int)(((long long)max_seq_len + st - 1) / st);
}

cudaError_t launch_cache_decode(const CacheAttnParams& p, cudaStream_t stream) {
  if (p.max_splits > 65535) return cudaErrorNotSupported;           // sequences beyond 2^28 tokens
  const bool w = p.weights != nullptr;
  CacheAttnParams q = p;                            // the finish kernel's
  q.merge_ctas = 0;
  if (p.max_splits > 1) {
    q.merge_warps = 1;                              // about four splits a warp
    while (q.merge_warps < kMergeWarps && q.merge_warps * 4 < p.max_splits) q.merge_warps *= 2;
    const int rows = kMergeWarps / q.merge_warps;
    const long long n = ((long long)p.num_seqs * p.H + rows - 1) / rows;
    if (n > 0x3fffffffLL) return cudaErrorNotSupported;
    q.merge_ctas = (int)n;
  }
  long long ctas = q.merge_ctas;
  if (w) {
    const int group = p.H / p.H_kv;
    q.token_lanes = 1;                              // at most 8 scores a lane, while lanes last
    while (q.token_lanes < 32 && q.token_lanes * 8 < group) q.token_lanes *= 2;
    q.range_tokens = q.token_lanes > 8 ? 128 : 1024 / q.token_lanes;
    ctas += (((long long)p.max_seq_len + q.range_tokens - 1) / q.range_tokens) * p.H_kv * p.num_seqs;
  }
  if (ctas > 0x7fffffffLL) return cudaErrorNotSupported;            // before anything is launched
  cudaError_t e;
  if (p.cache_dtype == PKV_I8)
    e = w ? launch_decode<PKV_I8, true>(p, stream) : launch_decode<PKV_I8, false>(p, stream);
  else if (p.cache_dtype == PKV_E4M3)
    e = w ? launch_decode<PKV_E4M3, true>(p, stream) : launch_decode<PKV_E4M3, false>(p, stream);
  else
    e = w ? launch_decode<PKV_BF16, true>(p, stream) : cudaErrorNotSupported;
  if (e != cudaSuccess || ctas == 0) return e;
  return launch_after(cache_finish_kernel, dim3((unsigned)ctas), kWeightThreads, q, stream);
}

}  // namespace pkv
