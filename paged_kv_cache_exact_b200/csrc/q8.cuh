// The 8-bit cache's number formats: what a code stands for, and the exact
// rounding of a quotient to a code.
//
//   value(t, h, c) = code(t, h, c) * scale(block of t, h)
//
// Codes are int8 in [-127, 127] or e4m3 (1 sign, 4 exponent bits with bias 7,
// 3 mantissa bits, largest 448, no infinities).  A scale is a float32 number
// >= 2^-126, or NaN for a block that took in a NaN or an infinity.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

template <int kCache> PKV_DEVINLINE constexpr float code_max() {
  return kCache == PKV_I8 ? 127.f : 448.f;
}

// Nearest e4m3 code (RNE, saturating).
PKV_DEVINLINE uint32_t f32_to_e4m3(float x) {
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %1, %2;\n\tcvt.u32.u16 %0, c;\n\t}"
      : "=r"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

// The code nearest to the real quotient num / den, ties to even.  `num` is a
// product that float64 holds exactly (a row's element, or a code times its
// old scale) and den a float32 number, so num / den differs from a tie by at
// least 2^-35 of itself or not at all: one float64 division decides.
template <int kCache>
__device__ __noinline__ uint32_t code_exact(double num, double den) {
  const double y = num / den;
  if (kCache == PKV_I8) {
    const double n = fmin(fmax(rint(y), -127.0), 127.0);
    return static_cast<uint32_t>(static_cast<int>(n)) & 0xffu;
  }
  // to float32 by round-to-odd, after which the rounding to e4m3 is the only one
  float f = __double2float_rz(y);
  if (static_cast<double>(f) != y) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f32_to_e4m3(f);
}

// Four codes (a word) from approximate quotients q (relative error <= 2^-22): q
// decides unless it lies next to a tie (or, for e4m3, in the subnormal range),
// where all four ask `exact(i)`.  That is about one element in 10^5 for int8 and
// one in 10^4 for e4m3, so the float64 division costs nothing on average.  int8
// rounds by adding 1.5 * 2^23, which leaves the integer in the low mantissa bits:
// conversion instructions run at a quarter of the rate.
template <int kCache, typename Exact>
PKV_DEVINLINE uint32_t codes_of4(const float (&q)[4], Exact exact) {
  bool near_tie;
  uint32_t word;
  if (kCache == PKV_I8) {
    float y[4], off = 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = q[i] + 12582912.f;
      off = fminf(off, fabsf(fabsf(q[i] - (y[i] - 12582912.f)) - 0.5f));
    }
    near_tie = off < 1e-4f;
    word = __byte_perm(__byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x0040),
                       __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x0040), 0x5410);
  } else {
    uint32_t tie = 0xffffffffu, small = 0xffffffffu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = __float_as_uint(q[i]);
      tie = min(tie, (b + 8u - 0x80000u) & 0xfffffu);                // 20 bits are dropped: a tie has 0x80000 there
      small = min(small, (b & 0x7fffffffu) - 1u);                    // zero is no trouble
    }
    near_tie = tie <= 16u || small < 0x3c800000u - 1u;               // 2^-6
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(word) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]));
  }
  if (near_tie) {
    word = 0;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) word |= exact(i) << (8 * i);
  }
  return word;
}

// The four values of a word of codes as float32 (exact).
template <int kCache>
PKV_DEVINLINE void values_of4(uint32_t w, float (&x)[4]) {
  if (kCache == PKV_I8) {
    const uint32_t u = w ^ 0x80808080u;                              // code + 128, in the mantissa of 2^23 + u
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.f;
  } else {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x[0]), "=f"(x[1]) : "r"(lo));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x[2]), "=f"(x[3]) : "r"(hi));
  }
}

// Four codes (one word) from scale s_old to scale s_new >= s_old;
// ratio = s_old / s_new rounded to float32.
template <int kCache>
PKV_DEVINLINE uint32_t requantize4(uint32_t w, float ratio, float s_old, float s_new) {
  float c[4], q[4];
  values_of4<kCache>(w, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = c[i] * ratio;
  return codes_of4<kCache>(q, [&](int i) {
    const float v = i == 0 ? c[0] : i == 1 ? c[1] : i == 2 ? c[2] : c[3];
    return code_exact<kCache>(static_cast<double>(v) * static_cast<double>(s_old), static_cast<double>(s_new));
  });
}

}  // namespace pkv
