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

// Exact rounding of a quotient num / den to a code.  An approximate quotient q
// (relative error <= 2^-22) finds the tie h nearest to it, the point half way
// between two neighbouring codes, and the sign of num - h * den says on which side
// of h the quotient lies:
//
// * ties are common, not rare: a scale is amax / qmax with amax a bf16 number, so
//   quotients of bf16 elements are ratios of small integers;
// * h has at most 9 significant bits, so near a tie num - h * den is exact in one
//   fused multiply-add (and one more term where num itself is the product of a
//   code and its old scale), and elsewhere its sign is not in doubt.
//
// h, moved a little to the quotient's side, is then rounded to nearest even.
// `residual(i, h)` has the sign of num_i - h * den.
template <int kCache, typename Residual>
PKV_DEVINLINE float settle_half(float q, int i, Residual residual) {
  // int8, or e4m3's subnormal codes in units of 2^-9: ties are halves
  const float unit = kCache == PKV_I8 ? 1.f : 0.001953125f;
  const float v = kCache == PKV_I8 ? q : q * 512.f;
  const float n = (v + 12582912.f) - 12582912.f;                     // nearest integer
  const float half = n + copysignf(0.5f, v - n);
  const float r = residual(i, half * unit);
  return (half + (r == 0.f ? 0.f : copysignf(0.0009765625f, r))) * unit;
}

// Four codes (a word) from approximate quotients.
template <int kCache, typename Residual>
PKV_DEVINLINE uint32_t codes_of4(float (&q)[4], Residual residual) {
  uint32_t word;
  if (kCache == PKV_I8) {
    // Few blocks have ties (127 is a prime): look for them first.  Rounding adds
    // 1.5 * 2^23, which leaves the integer in the low mantissa bits: conversion
    // instructions run at a quarter of the rate.
    float off = 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      off = fminf(off, fabsf(fabsf(q[i] - ((q[i] + 12582912.f) - 12582912.f)) - 0.5f));
    if (off < 4e-5f) {                                               // 127 * 2^-22 = 3.03e-5
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = settle_half<kCache>(q[i], i, residual);
    }
    uint32_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __float_as_uint(q[i] + 12582912.f);
    word = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
  } else {
    // A tie has 0x80000 in the 20 mantissa bits that are dropped: the one in q's
    // own cell decides every element, so there is nothing to look for.
    float x[4], least = fabsf(q[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float h = __uint_as_float((__float_as_uint(q[i]) & 0xfff00000u) | 0x80000u);
      const float r = residual(i, h);
      x[i] = h + (r == 0.f ? 0.f : copysignf(h * 9.5367432e-7f, r));
      least = fminf(least, fabsf(q[i]));
    }
    if (least < 0.015625f) {                                         // below 2^-6 codes are 2^-9 apart
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (fabsf(q[i]) < 0.015625f) x[i] = settle_half<kCache>(q[i], i, residual);
    }
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(word) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
  }
  return word;
}

// Scales below 2^-64 (and what they divide) are multiplied by 2^64 first, so that
// no residual is a subnormal number.
constexpr float kTinyScale = 5.42101086e-20f, kTinyLift = 1.8446744e19f;   // 2^-64, 2^64

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
  const float lift = s_new < kTinyScale ? kTinyLift : 1.f;
  const float a = s_old * lift, b = s_new * lift;
  float c[4], q[4];
  values_of4<kCache>(w, c);
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = c[i] * ratio;
  return codes_of4<kCache>(q, [&](int i, float h) {
    const float v = c[i], p = v * a;
    return fmaf(-h, b, p) + fmaf(v, a, -p);                          // p is rounded; its error is exact
  });
}

}  // namespace pkv
