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

// e4m3 pair <-> f16 pair / f32 pair (exact; RNE on the way to e4m3).
PKV_DEVINLINE uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}"
      : "=r"(r) : "r"(two_codes));
  return r;
}
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

// The same from an approximate quotient q (relative error <= 2^-22): q decides
// unless it lies next to a tie (or, for e4m3, in the subnormal range), where
// `exact` is asked.  That is about one element in 10^5 for int8 and one in
// 10^4 for e4m3, so the float64 division costs nothing on average.
template <int kCache, typename Exact>
PKV_DEVINLINE uint32_t code_of(float q, Exact exact) {
  if (kCache == PKV_I8) {
    const float n = rintf(q);
    if (fabsf(fabsf(q - n) - 0.5f) < 1e-4f) return exact();
    return static_cast<uint32_t>(static_cast<int>(n)) & 0xffu;
  }
  // 20 mantissa bits are dropped: a tie has 0x80000 there
  const uint32_t b = __float_as_uint(q);
  const bool near_tie = ((b + 8u - 0x80000u) & 0xfffffu) <= 16u;
  if (near_tie || (fabsf(q) < 0.015625f && q != 0.f)) return exact();
  return f32_to_e4m3(q);
}

// Value of a code as float32 (exact).
template <int kCache>
PKV_DEVINLINE float code_value(uint32_t code) {
  if (kCache == PKV_I8) return static_cast<float>(static_cast<int8_t>(code));
  const uint32_t h = e4m3x2_to_f16x2(code & 0xffu);
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// Four codes (one word) from scale s_old to scale s_new >= s_old;
// ratio = s_old / s_new rounded to float32.
template <int kCache>
PKV_DEVINLINE uint32_t requantize4(uint32_t w, float ratio, float s_old, float s_new) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float c = code_value<kCache>((w >> (8 * i)) & 0xffu);
    const uint32_t code = code_of<kCache>(c * ratio, [&] {
      return code_exact<kCache>(static_cast<double>(c) * static_cast<double>(s_old),
                                static_cast<double>(s_new));
    });
    r |= code << (8 * i);
  }
  return r;
}

}  // namespace pkv
