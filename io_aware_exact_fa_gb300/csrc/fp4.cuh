// 4-bit rows: groups of 16 neighbouring elements with one scale byte and 16 e2m1
// codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; element 2i in the lower
// half of byte i).
//
// A scale byte is the upper byte of an f16 without its sign: 5 exponent bits (bias
// 15) and 3 mantissa bits. A code has two significant bits and a scale four, so
// code * scale is exact in f16 (6 * 10240 is the largest, 2^-18 the least) and in
// bf16, and turning bytes into a product's operands is one conversion and one
// packed multiplication for each pair.
#pragma once

#include <cstdint>

#include "fa_ptx.cuh"

namespace fa {

constexpr float FP4_SCALE_MAX = 10240.f;          // 6 * 10240 < 65504, the largest f16
constexpr float FP4_SCALE_MIN = 1.f / 131072.f;   // 2^-17, the least scale byte
constexpr unsigned FP4_SCALE_NAN = 0xffu;

// Eight codes to four pairs of f16, in order.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t codes, uint32_t (&y)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
      : "r"(codes));
}

__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Byte `i` of `bytes` as a scale, in both halves of a pair.
template <int I>
__device__ __forceinline__ uint32_t fp4_scale2(uint32_t bytes) {
  return __byte_perm(bytes, 0u, 0x4040 | I * 0x0101) << 7;
}
// Two scale bytes (0 .. 255) as a pair.
__device__ __forceinline__ uint32_t fp4_scale_pair(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x5410) << 7; }

// The scale of a group whose largest bf16 magnitude has the bits `amax`: max / 6 rounded to nearest even with three
// mantissa bits, within [2^-17, 10240]; 0 for a group of zeros, NaN where an element is infinite or NaN. `inv` is what the
// elements are multiplied with.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax, float& inv) {
  inv = 0.f;
  if (amax >= 0x7f80u) return FP4_SCALE_NAN;
  const float y = __fdiv_rn(__uint_as_float(amax << 16), 6.f);
  // from 2^-14 on three mantissa bits, below the multiples of 2^-17 (the spacing of fp32 at 64). One rounding, of the
  // correctly rounded quotient: a bf16 value is never so close to 6 times a border that the quotient would round onto it.
  const uint32_t u = __float_as_uint(y);
  const float s = y >= 6.103515625e-5f ? __uint_as_float((u + 0x7ffffu + ((u >> 20) & 1u)) & ~0xfffffu)
                                       : __fadd_rn(__fadd_rn(y, 96.f), -96.f);
  const float c = fminf(fmaxf(s, FP4_SCALE_MIN), FP4_SCALE_MAX);
  if (amax == 0u) return 0u;
  inv = __frcp_rn(c);
  uint16_t h;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(h) : "f"(c));
  return static_cast<uint32_t>(h) >> 7;
}

// Eight bf16 values (pairs in order) to eight codes. x * inv is off from x / s by less than 2^-23 of it, and x / s (eight
// significant bits over four) is a border between two codes or at least 2^-10 away from it (255 2^-7 over 8
// from 1/4; every pair was looked at): rounding to a multiple of 2^-11 first (the spacing of fp32 at 6144) puts it back on
// the border, where the tie goes to the even code, and leaves the others on their side.
__device__ __forceinline__ uint32_t fp4_codes8(uint4 x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const uint64_t i2 = f2pack(inv, inv), up = f2pack(6144.f, 6144.f), down = f2pack(-6144.f, -6144.f);
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f2unpack(fadd2(ffma2(f2pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), i2, up), down), y[2 * i],
             y[2 * i + 1]);
  uint32_t c;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(c)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return c;
}

// Bits of the largest magnitude among eight bf16 values (infinities and NaN above all others).
__device__ __forceinline__ uint32_t bf16x8_amax_bits(uint4 x) {
  constexpr uint32_t MAG = 0x7fff7fffu;
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & MAG, x.y & MAG), __vmaxu2(x.z & MAG, x.w & MAG));
  return max(m & 0xffffu, m >> 16);
}

}  // namespace fa
