// Pages in 8 bits: E4M3 codes with a power-of-two scale for each block of 32
// tokens of a head.
#pragma once

#include <stdint.h>

namespace lynx {

// scale bytes s (the scale is 2^(s - 127)) that a block may have: what the codes stand for
// and that times 2^-64 are then BF16 numbers of full precision
constexpr int kScaleLo = 74, kScaleHi = 198;
constexpr int kScaleBytes = 16;   // of a page: the blocks of its keys, then of its values

#ifdef __CUDACC__
namespace {

// the scale of a byte; one outside kScaleLo..kScaleHi (of a block that nothing was written
// to) counts as the nearest
__device__ __forceinline__ float scale_of(int byte) {
  return __uint_as_float((uint32_t)min(max(byte, kScaleLo), kScaleHi) << 23);
}

// a factor of scores as a positive finite number: -inf (a masked score) times it is -inf, and 0 is 0
__device__ __forceinline__ float clamped(float f) { return fminf(fmaxf(f, 1.17549435e-38f), 3.402823466e38f); }

// the smallest scale byte with top <= 448 * 2^(s - 127); top = 1.m * 2^e is at most
// 1.75 * 2^(8 + s - 127) from s = e + 119 on, or from the one behind it for 1.m > 1.75
__device__ __forceinline__ int scale_byte(float top) {
  const int s = (int)((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 8;
  return min(max(s, kScaleLo), kScaleHi);
}

// two E4M3 codes (bits 0-7 and 8-15) as two FP16 values, exactly
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
  uint32_t d;
  asm("{\n\t.reg .b16 c, x;\n\tmov.b32 {c, x}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(d) : "r"(codes));
  return d;
}
// the same of bits 16-23 and 24-31
__device__ __forceinline__ uint32_t f16x2_of_high(uint32_t codes) {
  uint32_t d;
  asm("{\n\t.reg .b16 c, x;\n\tmov.b32 {x, c}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(d) : "r"(codes));
  return d;
}

}  // namespace
#endif

}  // namespace lynx
