// 8-bit floating-point blocks of 128 with one power-of-two scale (UE8M0: a byte b standing for
// 2^(b - 127)), shared by the FP8 linear layer and the 8-bit optimizer states.
//
// A block's exponent is the least e >= -127 with amax <= 1.75 * 2^(e + kTop): kTop = 8 for E4M3
// (largest value 448), 15 for E5M2 (57344); both formats' largest values have the mantissa 1.75, so
// one integer rule on the bit pattern of amax serves both.  A power-of-two scale makes x * 2^-e
// exact, so a code depends on x and e alone (no rounding of a reciprocal in between), costs
// no precision inside a binade (the formats are floating), and is what the tensor core multiplies in.
#pragma once
#include <stdint.h>

namespace nvfp4 {

constexpr int kFp8Block = 128;
constexpr int kTopE4M3 = 8, kTopE5M2 = 15;

// The scale byte of a block from the FP32 bit pattern of its largest finite magnitude.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax_bits, int top) {
  const int e = static_cast<int>(amax_bits >> 23) - top + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));  // at most 254 - 8 + 1
}
// 2^(b - 127); byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float fp8_scale_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b << 23);
}
// 2^(127 - b) for b <= 247, the largest byte a finite amax gives.
__device__ __forceinline__ float fp8_scale_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Two codes to FP32 (low byte first); both conversions are exact.
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
  float2 r;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return f16x2_to_f32x2(h);
}
__device__ __forceinline__ float2 e5m2x2_to_f32(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return f16x2_to_f32x2(h);
}

}  // namespace nvfp4
