// MX scale rule on fp32 values (blocks of 32 share 2^E, elements are e4m3 of
// v * 2^-E), for the kernels that quantize what they compute.
#pragma once

#include "common.cuh"

namespace fp8bw {

// The rule depends on a block's amax only through one small integer, so
// blocks reduce that integer instead of the amax.  With amax = 1.m * 2^(ef -
// 127) and 448 = 1.75 * 2^8:
//   RCEIL: E = ef - 135, plus one where 1.m > 1.75 -- the carry out of
//          m + 0x1FFFFF;     FLOOR: E = ef - 135
// so t = (bits(amax) + round) >> 23 is E + 135.  It grows with amax, and the
// clamp E >= -127 is t >= 8.  The largest t of a finite amax is 255, to which
// infinities and NaN (256 with some payloads) are clamped.  The E8M0 byte is
// t - 8, and 2^-E has the biased exponent 262 - t, in [7, 254]: a normal
// number.  mx_tile.cuh has the rule for two blocks at a time.
__device__ __forceinline__ uint32_t mx_round_f32(int mode) { return mode == 0 ? 0x1FFFFFu : 0u; }

// 2^E of an E8M0 byte (0 is 2^-127, a subnormal).
__device__ __forceinline__ float e8m0_value(uint32_t e8) {
  return __uint_as_float(e8 == 0 ? 0x00400000u : e8 << 23);
}

// Two e4m3 codes (low byte first) as fp32.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

// Four e4m3 codes, a's in the low byte.  One asm block, so that the two
// 16-bit halves are not widened before they are joined.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

}  // namespace fp8bw
