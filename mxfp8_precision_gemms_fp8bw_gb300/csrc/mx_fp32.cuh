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
// number.
__device__ __forceinline__ uint32_t mx_round_f32(int mode) { return mode == 0 ? 0x1FFFFFu : 0u; }
__device__ __forceinline__ uint32_t mx_t(uint32_t abs_bits, uint32_t round) {
  return min(max((abs_bits + round) >> 23, 8u), 255u);
}
__device__ __forceinline__ float mx_mul_of(uint32_t t) { return __uint_as_float((262u - t) << 23); }
__device__ __forceinline__ uint8_t mx_e8_of(uint32_t t) { return static_cast<uint8_t>(t - 8u); }
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

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

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return __byte_perm(cvt_e4m3x2(a, b), cvt_e4m3x2(c, d), 0x5410);
}

// A 32-row x 128-column fp32 tile, quantized both ways by 128 threads.
struct QuantTile {
  float v[32][129];
};

// Rowwise: warp w has rows 8w + [0, 8), lane l columns 4l + [0, 4), so eight
// lanes hold a block of 32.  Row r0 + r, columns c0 + ... of q [rows, ld].
__device__ __forceinline__ void quant_tile_rows(const QuantTile& t, int64_t r0, int64_t c0, int64_t ld, int64_t c_end,
                                                uint8_t* __restrict__ q, uint8_t* __restrict__ e8, uint32_t round) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t col = c0 + 4 * lane;
  for (int i = 0; i < 8; ++i) {
    const int r = warp * 8 + i;
    const float a = t.v[r][4 * lane], b = t.v[r][4 * lane + 1], c = t.v[r][4 * lane + 2], d = t.v[r][4 * lane + 3];
    uint32_t x = mx_t(max(max(abs_bits(a), abs_bits(b)), max(abs_bits(c), abs_bits(d))), round);
    for (int o = 1; o < 8; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    const float m = mx_mul_of(x);
    if (col < c_end) {
      *reinterpret_cast<uint32_t*>(q + (r0 + r) * ld + col) = e4m3x4(a * m, b * m, c * m, d * m);
      if ((lane & 7) == 0) e8[(r0 + r) * (ld / 32) + col / 32] = mx_e8_of(x);
    }
  }
}

// Colwise: thread i has column c0 + i, whose 32 rows are one block, written as
// 32 contiguous bytes of qT [columns, R].
__device__ __forceinline__ void quant_tile_cols(const QuantTile& t, int64_t r0, int64_t c0, int64_t R, int64_t c_end,
                                                uint8_t* __restrict__ qT, uint8_t* __restrict__ e8T, uint32_t round) {
  const int i = threadIdx.x;
  const int64_t col = c0 + i;
  if (col >= c_end) return;
  uint32_t a = 0;
  for (int r = 0; r < 32; ++r) a = max(a, abs_bits(t.v[r][i]));
  const uint32_t x = mx_t(a, round);
  const float m = mx_mul_of(x);
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    w[k] = e4m3x4(t.v[4 * k][i] * m, t.v[4 * k + 1][i] * m, t.v[4 * k + 2][i] * m, t.v[4 * k + 3][i] * m);
  uint4* out = reinterpret_cast<uint4*>(qT + col * R + r0);
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  e8T[col * (R / 32) + r0 / 32] = mx_e8_of(x);
}

}  // namespace fp8bw
