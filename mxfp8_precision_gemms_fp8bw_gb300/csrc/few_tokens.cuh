// Tokens as the products of a few of them read them: e4m3 codes in parts.
#pragma once

#include "few.h"
#include "mx_fp32.cuh"

namespace fp8bw {
namespace few {

constexpr uint32_t kAll = 0xffffffffu;

// A block of 32 values is the sum of parts, each a block of MXFP8 codes under a
// power of two of its own: the codes of the values, the codes of what those
// leave, and so on.  e4m3 has 4 significant bits and what rounding to the
// nearest leaves starts 5 bits further down.  So two parts hold the 8 bits of
// bf16 exactly down to 2^-12 of the block's largest value, and to 2^-21 of it
// below that; and five hold the 24 bits of fp32 exactly down to 2^-12 of the
// block's largest, and to 2^-36 of it below that: what the second product adds
// up has no fewer bits than the sums of the first.  With codes down to 2^E of
// a part that are 2^(E-9) apart, the largest of a block in [224, 448] 2^E, E
// falls by 4 from the first part to the second and by 5 from each of the
// others to the next, which keeps what is left under 448 2^E, so that the
// fifth's codes are 2^-28 of the first's power of two apart, and a value of 24
// bits from 2^-5 of it on, which is at most 2^-12 of the largest, is a multiple
// of that.  An infinity becomes a NaN, which e4m3 has.
//
// A third part of the tokens would bring 2^-21 to 2^-26 and take half as many
// columns again: 32 tokens of 8192 x 5120 in 4 bits 14.1 us where two take 12.7,
// 8 in 8 bits 14.2 and 13.6, one 9.4 and 9.1.  What two leave counts only where
// a weight is so small beside the block's largest element that its product is
// too: the largest's own rounding in an fp32 sum is 2^-24 of its product.
__device__ __forceinline__ float without_infinity(float v) {
  return fabsf(v) == INFINITY ? __uint_as_float(0x7FFFFFFFu) : v;
}

// E8M0 byte of a block's largest magnitude (as bits).
__device__ __forceinline__ uint32_t part_byte(uint32_t top) { return min(max((top + 0x1FFFFFu) >> 23, 8u), 255u) - 8u; }
__device__ __forceinline__ float part_factor(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }  // 2^-E

// Where element k of row r is in records of `rows` rows (few.h), and the scale of its block.
__device__ __forceinline__ uint8_t* code_at(uint8_t* records, int64_t rows, int64_t k, int r) {
  const int b = static_cast<int>(k & 127);
  return records + (k >> 7) * few_record(rows) + r * 128 + (((b >> 4) ^ (r & 7)) << 4) + (b & 15);
}
__device__ __forceinline__ uint8_t* scale_at(uint8_t* records, int64_t rows, int64_t k, int r) {
  return records + (k >> 7) * few_record(rows) + rows * 128 + (r >> 7) * 512 + (r & 31) * 16 + (r >> 5 & 3) * 4 + ((k & 127) >> 5);
}

// Eight values of a block that four neighbouring lanes hold, in kTokenParts parts: codes to code(part), and by the first of
// the four the block's byte to scale(part).
template <typename Code, typename Scale>
__device__ __forceinline__ void split8(uint4 v, Code&& code, Scale&& scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = without_infinity(bf16lo_to_f32(w[i]));
    f[2 * i + 1] = without_infinity(bf16hi_to_f32(w[i]));
  }
#pragma unroll
  for (int part = 0; part < kTokenParts; ++part) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(kAll, top, 1));
    top = max(top, __shfl_xor_sync(kAll, top, 2));
    const uint32_t byte = part_byte(top);
    const float down = part_factor(byte), up = e8m0_value(byte);
    uint2 q;
    q.x = e4m3x4(f[0] * down, f[1] * down, f[2] * down, f[3] * down);
    q.y = e4m3x4(f[4] * down, f[5] * down, f[6] * down, f[7] * down);
    *reinterpret_cast<uint2*>(code(part)) = q;
    if ((threadIdx.x & 3) == 0) *scale(part) = static_cast<uint8_t>(byte);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 g = e4m3x2_to_f32((i < 2 ? q.x : q.y) >> (i & 1) * 16);
      f[2 * i] -= g.x * up;
      f[2 * i + 1] -= g.y * up;
    }
  }
}

// Value k of column i of n, of a block that the warp holds, in kActParts parts.  Their powers of two go by the first one alone, as
// far down as they may have to, so that the block's maximum is taken once (one token over 64 experts 16.6 us, by every part's own
// maximum 17.0; 17 tokens 45.6 and 45.8).
__device__ __forceinline__ void split1(float v, uint8_t* records, int n, int64_t k, int i) {
  v = without_infinity(v);
  uint32_t byte = part_byte(__reduce_max_sync(kAll, __float_as_uint(v) & 0x7FFFFFFFu));
  v *= part_factor(byte);
#pragma unroll
  for (int part = 0; part < kActParts; ++part) {
    const uint32_t q = cvt_e4m3x2(v, 0.f);
    const int r = i * kActParts + part;
    *code_at(records, n * kActParts, k, r) = static_cast<uint8_t>(q);
    if ((threadIdx.x & 31) == 0) *scale_at(records, n * kActParts, k, r) = static_cast<uint8_t>(byte);
    const uint32_t down = min(byte, part == 0 ? 4u : 5u);  // less only below 2^-99
    byte -= down;
    v = (v - e4m3x2_to_f32(q).x) * __uint_as_float((127u + down) << 23);
  }
}

}  // namespace few
}  // namespace fp8bw
