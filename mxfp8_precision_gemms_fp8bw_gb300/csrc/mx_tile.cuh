// Register tiles of the kernels that quantize what they compute to MX codes.
//
// A warp owns 32 rows x 64 columns, a thread 8 rows x 8 columns of them: lane
// 8 i + j has rows 8 i + [0, 8) and columns 8 j + [0, 8).  A row block (32
// columns) is then four neighbouring lanes and a column block (32 rows) the
// four lanes 8 apart, so both block maxima are two shuffles, the tile is read
// once, and nothing goes through shared memory.  Every access is whole
// sectors: a row of bf16 is 128 contiguous bytes over its eight lanes, a row
// of codes 64, a column of codes 32.
#pragma once

#include "common.cuh"
#include "mx_fp32.cuh"

namespace fp8bw {

struct TileLane {
  int rg, cg;  // row group and column group of the lane
};
__device__ __forceinline__ TileLane tile_lane() {
  const int lane = threadIdx.x & 31;
  return TileLane{lane >> 3, lane & 7};
}

__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ void st_codes8(uint8_t* p, uint2 v) {
  asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int k) {
  return k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
}
__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t w) { return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w)); }

// The larger magnitude in each bf16 half; NaN stays NaN, the sign bits mean nothing.
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t absmax2_of8(const uint4& v) { return absmax2(absmax2(v.x, v.y), absmax2(v.z, v.w)); }
// Two such words a and b, each folded to one value: a's in the low half, b's in the high half.
__device__ __forceinline__ uint32_t fold2(uint32_t a, uint32_t b) {
  return absmax2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
}
// A block max in bf16 as the bits of the same fp32 value.
__device__ __forceinline__ uint32_t f32_bits_lo(uint32_t w) { return (w & 0x7FFFu) << 16; }
__device__ __forceinline__ uint32_t f32_bits_hi(uint32_t w) { return w & 0x7FFF0000u; }

// max over the lanes of a row block (xor 1, 2) or of a column block (xor 8, 16).
template <int kStep>
__device__ __forceinline__ uint32_t block_absmax2(uint32_t w) {
  w = absmax2(w, __shfl_xor_sync(0xffffffffu, w, kStep));
  return absmax2(w, __shfl_xor_sync(0xffffffffu, w, 2 * kStep));
}

// The larger magnitude of fp32 values; NaN stays NaN.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Of eight, with what is already there.
__device__ __forceinline__ float absmax8(float m, const float2 (&v)[4]) {
  m = absmax3(absmax3(m, v[0].x, v[0].y), v[1].x, v[1].y);
  return absmax3(absmax3(m, v[2].x, v[2].y), v[3].x, v[3].y);
}

// A bf16 half times the bf16 power of two m in fp32: exact, or rounded once
// where it falls below the fp32 range; adding -0 keeps the sign of a zero.
// One instruction on the packed pair, where unpacking first takes two.
template <int kHi>
__device__ __forceinline__ float half_times(uint32_t w, uint16_t m) {
  float r;
  if (kHi)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tfma.rn.f32.bf16 %0, hi, %2, %3;\n\t}"
        : "=f"(r) : "r"(w), "h"(m), "f"(-0.0f));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tfma.rn.f32.bf16 %0, lo, %2, %3;\n\t}"
        : "=f"(r) : "r"(w), "h"(m), "f"(-0.0f));
  return r;
}

// The scale rule on a block max held as bf16 magnitude bits (mx_t and
// mx_mul_of of mx_fp32.cuh, 16 bits down).
__device__ __forceinline__ uint32_t mx_t_bf16(uint32_t bits, uint32_t round) {
  return min(max((bits + (round >> 16)) >> 7, 8u), 255u);
}
__device__ __forceinline__ uint16_t mx_mul_bf16(uint32_t t) { return static_cast<uint16_t>((262u - t) << 7); }

// e4m3 codes of eight packed bf16 times m, of one row.
__device__ __forceinline__ uint2 codes8_row(const uint4& v, uint16_t m) {
  return make_uint2(e4m3x4(half_times<0>(v.x, m), half_times<1>(v.x, m), half_times<0>(v.y, m), half_times<1>(v.y, m)),
                    e4m3x4(half_times<0>(v.z, m), half_times<1>(v.z, m), half_times<0>(v.w, m), half_times<1>(v.w, m)));
}
// The same down column 2 k + kHi of eight rows.
template <int kHi>
__device__ __forceinline__ uint2 codes8_col(const uint4 (&v)[8], int k, uint16_t m) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = half_times<kHi>(word_of(v[i], k), m);
  return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
}

// e4m3 codes of eight fp32 values times m.
__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], float m) {
  const float2 mm = make_float2(m, m);
  const float2 a = __fmul2_rn(v[0], mm), b = __fmul2_rn(v[1], mm), c = __fmul2_rn(v[2], mm), d = __fmul2_rn(v[3], mm);
  return make_uint2(e4m3x4(a.x, a.y, b.x, b.y), e4m3x4(c.x, c.y, d.x, d.y));
}

// Scale bytes of a 128 x 128 tile: of each row's four 32-column blocks, and of
// each column's four 32-row blocks.  They leave as one word per row or column:
// as single bytes, straight from the lanes that have them, they took as many
// L1 tag cycles as all the codes.
struct ScaleTile {
  alignas(4) uint8_t row[128][4];
  alignas(4) uint8_t col[128][4];
};

// Line `i` (0 to 127; others do nothing) of one side: entries b0 .. b0 + 3 of
// line first + i of out [lines][per_line].
__device__ __forceinline__ void put_scales(const uint8_t (&side)[128][4], int i, int64_t first, int64_t lines,
                                           uint8_t* __restrict__ out, int b0, int per_line) {
  if (i < 0 || i >= 128 || first + i >= lines) return;
  uint8_t* to = out + (first + i) * per_line + b0;
  if ((per_line & 3) == 0) {
    *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(side[i]);
  } else {
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (b0 + b < per_line) to[b] = side[i][b];
  }
}

}  // namespace fp8bw
