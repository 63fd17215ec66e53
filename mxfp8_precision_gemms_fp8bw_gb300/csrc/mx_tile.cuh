// What the kernels that quantize gathered or computed values to MX codes share:
// loads and stores of 16 and 8 bytes, block maxima, and the scale rule and the
// conversion for several values at a time.
//
// The tile of moe_rows.cu: a warp owns 32 rows x 64 columns, a thread 8 rows x
// 8 columns of them: lane 8 i + j has rows 8 i + [0, 8) and columns 8 j + [0,
// 8).  A row block (32 columns) is then four neighbouring lanes and a column
// block (32 rows) the four lanes 8 apart, so both block maxima are two
// shuffles and the values are read once for both layouts.  A row of codes is
// 64 contiguous bytes over its eight lanes; column codes leave through shared
// memory.  (moe_swiglu.cu has more values live per element and half the tile
// per thread.)
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

// 16 bytes read once, or zeros where `live` is false (no branch around either).
__device__ __forceinline__ uint4 ld_once_v4(const void* p, bool live = true) {
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"(static_cast<int>(live)));
  return r;
}
// Codes go out with the streaming hint: nothing here reads them again, and
// without it they push what is still to be read out of L2 (130048 x 1024
// activations forward: 210 us without, 176 with).
__device__ __forceinline__ void st_codes8(uint8_t* p, uint2 v, bool live) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p st.global.cs.v2.u32 [%0], {%1, %2};\n\t}" ::"l"(p),
               "r"(v.x), "r"(v.y), "r"(static_cast<int>(live))
               : "memory");
}
__device__ __forceinline__ void st_codes4(uint8_t* p, uint32_t v, bool live) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.cs.u32 [%0], %1;\n\t}" ::"l"(p), "r"(v),
               "r"(static_cast<int>(live))
               : "memory");
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
// e4m3 codes of eight fp32 values times m, the values of one row in pairs as
// they were unpacked: two products per instruction.
__device__ __forceinline__ uint2 codes8(const float2 (&v)[4], float m) {
  const float2 mm = make_float2(m, m);
  const float2 a = __fmul2_rn(v[0], mm), b = __fmul2_rn(v[1], mm), c = __fmul2_rn(v[2], mm), d = __fmul2_rn(v[3], mm);
  return make_uint2(e4m3x4(a.x, a.y, b.x, b.y), e4m3x4(c.x, c.y, d.x, d.y));
}

// Two blocks' exponents in the halves of one word.  `raw` is (bits(amax) +
// round) >> 23 of mx_fp32.cuh before its clamp: it grows with the max, so the lanes
// of a block reduce it (__vmaxu2) and clamp once.
__device__ __forceinline__ uint32_t mx_raw2(float amax_lo, float amax_hi, uint32_t round) {  // both >= 0 or NaN
  return (__float_as_uint(amax_lo) + round) >> 23 | (((__float_as_uint(amax_hi) + round) >> 7) & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t mx_clamp2(uint32_t raw) { return __vminu2(__vmaxu2(raw, 0x00080008u), 0x00FF00FFu); }
// The same from two bf16 magnitudes in one word, whose sums cannot carry.
__device__ __forceinline__ uint32_t mx_t2(uint32_t w, uint32_t round) {
  return mx_clamp2((((w & 0x7FFF7FFFu) + (round >> 16) * 0x10001u) >> 7) & 0x01FF01FFu);
}
// 2^-E of both, as packed bf16 and as fp32.
__device__ __forceinline__ uint32_t mx_mul2(uint32_t t2) { return (0x01060106u - t2) << 7; }
__device__ __forceinline__ float2 mx_mul2_f32(uint32_t t2) { return bf16x2_to_f32(mx_mul2(t2)); }
// The E8M0 bytes of both, in the halves of a word.
__device__ __forceinline__ uint32_t mx_bytes2(uint32_t t2) { return t2 - 0x00080008u; }

// Packed bf16 products with powers of two: exact, or, far below the smallest
// e4m3 code, a zero or subnormal of the same sign.
__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// e4m3 codes of eight packed bf16 of one row times a packed pair of the scale.
__device__ __forceinline__ uint2 codes8_row(const uint4& v, uint32_t m2) {
  const uint32_t a = mul2_bf16(v.x, m2), b = mul2_bf16(v.y, m2), c = mul2_bf16(v.z, m2), d = mul2_bf16(v.w, m2);
  return make_uint2(e4m3x4(bf16lo_to_f32(a), bf16hi_to_f32(a), bf16lo_to_f32(b), bf16hi_to_f32(b)),
                    e4m3x4(bf16lo_to_f32(c), bf16hi_to_f32(c), bf16lo_to_f32(d), bf16hi_to_f32(d)));
}
// The same down columns 2 k (lo) and 2 k + 1 (hi) of eight rows, m2 their scales.
struct CodePair {
  uint2 lo, hi;
};
__device__ __forceinline__ CodePair pair_of_columns(const float2 (&p)[8]) {
  return CodePair{make_uint2(e4m3x4(p[0].x, p[1].x, p[2].x, p[3].x), e4m3x4(p[4].x, p[5].x, p[6].x, p[7].x)),
                  make_uint2(e4m3x4(p[0].y, p[1].y, p[2].y, p[3].y), e4m3x4(p[4].y, p[5].y, p[6].y, p[7].y))};
}
__device__ __forceinline__ CodePair codes8_cols(const uint4 (&v)[8], int k, uint32_t m2) {
  float2 p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = bf16x2_to_f32(mul2_bf16(word_of(v[i], k), m2));
  return pair_of_columns(p);
}

// Scale bytes of a 128 x 128 tile: of the rows' blocks (32 columns each) and of
// the columns' blocks (32 rows each).  Threads leave eight bytes at a time and
// they go out as one word per row or column: as single bytes, straight from
// the lanes that have them, they took as many L1 tag cycles as all the codes.
struct alignas(8) ScaleTile {
  uint8_t row[4][128];  // [block][row]
  uint8_t col[4][128];  // [block][column]
};

// The bytes of the thread's eight rows and columns, two to a word, from the
// first lane of each row block and of each column block; rt and ct are the
// thread's first row and column in the tile.
__device__ __forceinline__ void put_bytes(ScaleTile& s, int rt, int ct, const uint32_t (&rows)[4],
                                          const uint32_t (&cols)[4]) {
  if ((ct & 31) == 0)
    *reinterpret_cast<uint2*>(&s.row[ct / 32][rt]) =
        make_uint2(__byte_perm(rows[0], rows[1], 0x6420), __byte_perm(rows[2], rows[3], 0x6420));
  if ((rt & 31) == 0)
    *reinterpret_cast<uint2*>(&s.col[rt / 32][ct]) =
        make_uint2(__byte_perm(cols[0], cols[1], 0x6420), __byte_perm(cols[2], cols[3], 0x6420));
}

// One side by 128 threads, i = 0 to 127 (others do nothing): entries b0 .. b0 +
// 3 of lines first .. first + 127 of out [lines][per_line].  A word per line
// where lines are words; else four neighbouring lanes have a line's four
// bytes, which then still are one request (a thread per line, byte by byte,
// is four: 62 us for the two-layout kernel at 519 bytes per line against
// 54).
__device__ __forceinline__ void put_scales(const uint8_t (&side)[4][128], int i, int64_t first, int64_t lines,
                                           uint8_t* __restrict__ out, int b0, int per_line) {
  if (i < 0 || i >= 128) return;
  if ((per_line & 3) == 0) {
    if (first + i < lines)
      *reinterpret_cast<uint32_t*>(out + (first + i) * per_line + b0) =
          side[0][i] | side[1][i] << 8 | side[2][i] << 16 | static_cast<uint32_t>(side[3][i]) << 24;
  } else {
    const int b = i & 3;
    if (b0 + b >= per_line) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int line = j * 32 + i / 4;
      if (first + line < lines) out[(first + line) * per_line + b0 + b] = side[b][line];
    }
  }
}

}  // namespace fp8bw
