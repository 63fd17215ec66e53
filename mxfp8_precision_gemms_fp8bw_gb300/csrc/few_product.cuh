// The product of a few tokens with MX weights, as a stream of the weights
// through shared memory and the tensor cores.
#pragma once

#include "mx_weight.cuh"

namespace fp8bw {
namespace few {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kChunk = 128;       // weights of a row that a warp takes at a time: four blocks of 32
constexpr int kTileRows = 32;     // rows of a warp
constexpr int kRowPitch = 36;     // floats between the tokens of a warp's sums: lanes hit 32 banks

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 4 bytes, of which the last 4 - n become zeros without being read.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// c[16, 8] = a[16, 16] b[16, 8] (+ c), f16 into fp32.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- tokens

// Tokens are held in blocks of 32 as f16 under a common power of two, the
// exponent of the block's largest magnitude less 14: bf16 values are exact down
// to 2^-28 of it and rounded at 2^-39 of it below (an f16 subnormal), fp32
// values keep 11 bits.  The record of a block of n tokens is n rows of 32 f16,
// then n fp32 scales, padded to 16 bytes.
__host__ __device__ constexpr int record_bytes(int n) { return n * 64 + ((n * 4 + 15) & ~15); }

// Exponent field of the factor that brings a block into f16, from the exponent
// field of its largest magnitude (255 for infinities and NaN, which stay what
// they are; the finite rest of such a block becomes 0 beside them).
__device__ __forceinline__ uint32_t factor_field(uint32_t ef) { return min(268u - ef, 253u); }
__device__ __forceinline__ float of_field(uint32_t f) { return __uint_as_float(f << 23); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- weights

// One matrix of MX weights as a warp walks through it: 32 of its rows, in
// chunks of 128 weights.
//
// A chunk is copied to shared memory by 16-byte cp.async in the order it has in
// memory, 64 (4 bits) or 128 (8 bits) bytes of each row, and its four scale
// bytes a row by a 4-byte one.  Where the rows of scale bytes are no multiple
// of 4, the two words that hold a row's four bytes are copied and shifted on
// the way out; the last word is read no further than the array.
template <int kBits>
struct Weights {
  static constexpr int kRowBytes = 16 * kBits;
  static constexpr int kStage = kTileRows * kRowBytes + kTileRows * 8;  // codes, then 8 bytes of scales a row
  static constexpr int kCopies = kTileRows * kRowBytes / 512;
};

struct Matrix {
  const uint8_t* w;   // codes
  const uint8_t* e8;  // scales
  int64_t scale_end;  // bytes of e8
  int K;              // weights of a row
};

// The rows of a warp: `rows` of them from `row` on; those past the end of the
// matrix repeat the last and are never stored.
template <int kBits>
struct RowTile {
  const uint8_t* w;    // of the first row
  int64_t e8_at;       // offset of the first row's scales
  uint32_t last;       // index of the last valid row, at most 31
};

template <int kBits>
__device__ __forceinline__ RowTile<kBits> tile_at(const Matrix& m, int64_t row, int64_t end) {
  RowTile<kBits> t;
  t.w = m.w + row * (m.K / 8 * kBits);
  t.e8_at = row * (m.K / 32);
  const int64_t n = end - row;
  t.last = static_cast<uint32_t>(n < kTileRows ? n - 1 : kTileRows - 1);
  return t;
}

// Copies chunk `c` of the tile into the stage at `dst`.
template <int kBits>
__device__ __forceinline__ void copy_chunk(const Matrix& m, const RowTile<kBits>& t, int c, uint32_t dst, int lane) {
  using W = Weights<kBits>;
  constexpr int kPieces = W::kRowBytes / 16, kRowsPerCopy = 32 / kPieces;
  const int r0 = lane / kPieces, p = lane % kPieces;
  // 4 bits: two rows share 128 bytes, 8 bits: a row has 128.  The order of the
  // pieces changes with the row so that the reads below meet 32 banks.
  const uint32_t at = kBits == 4 ? (r0 >> 1) * 128 + (r0 & 1) * 64 + ((p ^ ((r0 >> 1) & 3)) << 4)
                                 : r0 * 128 + ((p ^ ((r0 & 3) << 1)) << 4);
  const uint32_t pitch = m.K / 8 * kBits, off = c * W::kRowBytes + p * 16;
  if (off < pitch) {  // the last chunk of a row may be short
#pragma unroll
    for (int i = 0; i < W::kCopies; ++i)
      cp_async16(dst + at + i * 512, t.w + (min(static_cast<uint32_t>(r0 + i * kRowsPerCopy), t.last) * pitch + off));
  }
  const int sp = m.K / 32;
  const int64_t s = t.e8_at + static_cast<int64_t>(min(static_cast<uint32_t>(lane), t.last)) * sp + c * 4;
  const uint32_t sdst = dst + kTileRows * W::kRowBytes + lane * 8;
  if ((sp & 3) == 0) {
    cp_async4(sdst, m.e8 + s, 4);
  } else {
    const int64_t word = s & ~int64_t{3}, left = m.scale_end - word;
    cp_async4(sdst, m.e8 + word, static_cast<uint32_t>(left < 4 ? left : 4));
    if (left > 4) cp_async4(sdst + 4, m.e8 + word + 4, static_cast<uint32_t>(left < 8 ? left - 4 : 4));
  }
}

// The chunk's products with n tokens, added to acc.  Of the 16 x 8 x 16 product, weights are the 16 rows and
// tokens the 8 columns; a lane's fragments are 8 consecutive weights of a block (lane % 4 says which) of rows lane / 4 + 8 q,
// and the same 8 of token lane / 4, so that a block of 32 is two products whose sum gets the block's two scales in
// fp32.  acc[q / 2][tile][..]: rows lane / 4 + 16 (q / 2) and + 8, tokens 2 (lane % 4) and + 1.
template <int kBits, int kTiles, bool kWhole>
__device__ __forceinline__ void multiply_chunk(const Matrix& m, const RowTile<kBits>& t, uint32_t stage, uint32_t tokens,
                                               uint32_t record, int n, int tiles, int blocks, int lane,
                                               float (&acc)[2][kTiles][4]) {
  using W = Weights<kBits>;
  const int g = lane >> 2, q4 = lane & 3;
  // scales: of four rows, four blocks each
  float s[4][4];
  {
    const int sp = m.K / 32;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t at = stage + kTileRows * W::kRowBytes + (g + 8 * q) * 8;
      uint32_t word;
      if ((sp & 3) == 0) {
        word = lds32(at);
      } else {
        const uint2 two = lds64(at);
        const uint32_t row = min(static_cast<uint32_t>(g + 8 * q), t.last);
        word = __funnelshift_r(two.x, two.y, ((static_cast<uint32_t>(t.e8_at) + row * sp) & 3) * 8);
      }
      e8m0x4_to_f32(word, s[q]);
    }
  }
  const uint32_t a_at = kBits == 4 ? stage + (g >> 1) * 128 + (g & 1) * 64 + (((g >> 1) & 3) << 4) + q4 * 4
                                   : stage + g * 128 + (((q4 >> 1) ^ ((g & 3) << 1)) << 4) + (q4 & 1) * 8;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!kWhole && j >= blocks) break;
    uint32_t a[4][4];  // [row][f16 pairs of its 8 weights]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (kBits == 4) {
        const uint32_t w = lds32((a_at ^ (j << 4)) + q * 512);
        a[q][0] = e2m1x2_to_f16x2<0>(w);
        a[q][1] = e2m1x2_to_f16x2<1>(w);
        a[q][2] = e2m1x2_to_f16x2<2>(w);
        a[q][3] = e2m1x2_to_f16x2<3>(w);
      } else {
        const uint2 w = lds64((a_at ^ (j << 5)) + q * 1024);
        a[q][0] = e4m3x2_to_f16x2<0>(w.x);
        a[q][1] = e4m3x2_to_f16x2<1>(w.x);
        a[q][2] = e4m3x2_to_f16x2<0>(w.y);
        a[q][3] = e4m3x2_to_f16x2<1>(w.y);
      }
    }
    const uint32_t rec = tokens + j * record;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      if (kTiles > 1 && i >= tiles) break;
      const uint4 b = lds128(rec + min(i * 8 + g, n - 1) * 64 + q4 * 16);
      const uint2 sx = lds64(rec + n * 64 + (i * 8 + q4 * 2) * 4);
      const float2 x = make_float2(__uint_as_float(sx.x), __uint_as_float(sx.y));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16(c, a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y);
        mma_f16(c, a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b.z, b.w);
        float(&d)[4] = acc[h][i];
        const float2 up = __ffma2_rn(make_float2(c[0], c[1]), __fmul2_rn(x, make_float2(s[2 * h][j], s[2 * h][j])),
                                     make_float2(d[0], d[1]));
        const float2 lo = __ffma2_rn(make_float2(c[2], c[3]),
                                     __fmul2_rn(x, make_float2(s[2 * h + 1][j], s[2 * h + 1][j])), make_float2(d[2], d[3]));
        d[0] = up.x;
        d[1] = up.y;
        d[2] = lo.x;
        d[3] = lo.y;
      }
    }
  }
}

}  // namespace few
}  // namespace fp8bw
