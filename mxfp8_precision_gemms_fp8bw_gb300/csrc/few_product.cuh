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
// Four 8 x 16-byte matrices, whose rows lanes 0-7, 8-15, ... point at; the lane gets bytes 4 (lane % 4).. of row lane / 4.
__device__ __forceinline__ void ldmatrix4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
// d[16, 8] = a[16, 16] b[16, 8] + c, f16 into fp32.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, "
      "%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// ---------------------------------------------------------------- tokens

// Tokens are held as f16 under a power of two that a run of them shares (32
// elements of the activation, a block's share of the contraction of x): the
// exponent of the largest magnitude less 14.  bf16 values are exact down to
// 2^-28 of the largest and rounded at 2^-39 of it below (an f16 subnormal),
// fp32 values keep 11 bits.  The record of 32 elements of n tokens is n rows of
// 32 f16; of the activation, n fp32 scales follow, padded to 16 bytes.
__host__ __device__ constexpr int record_bytes(int n, bool scaled) { return n * 64 + (scaled ? (n * 4 + 15) & ~15 : 0); }

// Where element e of 32 stands in its row, so that a lane's eight are side by
// side: those whose weights ldmatrix gives it, 8 l .. of 4-bit weights, and
// 4 l .. and 16 + 4 l .. of 8-bit ones.
template <int kBits>
__device__ __forceinline__ int place_of(int e) {
  return kBits == 4 ? e : ((e >> 2) & 3) * 8 + (e >> 4) * 4 + (e & 3);
}

// Exponent field of the factor that brings values into f16, from the exponent
// field of the largest magnitude (255 for infinities and NaN, which stay what
// they are; the finite rest becomes 0 beside them).
__device__ __forceinline__ uint32_t factor_field(uint32_t ef) { return min(268u - ef, 253u); }
__device__ __forceinline__ float of_field(uint32_t f) { return __uint_as_float(f << 23); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t largest(uint4 v) {  // of eight bf16 magnitudes, as two halves
  return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}
__device__ __forceinline__ uint4 to_f16(uint4 v, float f) {
  return make_uint4(pack_f16x2(bf16lo_to_f32(v.x) * f, bf16hi_to_f32(v.x) * f),
                    pack_f16x2(bf16lo_to_f32(v.y) * f, bf16hi_to_f32(v.y) * f),
                    pack_f16x2(bf16lo_to_f32(v.z) * f, bf16hi_to_f32(v.z) * f),
                    pack_f16x2(bf16lo_to_f32(v.w) * f, bf16hi_to_f32(v.w) * f));
}
// Elements 8 i .. of a row of 32, in their places.
template <int kBits>
__device__ __forceinline__ void store_f16(uint8_t* row, int i, uint4 h) {
  if constexpr (kBits == 4) {
    *reinterpret_cast<uint4*>(row + i * 16) = h;
  } else {
    *reinterpret_cast<uint2*>(row + place_of<8>(i * 8) * 2) = make_uint2(h.x, h.y);
    *reinterpret_cast<uint2*>(row + place_of<8>(i * 8 + 4) * 2) = make_uint2(h.z, h.w);
  }
}

// ---------------------------------------------------------------- weights

// A matrix of MX weights as a warp walks through it: 32 of its rows, in chunks
// of 128 weights.
//
// A chunk is copied to shared memory by 16-byte cp.async as it lies in memory,
// 64 (4 bits) or 128 (8 bits) bytes of each row, and its four scale bytes a
// row by a 4-byte one.  Where the rows of scale bytes are no multiple of 4, the
// two words that hold a row's four bytes are copied and shifted on the way out;
// the last word is read no further than the array.
struct Matrix {
  const uint8_t* w;   // codes
  const uint8_t* e8;  // scales
  int64_t scale_end;  // bytes of e8
  int K;              // weights of a row
};

template <int kBits>
struct Weights {
  static constexpr int kRowBytes = 16 * kBits;
  static constexpr int kScales = kTileRows * kRowBytes;  // in a stage: codes, then 8 bytes of scales a row
  static constexpr int kStage = kScales + kTileRows * 8;
  static constexpr int kCopies = kScales / 512;
  static constexpr int kPieces = kRowBytes / 16;

  // Fixed for the warp: where the lane's pieces are in the tile and the stage.
  uint32_t from[kCopies], scale_from, to, pitch;
  uint32_t read, scale_read;  // for multiply_chunk
  int last, scale_pitch;      // the tile's last valid row; rows past it repeat it and are never stored
  const uint8_t* scales;
  int64_t scale_end;

  __device__ __forceinline__ Weights(const Matrix& m, int last_row, int lane) {
    last = last_row;
    pitch = m.K / 8 * kBits;
    scale_pitch = m.K / 32;
    scales = m.e8;
    scale_end = m.scale_end;
    const int r0 = lane / kPieces, p = lane % kPieces;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) from[i] = min(r0 + i * (32 / kPieces), last) * pitch + p * 16;
    scale_from = min(lane, last) * scale_pitch;
    // The order of a row's pieces changes with the row, so that the eight rows
    // of a matrix of ldmatrix lie in 32 banks.  4 bits: two rows to 128 bytes.
    to = kBits == 4 ? (r0 >> 1) * 128 + (r0 & 1) * 64 + ((p ^ ((r0 >> 1) & 3)) << 4) : r0 * 128 + ((p ^ r0) << 4);
    read = kBits == 4 ? (lane >> 1) * 128 + (lane & 1) * 64 + (((lane >> 1) & 3) << 4) : lane * 128 + ((lane & 7) << 4);
    scale_read = kScales + (lane >> 2) * 8;
  }

  // Copies chunk c of the tile, whose codes begin at w and scales at byte e8_at, into a stage.
  __device__ __forceinline__ void copy(const uint8_t* w, int64_t e8_at, int c, uint32_t stage, int lane) const {
    const uint32_t off = c * kRowBytes;
    if (off + lane % kPieces * 16 < pitch) {  // the last chunk of a row may be short
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        cp_async16(stage + (kBits == 4 ? to : to ^ ((i & 1) << 6)) + i * 512, w + (from[i] + off));
    }
    const int64_t s = e8_at + (scale_from + c * 4);
    const uint32_t dst = stage + kScales + lane * 8;
    if ((scale_pitch & 3) == 0) {
      cp_async4(dst, scales + s, 4);
    } else {
      const int64_t word = s & ~int64_t{3}, left = scale_end - word;
      cp_async4(dst, scales + word, static_cast<uint32_t>(left < 4 ? left : 4));
      if (left > 4) cp_async4(dst + 4, scales + word + 4, static_cast<uint32_t>(left < 8 ? left - 4 : 4));
    }
  }

  // The four scale bytes of row lane / 4 + 8 q.
  __device__ __forceinline__ uint32_t scale_word(uint32_t stage, int64_t e8_at, int q, int lane) const {
    if ((scale_pitch & 3) == 0) return lds32(stage + scale_read + q * 64);
    const uint2 two = lds64(stage + scale_read + q * 64);
    const uint32_t row = min((lane >> 2) + 8 * q, last);
    return __funnelshift_r(two.x, two.y, ((static_cast<uint32_t>(e8_at) + row * scale_pitch) & 3) * 8);
  }

  // The 32 rows' weights of block j as f16: a[q] are those of row lane / 4 + 8 q, eight of them.
  __device__ __forceinline__ void block(uint32_t stage, int j, uint32_t (&a)[4][4]) const {
    uint32_t w[4];
    if constexpr (kBits == 4) {
      ldmatrix4((stage + read) ^ (j << 4), w);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q][0] = e2m1x2_to_f16x2<0>(w[q]);
        a[q][1] = e2m1x2_to_f16x2<1>(w[q]);
        a[q][2] = e2m1x2_to_f16x2<2>(w[q]);
        a[q][3] = e2m1x2_to_f16x2<3>(w[q]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ldmatrix4((stage + read) ^ ((2 * j + h) << 4), w);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          a[q][2 * h] = e4m3x2_to_f16x2<0>(w[q]);
          a[q][2 * h + 1] = e4m3x2_to_f16x2<1>(w[q]);
        }
      }
    }
  }
};

// The products of a chunk with kTiles * 8 tokens, added to acc.  Weights are
// the 16 rows and tokens the 8 columns of m16n8k16; a lane's fragments are
// eight weights of a block and the same eight of token lane / 4, so that a block
// of 32 is two products, whose sum gets the block's scales in fp32.
// acc[h][i]: rows lane / 4 + 16 h (and + 8), tokens 8 i + 2 (lane % 4) (and + 1).
//   tokens: the chunk's first record; at[i]: the lane's token in a record;
//   scale_at: of the lane's first scale in a record (kScaled)
template <int kBits, int kTiles, int kAcc, bool kScaled, bool kWhole>
__device__ __forceinline__ void multiply_chunk(const Weights<kBits>& W, uint32_t stage, int64_t e8_at, uint32_t tokens,
                                               uint32_t record, const uint32_t (&at)[kAcc], uint32_t scale_at, int blocks,
                                               int lane, float (&acc)[2][kAcc][4]) {
  float s[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) e8m0x4_to_f32(W.scale_word(stage, e8_at, q, lane), s[q]);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!kWhole && j >= blocks) break;
    uint32_t a[4][4];
    W.block(stage, j, a);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const uint4 b = lds128(tokens + at[i]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float c[4];
        mma_f16(c, a[2 * h][0], a[2 * h + 1][0], a[2 * h][1], a[2 * h + 1][1], b.x, b.y, 0.f, 0.f, 0.f, 0.f);
        mma_f16(c, a[2 * h][2], a[2 * h + 1][2], a[2 * h][3], a[2 * h + 1][3], b.z, b.w, c[0], c[1], c[2], c[3]);
        float(&d)[4] = acc[h][i];
        if constexpr (kScaled) {
          const uint2 sx = lds64(tokens + scale_at + i * 32);
          const float2 x = make_float2(__uint_as_float(sx.x), __uint_as_float(sx.y));
          const float2 up = __ffma2_rn(make_float2(c[0], c[1]), __fmul2_rn(x, make_float2(s[2 * h][j], s[2 * h][j])),
                                       make_float2(d[0], d[1]));
          const float2 lo = __ffma2_rn(make_float2(c[2], c[3]),
                                       __fmul2_rn(x, make_float2(s[2 * h + 1][j], s[2 * h + 1][j])),
                                       make_float2(d[2], d[3]));
          d[0] = up.x, d[1] = up.y, d[2] = lo.x, d[3] = lo.y;
        } else {
          d[0] = fmaf(c[0], s[2 * h][j], d[0]);
          d[1] = fmaf(c[1], s[2 * h][j], d[1]);
          d[2] = fmaf(c[2], s[2 * h + 1][j], d[2]);
          d[3] = fmaf(c[3], s[2 * h + 1][j], d[3]);
        }
      }
    }
    tokens += record;
  }
}

}  // namespace few
}  // namespace fp8bw
