// MXFP4 weights: bf16 to e2m1 codes with E8M0 scales, and those codes widened
// to e4m3.
#include "common.cuh"
#include "launch.h"

namespace fp8bw {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kThreads = 256;

// Blocks of 32 do not cross rows and rows are dense, so both kernels see one
// long run of blocks.  Both are bound by memory: codes of 8 x 8192 x 5120
// weights take 135 us (6.4 TB/s, 0.94 of the copy bandwidth), widening them 83
// (6.1 TB/s).  Four lanes hold a block, 8 weights (16 bytes) each, and a warp
// takes 1024 weights at a time in four requests.
//
// The exponent comes from the block's largest magnitude as an integer: with
// bf16 bits amax = 1.m * 2^(ef - 127), m of 7 bits, 6 = 1.5 * 2^2,
//   RCEIL: E = ef - 129, plus one where 1.m > 1.5 -- the carry out of m + 0x3F
//   FLOOR: E = ef - 129
// and the E8M0 byte is E + 127, at least 0.  The largest finite amax gives 253
// (E = 126), so 2^-E is a normal number throughout.
__global__ void __launch_bounds__(kThreads) mxfp4_quant_kernel(const uint4* __restrict__ w, int64_t blocks, uint32_t round,
                                                               uint32_t* __restrict__ q, uint8_t* __restrict__ e8) {
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t b0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * 32; b0 < blocks;
       b0 += warps * 32) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = b0 + i * 8 + lane / 4;
      v[i] = at < blocks ? __ldcs(w + at * 4 + (lane & 3)) : make_uint4(0, 0, 0, 0);
    }
    uint32_t mine = 0;  // the scale byte that this lane writes: of the block lane / 4 of request lane % 4
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = b0 + i * 8 + lane / 4;
      uint32_t m = __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                            __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
      m = max(m & 0xFFFFu, m >> 16);
      m = max(m, __shfl_xor_sync(kAll, m, 1));
      m = max(m, __shfl_xor_sync(kAll, m, 2));
      const uint32_t t = (m + round) >> 7;
      const uint32_t byte = m >= 0x7F80u ? 255u : t < 2 ? 0u : t - 2;
      if ((lane & 3) == i) mine = byte;
      const float s = __uint_as_float((254u - min(byte, 253u)) << 23);
      const uint32_t words[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t out = 0;
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16lo_to_f32(words[j]) * s;
        f[2 * j + 1] = bf16hi_to_f32(words[j]) * s;
      }
      asm("{\n\t.reg .b8 a, b, c, d;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
          "mov.b32 %0, {a, b, c, d};\n\t}"
          : "=r"(out)
          : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
      if (at < blocks) q[at * 4 + (lane & 3)] = out;
    }
    const int64_t at = b0 + (lane & 3) * 8 + lane / 4;
    if (at < blocks) e8[at] = static_cast<uint8_t>(mine);
  }
}

// e4m3 of the four e2m1 codes in the low 16 bits.  The magnitudes are a byte
// permutation whose selectors are the codes; selectors with bit 3 set
// replicate a byte's top bit, which turns 0x80 into 0xff where the code is
// negative.
__device__ __forceinline__ uint32_t widen4(uint32_t codes) {
  const uint32_t size = __byte_perm(0x3C383000u, 0x4C484440u, codes & 0x7777u);
  uint32_t sign;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(codes));
  return size | ((sign << 1) & 0x80808080u);
}

__global__ void __launch_bounds__(kThreads)
    mxfp4_widen_kernel(const uint2* __restrict__ q4, int64_t n, uint4* __restrict__ q8) {  // n: runs of 16 codes
  constexpr int kRuns = 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i0 < n; i0 += step * kRuns) {
    uint2 v[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if (i0 + i * step < n) v[i] = __ldcs(q4 + i0 + i * step);
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if (i0 + i * step < n)
        q8[i0 + i * step] = make_uint4(widen4(v[i].x), widen4(v[i].x >> 16), widen4(v[i].y), widen4(v[i].y >> 16));
  }
}

unsigned grid_of(int64_t work, int num_sms, int per_sm) {
  const int64_t most = static_cast<int64_t>(num_sms) * per_sm;
  return static_cast<unsigned>(work < most ? work : most);
}

}  // namespace

cudaError_t launch_mxfp4_quant_row(const uint16_t* w, int64_t n, uint8_t* q, uint8_t* e8, int mode, int num_sms,
                                   cudaStream_t st) {
  const int64_t blocks = n / 32, per = 32 * (kThreads / 32);
  mxfp4_quant_kernel<<<grid_of((blocks + per - 1) / per, num_sms, 8), kThreads, 0, st>>>(
      reinterpret_cast<const uint4*>(w), blocks, mode == 0 ? 0x3Fu : 0u, reinterpret_cast<uint32_t*>(q), e8);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_to_mxfp8(const uint8_t* q4, int64_t n, uint8_t* q8, int num_sms, cudaStream_t st) {
  const int64_t runs = n / 16;
  mxfp4_widen_kernel<<<grid_of((runs + kThreads - 1) / kThreads, num_sms, 8), kThreads, 0, st>>>(
      reinterpret_cast<const uint2*>(q4), runs, reinterpret_cast<uint4*>(q8));
  return cudaGetLastError();
}

}  // namespace fp8bw
