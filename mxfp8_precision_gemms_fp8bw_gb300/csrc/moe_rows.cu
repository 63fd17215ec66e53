// Rows of the experts: gathering tokens into them as MX codes, and summing
// them back into the tokens.
#include "common.cuh"
#include "launch.h"
#include "mx_tile.cuh"

namespace fp8bw {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

constexpr int kGatherWarps = 8;

// MX codes of gathered rows, v_p = w_p * x[src_p / top_k], in both layouts.
// A warp's 32-row x 64-column tile lives in registers (mx_tile.cuh); a block
// has 128 x 128, so that the codes of its rows and of its columns fill whole
// 128-byte lines.  The blocks of one 128-column stripe run one after another:
// a token is gathered up to top_k times, and a stripe of x stays in L2 between
// them (with the columns fastest, 5120 of them and 8192 x 2 entries, x came
// from DRAM 1.9 times).  Without weights the maxima are taken on packed bf16 pairs.  With
// them the max of a row block is still the bf16 max, times |w| (rounding is
// monotonic, so the product of the max is the max of the products); a column
// block mixes weights and takes the max of the fp32 products.
template <bool kWeighted>
__global__ void __launch_bounds__(kGatherWarps * 32)
    gather_quant_kernel(const uint16_t* __restrict__ x, const float* __restrict__ weights,
                        const int32_t* __restrict__ src_of, uint32_t entries, uint32_t top_k, int P, int C, int bands,
                        uint8_t* __restrict__ q, uint8_t* __restrict__ e8, uint8_t* __restrict__ qT,
                        uint8_t* __restrict__ e8T, int mode, int* status) {
  __shared__ ScaleTile scales;
  const TileLane t = tile_lane();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stripe = blockIdx.x / bands;
  const int c0 = stripe * 128 + (warp & 1) * 64 + t.cg * 8;
  const int64_t rb = static_cast<int64_t>(blockIdx.x - stripe * bands) * 128;
  const int64_t rw = rb + (warp >> 1) * 32;
  const bool row_ok = rw < P;            // P % 32 == 0: a warp's rows are all in or all out
  const bool col_ok = row_ok && c0 < C;  // C % 32 == 0: so are the columns of a block
  // Lane l looks up row l of the warp's 32; shuffles hand the token and the weight to the row's eight lanes.
  const uint32_t src = row_ok ? static_cast<uint32_t>(src_of[rw + lane]) : 0xffffffffu;
  uint32_t token = 0xffffffffu;
  float weight = 0.f;
  if (src < entries) {
    token = src / top_k;
    if (kWeighted) weight = weights[src];
  } else if (src != 0xffffffffu) {
    atomicExch(status, kStatusShape);
  }
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t from = __shfl_sync(kAll, token, t.rg * 8 + i);
    v[i] = make_uint4(0, 0, 0, 0);
    if (from != 0xffffffffu && col_ok) v[i] = ld_once_v4(x + (static_cast<uint64_t>(from) * static_cast<uint32_t>(C) + c0));
  }
  const uint32_t round = mx_round_f32(mode);
  const int64_t r0 = rw + t.rg * 8;
  uint8_t* qrow = q + r0 * C + c0;
  // Where the thread's row and column blocks have their scale bytes.
  uint8_t* erow = &scales.row[(warp >> 1) * 32 + t.rg * 8][(warp & 1) * 2 + (t.cg >> 2)];
  uint8_t* ecol = &scales.col[(warp & 1) * 64 + t.cg * 8][warp >> 1];
  uint8_t* qcol = qT + static_cast<int64_t>(c0) * P + r0;

  uint32_t m[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) m[p] = block_absmax2<1>(fold2(absmax2_of8(v[2 * p]), absmax2_of8(v[2 * p + 1])));

  if (!kWeighted) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = mx_t_bf16((m[i >> 1] >> (i & 1) * 16) & 0x7FFFu, round);
      if (col_ok) st_codes8(qrow + static_cast<int64_t>(i) * C, codes8_row(v[i], mx_mul_bf16(e)));
      if ((t.cg & 3) == 0) erow[4 * i] = mx_e8_of(e);
    }
    if (qT != nullptr) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // columns c0 + 2k and c0 + 2k + 1
      uint32_t a = word_of(v[0], k);
#pragma unroll
      for (int i = 1; i < 8; ++i) a = absmax2(a, word_of(v[i], k));
      a = block_absmax2<8>(a);
      const uint32_t lo = mx_t_bf16(a & 0x7FFFu, round), hi = mx_t_bf16((a >> 16) & 0x7FFFu, round);
      if (col_ok) {
        st_codes8(qcol + static_cast<int64_t>(2 * k) * P, codes8_col<0>(v, k, mx_mul_bf16(lo)));
        st_codes8(qcol + static_cast<int64_t>(2 * k + 1) * P, codes8_col<1>(v, k, mx_mul_bf16(hi)));
      }
      if (t.rg == 0) {
        ecol[8 * k] = mx_e8_of(lo);
        ecol[8 * k + 4] = mx_e8_of(hi);
      }
    }
    }
  } else {
  // Weighted: the products stay in registers between the two passes.
  float2 f[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = __shfl_sync(kAll, weight, t.rg * 8 + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[i][k] = __fmul2_rn(bf16x2_to_f32(word_of(v[i], k)), make_float2(w, w));
    const uint32_t amax = (i & 1) ? f32_bits_hi(m[i >> 1]) : f32_bits_lo(m[i >> 1]);
    const uint32_t e = mx_t(abs_bits(__uint_as_float(amax) * w), round);
    if (col_ok) st_codes8(qrow + static_cast<int64_t>(i) * C, codes8(f[i], mx_mul_of(e)));
    if ((t.cg & 3) == 0) erow[4 * i] = mx_e8_of(e);
  }
  if (qT != nullptr) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 lo[4] = {{f[0][k].x, f[1][k].x}, {f[2][k].x, f[3][k].x}, {f[4][k].x, f[5][k].x}, {f[6][k].x, f[7][k].x}};
    const float2 hi[4] = {{f[0][k].y, f[1][k].y}, {f[2][k].y, f[3][k].y}, {f[4][k].y, f[5][k].y}, {f[6][k].y, f[7][k].y}};
    // The exponent grows with the max, so the lanes reduce both columns' exponents in one word.
    uint32_t e = mx_t(abs_bits(absmax8(0.f, lo)), round) | mx_t(abs_bits(absmax8(0.f, hi)), round) << 16;
    e = __vmaxu2(e, __shfl_xor_sync(kAll, e, 8));
    e = __vmaxu2(e, __shfl_xor_sync(kAll, e, 16));
    const uint32_t el = e & 0xFFFFu, eh = e >> 16;
    if (col_ok) {
      st_codes8(qcol + static_cast<int64_t>(2 * k) * P, codes8(lo, mx_mul_of(el)));
      st_codes8(qcol + static_cast<int64_t>(2 * k + 1) * P, codes8(hi, mx_mul_of(eh)));
    }
    if (t.rg == 0) {
      ecol[8 * k] = mx_e8_of(el);
      ecol[8 * k + 4] = mx_e8_of(eh);
    }
  }
  }
  }
  __syncthreads();
  put_scales(scales.row, threadIdx.x, rb, P, e8, stripe * 4, C / 32);
  if (qT != nullptr) put_scales(scales.col, threadIdx.x - 128, stripe * 128, C, e8T, static_cast<int>(rb / 32), P / 32);
}

__device__ __forceinline__ int64_t checked_row(const int32_t* row_of, int64_t i, int64_t P, int* status) {
  int64_t r = row_of[i];
  if (r < -1 || r >= P) {
    atomicExch(status, kStatusShape);
    r = -1;
  }
  return r;
}

// A thread per 8 columns of a token.
__global__ void __launch_bounds__(256)
    combine_kernel(const uint16_t* __restrict__ y, const float* __restrict__ weights,
                   const int32_t* __restrict__ row_of, const uint16_t* base, int64_t chunks, int64_t total, int top_k,
                   int64_t P, uint16_t* out, int* status) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t t = i / chunks;
  float acc[8] = {};
  if (base != nullptr) {
    const uint4 b = reinterpret_cast<const uint4*>(base)[i];
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
    for (int k = 0; k < 4; ++k) {
      acc[2 * k] = bf16lo_to_f32(w[k]);
      acc[2 * k + 1] = bf16hi_to_f32(w[k]);
    }
  }
  for (int j = 0; j < top_k; ++j) {
    const int64_t r = checked_row(row_of, t * top_k + j, P, status);
    if (r < 0) continue;
    const float m = weights != nullptr ? weights[t * top_k + j] : 1.f;
    const uint4 v = reinterpret_cast<const uint4*>(y)[r * chunks + i % chunks];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    for (int k = 0; k < 4; ++k) {
      acc[2 * k] += m * bf16lo_to_f32(w[k]);
      acc[2 * k + 1] += m * bf16hi_to_f32(w[k]);
    }
  }
  reinterpret_cast<uint4*>(out)[i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

// A warp per entry.
__global__ void __launch_bounds__(256)
    combine_dweights_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y,
                            const int32_t* __restrict__ row_of, int64_t entries, int top_k, int64_t P, int64_t chunks,
                            float* __restrict__ dweights, int* status) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= entries) return;
  const int64_t r = checked_row(row_of, i, P, status);
  float acc = 0.f;
  if (r >= 0) {
    for (int64_t c = lane; c < chunks; c += 32) {
      const uint4 a = reinterpret_cast<const uint4*>(dout)[i / top_k * chunks + c];
      const uint4 b = reinterpret_cast<const uint4*>(y)[r * chunks + c];
      const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
      for (int k = 0; k < 4; ++k) {
        acc = fmaf(bf16lo_to_f32(u[k]), bf16lo_to_f32(v[k]), acc);
        acc = fmaf(bf16hi_to_f32(u[k]), bf16hi_to_f32(v[k]), acc);
      }
    }
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kAll, acc, o);
  }
  if (lane == 0) dweights[i] = acc;
}

}  // namespace

cudaError_t launch_moe_gather_quant(const MoeGatherArgs& a, cudaStream_t st) {
  const int64_t bands = (a.P + 127) / 128, blocks = bands * ((a.C + 127) / 128);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    kernel<<<dim3(static_cast<unsigned>(blocks)), kGatherWarps * 32, 0, st>>>(
        a.x, a.weights, a.src_of, static_cast<uint32_t>(a.M * a.top_k), static_cast<uint32_t>(a.top_k),
        static_cast<int>(a.P), static_cast<int>(a.C), static_cast<int>(bands), a.q, a.e8, a.qT, a.e8T, a.mode, a.status);
    return cudaGetLastError();
  };
  return a.weights != nullptr ? go(gather_quant_kernel<true>) : go(gather_quant_kernel<false>);
}

cudaError_t launch_moe_combine(const MoeCombineArgs& a, cudaStream_t st) {
  const int64_t chunks = a.C / 8, total = a.M * chunks;
  combine_kernel<<<dim3(static_cast<unsigned>((total + 255) / 256)), 256, 0, st>>>(
      a.y, a.weights, a.row_of, a.base, chunks, total, static_cast<int>(a.top_k), a.P, a.out, a.status);
  return cudaGetLastError();
}

cudaError_t launch_moe_combine_dweights(const MoeCombineArgs& a, cudaStream_t st) {
  const int64_t entries = a.M * a.top_k;
  combine_dweights_kernel<<<dim3(static_cast<unsigned>((entries + 7) / 8)), 256, 0, st>>>(
      a.dout, a.y, a.row_of, entries, static_cast<int>(a.top_k), a.P, a.C / 8, a.dweights, a.status);
  return cudaGetLastError();
}

}  // namespace fp8bw
