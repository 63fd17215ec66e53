// Rows of the experts: gathering tokens into them as MX codes, and summing
// them back into the tokens.
#include "common.cuh"
#include "launch.h"
#include "mx_fp32.cuh"

namespace fp8bw {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// 32 rows x 128 columns per CTA.
__global__ void __launch_bounds__(128)
    gather_quant_kernel(const uint16_t* __restrict__ x, const float* __restrict__ weights,
                        const int32_t* __restrict__ src_of, int64_t entries, int top_k, int64_t P, int64_t C,
                        uint8_t* __restrict__ q, uint8_t* __restrict__ e8, uint8_t* __restrict__ qT,
                        uint8_t* __restrict__ e8T, int mode, int* status) {
  __shared__ QuantTile t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 128, r0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int64_t col = c0 + 4 * lane;
  for (int i = 0; i < 8; ++i) {
    const int r = warp * 8 + i;
    int64_t src = src_of[r0 + r];
    if (src < -1 || src >= entries) {
      atomicExch(status, kStatusShape);
      src = -1;
    }
    uint2 w = make_uint2(0, 0);
    if (src >= 0 && col < C) w = *reinterpret_cast<const uint2*>(x + src / top_k * C + col);
    const float m = weights != nullptr && src >= 0 ? weights[src] : 1.f;
    t.v[r][4 * lane] = bf16lo_to_f32(w.x) * m;
    t.v[r][4 * lane + 1] = bf16hi_to_f32(w.x) * m;
    t.v[r][4 * lane + 2] = bf16lo_to_f32(w.y) * m;
    t.v[r][4 * lane + 3] = bf16hi_to_f32(w.y) * m;
  }
  __syncthreads();
  const uint32_t round = mx_round_f32(mode);
  quant_tile_rows(t, r0, c0, C, C, q, e8, round);
  if (qT != nullptr) quant_tile_cols(t, r0, c0, P, C, qT, e8T, round);
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
  const dim3 grid(static_cast<unsigned>(a.P / 32), static_cast<unsigned>((a.C + 127) / 128));
  gather_quant_kernel<<<grid, 128, 0, st>>>(a.x, a.weights, a.src_of, a.M * a.top_k, static_cast<int>(a.top_k), a.P,
                                            a.C, a.q, a.e8, a.qT, a.e8T, a.mode, a.status);
  return cudaGetLastError();
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
