// The gated activation of an MXFP8 layer, held as MX codes, with its input
// kept in 8 bits, and its gradient from those 8 bits.
#include "common.cuh"
#include "launch.h"
#include "mx_fp32.cuh"

namespace fp8bw {
namespace {

__device__ __forceinline__ float sigmoid_f32(float x) { return 1.f / (1.f + __expf(-x)); }

// 32 rows x 128 columns of a per CTA; the same columns of gate and up.
__global__ void __launch_bounds__(128)
    swiglu_kernel(const uint16_t* __restrict__ h, int64_t R, int64_t F, uint8_t* __restrict__ aq,
                  uint8_t* __restrict__ ae, uint8_t* __restrict__ aqT, uint8_t* __restrict__ aeT,
                  uint8_t* __restrict__ hq, uint8_t* __restrict__ he, int mode) {
  __shared__ QuantTile gate, up;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 128, r0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int64_t col = c0 + 4 * lane;
  const uint32_t round = mx_round_f32(mode);
  for (int i = 0; i < 8; ++i) {
    const int r = warp * 8 + i;
    uint2 g = make_uint2(0, 0), u = g;
    if (col < F) {
      g = *reinterpret_cast<const uint2*>(h + (r0 + r) * 2 * F + col);
      u = *reinterpret_cast<const uint2*>(h + (r0 + r) * 2 * F + F + col);
    }
    const float gv[4] = {bf16lo_to_f32(g.x), bf16hi_to_f32(g.x), bf16lo_to_f32(g.y), bf16hi_to_f32(g.y)};
    const float uv[4] = {bf16lo_to_f32(u.x), bf16hi_to_f32(u.x), bf16lo_to_f32(u.y), bf16hi_to_f32(u.y)};
    for (int k = 0; k < 4; ++k) {
      gate.v[r][4 * lane + k] = gv[k];
      up.v[r][4 * lane + k] = uv[k];
    }
  }
  __syncthreads();
  if (hq != nullptr) {
    quant_tile_rows(gate, r0, c0, 2 * F, F, hq, he, round);
    quant_tile_rows(up, r0, F + c0, 2 * F, 2 * F, hq, he, round);
  }
  for (int i = threadIdx.x; i < 32 * 128; i += 128) {
    const float g = gate.v[i >> 7][i & 127];
    gate.v[i >> 7][i & 127] = g * sigmoid_f32(g) * up.v[i >> 7][i & 127];
  }
  __syncthreads();
  quant_tile_rows(gate, r0, c0, F, F, aq, ae, round);
  if (aqT != nullptr) quant_tile_cols(gate, r0, c0, R, F, aqT, aeT, round);
}

__global__ void __launch_bounds__(128)
    swiglu_bwd_kernel(const uint16_t* __restrict__ da, const uint8_t* __restrict__ hq, const uint8_t* __restrict__ he,
                      int64_t R, int64_t F, uint8_t* __restrict__ dq, uint8_t* __restrict__ de,
                      uint8_t* __restrict__ dqT, uint8_t* __restrict__ deT, int mode) {
  __shared__ QuantTile dgate, dup;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 128, r0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int64_t col = c0 + 4 * lane;
  const uint32_t round = mx_round_f32(mode);
  for (int i = 0; i < 8; ++i) {
    const int r = warp * 8 + i;
    const int64_t row = r0 + r;
    float g[4] = {}, u[4] = {}, d[4] = {};
    if (col < F) {
      const uint32_t gc = *reinterpret_cast<const uint32_t*>(hq + row * 2 * F + col);
      const uint32_t uc = *reinterpret_cast<const uint32_t*>(hq + row * 2 * F + F + col);
      const float gs = e8m0_value(he[row * (2 * F / 32) + col / 32]);
      const float us = e8m0_value(he[row * (2 * F / 32) + (F + col) / 32]);
      const uint2 w = *reinterpret_cast<const uint2*>(da + row * F + col);
      const float2 g0 = e4m3x2_to_f32(gc & 0xFFFF), g1 = e4m3x2_to_f32(gc >> 16);
      const float2 u0 = e4m3x2_to_f32(uc & 0xFFFF), u1 = e4m3x2_to_f32(uc >> 16);
      g[0] = g0.x * gs, g[1] = g0.y * gs, g[2] = g1.x * gs, g[3] = g1.y * gs;
      u[0] = u0.x * us, u[1] = u0.y * us, u[2] = u1.x * us, u[3] = u1.y * us;
      d[0] = bf16lo_to_f32(w.x), d[1] = bf16hi_to_f32(w.x), d[2] = bf16lo_to_f32(w.y), d[3] = bf16hi_to_f32(w.y);
    }
    for (int k = 0; k < 4; ++k) {
      const float sig = sigmoid_f32(g[k]);
      dgate.v[r][4 * lane + k] = d[k] * u[k] * sig * (1.f + g[k] * (1.f - sig));
      dup.v[r][4 * lane + k] = d[k] * g[k] * sig;
    }
  }
  __syncthreads();
  quant_tile_rows(dgate, r0, c0, 2 * F, F, dq, de, round);
  quant_tile_rows(dup, r0, F + c0, 2 * F, 2 * F, dq, de, round);
  quant_tile_cols(dgate, r0, c0, R, F, dqT, deT, round);
  quant_tile_cols(dup, r0, F + c0, R, 2 * F, dqT, deT, round);
}

dim3 grid_of(int64_t R, int64_t F) {
  return dim3(static_cast<unsigned>(R / 32), static_cast<unsigned>((F + 127) / 128));
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t st) {
  swiglu_kernel<<<grid_of(a.R, a.F), 128, 0, st>>>(a.h, a.R, a.F, a.aq, a.ae, a.aqT, a.aeT, a.hq, a.he, a.mode);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t st) {
  swiglu_bwd_kernel<<<grid_of(a.R, a.F), 128, 0, st>>>(a.da, a.hq, a.he, a.R, a.F, a.dq, a.de, a.dqT, a.deT, a.mode);
  return cudaGetLastError();
}

}  // namespace fp8bw
