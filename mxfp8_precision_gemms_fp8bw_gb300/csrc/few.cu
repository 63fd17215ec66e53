// Products of a few tokens with MX weights: a linear, and a mixture-of-experts
// layer.  The plain way: a warp per row of the weights, fp32 throughout.
#include "launch.h"
#include "mx_weight.cuh"

namespace fp8bw {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ float2 half2_to_f32(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h));
  return r;
}

__device__ __forceinline__ float value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float value(const uint16_t* p, int64_t i) { return __uint_as_float(uint32_t{p[i]} << 16); }

// sum over k of W[row, k] v[k], by a warp.
template <int kBits, typename T>
__device__ float row_dot(const uint8_t* w, const uint8_t* e8, int64_t row, int64_t K, const T* v, int lane) {
  float sum = 0.f;
  for (int64_t g = lane; g < K / 32; g += 32) {
    float part = 0.f, s[4];
    const uint32_t* words = reinterpret_cast<const uint32_t*>(w + (row * K + g * 32) / 8 * kBits);
    for (int i = 0; i < kBits; ++i) {  // words of the block
      const uint32_t c = words[i];
      const int64_t k = g * 32 + i * (32 / kBits);
      float2 p[4];
      if (kBits == 4) {
        p[0] = half2_to_f32(e2m1x2_to_f16x2<0>(c));
        p[1] = half2_to_f32(e2m1x2_to_f16x2<1>(c));
        p[2] = half2_to_f32(e2m1x2_to_f16x2<2>(c));
        p[3] = half2_to_f32(e2m1x2_to_f16x2<3>(c));
      } else {
        p[0] = half2_to_f32(e4m3x2_to_f16x2<0>(c));
        p[1] = half2_to_f32(e4m3x2_to_f16x2<1>(c));
      }
      for (int j = 0; j < 16 / kBits; ++j)
        part += p[j].x * value(v, k + 2 * j) + p[j].y * value(v, k + 2 * j + 1);
    }
    e8m0x4_to_f32(e8[row * (K / 32) + g], s);
    sum += part * s[0];
  }
  return warp_sum(sum);
}

template <int kBits>
__global__ void __launch_bounds__(kWarps * 32) linear_kernel(FewLinearArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (n >= a.N) return;
  for (int64_t t = 0; t < a.M; ++t) {
    const float y = row_dot<kBits>(a.w, a.e8, n, a.K, a.x + t * a.K, lane);
    if (lane == 0) a.y[t * a.N + n] = static_cast<uint16_t>(pack_bf16x2(y, 0.f) & 0xFFFFu);
  }
}

__global__ void __launch_bounds__(kWarps * 32) logits_kernel(FewMoeArgs a, float* logits) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32, E = a.route.E;
  if (i >= a.route.M * E) return;
  float sum = 0.f;
  for (int64_t c = lane; c < a.C; c += 32) sum += value(a.x, i / E * a.C + c) * a.router[i % E * a.C + c];
  sum = warp_sum(sum);
  if (lane == 0) logits[i] = sum;
}

template <int kBits>
__global__ void __launch_bounds__(kWarps * 32) up_kernel(FewMoeArgs a, const int32_t* experts, float* act) {
  const int lane = threadIdx.x & 31;
  const int64_t f = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32, entry = blockIdx.y;
  const int64_t e = experts[entry];
  if (f >= a.F || e < 0) return;
  const uint16_t* x = a.x + entry / a.route.top_k * a.C;
  const float gate = row_dot<kBits>(a.w13, a.e13, e * 2 * a.F + f, a.C, x, lane);
  const float up = row_dot<kBits>(a.w13, a.e13, e * 2 * a.F + a.F + f, a.C, x, lane);
  if (lane == 0) act[entry * a.F + f] = gate / (1.f + expf(-gate)) * up;
}

template <int kBits>
__global__ void __launch_bounds__(kWarps * 32)
    down_kernel(FewMoeArgs a, const int32_t* experts, const float* weights, const float* act) {
  const int lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32, t = blockIdx.y;
  if (c >= a.C) return;
  float sum = 0.f;
  for (int64_t entry = t * a.route.top_k; entry < (t + 1) * a.route.top_k; ++entry) {
    const int64_t e = experts[entry];
    if (e >= 0) sum += weights[entry] * row_dot<kBits>(a.w2, a.e2, e * a.C + c, a.F, act + entry * a.F, lane);
  }
  if (lane == 0) a.y[t * a.C + c] = static_cast<uint16_t>(pack_bf16x2(sum, 0.f) & 0xFFFFu);
}

unsigned blocks_of(int64_t warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

struct Scratch {
  float* logits;
  int32_t* experts;
  float* weights;
  float* act;
  size_t bytes;
};

Scratch scratch_of(void* p, int64_t M, int64_t E, int64_t k, int64_t F) {
  const auto up = [](int64_t n) { return (n * 4 + 255) / 256 * 256; };
  char* b = static_cast<char*>(p);
  Scratch s{};
  s.logits = reinterpret_cast<float*>(b);
  s.experts = reinterpret_cast<int32_t*>(b + up(M * E));
  s.weights = reinterpret_cast<float*>(b + up(M * E) + up(M * k));
  s.act = reinterpret_cast<float*>(b + up(M * E) + 2 * up(M * k));
  s.bytes = up(M * E) + 2 * up(M * k) + up(M * k * F);
  return s;
}

}  // namespace

cudaError_t launch_few_linear(const FewLinearArgs& a, cudaStream_t st) {
  if (a.bits == 4)
    linear_kernel<4><<<blocks_of(a.N), kWarps * 32, 0, st>>>(a);
  else
    linear_kernel<8><<<blocks_of(a.N), kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

size_t few_moe_workspace_bytes(int64_t M, int64_t E, int64_t top_k, int64_t, int64_t F) {
  return scratch_of(nullptr, M, E, top_k, F).bytes;
}

cudaError_t launch_few_moe(const FewMoeArgs& a, cudaStream_t st) {
  const Scratch s = scratch_of(a.workspace, a.route.M, a.route.E, a.route.top_k, a.F);
  logits_kernel<<<blocks_of(a.route.M * a.route.E), kWarps * 32, 0, st>>>(a, s.logits);
  MoeRouteArgs r = a.route;
  r.logits = s.logits;
  r.experts = s.experts;
  r.weights = s.weights;
  if (const cudaError_t e = launch_moe_route(r, st)) return e;
  const dim3 up(blocks_of(a.F), static_cast<unsigned>(r.M * r.top_k)), down(blocks_of(a.C), static_cast<unsigned>(r.M));
  if (a.bits == 4) {
    up_kernel<4><<<up, kWarps * 32, 0, st>>>(a, s.experts, s.act);
    down_kernel<4><<<down, kWarps * 32, 0, st>>>(a, s.experts, s.weights, s.act);
  } else {
    up_kernel<8><<<up, kWarps * 32, 0, st>>>(a, s.experts, s.act);
    down_kernel<8><<<down, kWarps * 32, 0, st>>>(a, s.experts, s.weights, s.act);
  }
  return cudaGetLastError();
}

}  // namespace fp8bw
