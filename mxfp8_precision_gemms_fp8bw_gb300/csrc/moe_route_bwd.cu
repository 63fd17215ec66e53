// The gradient of routing (moe_route.cu).
#include "route_row.cuh"

namespace fp8bw {
namespace {

template <typename T, int L, int V>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_bwd_kernel(const float* __restrict__ dw, const T* __restrict__ logits, const int32_t* __restrict__ experts,
                     RouteShape p, T* __restrict__ dlogits, int* status) {
  constexpr int kRowsPerWarp = 32 / L;
  constexpr int K = (32 + L - 1) / L;
  extern __shared__ uint32_t staged[];
  const int l = threadIdx.x & (L - 1), mine = threadIdx.x / L;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRouteWarps * kRowsPerWarp) + mine;
  const bool live = row < p.M;
  float x[V], s[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    x[v] = live && e < p.E ? logit_at(logits, row * p.E + e) : -INFINITY;
  }
  int at[K];
  float ds[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int c = j * L + l;
    at[j] = -1;
    ds[j] = 0.f;
    if (j * L >= p.k) continue;
    at[j] = live && c < p.k ? experts[row * p.k + c] : -1;
    if (at[j] < -1 || at[j] >= p.E) {
      atomicExch(status, kStatusShape);
      at[j] = -1;
    }
    ds[j] = at[j] >= 0 ? dw[row * p.k + c] * p.scale : 0.f;
  }
  scores_of<L, V, false>(x, p.score, s);
  // The chosen scores come by way of shared memory.
  float* scores = reinterpret_cast<float*>(staged) + mine * (p.E | 8);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * L + l < p.E) scores[v * L + l] = s[v];
  __syncwarp();
  float cs[K], sum = 0.f, dot = 0.f;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    cs[j] = 0.f;
    if (j * L >= p.k) continue;
    cs[j] = at[j] >= 0 ? scores[at[j]] : 0.f;
    sum += cs[j];
    dot += at[j] >= 0 ? ds[j] * cs[j] : 0.f;
  }
  if (p.renorm) {
    sum = lanes_sum<L>(sum) + 1e-20f;
    dot = lanes_sum<L>(dot);
    float rest = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j * L >= p.k) continue;
      ds[j] = at[j] >= 0 ? (ds[j] - dot / sum) / sum : 0.f;
      rest += at[j] >= 0 ? ds[j] * cs[j] : 0.f;
    }
    dot = rest;
  }
  dot = lanes_sum<L>(dot);
  // What every expert gets, then, behind the barrier, what the chosen ones get in its place.
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    if (live && e < p.E) put_logit(dlogits, row * p.E + e, p.score != 0 ? 0.f * s[v] : s[v] * (0.f - dot));
  }
  __syncwarp();
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (at[j] >= 0)
      put_logit(dlogits, row * p.E + at[j], p.score != 0 ? ds[j] * cs[j] * (1.f - cs[j]) : cs[j] * (ds[j] - dot));
}

template <typename T>
cudaError_t route_bwd_of(const MoeRouteArgs& a, cudaStream_t st) {
  return for_experts(a.E, [&](auto lanes, auto width) {
    constexpr int L = decltype(lanes)::value, V = decltype(width)::value;
    const dim3 grid(static_cast<unsigned>((a.M + kRouteRows<L> - 1) / kRouteRows<L>));
    route_bwd_kernel<T, L, V><<<grid, kRouteWarps * 32, staged_bytes<L>(a.E), st>>>(
        a.dweights, static_cast<const T*>(a.logits), a.experts_in, shape_of(a), static_cast<T*>(a.dlogits), a.status);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_moe_route_bwd(const MoeRouteArgs& a, cudaStream_t st) {
  return a.bf16 ? route_bwd_of<uint16_t>(a, st) : route_bwd_of<float>(a, st);
}

}  // namespace fp8bw
