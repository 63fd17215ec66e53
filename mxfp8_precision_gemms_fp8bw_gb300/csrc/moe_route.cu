// Routing of a mixture-of-experts layer: scores, the choice of experts and
// its gradient, and the sort of the choices into expert groups.
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace fp8bw {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLowest = -3.4028234663852886e38f;

__device__ __forceinline__ float logit_at(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit_at(const uint16_t* p, int64_t i) { return __uint_as_float(uint32_t{p[i]} << 16); }
__device__ __forceinline__ void put_logit(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put_logit(uint16_t* p, int64_t i, float v) {
  p[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xFFFFu);
}

// Keys as unsigned integers of the same order: 0 is a masked expert, below
// the lowest finite key (0x00800000), and NaN is above everything.
__device__ __forceinline__ uint32_t ordered(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t b = __float_as_uint(f + 0.f);  // -0 becomes +0
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  if (u == 0xffffffffu) return __uint_as_float(0x7FFFFFFFu);
  return __uint_as_float((u >> 31) ? u & 0x7FFFFFFFu : ~u);
}

// The scores of one row; a lane holds experts v * 32 + lane.  Divisions and
// exponentials are the correctly rounded or library forms and the sum runs by
// halves (first over v, then over lanes), because the choice has to come out
// the same however the row is split.
template <int V>
__device__ __forceinline__ void scores_of(const float (&x)[V], int E, int lane, int score, float (&s)[V]) {
  if (score != 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 1.f / (1.f + expf(-x[v]));
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  const bool empty = top == -INFINITY;
  // NaN in the row makes every score NaN through the sum; an empty row has none.
  float part[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = empty ? (x[v] != x[v] ? x[v] : 0.f) : expf(x[v] - top);
    part[v] = s[v];
  }
#pragma unroll
  for (int h = V / 2; h > 0; h /= 2)
#pragma unroll
    for (int v = 0; v < h; ++v) part[v] += part[v + h];
  float total = part[0];
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = empty ? s[v] + total : s[v] / total;
}

struct RouteShape {
  int64_t M;
  int E, k, groups, kept, group_top, score, renorm;
  float scale;
};

constexpr int kRouteWarps = 4;

template <typename T, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const T* __restrict__ logits,
                                                                 const float* __restrict__ bias, RouteShape p,
                                                                 int32_t* __restrict__ experts,
                                                                 float* __restrict__ weights) {
  extern __shared__ uint32_t staged[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (row >= p.M) return;
  float x[V], s[V];
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + lane;
    x[v] = e < p.E ? logit_at(logits, row * p.E + e) : -INFINITY;
  }
  scores_of<V>(x, p.E, lane, p.score, s);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + lane;
    const float b = bias != nullptr && e < p.E ? bias[e] : 0.f;
    const bool masked = e >= p.E || x[v] == -INFINITY || b == -INFINITY;
    key[v] = masked ? 0u : ordered(s[v] + b);
  }

  if (p.groups > 1) {
    // Lane g scores group g from the keys in shared memory.
    uint32_t* mine = staged + warp * p.E;
    const int size = p.E / p.groups;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane < p.E) mine[v * 32 + lane] = key[v];
    __syncwarp();
    uint32_t best = 0, second = 0;
    if (lane < p.groups) {
      for (int i = 0; i < size; ++i) {
        const uint32_t u = mine[lane * size + i];
        second = max(second, min(best, u));
        best = max(best, u);
      }
    }
    uint32_t total = best;
    if (p.group_top == 2 && second != 0 && best != 0) {
      const float sum = unordered(best) + unordered(second);
      total = ordered(sum < kLowest ? kLowest : sum);
    }
    uint32_t kept = 0;
    for (int i = 0; i < p.kept; ++i) {
      const uint32_t m = __reduce_max_sync(kAll, total);
      if (m == 0) break;
      const int g = __ffs(__ballot_sync(kAll, total == m)) - 1;
      kept |= 1u << g;
      if (lane == g) total = 0;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      if (e < p.E && !((kept >> (e / size)) & 1u)) key[v] = 0;
    }
  }

  int chosen = -1;
  float cs = 0.f;
  for (int j = 0; j < p.k; ++j) {
    uint32_t local = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) local = max(local, key[v]);
    const uint32_t m = __reduce_max_sync(kAll, local);
    if (m == 0) break;
    uint32_t e = 0xffffffffu;
    float sv = 0.f;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (key[v] == m) {
        e = v * 32 + lane;
        sv = s[v];
      }
    const uint32_t win = __reduce_min_sync(kAll, e);
    sv = __shfl_sync(kAll, sv, win & 31);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane == static_cast<int>(win)) key[v] = 0;
    if (lane == j) {
      chosen = static_cast<int>(win);
      cs = sv;
    }
  }
  float w = cs * p.scale;
  if (p.renorm) {
    float total = cs;
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    w = cs / (total + 1e-20f) * p.scale;
  }
  if (lane < p.k) {
    experts[row * p.k + lane] = chosen;
    weights[row * p.k + lane] = w;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_bwd_kernel(const float* __restrict__ dw, const T* __restrict__ logits, const int32_t* __restrict__ experts,
                     RouteShape p, T* __restrict__ dlogits, int* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (row >= p.M) return;
  float x[V], s[V], g[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + lane;
    x[v] = e < p.E ? logit_at(logits, row * p.E + e) : -INFINITY;
    g[v] = 0.f;
  }
  scores_of<V>(x, p.E, lane, p.score, s);
  int mine = lane < p.k ? experts[row * p.k + lane] : -1;
  if (mine < -1 || mine >= p.E) {
    atomicExch(status, kStatusShape);
    mine = -1;
  }
  // Lane j holds choice j: its score and the gradient of its score.
  float cs = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float t = __shfl_sync(kAll, s[v], mine & 31);
    if (mine >= 0 && (mine >> 5) == v) cs = t;
  }
  float ds = mine >= 0 ? dw[row * p.k + lane] * p.scale : 0.f;
  if (p.renorm) {
    float total = cs, dot = mine >= 0 ? ds * cs : 0.f;
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(kAll, total, o);
      dot += __shfl_xor_sync(kAll, dot, o);
    }
    total += 1e-20f;
    ds = mine >= 0 ? (ds - dot / total) / total : 0.f;
  }
  for (int j = 0; j < p.k; ++j) {
    const int e = __shfl_sync(kAll, mine, j);
    const float d = __shfl_sync(kAll, ds, j);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * 32 + lane == e) g[v] = d;
  }
  float dot = mine >= 0 ? ds * cs : 0.f;
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * 32 + lane;
    const float d = p.score != 0 ? g[v] * s[v] * (1.f - s[v]) : s[v] * (g[v] - dot);
    if (e < p.E) put_logit(dlogits, row * p.E + e, d);
  }
}

// One CTA: per-warp counts of contiguous runs of entries, their prefix over
// warps and experts, then the entries take their rows in order.
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ int checked_expert(const int32_t* experts, int64_t i, int64_t N, int E, int* status) {
  int e = i < N ? experts[i] : -1;
  if (e < -1 || e >= E) {
    atomicExch(status, kStatusShape);
    e = -1;
  }
  return e;
}

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int32_t* __restrict__ experts, int64_t N, int E, int64_t P, int32_t* __restrict__ group_end,
                int32_t* __restrict__ counts, int32_t* __restrict__ row_of, int32_t* __restrict__ src_of, int* status) {
  extern __shared__ int next[];  // [kPlanWarps][E], then the group starts [E + 1]
  int* start = next + kPlanWarps * E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kPlanWarps * E; i += kPlanThreads) next[i] = 0;
  __syncthreads();
  const int64_t run = (N + kPlanThreads - 1) / kPlanThreads * 32;  // entries of a warp
  const int64_t first = warp * run, last = min(first + run, N);
  int* my = next + warp * E;
  for (int64_t i0 = first; i0 < last; i0 += 32) {
    const int e = checked_expert(experts, i0 + lane, last, E, status);
    const uint32_t same = __match_any_sync(kAll, e);
    if (e >= 0 && lane == __ffs(same) - 1) my[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e < E; e += kPlanThreads) {
    int sum = 0;
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = next[w * E + e];
      next[w * E + e] = sum;
      sum += c;
    }
    counts[e] = sum;
    start[e + 1] = sum;
  }
  __syncthreads();
  if (tid == 0) {
    int at = 0;
    start[0] = 0;
    for (int e = 0; e < E; ++e) {
      at += (start[e + 1] + 31) & ~31;
      start[e + 1] = at;
      group_end[e] = e + 1 == E ? static_cast<int>(P) : at;
    }
  }
  __syncthreads();
  for (int64_t i0 = first; i0 < last; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = checked_expert(experts, i, last, E, status);
    const uint32_t same = __match_any_sync(kAll, e);
    int row = -1;
    if (e >= 0) row = start[e] + my[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) my[e] += __popc(same);
    __syncwarp();
    if (i < last) row_of[i] = row;
    if (row >= 0) src_of[row] = static_cast<int32_t>(i);
  }
  __syncthreads();
  for (int e = warp; e < E; e += kPlanWarps) {  // the empty rows of each group
    const int used = start[e] + next[(kPlanWarps - 1) * E + e];
    if (used + lane < start[e + 1]) src_of[used + lane] = -1;
  }
  for (int64_t p = start[E] + tid; p < P; p += kPlanThreads) src_of[p] = -1;
}

template <typename T>
cudaError_t route_of(const MoeRouteArgs& a, cudaStream_t st) {
  const RouteShape p{a.M,
                     static_cast<int>(a.E),
                     static_cast<int>(a.top_k),
                     static_cast<int>(a.groups),
                     static_cast<int>(a.groups_kept),
                     static_cast<int>(a.group_top),
                     a.score,
                     a.renorm,
                     a.scale};
  const dim3 grid(static_cast<unsigned>((a.M + kRouteWarps - 1) / kRouteWarps));
  const T* logits = static_cast<const T*>(a.logits);
  auto go = [&](auto W) {
    constexpr int V = decltype(W)::value;
    if (a.dlogits != nullptr) {
      route_bwd_kernel<T, V><<<grid, kRouteWarps * 32, 0, st>>>(a.dweights, logits, a.experts_in, p,
                                                               static_cast<T*>(a.dlogits), a.status);
    } else {
      const size_t smem = a.groups > 1 ? kRouteWarps * a.E * sizeof(uint32_t) : 0;
      route_kernel<T, V><<<grid, kRouteWarps * 32, smem, st>>>(logits, a.bias, p, a.experts, a.weights);
    }
    return cudaGetLastError();
  };
  if (a.E <= 32) return go(std::integral_constant<int, 1>{});
  if (a.E <= 64) return go(std::integral_constant<int, 2>{});
  if (a.E <= 128) return go(std::integral_constant<int, 4>{});
  if (a.E <= 256) return go(std::integral_constant<int, 8>{});
  if (a.E <= 512) return go(std::integral_constant<int, 16>{});
  return go(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t st) {
  return a.bf16 ? route_of<uint16_t>(a, st) : route_of<float>(a, st);
}

size_t moe_plan_workspace_bytes(int64_t, int64_t, int64_t) { return 16; }

cudaError_t launch_moe_plan(const MoePlanArgs& a, cudaStream_t st) {
  const size_t smem = (kPlanWarps * a.E + a.E + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  plan_kernel<<<1, kPlanThreads, smem, st>>>(a.experts, a.M * a.top_k, static_cast<int>(a.E), a.P, a.group_end,
                                             a.counts, a.row_of, a.src_of, a.status);
  return cudaGetLastError();
}

}  // namespace fp8bw
