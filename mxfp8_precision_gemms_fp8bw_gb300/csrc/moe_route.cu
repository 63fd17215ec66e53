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

// ---------------------------------------------------------------- plan
//
// A stable counting sort in which the entries keep their order: block b owns
// `chunk` consecutive entries and each of its warps a consecutive run of
// them, so an entry's row is the start of its group + the entries of its
// expert in earlier blocks + in earlier warps + before it in its own run (the
// lower lanes of the same 32 that have the same expert, by a warp match).
// Nothing depends on the order in which blocks or atomics come.
//
// It reads and writes a few bytes per entry and is bound by latency: one
// launch while one block suffices, two beyond that (counts per block, then
// the rows), of which the second starts under the first and counts its own
// runs meanwhile.
constexpr int kPlanChunk = 2048;     // entries per block, more where that would be over kPlanBlocks blocks
constexpr int kPlanBlocks = 152;
constexpr int kPlanHistogram = 1 << 14;  // blocks * E of the counts: every block reads them all

struct PlanShape {
  int64_t N, chunk, P;
  int E, blocks, threads;
};

PlanShape plan_shape(int64_t M, int64_t E, int64_t top_k, int64_t P) {
  PlanShape s{};
  s.N = M * top_k;
  s.E = static_cast<int>(E);
  s.P = P;
  int64_t blocks = (s.N + kPlanChunk - 1) / kPlanChunk;
  if (blocks > kPlanBlocks) blocks = kPlanBlocks;
  if (blocks > kPlanHistogram / E) blocks = kPlanHistogram / E;
  if (s.N <= 2 * kPlanChunk) blocks = 1;
  s.blocks = static_cast<int>(blocks);
  s.chunk = (s.N + blocks - 1) / blocks;
  s.threads = s.N <= 1024 ? 256 : 1024;
  return s;
}

__device__ __forceinline__ int checked_expert(const int32_t* experts, int64_t i, int64_t last, int E, int* status) {
  int e = i < last ? experts[i] : -1;
  if (e < -1 || e >= E) {
    atomicExch(status, kStatusShape);
    e = -1;
  }
  return e;
}

__global__ void __launch_bounds__(1024)
    plan_count_kernel(const int32_t* __restrict__ experts, PlanShape s, int32_t* __restrict__ histogram, int* status) {
  extern __shared__ int smem[];  // [E]
  asm volatile("griddepcontrol.launch_dependents;");
  for (int e = threadIdx.x; e < s.E; e += s.threads) smem[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * s.chunk, last = min(first + s.chunk, s.N);
  for (int64_t i0 = first + (threadIdx.x & ~31); i0 < last; i0 += s.threads) {
    const int lane = threadIdx.x & 31;
    const int e = checked_expert(experts, i0 + lane, last, s.E, status);
    const uint32_t same = __match_any_sync(kAll, e);
    if (e >= 0 && lane == __ffs(same) - 1) atomicAdd(&smem[e], __popc(same));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < s.E; e += s.threads) histogram[static_cast<int64_t>(blockIdx.x) * s.E + e] = smem[e];
}

__global__ void __launch_bounds__(1024)
    plan_place_kernel(const int32_t* __restrict__ experts, PlanShape s, const int32_t* histogram,
                      int32_t* __restrict__ group_end, int32_t* __restrict__ counts, int32_t* __restrict__ row_of,
                      int32_t* __restrict__ src_of, int* status) {
  extern __shared__ int smem[];
  const int E = s.E, T = s.threads, warps = T / 32;
  int* next = smem;               // [warps][E]: the next row of an expert in a warp's run, less the group's start
  int* start = next + warps * E;  // [E + 1]: the groups' first rows
  int* total = start + E + 1;     // [E]: entries of an expert
  int* sums = total + E;          // [33]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < warps * E; i += T) next[i] = 0;
  for (int e = tid; e < E; e += T) total[e] = start[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * s.chunk, last = min(first + s.chunk, s.N);
  const int64_t run = (s.chunk + T - 1) / T * 32;
  const int64_t mine = first + warp * run, end = min(mine + run, last);
  int* my = next + warp * E;
  for (int64_t i0 = mine; i0 < end; i0 += 32) {
    const int e = checked_expert(experts, i0 + lane, end, E, status);
    const uint32_t same = __match_any_sync(kAll, e);
    if (e >= 0 && lane == __ffs(same) - 1) my[e] += __popc(same);
    __syncwarp();
  }
  if (s.blocks > 1) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Threads in E columns and as many slices of blocks as fit; start[] holds
    // the entries in earlier blocks for now.
    const int slices = max(T / E, 1);
    for (int i = tid; i < slices * E; i += T) {
      const int e = i % E;
      int all = 0, before = 0;
      for (int b = i / E; b < s.blocks; b += slices) {
        const int c = histogram[b * E + e];
        all += c;
        before += b < static_cast<int>(blockIdx.x) ? c : 0;
      }
      atomicAdd(&total[e], all);
      atomicAdd(&start[e], before);
    }
  }
  __syncthreads();
  // Exclusive prefix over the warps, then over the experts' padded totals.
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += T) {
    const int e = e0 + tid;
    int padded = 0;
    if (e < E) {
      int sum = start[e];
      for (int w = 0; w < warps; ++w) {
        const int c = next[w * E + e];
        next[w * E + e] = sum;
        sum += c;
      }
      if (s.blocks == 1) total[e] = sum;
      padded = (total[e] + 31) & ~31;
    }
    int up = padded;
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(kAll, up, o);
      if (lane >= o) up += t;
    }
    if (lane == 31) sums[warp] = up;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
      before += w < warp ? sums[w] : 0;
      all += sums[w];
    }
    if (e < E) start[e] = carry + before + up - padded;
    carry += all;
    if (e == E - 1) start[E] = carry;
    if (e < E && blockIdx.x == 0) {
      counts[e] = total[e];
      group_end[e] = e + 1 == E ? static_cast<int>(s.P) : start[e] + padded;
    }
    __syncthreads();
  }
  for (int64_t i0 = mine; i0 < end; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = checked_expert(experts, i, end, E, status);
    const uint32_t same = __match_any_sync(kAll, e);
    int row = -1;
    if (e >= 0) row = start[e] + my[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) my[e] += __popc(same);
    __syncwarp();
    if (i < end) row_of[i] = row;
    if (row >= 0) src_of[row] = static_cast<int32_t>(i);
  }
  // The empty rows: of each group, and behind the last one.
  const int workers = warps * s.blocks;
  for (int e = blockIdx.x * warps + warp; e < E; e += workers) {
    const int used = start[e] + total[e];
    if (used + lane < start[e + 1]) src_of[used + lane] = -1;
  }
  for (int64_t p = start[E] + static_cast<int64_t>(blockIdx.x) * T + tid; p < s.P; p += static_cast<int64_t>(s.blocks) * T)
    src_of[p] = -1;
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

size_t moe_plan_workspace_bytes(int64_t M, int64_t E, int64_t top_k) {
  const PlanShape s = plan_shape(M, E, top_k, 0);
  const size_t n = s.blocks > 1 ? static_cast<size_t>(s.blocks) * s.E * sizeof(int32_t) : 0;
  return n < 16 ? 16 : n;
}

cudaError_t launch_moe_plan(const MoePlanArgs& a, cudaStream_t st) {
  const PlanShape s = plan_shape(a.M, a.E, a.top_k, a.P);
  int32_t* histogram = static_cast<int32_t*>(a.workspace);
  if (s.blocks > 1) {
    plan_count_kernel<<<s.blocks, s.threads, s.E * sizeof(int), st>>>(a.experts, s, histogram, a.status);
    if (const cudaError_t e = cudaGetLastError()) return e;
  }
  const size_t smem = (s.threads / 32 * s.E + 2 * s.E + 1 + 33) * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(plan_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute overlap{};
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(s.blocks);
  cfg.blockDim = dim3(s.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &overlap;
  cfg.numAttrs = s.blocks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, plan_place_kernel, a.experts, s, static_cast<const int32_t*>(histogram), a.group_end,
                            a.counts, a.row_of, a.src_of, a.status);
}

}  // namespace fp8bw
