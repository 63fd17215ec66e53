// Routing of a mixture-of-experts layer: the choice of experts, and the sort of
// the choices into expert groups.
#include "route_row.cuh"

namespace fp8bw {
namespace {

template <typename T, int L, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const T* __restrict__ logits,
                                                                 const float* __restrict__ bias, RouteShape p,
                                                                 int32_t* __restrict__ experts,
                                                                 float* __restrict__ weights) {
  extern __shared__ uint32_t staged[];
  const int mine = threadIdx.x / L;  // the row in the block
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteRows<L> + mine;
  // all lanes go through the shuffles
  route_row<T, L, V>(logits, bias, p, row, row < p.M, mine, staged, experts, weights);
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
// runs meanwhile.  16384 entries over 8 experts take 9.5 us, 127992 over 64
// 12.7 us; one block for all of them took 20 and 196.
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
  return for_experts(a.E, [&](auto lanes, auto width) {
    constexpr int L = decltype(lanes)::value, V = decltype(width)::value;
    const dim3 grid(static_cast<unsigned>((a.M + kRouteRows<L> - 1) / kRouteRows<L>));
    route_kernel<T, L, V><<<grid, kRouteWarps * 32, a.groups > 1 ? staged_bytes<L>(a.E) : 0, st>>>(
        static_cast<const T*>(a.logits), a.bias, shape_of(a), a.experts, a.weights);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteArgs& a, cudaStream_t st) {
  return a.bf16 ? route_of<uint16_t>(a, st) : route_of<float>(a, st);
}

size_t moe_plan_workspace_bytes(int64_t M, int64_t E, int64_t top_k) {
  const PlanShape s = plan_shape(M, E, top_k, 0);
  return s.blocks > 1 ? static_cast<size_t>(s.blocks) * s.E * sizeof(int32_t) : 0;
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
