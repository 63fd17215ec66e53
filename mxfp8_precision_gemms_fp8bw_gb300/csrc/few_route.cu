// The first kernel of the mixture-of-experts layer for a few tokens: router
// logits, the choice of experts, and the plan of the products.
#include <cooperative_groups.h>

#include "few.h"
#include "few_tokens.cuh"
#include "route_row.cuh"

namespace fp8bw {
namespace {

namespace cg = cooperative_groups;

// One cluster.  Each block takes a share of the features: its warps, four
// experts and eight tokens at a time, multiply fp32 router rows with tokens in
// shared memory, so that the router is read once, by all blocks together.
// (Where that is fewer than 16 pieces of work, warps share the features too.)
// The shares of a token's logits then meet in one block (distributed shared
// memory, in the order of the blocks), which makes the choice as fp8bw_moe_route
// does; and the first block sorts the choices.  An expert's tokens are a
// 32-bit mask, whose bits below a token give its place.
constexpr int kBlocks = 8, kWarps = 16, kThreads = kWarps * 32;
constexpr int kMostRows = kFewTokens / kBlocks;  // tokens whose choice a block makes

struct RouteFew {
  const uint16_t* x;
  const float* router;
  const float* bias;
  RouteShape how;  // M rows
  int C, share;    // features, and of a block: a multiple of 8
  int width;       // features in shared memory at a time: a multiple of 128
  int slices;      // warps that share four experts and eight tokens
  FewPlan* plan;
  FewRows held;    // the tokens as the first product reads them
};

struct Layout {  // floats of shared memory
  int tokens, partial, logits, staged, experts, weights, all_experts, all_weights, masks, starts, total;
};
__host__ __device__ inline Layout layout_of(int M, int E, int k, int width, int slices) {
  Layout l{};
  l.tokens = 0;
  l.partial = M * width / 2;  // bf16
  l.logits = l.partial + slices * M * E;
  l.staged = l.logits + kMostRows * E;
  l.experts = l.staged + kMostRows * (E | 8);
  l.weights = l.experts + kMostRows * k;
  l.all_experts = l.weights + kMostRows * k;
  l.all_weights = l.all_experts + M * k;
  l.masks = l.all_weights + M * k;
  l.starts = l.masks + E;
  l.total = l.starts + E + 32;
  return l;
}

// Adds each of 32 values over the warp; lane l returns the sum of v[l].
__device__ __forceinline__ float sum_each(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool high = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = high ? v[i] : v[i + o], keep = high ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(kAll, give, o);
    }
  }
  return v[0];
}

template <int L, int V>
__global__ void __launch_bounds__(kThreads) few_route_kernel(const __grid_constant__ RouteFew p) {
  extern __shared__ __align__(16) float smem[];
  cg::cluster_group cluster = cg::this_cluster();
  const int M = static_cast<int>(p.how.M), E = p.how.E, k = p.how.k;
  const int rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Layout at = layout_of(M, E, k, p.width, p.slices);
  asm volatile("griddepcontrol.launch_dependents;");  // they wait for this kernel's end before they read the plan

  // Logits of this block's features.
  uint2* const tokens = reinterpret_cast<uint2*>(smem + at.tokens);  // four bf16 each
  float* const partial = smem + at.partial;
  const int first = rank * p.share, last = min(first + p.share, p.C);
  const int tiles = (M + 7) / 8, work = (E + 3) / 4 * tiles * p.slices;
  const int steps = max((last - first + p.width - 1) / p.width, 1);
  for (int s = 0; s < steps; ++s) {
    const int c0 = first + s * p.width, n = min(p.width, max(last - c0, 0));  // n: a multiple of 8
    if (s > 0) __syncthreads();
    for (int t = warp; t < M; t += kWarps)
      for (int c = lane * 8; c < n; c += 256)
        *reinterpret_cast<uint4*>(tokens + (t * p.width + c) / 4) =
            __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.C + c0 + c));
    __syncthreads();
    for (int w = warp; w < work; w += kWarps) {
      const int slice = w % p.slices, t0 = w / p.slices % tiles * 8, e0 = w / p.slices / tiles * 4;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 2
      for (int c = slice * 128 + lane * 4; c < n; c += p.slices * 128) {
        float4 r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          r[i] = e0 + i < E ? __ldg(reinterpret_cast<const float4*>(p.router + static_cast<int64_t>(e0 + i) * p.C + c0 + c))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (t0 + j >= M) break;
          const uint2 x = tokens[((t0 + j) * p.width + c) / 4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[i * 8 + j] = fmaf(r[i].x, bf16lo_to_f32(x.x),
                                fmaf(r[i].y, bf16hi_to_f32(x.x),
                                     fmaf(r[i].z, bf16lo_to_f32(x.y), fmaf(r[i].w, bf16hi_to_f32(x.y), v[i * 8 + j]))));
        }
      }
      const float sum = sum_each(v);
      const int e = e0 + lane / 8, t = t0 + lane % 8;
      if (e < E && t < M) {
        float* to = partial + (slice * M + t) * E + e;
        *to = s > 0 ? *to + sum : sum;
      }
    }
  }
  cluster.sync();

  // The choice for tokens rank, rank + kBlocks, ...
  const int rows = rank < M ? (M - rank + kBlocks - 1) / kBlocks : 0;
  float* const logits = smem + at.logits;
  for (int i = tid; i < rows * E; i += kThreads) {
    const int row = i / E, e = i - row * E;
    float sum = 0.f;
    for (int b = 0; b < kBlocks; ++b) {
      const float* from = cluster.map_shared_rank(partial, b) + (rank + row * kBlocks) * E + e;
      for (int s = 0; s < p.slices; ++s) sum += from[s * M * E];
    }
    logits[i] = sum;
  }
  __syncthreads();
  int32_t* const experts = reinterpret_cast<int32_t*>(smem + at.experts);
  float* const weights = smem + at.weights;
  constexpr int kChoosers = L == 8 ? 1 : kMostRows;  // warps that choose; the others bring the tokens into e4m3
  if (warp >= kChoosers) {
    const int pieces = p.C / 8;  // of 8 values
    for (int r = 0; r < rows; ++r) {
      const int64_t t = rank + r * kBlocks;
      const uint4* row = reinterpret_cast<const uint4*>(p.x + t * p.C);
      uint8_t* to = p.held.codes + t * kTokenParts * p.held.pitch;
      uint8_t* scales = p.held.scales + t * kTokenParts * (p.held.pitch / 32);
#pragma unroll 2
      for (int i0 = (warp - kChoosers) * 32; i0 < pieces; i0 += (kWarps - kChoosers) * 32) {
        const int i = i0 + lane < pieces ? i0 + lane : i0 + lane % 4;  // past the end the same four again
        few::split8(__ldg(row + i), to + i * 8, scales + i / 4, p.held.pitch);
      }
    }
  } else if (warp * (32 / L) < rows) {
    const int row = tid / L;
    route_row<float, L, V>(logits, p.bias, p.how, row, row < rows, row, reinterpret_cast<uint32_t*>(smem + at.staged), experts,
                           weights);
  }
  __syncthreads();
  {
    int32_t* to = cluster.map_shared_rank(reinterpret_cast<int32_t*>(smem + at.all_experts), 0);
    float* tow = cluster.map_shared_rank(smem + at.all_weights, 0);
    for (int i = tid; i < rows * k; i += kThreads) {
      const int entry = (rank + i / k * kBlocks) * k + i % k;
      to[entry] = experts[i];
      tow[entry] = weights[i];
    }
  }
  cluster.sync();
  if (rank != 0) return;

  // The plan.
  uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + at.masks);
  int* const starts = reinterpret_cast<int*>(smem + at.starts);
  int* const sums = starts + E;
  const int32_t* chosen = reinterpret_cast<const int32_t*>(smem + at.all_experts);
  const float* given = smem + at.all_weights;
  for (int e = tid; e < E; e += kThreads) masks[e] = 0;
  __syncthreads();
  for (int i = tid; i < M * k; i += kThreads)
    if (chosen[i] >= 0) atomicOr(masks + chosen[i], 1u << (i / k));
  __syncthreads();
  int before = 0;  // slots in the upper half word, choices in the lower
  FewSlot* slots = few_slots(p.plan, M * k);
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + tid;
    const uint32_t mask = e < E ? masks[e] : 0;
    const int mine = mask != 0 ? (1 << 16) | __popc(mask) : 0;
    int up = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(kAll, up, o);
      if (lane >= o) up += t;
    }
    if (lane == 31) sums[warp] = up;
    __syncthreads();
    int all = 0, earlier = before;
    for (int w = 0; w < kWarps; ++w) {
      earlier += w < warp ? sums[w] : 0;
      all += sums[w];
    }
    earlier += up - mine;
    if (mask != 0) {
      slots[earlier >> 16] = FewSlot{e, earlier & 0xFFFF, mask, __popc(mask)};
      starts[e] = earlier & 0xFFFF;
    }
    before += all;
    __syncthreads();
  }
  if (tid == 0) p.plan->active = before >> 16;
  float* const out = few_weights(p.plan);
  for (int i = tid; i < M * k; i += kThreads) {
    const int e = chosen[i];
    if (e >= 0) out[starts[e] + __popc(masks[e] & ((1u << (i / k)) - 1))] = given[i];
  }
}

}  // namespace

cudaError_t launch_few_route(const FewMoeArgs& a, FewPlan* plan, const FewRows& tokens, cudaStream_t st) {
  RouteFew p{};
  p.x = a.x;
  p.router = a.router;
  p.bias = a.route.bias;
  p.how = shape_of(a.route);
  p.C = static_cast<int>(a.C);
  p.share = (p.C + 8 * kBlocks - 1) / (8 * kBlocks) * 8;
  const int M = static_cast<int>(a.route.M), E = p.how.E;
  // Tokens in shared memory: 64 KB, or 32 beside the logits of very many experts.
  const int most = (M * E <= 16384 ? 32768 : 16384) / M / 128 * 128, want = (p.share + 127) / 128 * 128;
  p.width = want < most ? want : most;
  const int work = (E + 3) / 4 * ((M + 7) / 8);
  p.slices = 1;
  while (2 * p.slices * work <= kWarps && 2 * p.slices * 128 <= p.width) p.slices *= 2;
  p.plan = plan;
  p.held = tokens;
  const int smem = layout_of(M, E, p.how.k, p.width, p.slices).total * 4;
  return for_experts(E, [&](auto lanes, auto width) {
    constexpr int L = decltype(lanes)::value, V = decltype(width)::value;
    auto* kernel = few_route_kernel<L, V>;
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kBlocks;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kBlocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  });
}

}  // namespace fp8bw
