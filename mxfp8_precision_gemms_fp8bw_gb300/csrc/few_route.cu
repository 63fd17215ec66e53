// The first kernel of the mixture-of-experts layer for a few tokens: router
// logits, the choice of experts, and the plan of the products.
#include "few.h"
#include "few_tokens.cuh"
#include "route_row.cuh"

namespace fp8bw {
namespace {

// One cluster of eight blocks, a few microseconds of latencies: the kernel runs
// once through its code, which is kept short (instructions come from memory
// too), and blocks send each other what they have rather than fetch it.
//
//   1. Each block takes an eighth of the features.  A warp takes four experts
//      and eight tokens at a time (where that is fewer than 16 pieces of work,
//      warps share the features as well), and sends each logit's share to the
//      block that makes the token's choice.
//   2. Block r adds up the shares of tokens r, r + 8, .. in the order of the
//      blocks, and a warp chooses for each, as fp8bw_moe_route does, while the
//      others bring the tokens into e4m3 for the first product.
//   3. The first block sorts the choices.  An expert's tokens are a 32-bit mask,
//      whose bits below a token give its place.
constexpr int kBlocks = 8, kWarps = 16, kThreads = kWarps * 32;
constexpr int kMostRows = kFewTokens / kBlocks;  // tokens of a block

struct RouteFew {
  const uint16_t* x;
  const float* router;
  const float* bias;
  RouteShape how;  // M rows
  int C, share;    // features, and of a block: a multiple of 8
  int slices;      // warps that share four experts and eight tokens
  FewPlan* plan;
  uint8_t* held;   // the tokens as the first product reads them
};

// A power of two, at least 32, that E is not above.
__host__ __device__ inline int padded(int E) {
  int P = 32;
  while (P < E) P *= 2;
  return P;
}

struct Layout {  // words of shared memory
  int partial, received, scores, keys, experts, weights, masks, starts, total;
};
__host__ __device__ inline Layout layout_of(int M, int E, int k, int slices) {
  Layout l{};
  l.partial = 0;
  l.received = slices > 1 ? slices * M * E : 0;  // [rows][blocks][E]
  l.scores = l.received + kMostRows * kBlocks * E;
  l.keys = l.scores + kMostRows * E;
  l.experts = l.keys + kMostRows * padded(E);    // first the exponentials that are summed up
  l.weights = l.experts + M * k;
  l.masks = l.weights + M * k;
  l.starts = l.masks + E;
  l.total = l.starts + E;
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

__device__ __forceinline__ void store_remote(uint32_t mine, int rank, uint32_t v) {  // to the same place of another block
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The choice of one row by a warp: the rule, the keys and the scores of
// route_row, bit for bit (the softmax's sum by halves of the row's indexes),
// with the row in shared memory.  s: logits, then scores; key: P words.
// Lane c < k returns choice c and the sum over all choices' scores.
struct Choice {
  int expert;
  float score, sum;
};
__device__ Choice choose_row(float* s, uint32_t* key, const float* bias, const RouteShape& p) {
  const int lane = threadIdx.x & 31, E = p.E;
  float top = -INFINITY;
  for (int e = lane; e < E; e += 32) top = fmaxf(top, s[e]);
  uint32_t masked = 0;  // of the lane's experts, those whose logit is -inf
  for (int e = lane, i = 0; e < E; e += 32, ++i) masked |= s[e] == -INFINITY ? 1u << i : 0u;
  if (p.score == 0) {
    top = lanes_reduce<32>(top, [](float a, float b) { return fmaxf(a, b); });
    if (top == -INFINITY) top = 0.f;
    float* part = reinterpret_cast<float*>(key);
    const int P = padded(E);
    for (int e = lane; e < P; e += 32) part[e] = e < E ? expf(s[e] - top) : 0.f;
    for (int e = lane; e < E; e += 32) s[e] = part[e];
    for (int h = P / 2; h >= 32; h /= 2)  // a lane adds what it wrote itself
      for (int e = lane; e < h; e += 32) part[e] += part[e + h];
    float total = lanes_sum<32>(part[lane]);
    if (total == 0.f) total = 1.f;
    for (int e = lane; e < E; e += 32) s[e] = __fdiv_rn(s[e], total);
  } else {
    for (int e = lane; e < E; e += 32) s[e] = sigmoid_of(s[e]);
  }
  for (int e = lane, i = 0; e < E; e += 32, ++i) {
    const float b = bias != nullptr ? __uint_as_float(load_after(reinterpret_cast<const uint32_t*>(bias + e))) : 0.f;
    key[e] = ((masked >> i) & 1) || b == -INFINITY ? 0u : ordered(s[e] + b);
  }
  __syncwarp();
  if (p.groups > 1) {
    const int size = E / p.groups;
    uint32_t total = 0;
    if (lane < p.groups) {
      uint32_t best = 0, second = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t u = key[lane * size + i];
        second = max(second, min(best, u));
        best = max(best, u);
      }
      total = best;
      if (p.group_top == 2 && second != 0) {
        const float sum = unordered(best) + unordered(second);
        total = ordered(sum < kLowest ? kLowest : sum);
      }
    }
    int before = 0;  // groups that come first
    for (int g = 0; g < p.groups; ++g) {
      const uint32_t other = __shfl_sync(kAll, total, g);
      before += other > total || (other == total && g < lane);
    }
    const uint32_t kept = __ballot_sync(kAll, lane < p.groups && total != 0 && before < p.kept);
    for (int e = lane; e < E; e += 32)
      if (!((kept >> (e / size)) & 1)) key[e] = 0;
  }
  Choice mine{-1, 0.f, 0.f};
  uint32_t best = 0;  // of the lane's keys
  int at = 0;
  for (int e = lane; e < E; e += 32)
    if (key[e] > best) best = key[e], at = e;
#pragma unroll 1
  for (int c = 0; c < p.k; ++c) {
    const uint32_t most = __reduce_max_sync(kAll, best);
    if (most == 0) break;
    const int e = __reduce_min_sync(kAll, best == most ? at : E);
    if (lane == c) mine.expert = e;
    if (best == most && at == e) {
      key[e] = 0;
      best = 0;
      for (int i = lane; i < E; i += 32)
        if (key[i] > best) best = key[i], at = i;
    }
  }
  __syncwarp();
  mine.score = mine.expert >= 0 ? s[mine.expert] : 0.f;
  mine.sum = lanes_sum<32>(mine.score);
  return mine;
}

__global__ void __launch_bounds__(kThreads) few_route_kernel(const __grid_constant__ RouteFew p) {
  extern __shared__ __align__(16) float smem[];
  const int M = static_cast<int>(p.how.M), E = p.how.E, k = p.how.k;
  const int rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Layout at = layout_of(M, E, k, p.slices);
  asm volatile("griddepcontrol.launch_dependents;");  // they wait for this kernel's end before they read the plan
  cluster_arrive();  // blocks may write to each other's memory once they run
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // 1. Logits.
  uint32_t* const received = reinterpret_cast<uint32_t*>(smem + at.received);
  const auto send = [&](int t, int e, float v) {
    store_remote(smem_u32(received + (t / kBlocks * kBlocks + rank) * E + e), t % kBlocks, __float_as_uint(v));
  };
  const int first = rank * p.share, last = min(first + p.share, p.C);
  const int tiles = (M + 7) / 8, work = (E + 3) / 4 * tiles * p.slices;
  bool together = false;
#pragma unroll 1
  for (int w = warp; w < work; w += kWarps) {
    const int slice = w % p.slices, t0 = w / p.slices % tiles * 8, e0 = w / p.slices / tiles * 4;
    float v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 2
    for (int c = first + slice * 128 + lane * 4; c < last; c += p.slices * 128) {
      float4 r[4];
      uint2 x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w = load_after(reinterpret_cast<const uint4*>(p.router + static_cast<int64_t>(min(e0 + i, E - 1)) * p.C + c));
        r[i] = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (t0 + j < M) x[j] = load_after(reinterpret_cast<const uint2*>(p.x + static_cast<int64_t>(t0 + j) * p.C + c));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (t0 + j >= M) break;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i * 8 + j] = fmaf(r[i].x, bf16lo_to_f32(x[j].x),
                              fmaf(r[i].y, bf16hi_to_f32(x[j].x),
                                   fmaf(r[i].z, bf16lo_to_f32(x[j].y), fmaf(r[i].w, bf16hi_to_f32(x[j].y), v[i * 8 + j]))));
      }
    }
    const float sum = sum_each(v);
    const int e = e0 + lane / 8, t = t0 + lane % 8;
    if (p.slices > 1) {
      if (e < E && t < M) smem[at.partial + (slice * M + t) * E + e] = sum;
      continue;
    }
    if (!together) cluster_wait();  // all blocks run
    together = true;
    if (e < E && t < M) send(t, e, sum);
    __syncwarp();
  }
  if (!together) cluster_wait();
  if (p.slices > 1) {
    __syncthreads();
    for (int i = tid; i < M * E; i += kThreads) {
      float sum = 0.f;
      for (int s = 0; s < p.slices; ++s) sum += smem[at.partial + s * M * E + i];
      send(i / E, i % E, sum);
    }
    __syncwarp();
  }
  cluster_arrive();
  cluster_wait();

  // 2. The choice for tokens rank, rank + kBlocks, ..: a warp each.
  const int rows = rank < M ? (M - rank + kBlocks - 1) / kBlocks : 0;
  uint32_t* const experts = reinterpret_cast<uint32_t*>(smem + at.experts);
  uint32_t* const weights = reinterpret_cast<uint32_t*>(smem + at.weights);
  if (warp < rows) {
    float* const s = smem + at.scores + warp * E;
    for (int e = lane; e < E; e += 32) {
      float sum = 0.f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) sum += __uint_as_float(received[(warp * kBlocks + b) * E + e]);
      s[e] = sum;
    }
    const Choice c = choose_row(s, reinterpret_cast<uint32_t*>(smem + at.keys) + warp * padded(E), p.bias, p.how);
    if (M == 1) {  // the choices are the slots
      const uint32_t some = __ballot_sync(kAll, c.expert >= 0);
      const int at = __popc(some & ((1u << lane) - 1));
      if (c.expert >= 0) {
        few_slots(p.plan, k)[at] = FewSlot{c.expert, at, 1, 1};
        few_weights(p.plan)[at] = (p.how.renorm ? c.score / (c.sum + 1e-20f) : c.score) * p.how.scale;
      }
      if (lane == 0) p.plan->active = __popc(some);
    } else if (lane < k) {
      const float w = (p.how.renorm ? c.score / (c.sum + 1e-20f) : c.score) * p.how.scale;
      const int entry = (rank + warp * kBlocks) * k + lane;
      store_remote(smem_u32(experts + entry), 0, static_cast<uint32_t>(c.expert));
      store_remote(smem_u32(weights + entry), 0, __float_as_uint(c.expert >= 0 ? w : 0.f));
    }
  } else if (warp >= kMostRows) {
    const int pieces = p.C / 8;  // of 8 values
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
      const int t = rank + r * kBlocks;
      const uint4* row = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.C);
#pragma unroll 1
      for (int i0 = (warp - kMostRows) * 32; i0 < pieces; i0 += (kWarps - kMostRows) * 32) {
        const int i = i0 + lane < pieces ? i0 + lane : i0 + lane % 4;  // past the end the same four again
        few::split8(
            load_after(row + i), [&](int part) { return few::code_at(p.held, M * kTokenParts, i * 8, t * kTokenParts + part); },
            [&](int part) { return few::scale_at(p.held, M * kTokenParts, i * 8, t * kTokenParts + part); });
      }
    }
  }
  if (M == 1) return;
  __syncwarp();
  cluster_arrive();
  if (rank != 0) return;
  uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + at.masks);
  for (int e = tid; e < E; e += kThreads) masks[e] = 0;
  cluster_wait();
  __syncthreads();

  // 3. The plan.
  int* const starts = reinterpret_cast<int*>(smem + at.starts);
  for (int i = tid; i < M * k; i += kThreads)
    if (static_cast<int>(experts[i]) >= 0) atomicOr(masks + experts[i], 1u << (i / k));
  __syncthreads();
  if (warp == 0) {
    FewSlot* slots = few_slots(p.plan, M * k);
    int before = 0;  // slots in the upper half word, choices in the lower
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const uint32_t mask = e < E ? masks[e] : 0;
      const int mine = mask != 0 ? (1 << 16) | __popc(mask) : 0;
      int up = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(kAll, up, o);
        if (lane >= o) up += t;
      }
      const int earlier = before + up - mine;
      if (mask != 0) {
        slots[earlier >> 16] = FewSlot{e, earlier & 0xFFFF, mask, __popc(mask)};
        starts[e] = earlier & 0xFFFF;
      }
      before += __shfl_sync(kAll, up, 31);
    }
    if (lane == 0) p.plan->active = before >> 16;
  }
  __syncthreads();
  float* const out = few_weights(p.plan);
  for (int i = tid; i < M * k; i += kThreads) {
    const int e = static_cast<int>(experts[i]);
    if (e >= 0) out[starts[e] + __popc(masks[e] & ((1u << (i / k)) - 1))] = __uint_as_float(weights[i]);
  }
}

}  // namespace

cudaError_t launch_few_route(const FewMoeArgs& a, FewPlan* plan, uint8_t* tokens, cudaStream_t st) {
  RouteFew p{};
  p.x = a.x;
  p.router = a.router;
  p.bias = a.route.bias;
  p.how = shape_of(a.route);
  p.C = static_cast<int>(a.C);
  p.share = (p.C + 8 * kBlocks - 1) / (8 * kBlocks) * 8;
  const int M = static_cast<int>(a.route.M), E = p.how.E;
  const int work = (E + 3) / 4 * ((M + 7) / 8);
  p.slices = 1;
  while (2 * p.slices * work <= kWarps && 2 * p.slices * 128 <= p.share + 127) p.slices *= 2;
  p.plan = plan;
  p.held = tokens;
  const int smem = layout_of(M, E, p.how.k, p.slices).total * 4;
  static thread_local bool allowed[64] = {};  // by device
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev >= 64 || !allowed[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(few_route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = true;
  }
  cudaLaunchAttribute attrs[2]{};
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = kBlocks;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // it waits itself
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kBlocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, few_route_kernel, p);
}

}  // namespace fp8bw
