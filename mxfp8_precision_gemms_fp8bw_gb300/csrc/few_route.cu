// The first kernel of the mixture-of-experts layer for a few tokens: router
// logits, the choice of experts, and the plan of the products.
#include "few.h"
#include "few_tokens.cuh"
#include "route_row.cuh"

namespace fp8bw {
namespace {

// One cluster of sixteen blocks, a few microseconds of latencies: the kernel runs
// once through its code, which is kept short (instructions come from memory
// too), and blocks send each other what they have rather than fetch it.  5 us
// for one token, 8 for 17 of 64 experts and for 32 of 8 (5120 features), half of
// it steps 2 and 3; with eight blocks and rows kept in shared memory for the
// choice it took 7, 18 and 14.
//
//   1. Each block takes a sixteenth of the features.  A warp takes 16 experts
//      and all tokens (where those are fewer than 16 pieces of work, warps share
//      the features as well), and sends each logit's share to the block that
//      makes the token's choice.  The products are the tensor core's: a weight
//      of the router, fp32, is the sum of three bf16, exactly, a token's value is
//      one, products of two are exact and sums fp32 (16 features by the tensor
//      core, those then added as ever): 2.2 us for 17 tokens and 64
//      experts of 2048 features, 1.0 for one token.  Fused multiply-adds took 5.5
//      (shared memory or the cache, whichever the operands came from, had more to
//      hand out than this step has time for) and 0.7.
//   2. Block r adds up the shares of tokens r and r + 16 in the order of the
//      blocks, and a warp chooses for each, as fp8bw_moe_route does, while the
//      others bring the block's features into e4m3 for the first product.
//   3. The first block sorts the choices.  An expert's tokens are a 32-bit mask,
//      whose bits below a token give its place.
constexpr int kBlocks = 16, kWarps = 16, kThreads = kWarps * 32;
constexpr int kMostRows = kFewTokens / kBlocks;  // tokens of a block

int share_of(int64_t C) { return static_cast<int>((C + 32 * kBlocks - 1) / (32 * kBlocks) * 32); }

struct RouteFew {
  const uint16_t* x;
  const float* router;
  const float* bias;
  RouteShape how;  // M rows
  int C, share;    // features, and of a block: a multiple of 32
  int slices;      // warps that share 16 experts
  FewPlan* plan;
  uint8_t* held;   // the tokens as the first product reads them
};

struct Layout {  // words of shared memory
  int partial, received, keys, experts, weights, masks, starts, total;
};
__host__ __device__ inline Layout layout_of(int M, int E, int k, int slices, int groups) {
  Layout l{};
  l.partial = 0;
  l.received = slices > 1 ? slices * M * E : 0;  // [rows][blocks][E]
  l.keys = l.received + kMostRows * kBlocks * E;
  l.experts = l.keys + (groups > 1 ? kMostRows * E : 0);
  l.weights = l.experts + M * k;
  l.masks = l.weights + M * k;
  l.starts = l.masks + E;
  l.total = l.starts + E;
  return l;
}

// Two values as pairs of bf16: the upper, middle and lower eight bits of their significands.  An infinity is the first's
// alone.
__device__ __forceinline__ void thirds(float a, float b, uint32_t (&out)[3]) {
  const auto pair = [](float lo, float hi) { return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632); };
  const auto cut = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xFFFF0000u); };
  const auto rest = [](float v, float first) { return fabsf(v) == INFINITY ? 0.f : v - first; };
  out[0] = pair(a, b);
  a = rest(a, cut(a)), b = rest(b, cut(b));
  out[1] = pair(a, b);
  out[2] = pair(a - cut(a), b - cut(b));
}

// Two bf16 whose infinities have become NaN (times 0, and that on top): a token with one has no logit that means anything, and
// one of -inf would leave the token without the expert.
__device__ __forceinline__ uint32_t finite_or_nan(uint32_t v) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %1;" : "=r"(d) : "r"(v), "r"(0u));
  return d;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void store_remote(uint32_t mine, int rank, uint32_t v) {  // to the same place of another block
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void or_remote(uint32_t mine, int rank, uint32_t v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(mine), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// Loads behind the wait for the kernel before, like load_after, of what several warps of the block read: by its cache.
__device__ __forceinline__ uint4 load_shared_after(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_shared_after(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

// The choice of one row by a warp: the rule, the keys and the scores of
// route_row, bit for bit (the softmax's sum by halves of the row's indexes).
// s: the logits, bias: what is added for the choice, both of experts lane + 32 i.
// key: E words of shared memory, where there are groups.
// Lane c < k returns choice c and the sum over all choices' scores.
struct Choice {
  int expert;
  float score, sum;
};
template <int kPer>
__device__ __forceinline__ Choice choose_row(float (&s)[kPer], const float (&bias)[kPer], uint32_t* key, const RouteShape& p) {
  const int lane = threadIdx.x & 31, E = p.E;
  uint32_t masked = 0, u[kPer];  // of the lane's experts, those whose logit is -inf; keys
#pragma unroll
  for (int i = 0; i < kPer; ++i) masked |= s[i] == -INFINITY ? 1u << i : 0u;
  if (p.score == 0) {
    float top = s[0], part[kPer];
#pragma unroll
    for (int i = 1; i < kPer; ++i) top = fmaxf(top, s[i]);
    top = lanes_reduce<32>(top, [](float a, float b) { return fmaxf(a, b); });
    if (top == -INFINITY) top = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s[i] = part[i] = lane + 32 * i < E ? expf(s[i] - top) : 0.f;
#pragma unroll
    for (int h = kPer / 2; h >= 1; h /= 2)  // past the row zeros, which change no sum
#pragma unroll
      for (int i = 0; i < h; ++i) part[i] += part[i + h];
    float total = lanes_sum<32>(part[0]);
    if (total == 0.f) total = 1.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) s[i] = __fdiv_rn(s[i], total);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) s[i] = sigmoid_of(s[i]);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    u[i] = lane + 32 * i >= E || ((masked >> i) & 1) || bias[i] == -INFINITY ? 0u : ordered(s[i] + bias[i]);
  if (p.groups > 1) {
    const int size = E / p.groups;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < E) key[lane + 32 * i] = u[i];
    __syncwarp();
    uint32_t total = 0;
    if (lane < p.groups) {
      uint32_t best = 0, second = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t v = key[lane * size + i];
        second = max(second, min(best, v));
        best = max(best, v);
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
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < E && !((kept >> ((lane + 32 * i) / size)) & 1)) u[i] = 0;
  }
  Choice mine{-1, 0.f, 0.f};
#pragma unroll 1
  for (int c = 0; c < p.k; ++c) {
    uint32_t best = u[0];  // of the lane's keys
    int at = 0;
    float score = s[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i)
      if (u[i] > best) best = u[i], at = i, score = s[i];
    const uint32_t most = __reduce_max_sync(kAll, best);
    if (most == 0) break;
    const int e = __reduce_min_sync(kAll, best == most ? lane + 32 * at : E);
    score = __shfl_sync(kAll, score, e & 31);
    if (lane == c) mine.expert = e, mine.score = score;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i == e) u[i] = 0;
  }
  mine.sum = lanes_sum<32>(mine.score);
  return mine;
}

// kPer: experts that a lane chooses from, E <= 32 kPer.
template <int kPer>
__global__ void __launch_bounds__(kThreads, kPer == 32 ? 1 : 2) few_route_kernel(const __grid_constant__ RouteFew p) {
  extern __shared__ __align__(16) float smem[];
  const int M = static_cast<int>(p.how.M), E = p.how.E, k = p.how.k;
  const int rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Layout at = layout_of(M, E, k, p.slices, p.how.groups);
  const int first = min(rank * p.share, p.C), last = min(first + p.share, p.C);
  uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + at.masks);
  asm volatile("griddepcontrol.launch_dependents;");  // they wait for this kernel's end before they read the plan
  if (rank == 0)
    for (int e = tid; e < E; e += kThreads) masks[e] = 0;
  cluster_arrive();  // blocks may write to each other's memory once they run
  // What the block will read comes nearer while the kernel before may still run: only into the cache that all share.
  const int lines = (last - first + 31) / 32;
  for (int i = tid; i < E * lines; i += kThreads)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.router + static_cast<int64_t>(i / lines) * p.C + first + i % lines * 32));
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // 1. Logits.
  uint32_t* const received = reinterpret_cast<uint32_t*>(smem + at.received);
  const auto send = [&](int t, int e, float v) {
    store_remote(smem_u32(received + (t / kBlocks * kBlocks + rank) * E + e), t % kBlocks, __float_as_uint(v));
  };
  const int work = (E + 15) / 16 * p.slices, tiles = (M + 7) / 8;
  const int g = lane / 4, q = lane % 4;
  bool together = false;
#pragma unroll 1
  for (int w = warp; w < work; w += kWarps) {
    const int slice = w % p.slices, e0 = w / p.slices * 16;
    float v[4][4] = {};  // experts e0 + g (and + 8 as the upper two), tokens 8 tile + 2 q and the one after
#pragma unroll 1
    for (int c = first + slice * 16 + q * 4; c < last; c += p.slices * 16) {
      // The sum goes over 16 features at a time, in an order that suits the loads: a lane has four next to each other.
      uint4 r[2];
      uint2 x[4] = {};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        r[h] = load_shared_after(reinterpret_cast<const uint4*>(p.router + static_cast<int64_t>(min(e0 + g + h * 8, E - 1)) * p.C + c));
#pragma unroll
      for (int t = 0; t < 4; ++t)  // past the last token that one again
        if (t < tiles) x[t] = load_shared_after(reinterpret_cast<const uint2*>(p.x + static_cast<int64_t>(min(t * 8 + g, M - 1)) * p.C + c));
#pragma unroll
      for (int t = 0; t < 4; ++t) x[t].x = finite_or_nan(x[t].x), x[t].y = finite_or_nan(x[t].y);
      uint32_t part[4][3];  // as the product takes them: rows g, g + 8, features 4 q and the next; the two after those
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        thirds(__uint_as_float(r[h].x), __uint_as_float(r[h].y), part[h]);
        thirds(__uint_as_float(r[h].z), __uint_as_float(r[h].w), part[2 + h]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if (t >= tiles) break;
        // 16 features alone: the tensor core cuts off what is below the last bit of the largest term, which on top of the sum
        // so far would be of the whole logit.  That one is rounded to the nearest.
        float f[4] = {};
#pragma unroll
        for (int i = 2; i >= 0; --i) {
          const uint32_t a[4] = {part[0][i], part[1][i], part[2][i], part[3][i]};
          mma_bf16(f, a, x[t].x, x[t].y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[t][i] += f[i];
      }
    }
    const auto each = [&](auto&& to) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int token = t * 8 + q * 2 + i % 2, e = e0 + g + i / 2 * 8;
          if (token < M && e < E) to(token, e, v[t][i]);
        }
    };
    if (p.slices > 1) {
      each([&](int t, int e, float sum) { smem[at.partial + (slice * M + t) * E + e] = sum; });
      continue;
    }
    if (!together) cluster_wait();  // all blocks run
    together = true;
    each(send);
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

  // 2. The choice for tokens rank and rank + kBlocks: a warp each.
  uint32_t* const experts = reinterpret_cast<uint32_t*>(smem + at.experts);
  uint32_t* const weights = reinterpret_cast<uint32_t*>(smem + at.weights);
  if (warp < kMostRows) {
    const int t = rank + warp * kBlocks;
    float s[kPer], bias[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      bias[i] = p.bias != nullptr && t < M && lane + 32 * i < E
                    ? __uint_as_float(load_after(reinterpret_cast<const uint32_t*>(p.bias + lane + 32 * i))) : 0.f;
    cluster_wait();
    if (t < M) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        float sum = 0.f;
        if (lane + 32 * i < E)
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) sum += __uint_as_float(received[(warp * kBlocks + b) * E + lane + 32 * i]);
        s[i] = lane + 32 * i < E ? sum : -INFINITY;
      }
      const Choice c = choose_row(s, bias, reinterpret_cast<uint32_t*>(smem + at.keys) + warp * E, p.how);
      const float w = (p.how.renorm ? c.score / (c.sum + 1e-20f) : c.score) * p.how.scale;
      if (M == 1) {  // the choices are the slots
        const uint32_t some = __ballot_sync(kAll, c.expert >= 0);
        const int place = __popc(some & ((1u << lane) - 1));
        if (c.expert >= 0) {
          few_slots(p.plan, k)[place] = FewSlot{c.expert, place, 1, 1};
          few_weights(p.plan)[place] = w;
        }
        if (lane == 0) p.plan->active = __popc(some), p.plan->most = 1;
      } else if (lane < k) {
        store_remote(smem_u32(experts + t * k + lane), 0, static_cast<uint32_t>(c.expert));
        if (c.expert >= 0) {
          store_remote(smem_u32(weights + t * k + lane), 0, __float_as_uint(w));
          or_remote(smem_u32(masks + c.expert), 0, 1u << t);
        }
      }
    }
  } else {
    const int pieces = (last - first) / 8, all = pieces * M;  // of 8 values
#pragma unroll 1
    for (int i0 = (warp - kMostRows) * 32; i0 < all; i0 += (kWarps - kMostRows) * 32) {
      const int i = i0 + lane < all ? i0 + lane : i0 + lane % 4;  // past the end the same four again
      const int t = i / pieces, c = first + i % pieces * 8;
      few::split8(
          load_shared_after(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.C + c)),
          [&](int part) { return few::code_at(p.held, M * kTokenParts, c, t * kTokenParts + part); },
          [&](int part) { return few::scale_at(p.held, M * kTokenParts, c, t * kTokenParts + part); });
    }
    cluster_wait();
  }
  if (M == 1) return;
  __syncwarp();
  cluster_arrive();
  if (rank != 0) return;
  cluster_wait();

  // 3. The plan.
  int* const starts = reinterpret_cast<int*>(smem + at.starts);
  if (warp == 0) {
    FewSlot* slots = few_slots(p.plan, M * k);
    int before = 0, most = 0;  // before: slots in the upper half word, choices in the lower
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const uint32_t mask = e < E ? masks[e] : 0;
      const int mine = mask != 0 ? (1 << 16) | __popc(mask) : 0;
      most = max(most, __popc(mask));
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
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) p.plan->active = before >> 16, p.plan->most = most;
  }
  __syncthreads();
  float* const out = few_weights(p.plan);
  for (int i = tid; i < M * k; i += kThreads) {
    const int e = static_cast<int>(experts[i]);
    if (e >= 0) out[starts[e] + __popc(masks[e] & ((1u << (i / k)) - 1))] = __uint_as_float(weights[i]);
  }
}

}  // namespace

template <int kPer>
static cudaError_t launch(const RouteFew& p, int smem, cudaStream_t st) {
  auto* kernel = few_route_kernel<kPer>;
  static thread_local bool allowed[64] = {};  // by device
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev >= 64 || !allowed[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int few_route_slices(int64_t E, int64_t C) {
  const int most = share_of(C) / 16, work = static_cast<int>((E + 15) / 16);
  return work >= kWarps ? 1 : kWarps / work < most ? kWarps / work : most;
}

cudaError_t launch_few_route(const FewMoeArgs& a, FewPlan* plan, uint8_t* tokens, cudaStream_t st) {
  RouteFew p{};
  p.x = a.x;
  p.router = a.router;
  p.bias = a.route.bias;
  p.how = shape_of(a.route);
  p.C = static_cast<int>(a.C);
  p.share = share_of(a.C);
  const int M = static_cast<int>(a.route.M), E = p.how.E;
  p.slices = few_route_slices(E, a.C);
  p.plan = plan;
  p.held = tokens;
  const int smem = layout_of(M, E, p.how.k, p.slices, p.how.groups).total * 4;
  return E <= 64 ? launch<2>(p, smem, st) : E <= 256 ? launch<8>(p, smem, st) : launch<32>(p, smem, st);
}

}  // namespace fp8bw
