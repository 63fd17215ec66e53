// Routing of a mixture-of-experts layer: the choice of experts, and the sort of
// the choices into expert groups.
#include "route_row.cuh"

namespace fp8bw {
namespace {

// The largest key of the row and where it is, the lowest place of equal ones;
// key 0 where nothing is left.
struct Best {
  uint32_t key;
  int at;
};
template <int L, int V>
__device__ __forceinline__ Best best_of(const uint32_t (&key)[V], int l) {
  Best b{key[0], 0};
#pragma unroll
  for (int v = 1; v < V; ++v)
    if (key[v] > b.key) b = Best{key[v], v};
  b.at = b.at * L + l;
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    const Best c{__shfl_xor_sync(kAll, b.key, o), __shfl_xor_sync(kAll, b.at, o)};
    if (c.key > b.key || (c.key == b.key && c.at < b.at)) b = c;
  }
  return b;
}

template <typename T, int L, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const T* __restrict__ logits,
                                                                 const float* __restrict__ bias, RouteShape p,
                                                                 int32_t* __restrict__ experts,
                                                                 float* __restrict__ weights) {
  constexpr int kRowsPerWarp = 32 / L;
  extern __shared__ uint32_t staged[];
  const int l = threadIdx.x & (L - 1), mine = threadIdx.x / L;  // the lane in its row, the row in the block
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRouteWarps * kRowsPerWarp) + mine;
  const bool live = row < p.M;  // all lanes go through the shuffles
  float x[V], s[V];
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    x[v] = live && e < p.E ? logit_at(logits, row * p.E + e) : -INFINITY;
  }
  const RowScale scale = scores_of<L, V, true>(x, p.score, s);
  if (bias == nullptr && p.groups == 1) {
    // Scores are not negative, and NaN comes as 0x7fffffff: their bits order them.
#pragma unroll
    for (int v = 0; v < V; ++v)  // x is -inf past the last expert
      key[v] = x[v] == -INFINITY ? 0u : __float_as_uint(s[v]) + 1u;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float b = bias != nullptr && v * L + l < p.E ? bias[v * L + l] : 0.f;
      key[v] = x[v] == -INFINITY || b == -INFINITY ? 0u : ordered(s[v] + b);
    }
  }

  if (p.groups > 1) {
    // Lane l scores groups l, l + L, ... from the keys in shared memory; each
    // starts at another place of its group, so that lanes hit other banks.
    constexpr int G = (32 + L - 1) / L;
    uint32_t* keys = staged + mine * (p.E | 8);
    const int size = p.E / p.groups;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * L + l < p.E) keys[v * L + l] = key[v];
    __syncwarp();
    uint32_t total[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int g = j * L + l;
      uint32_t best = 0, second = 0;
      if (g < p.groups) {
        int at = g % size;
#pragma unroll 4
        for (int i = 0; i < size; ++i) {
          const uint32_t u = keys[g * size + at];
          second = max(second, min(best, u));
          best = max(best, u);
          at = at + 1 == size ? 0 : at + 1;
        }
      }
      total[j] = best;
      if (p.group_top == 2 && second != 0) {
        const float sum = unordered(best) + unordered(second);
        total[j] = ordered(sum < kLowest ? kLowest : sum);
      }
    }
    uint32_t kept = 0;
#pragma unroll 1
    for (int i = 0; i < p.kept; ++i) {
      const Best b = best_of<L, G>(total, l);
      if (b.key != 0) kept |= 1u << b.at;
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (j * L + l == b.at) total[j] = 0;
    }
    const uint32_t per = (0xffffffffu / static_cast<uint32_t>(size)) + 1;  // e / size = (e * per) >> 32 for e, size <= 1024
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t g = size == 1 ? v * L + l : __umulhi(v * L + l, per);
      if (v * L + l < p.E && !((kept >> g) & 1u)) key[v] = 0;
    }
  }

  // Choice j is kept by lane j % L.
  constexpr int K = (32 + L - 1) / L;
  int chosen[K];
#pragma unroll
  for (int j = 0; j < K; ++j) chosen[j] = -1;
  bool done = false;
  if constexpr (L == 8 && V > 4) {
    // Looking through all V keys again for every choice costs more than all
    // the scores.  At least k experts are not below the k-th largest of the
    // lanes' maxima, and for a k well below the lanes rarely more than twice
    // as many: those go into a short list, whose members then rank each other.
    // The list costs about three choices of the loop below; the eighth of eight
    // lanes' maxima is so low that most warps hold a row with too many
    // candidates, and pay for both, and with more keys to a lane so is the
    // seventh.  127999 rows, list against loop:
    // 160 experts 41.3 us against 39.3 for k = 2, 41.3 and 45.4 (3), 49.5 and
    // 61.8 (6), 65.9 and 68.0 (7), 81 and 74 (8); 64 experts 24.9 and 23.7
    // (3), 24.9 and 27.0 (4), 29.4 and 33.1 (6), 43 and 39 (8); 256 experts
    // 62 and 58 (2), 62 and 66 (3), 78 and 93 (6), 111 and 103 (7); 32 experts
    // 20.8 and 18.7 (3), 24.9 and 22.9 (6).
    if (p.k >= 3 && p.k <= (V > 24 ? 6 : 7)) {
      __shared__ uint2 lists[kRouteWarps * kRowsPerWarp][2 * L];
      __shared__ int16_t orders[kRouteWarps * kRowsPerWarp][L];
      uint32_t most = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) most = max(most, key[v]);
      int rank = 0;  // of the lane's maximum, the lower lane first among equals
#pragma unroll
      for (int o = 1; o < L; ++o) {
        const uint32_t other = __shfl_xor_sync(kAll, most, o);
        rank += other > most || (other == most && (l ^ o) < l);
      }
      const uint32_t holder = __ballot_sync(kAll, rank == p.k - 1) >> (threadIdx.x & 31 & ~(L - 1)) & ((1u << L) - 1);
      const uint32_t least = max(__shfl_sync(kAll, most, __ffs(holder) - 1, L), 1u);
      int count = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) count += key[v] >= least;
      int up = count;
#pragma unroll
      for (int o = 1; o < L; o <<= 1) {
        const int t = __shfl_up_sync(kAll, up, o, L);
        if (l >= o) up += t;
      }
      const int all = __shfl_sync(kAll, up, L - 1, L);
      if (__all_sync(kAll, all <= 2 * L)) {
        done = true;
        uint2* list = lists[mine];
        uint32_t to = smem_u32(list + up - count);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool in = key[v] >= least;
          asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p st.shared.v2.u32 [%0], {%1, %2};\n\t}" ::"r"(to),
                       "r"(key[v]), "r"(v * L + l), "r"(static_cast<int>(in))
                       : "memory");
          to += in ? sizeof(uint2) : 0;
        }
        __syncwarp();
        // Every candidate's rank among them, by reading the list.
        int16_t* order = orders[mine];
        for (int i = l; i < all; i += L) {
          const uint2 c = list[i];
          int before = 0;
#pragma unroll
          for (int j = 0; j < 2 * L; ++j) {
            const uint2 o = j < all ? list[j] : make_uint2(0, 0);
            before += o.x > c.x || (o.x == c.x && o.y < c.y);
          }
          if (before < p.k) order[before] = static_cast<int16_t>(c.y);
        }
        __syncwarp();
        if (l < p.k && l < all) chosen[0] = order[l];
      }
    }
  }
  if (!done) {
#pragma unroll 1
    for (int c = 0; c < p.k; ++c) {
      const Best b = best_of<L, V>(key, l);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * L + l == b.at) key[v] = 0;
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (c == j * L + l && b.key != 0) chosen[j] = b.at;
    }
  }
  // Weights from the scores without the bias, computed again for the few chosen.
  float cs[K], sum = 0.f;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    cs[j] = 0.f;
    if (j * L >= p.k) continue;
    cs[j] = chosen[j] >= 0 ? score_at(logit_at(logits, row * p.E + chosen[j]), p.score, scale) : 0.f;
    sum += cs[j];
  }
  sum = lanes_sum<L>(sum);
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int c = j * L + l;
    if (j * L < p.k && live && c < p.k) {
      experts[row * p.k + c] = chosen[j];
      const float w = (p.renorm ? cs[j] / (sum + 1e-20f) : cs[j]) * p.scale;
      weights[row * p.k + c] = chosen[j] >= 0 ? w : 0.f;  // also beside a NaN, which makes the sum NaN
    }
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
