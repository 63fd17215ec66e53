// Products of a few tokens with MX weights: a linear, and the two products of
// a mixture-of-experts layer.
#include <cooperative_groups.h>

#include "few.h"
#include "few_product.cuh"
#include "launch.h"

namespace fp8bw {
namespace {

using namespace few;
namespace cg = cooperative_groups;

// A block owns a run of rows and walks through its share of the contraction in
// units: parts of K of one matrix.  Its warps are row_warps (32 rows each) times
// as many shares of every unit's chunks; the shares' sums meet in shared memory,
// and those of the `splits` blocks of a cluster, which take every splits-th
// unit, through distributed shared memory.  All orders are fixed.
//
//   kLinear  one matrix                                   y
//   kUp      the matrix of one active expert (grid.y), rows in pairs of gate
//            and up                                       records of the activation
//   kDown    the matrices of all active experts, one unit behind the other
//                                                         y
enum Mode { kLinear, kUp, kDown };

struct Product {
  Matrix m;
  int64_t rows;         // of a matrix; kUp: 2F
  int M;
  int row_warps, part, parts, splits;
  uint32_t buffer;      // bytes of tokens in shared memory at a time
  const uint16_t* x;    // bf16 [M, K]; kDown: none
  const FewPlan* plan;  // kUp, kDown
  int choices;          // of the plan
  uint8_t* act;         // records of the activation: written by kUp, read by kDown
  uint16_t* y;          // bf16 [M, rows]
};

template <int kBits>
constexpr int kStages = kBits == 4 ? 4 : 3;
template <int kBits>
constexpr uint32_t kRing = kWarps * kStages<kBits> * Weights<kBits>::kStage;
constexpr uint32_t kSlack = 128;  // lanes without a token read past the last record

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Tokens x[list[i]][k0 .. k0 + len) as records at `to`.
__device__ void convert_tokens(const uint16_t* __restrict__ x, int K, const int* list, int n, int k0, int len, uint8_t* to) {
  const int per = len / 8, total = n * per, record = record_bytes(n);
  for (int i0 = threadIdx.x & ~31; i0 < total; i0 += kThreads) {
    const int i = i0 + (threadIdx.x & 31);
    const int token = i / per, k8 = i - token * per;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (i < total) v = __ldg(reinterpret_cast<const uint4*>(x + static_cast<int64_t>(list ? list[token] : token) * K + k0) + k8);
    uint32_t top = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    top = max(top & 0xFFFFu, top >> 16);
    top = max(top, __shfl_xor_sync(kAll, top, 1));
    top = max(top, __shfl_xor_sync(kAll, top, 2));
    const uint32_t field = factor_field(top >> 7);
    const float f = of_field(field);
    const uint4 h = make_uint4(pack_f16x2(bf16lo_to_f32(v.x) * f, bf16hi_to_f32(v.x) * f),
                               pack_f16x2(bf16lo_to_f32(v.y) * f, bf16hi_to_f32(v.y) * f),
                               pack_f16x2(bf16lo_to_f32(v.z) * f, bf16hi_to_f32(v.z) * f),
                               pack_f16x2(bf16lo_to_f32(v.w) * f, bf16hi_to_f32(v.w) * f));
    if (i < total) {
      uint8_t* r = to + (k8 >> 2) * record;
      *reinterpret_cast<uint4*>(r + token * 64 + (k8 & 3) * 16) = h;
      if ((k8 & 3) == 0) *reinterpret_cast<float*>(r + n * 64 + token * 4) = of_field(254u - field);
    }
  }
}

template <Mode kMode, int kBits, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const __grid_constant__ Product p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_list[kWarps][32];
  using W = Weights<kBits>;
  constexpr int kDepth = kStages<kBits>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int shares = kWarps / p.row_warps, rw = warp % p.row_warps, share = warp / p.row_warps;
  const int R = p.row_warps * kTileRows;
  const int rank = blockIdx.x % p.splits;
  const int64_t block = blockIdx.x / p.splits;
  const int K = p.m.K;

  // What the plan says.  The plan is older than the kernel before this one, which waited for it before it let this one
  // start, so kDown reads it, and starts on the weights, while that kernel still runs.
  int slots = 1;
  FewSlot one{0, 0, 0, p.M};
  FewSlot* table = nullptr;
  if constexpr (kMode == kUp) {
    grid_wait();
    grid_release();
    if (static_cast<int>(blockIdx.y) >= few_active(p.plan)) return;
    one = few_slot(p.plan, p.choices, blockIdx.y);
    if ((one.mask >> lane) & 1) s_list[warp][__popc(one.mask & ((1u << lane) - 1))] = lane;
  } else if constexpr (kMode == kDown) {
    slots = few_active(p.plan);
    table = reinterpret_cast<FewSlot*>(smem + kRing<kBits> + 2 * p.buffer + kSlack +
                                       (p.M > 1 ? kWarps * p.M * kRowPitch * 4 : 0));
    for (int i = threadIdx.x; i < slots; i += kThreads) table[i] = few_slot(p.plan, p.choices, i);
  }
  __syncthreads();
  const auto slot_of = [&](int u) { return kMode == kDown ? table[u / p.parts] : one; };
  const int units = slots * p.parts;
  const auto length = [&](int u) { return min(p.part, K - u % p.parts * p.part); };
  const auto chunks = [&](int u) { return (length(u) + kChunk - 1) / kChunk; };

  // The warp's rows in the matrix of a unit.
  int64_t row0;
  if constexpr (kMode == kUp) {
    const int half = p.row_warps / 2;
    row0 = (block * half + rw % half) * kTileRows;
    row0 = (row0 < p.rows / 2 ? row0 : p.rows / 2 - kTileRows) + (rw >= half ? p.rows / 2 : 0);
  } else {
    row0 = block * R + rw * kTileRows;
    row0 = row0 < p.rows ? row0 : p.rows - 1;
  }
  const auto tile_of = [&](int u) {
    const int64_t first = slot_of(u).expert * p.rows;
    return tile_at<kBits>(p.m, first + row0, first + p.rows);
  };

  // The stream of weights: the warp's chunks of unit after unit, kDepth - 1 of them under way.
  const uint32_t ring = smem_u32(smem) + warp * kDepth * W::kStage;
  int load_u = rank - p.splits, load_c = 0, load_n = 0, load_first = 0;  // the unit, its next chunk, its chunks, where it begins
  RowTile<kBits> load_tile{};
  const auto next_unit = [&]() {
    do {
      load_u += p.splits;
      if (load_u >= units) return;
      load_n = chunks(load_u);
      load_c = share;
    } while (load_c >= load_n);
    load_first = load_u % p.parts * p.part / kChunk;
    load_tile = tile_of(load_u);
  };
  next_unit();
  const auto fetch = [&](int stage) {
    if (load_u < units) {
      copy_chunk<kBits>(p.m, load_tile, load_first + load_c, ring + stage * W::kStage, lane);
      load_c += shares;
      if (load_c >= load_n) next_unit();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch(i);

  // Tokens: as many units at a time as fit.
  uint8_t* const tokens = smem + kRing<kBits>;
  const auto bytes = [&](int u) { return static_cast<uint32_t>(length(u) / 32 * record_bytes(slot_of(u).n)); };
  const auto pass_end = [&](int u) {
    uint32_t used = 0;
    for (int v = u; v < units; v += p.splits) {
      used += bytes(v);
      if (v != u && used > p.buffer) return v;
    }
    return units;
  };
  const auto bring = [&](int from, int end, uint8_t* to) {
    for (int u = from; u < end; u += p.splits) {
      const FewSlot s = slot_of(u);
      if constexpr (kMode == kDown) {
        const uint8_t* src = p.act + few_act_at(s.start, K) + static_cast<int64_t>(u % p.parts * p.part / 32) * record_bytes(s.n);
        const uint32_t n = bytes(u), dst = smem_u32(to);
        for (uint32_t i = threadIdx.x * 16; i < n; i += kThreads * 16) cp_async16(dst + i, src + i);
      } else {
        convert_tokens(p.x, K, kMode == kUp ? s_list[warp] : nullptr, s.n, u % p.parts * p.part, length(u), to);
      }
      to += bytes(u);
    }
  };

  float* const sums = reinterpret_cast<float*>(kMode == kDown && p.M > 1 ? smem + kRing<kBits> + 2 * p.buffer + kSlack : smem);
  float* const mine = sums + warp * p.M * kRowPitch;
  if (kMode == kDown && p.M > 1)
    for (int i = lane; i < p.M * kRowPitch; i += 32) mine[i] = 0.f;

  float acc[2][kTiles][4] = {};
  int step = 0, since = 0, which = 0;
  if constexpr (kMode == kDown) {
    grid_wait();
    if (rank < units) bring(rank, pass_end(rank), tokens);
  }
  for (int u0 = rank; u0 < units;) {
    const int u1 = pass_end(u0);
    uint32_t at;
    if constexpr (kMode == kDown) {
      // Tokens came with the chunk copies of kDepth steps ago, or are waited for.
      if (since < kDepth) asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
      at = smem_u32(tokens + which * p.buffer);
      which ^= 1;
      if (u1 < units) bring(u1, pass_end(u1), tokens + which * p.buffer);
      since = 0;
    } else {
      if (u0 != rank) __syncthreads();
      bring(u0, u1, tokens);
      __syncthreads();
      at = smem_u32(tokens);
    }
    for (int u = u0; u < u1; u += p.splits) {
      const FewSlot s = slot_of(u);
      const int record = record_bytes(s.n), tiles = (s.n + 7) / 8, len = length(u), count = chunks(u);
      const RowTile<kBits> tile = tile_of(u);
      for (int c = share; c < count; c += shares) {
        cp_async_wait<kDepth - 2>();
        __syncwarp();  // the chunk is there for all lanes, and the stage read in the last step is free
        fetch((step + kDepth - 1) % kDepth);
        const uint32_t stage = ring + step % kDepth * W::kStage, t = at + c * 4 * record;
        const int blocks = len / 32 - c * 4;
        if (blocks >= 4)
          multiply_chunk<kBits, kTiles, true>(p.m, tile, stage, t, record, s.n, tiles, 4, lane, acc);
        else
          multiply_chunk<kBits, kTiles, false>(p.m, tile, stage, t, record, s.n, tiles, blocks, lane, acc);
        ++step;
        ++since;
      }
      at += bytes(u);
      if constexpr (kMode == kDown) {
        // Another expert has other tokens in the columns.
        if (p.M > 1 && (u + p.splits >= units || (u + p.splits) / p.parts != u / p.parts)) {
          if ((s.mask >> lane) & 1) s_list[warp][__popc(s.mask & ((1u << lane) - 1))] = lane;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int column = i * 8 + q4 * 2 + e;
              float* to = mine + s_list[warp][column & 31] * kRowPitch + g;
              if (column < s.n)
#pragma unroll
                for (int h = 0; h < 4; ++h) to[8 * h] += acc[h / 2][i][(h & 1) * 2 + e];
#pragma unroll
              for (int h = 0; h < 4; ++h) acc[h / 2][i][(h & 1) * 2 + e] = 0.f;
            }
          __syncwarp();
        }
      }
    }
    u0 = u1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // The sums of the warps' shares, then of the cluster's blocks.
  const int n = kMode == kUp ? one.n : p.M;
  if (kMode != kDown || p.M == 1) {
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int column = i * 8 + q4 * 2 + e;
        if (column < n)
#pragma unroll
          for (int h = 0; h < 4; ++h) mine[column * kRowPitch + g + 8 * h] = acc[h / 2][i][(h & 1) * 2 + e];
      }
    __syncthreads();
  }
  const auto block_sum = [&](int token, int row) {
    float v = 0.f;
    const float* from = sums + (row / kTileRows * p.M + token) * kRowPitch + row % kTileRows;
    for (int i = 0; i < shares; ++i) v += from[i * p.row_warps * p.M * kRowPitch];
    return v;
  };
  float* const part = reinterpret_cast<float*>(smem) + (reinterpret_cast<uint8_t*>(sums) == smem ? kWarps * p.M * kRowPitch : 0);
  cg::cluster_group cluster = cg::this_cluster();
  if (p.splits > 1) {
    for (int i = threadIdx.x; i < n * R; i += kThreads) part[i] = block_sum(i / R, i % R);
    cluster.sync();
  }
  const auto total = [&](int token, int row) {
    if (p.splits == 1) return block_sum(token, row);
    float v = 0.f;
    for (int r = 0; r < p.splits; ++r) v += cluster.map_shared_rank(part, r)[token * R + row];
    return v;
  };
  if constexpr (kMode == kUp) {
    // A warp per token and block of 32 of the activation.
    const int groups = p.row_warps / 2, F = static_cast<int>(p.rows / 2), record = record_bytes(n);
    const float* weights = few_weights(p.plan) + one.start;
    uint8_t* to = p.act + few_act_at(one.start, F);
    for (int i = rank * kWarps + warp; i < n * groups; i += p.splits * kWarps) {
      const int token = i / groups, gi = i % groups;
      const int64_t f = (block * groups + gi) * kTileRows;
      if (f >= F) continue;
      const float gate = total(token, gi * kTileRows + lane), up = total(token, (groups + gi) * kTileRows + lane);
      const float a = gate / (1.f + expf(-gate)) * up;
      uint32_t top = __float_as_uint(a) & 0x7FFFFFFFu;
      top = __reduce_max_sync(kAll, top);
      const uint32_t field = factor_field(top >> 23);
      uint8_t* r = to + f / 32 * record;
      reinterpret_cast<uint16_t*>(r + token * 64)[lane] = static_cast<uint16_t>(pack_f16x2(a * of_field(field), 0.f));
      if (lane == 0) *reinterpret_cast<float*>(r + n * 64 + token * 4) = of_field(254u - field) * weights[token];
    }
  } else {
    for (int i = rank * kThreads + threadIdx.x; i < n * R; i += p.splits * kThreads) {
      const int token = i / R, row = i % R;
      const int64_t at = block * R + row;
      if (at < p.rows)
        p.y[token * p.rows + at] = static_cast<uint16_t>(pack_bf16x2(total(token, row), 0.f) & 0xFFFFu);
    }
  }
  if (p.splits > 1) cluster.sync();  // a block's shared memory is read until then
}

// ---------------------------------------------------------------- launches

struct Shape {
  int row_warps, splits, part, parts;
  uint32_t buffer, smem;
};

constexpr uint32_t kMostSmem = 227 * 1024 - 2048;

// How a product of `rows` rows (of one matrix) is cut.  matrices: how many lie behind each other along the contraction
// (kDown), copies: how many share the grid (kUp).
Shape shape_of(Mode mode, int bits, int M, int64_t rows, int K, int matrices, int copies, int num_sms) {
  Shape s{};
  const uint32_t ring = bits == 4 ? kRing<4> : kRing<8>;
  s.row_warps = M <= 4 ? 1 : M <= 16 ? 2 : 4;
  if (mode == kUp && s.row_warps < 2) s.row_warps = 2;
  const int64_t blocks = (rows + s.row_warps * kTileRows - 1) / (s.row_warps * kTileRows) * copies;
  const int chunks = (K + kChunk - 1) / kChunk, shares = kWarps / s.row_warps;
  s.splits = 1;
  while (s.splits < 8 && blocks * s.splits < num_sms && static_cast<int64_t>(chunks) * matrices >= 2 * s.splits * shares)
    s.splits *= 2;
  const int record = record_bytes(M), buffers = mode == kDown ? 2 : 1;
  const uint32_t fixed = ring + kSlack + (mode == kDown && M > 1 ? kWarps * M * kRowPitch * 4 : 0) +
                         (mode == kDown ? matrices * sizeof(FewSlot) : 0);
  // Two blocks an SM where that leaves room for some tokens.
  uint32_t room = (kMostSmem / 2 > fixed + 16 * 1024 ? kMostSmem / 2 : kMostSmem) - fixed;
  room = room / buffers / 128 * 128;
  const int most = static_cast<int>(room / record) / 4 * kChunk;  // weights of a row whose tokens fit
  const int64_t even = (static_cast<int64_t>(chunks) * matrices + s.splits - 1) / s.splits;  // chunks of a block
  s.part = static_cast<int>(even < chunks ? even : chunks) * kChunk;
  if (mode == kDown && s.part > 8 * kChunk) s.part = 8 * kChunk;
  if (s.part > most) s.part = most;
  s.parts = (K + s.part - 1) / s.part;
  const int64_t units = (static_cast<int64_t>(s.parts) * matrices + s.splits - 1) / s.splits;
  const int64_t want = units * (s.part / 32) * record;
  s.buffer = static_cast<uint32_t>(want < room ? (want + 127) / 128 * 128 : room);
  s.smem = fixed + buffers * s.buffer;
  return s;
}

template <Mode kMode, int kBits, int kTiles>
cudaError_t launch(const Product& p, const Shape& s, dim3 grid, bool overlap, cudaStream_t st) {
  static thread_local uint32_t allowed[64] = {};  // by device
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  auto* kernel = few_kernel<kMode, kBits, kTiles>;
  if (dev >= 64 || allowed[dev] < s.smem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostSmem));
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = kMostSmem;
  }
  cudaLaunchAttribute attrs[2]{};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = st;
  cfg.attrs = attrs;
  if (s.splits > 1) {
    attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attrs[cfg.numAttrs].val.clusterDim.x = s.splits;
    attrs[cfg.numAttrs].val.clusterDim.y = 1;
    attrs[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (overlap) {
    attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <Mode kMode>
cudaError_t launch_product(Product p, int bits, int matrices, int copies, int num_sms, cudaStream_t st) {
  const Shape s = shape_of(kMode, bits, p.M, p.rows, p.m.K, matrices, copies, num_sms);
  p.row_warps = s.row_warps;
  p.part = s.part;
  p.parts = s.parts;
  p.splits = s.splits;
  p.buffer = s.buffer;
  const int64_t blocks = (p.rows + s.row_warps * kTileRows - 1) / (s.row_warps * kTileRows);
  const dim3 grid(static_cast<unsigned>(blocks * s.splits), static_cast<unsigned>(copies));
  const bool overlap = kMode != kLinear;
  const int tiles = p.M <= 8 ? 1 : p.M <= 16 ? 2 : 4;
  if (bits == 4)
    return tiles == 1   ? launch<kMode, 4, 1>(p, s, grid, overlap, st)
           : tiles == 2 ? launch<kMode, 4, 2>(p, s, grid, overlap, st)
                        : launch<kMode, 4, 4>(p, s, grid, overlap, st);
  return tiles == 1   ? launch<kMode, 8, 1>(p, s, grid, overlap, st)
         : tiles == 2 ? launch<kMode, 8, 2>(p, s, grid, overlap, st)
                      : launch<kMode, 8, 4>(p, s, grid, overlap, st);
}

}  // namespace

cudaError_t launch_few_linear(const FewLinearArgs& a, cudaStream_t st) {
  Product p{};
  p.m = Matrix{a.w, a.e8, a.N * (a.K / 32), static_cast<int>(a.K)};
  p.rows = a.N;
  p.M = static_cast<int>(a.M);
  p.x = a.x;
  p.y = a.y;
  return launch_product<kLinear>(p, a.bits, 1, 1, a.num_sms, st);
}

size_t few_moe_workspace_bytes(int64_t M, int64_t, int64_t top_k, int64_t, int64_t F) {
  return few_plan_bytes(M, top_k) + few_act_at(M * top_k, F);
}

cudaError_t launch_few_moe(const FewMoeArgs& a, cudaStream_t st) {
  const int64_t E = a.route.E, M = a.route.M, k = a.route.top_k;
  const int active = static_cast<int>(E < M * k ? E : M * k);
  FewPlan* plan = static_cast<FewPlan*>(a.workspace);
  uint8_t* act = static_cast<uint8_t*>(a.workspace) + few_plan_bytes(M, k);
  if (const cudaError_t e = launch_few_route(a, plan, st)) return e;
  Product up{};
  up.m = Matrix{a.w13, a.e13, E * 2 * a.F * (a.C / 32), static_cast<int>(a.C)};
  up.rows = 2 * a.F;
  up.M = static_cast<int>(M);
  up.x = a.x;
  up.plan = plan;
  up.choices = static_cast<int>(M * k);
  up.act = act;
  if (const cudaError_t e = launch_product<kUp>(up, a.bits, 1, active, a.num_sms, st)) return e;
  Product down{};
  down.m = Matrix{a.w2, a.e2, E * a.C * (a.F / 32), static_cast<int>(a.F)};
  down.rows = a.C;
  down.M = static_cast<int>(M);
  down.plan = plan;
  down.choices = static_cast<int>(M * k);
  down.act = act;
  down.y = a.y;
  return launch_product<kDown>(down, a.bits, active, 1, a.num_sms, st);
}

}  // namespace fp8bw
