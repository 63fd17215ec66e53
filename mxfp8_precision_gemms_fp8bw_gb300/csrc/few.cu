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

// A block owns a run of rows and walks through its share of the contraction.
// Its warps are row_warps (32 rows each) times as many shares of the chunks;
// the shares' sums meet in shared memory, and those of the `splits` blocks of a
// cluster, which split the contraction, through distributed shared memory.  All
// orders are fixed.
//
//   kLinear  one matrix                                   y
//   kUp      the matrix of one active expert (grid.y), rows in pairs of gate
//            and up                                       records of the activation
//   kDown    the matrices of all active experts, one behind the other
//                                                         y
enum Mode { kLinear, kUp, kDown };

struct Product {
  Matrix m;
  int64_t rows;         // of a matrix; kUp: 2F
  int M;
  int row_warps, splits;
  int part, parts;      // chunks whose tokens are in shared memory at a time; kDown: parts of a matrix
  int share;            // chunks (kDown: parts) of a block
  uint32_t buffer;      // bytes of tokens in shared memory at a time, of which there are two
  uint32_t sums_at;     // where the sums are; 0 puts them over the stages, once the stream has ended
  uint32_t table_at;    // kDown: where the slots are
  const uint16_t* x;    // kLinear with few elements: bf16 [M, K], converted here
  FewTokens t;          // kLinear otherwise, kUp
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
constexpr int kInline = 8;        // 16-byte pieces of tokens that a thread converts where the kernel does
constexpr int64_t kMostInline = kInline * 8 * kThreads;

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// x as FewTokens holds it, a token to a block.
template <int kBits>
__global__ void __launch_bounds__(kThreads) few_tokens_kernel(const uint16_t* __restrict__ x, int K, FewTokens t) {
  __shared__ uint32_t top;
  grid_release();
  const uint4* row = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(blockIdx.x) * K);
  uint8_t* to = t.rows + static_cast<int64_t>(blockIdx.x) * K * 2;
  if (threadIdx.x == 0) top = 0;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < K / 8; i += kThreads) m = __vmaxu2(m, largest(__ldg(row + i)));
  m = __reduce_max_sync(kAll, max(m & 0xFFFFu, m >> 16));
  if ((threadIdx.x & 31) == 0) atomicMax(&top, m);  // a maximum does not depend on the order
  __syncthreads();
  const uint32_t field = factor_field(top >> 7);
  if (threadIdx.x == 0) t.scales[blockIdx.x] = of_field(254u - field);
#pragma unroll 4
  for (int i = threadIdx.x; i < K / 8; i += kThreads)
    store_f16<kBits>(to + i / 4 * 64, i & 3, to_f16(__ldg(row + i), of_field(field)));
}

template <Mode kMode, int kBits, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) few_kernel(const __grid_constant__ Product p) {
  constexpr bool kScaled = kMode == kDown;
  constexpr int kDepth = kStages<kBits>;
  constexpr int kStage = Weights<kBits>::kStage;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_list[kMode == kDown ? kWarps : 1][32];
  __shared__ uint32_t s_top[kMode == kLinear ? 32 : 1];
  __shared__ float s_scale[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int shares = kWarps / p.row_warps, rw = warp & (p.row_warps - 1), share = warp / p.row_warps;
  const int R = p.row_warps * kTileRows;
  const int rank = blockIdx.x & (p.splits - 1), block = blockIdx.x / p.splits;
  const int K = p.m.K;

  // What the plan says.  The plan is older than the kernel before this one, which waited for it before it let this one
  // start, so kDown reads it, and starts on the weights, while that kernel still runs.
  int slots = 1;
  FewSlot one{0, 0, 0, p.M};
  const FewSlot* table = nullptr;
  if constexpr (kMode == kUp) {
    grid_wait();
    grid_release();
    if (static_cast<int>(blockIdx.y) >= few_active(p.plan)) return;
    one = few_slot(p.plan, p.choices, blockIdx.y);
    if (warp == 0 && ((one.mask >> lane) & 1)) {
      const int column = __popc(one.mask & ((1u << lane) - 1));
      s_list[0][column] = lane;
      s_scale[column] = __ldcg(p.t.scales + lane);
    }
  } else if constexpr (kMode == kDown) {
    slots = few_active(p.plan);
    FewSlot* to = reinterpret_cast<FewSlot*>(smem + p.table_at);
    for (int i = threadIdx.x; i < slots; i += kThreads) to[i] = few_slot(p.plan, p.choices, i);
    table = to;
  } else {
    if (warp == 0) s_top[lane] = 0, s_list[0][lane] = lane;
  }

  // The warp's rows in a matrix.
  int64_t row0;
  if constexpr (kMode == kUp) {
    const int half = p.row_warps / 2, F = static_cast<int>(p.rows / 2);
    row0 = min((block * half + (rw & (half - 1))) * kTileRows, F - kTileRows) + (rw >= half ? F : 0);
  } else {
    row0 = min(static_cast<int64_t>(block) * R + rw * kTileRows, p.rows - 1);
  }
  const Weights<kBits> W(p.m, static_cast<int>(min(p.rows - row0, int64_t{kTileRows})) - 1, lane);

  // The stream of weights: the warp's chunks, kDepth - 1 of them under way.
  const uint32_t ring = smem_u32(smem) + warp * (kDepth * kStage);
  const int begin = kMode == kDown ? 0 : rank * p.share, end = kMode == kDown ? 0 : min(begin + p.share, (K + kChunk - 1) / kChunk);
  int64_t e8_at = (one.expert * p.rows + row0) * W.scale_pitch;
  const uint8_t* load_w = p.m.w + (one.expert * p.rows + row0) * W.pitch;
  int64_t load_e8 = e8_at;
  int load_c = begin + share, load_end = end;
  // kDown: parts u of all matrices, part u % parts of the matrix of slot u / parts
  int load_u = 0, u_end = 0, u_begin = 0;
  struct Part {
    FewSlot slot;
    int first, blocks;  // in chunks, in blocks of 32
  };
  const auto part_at = [&](int u) {
    const int i = p.parts == 1 ? u : u / p.parts;
    Part v;
    v.slot = table[i];
    v.first = (u - i * p.parts) * p.part;
    v.blocks = min(p.part * 4, K / 32 - v.first * 4);
    return v;
  };
  const auto next_part = [&]() {
    while (load_u < u_end) {
      const Part v = part_at(load_u);
      ++load_u;
      load_c = v.first + share;
      load_end = v.first + (v.blocks + 3) / 4;
      const int64_t row = v.slot.expert * p.rows + row0;
      load_w = p.m.w + row * W.pitch;
      load_e8 = row * W.scale_pitch;
      if (load_c < load_end) return;
    }
  };
  if constexpr (kMode == kDown) {
    __syncthreads();  // the table
    u_begin = min(slots * p.parts * rank / p.splits, slots * p.parts);
    u_end = slots * p.parts * (rank + 1) / p.splits;
    load_u = u_begin;
    next_part();
  }
  const auto fetch = [&](uint32_t stage) {
    if (load_c < load_end) {
      W.copy(load_w, load_e8, load_c, stage, lane);
      load_c += shares;
      if (kMode == kDown && load_c >= load_end) next_part();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch(ring + i * kStage);
  uint32_t stage = ring, free_stage = ring + (kDepth - 1) * kStage;  // to be read next, to be filled next

  uint8_t* const tokens = smem + kRing<kBits>;
  const bool apart = kMode == kDown && p.M > 1;
  float* const sums = reinterpret_cast<float*>(smem + p.sums_at);
  float* const mine = sums + warp * p.M * kRowPitch;
  if (apart)
    for (int i = lane; i < p.M * kRowPitch; i += 32) mine[i] = 0.f;

  float acc[2][kTiles][4] = {};
  // acc to the warp's sums, of the tokens in its columns; acc is 0 after it.
  const auto put = [&](uint32_t mask, int n) {
    if (apart) {
      if ((mask >> lane) & 1) s_list[warp % (kMode == kDown ? kWarps : 1)][__popc(mask & ((1u << lane) - 1))] = lane;
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int column = i * 8 + q4 * 2 + e;
        if (column < n) {
          const int token = apart ? s_list[warp % (kMode == kDown ? kWarps : 1)][column] : column;
          const float f = kMode == kDown ? 1.f : s_scale[column];
          float* to = mine + token * kRowPitch + g;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float v = acc[h / 2][i][(h & 1) * 2 + e] * f;
            to[8 * h] = apart ? to[8 * h] + v : v;
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) acc[h / 2][i][(h & 1) * 2 + e] = 0.f;
      }
    if (apart) __syncwarp();
  };
  // Chunks of this warp from c to last, whose tokens are records at `at` for chunk `from` on.
  int since = 0;
  const auto multiply = [&](int c, int last, int from, int n, uint32_t at) {
    const int record = record_bytes(n, kScaled), tiles = (n + 7) / 8;
    uint32_t columns[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) columns[i] = min(i * 8 + g, n - 1) * 64 + q4 * 16;
    const uint32_t scale_at = n * 64 + q4 * 8;
    at += (c - from) * 4 * record;
    for (; c < last; c += shares) {
      cp_async_wait<kDepth - 2>();
      __syncwarp();  // the chunk is there for all lanes, and the stage read in the last step is free
      fetch(free_stage);
      const int blocks = K / 32 - c * 4;
      if (blocks < 4)
        multiply_chunk<kBits, kTiles, kTiles, kScaled, false>(W, stage, e8_at, at, record, columns, scale_at, blocks, lane, acc);
      else if (kTiles == 1 || tiles == 1)
        multiply_chunk<kBits, 1, kTiles, kScaled, true>(W, stage, e8_at, at, record, columns, scale_at, 4, lane, acc);
      else if (kTiles == 2 || tiles == 2)
        multiply_chunk<kBits, kTiles < 2 ? kTiles : 2, kTiles, kScaled, true>(W, stage, e8_at, at, record, columns, scale_at, 4,
                                                                             lane, acc);
      else if (tiles == 3)
        multiply_chunk<kBits, kTiles < 3 ? kTiles : 3, kTiles, kScaled, true>(W, stage, e8_at, at, record, columns, scale_at, 4,
                                                                             lane, acc);
      else
        multiply_chunk<kBits, kTiles, kTiles, kScaled, true>(W, stage, e8_at, at, record, columns, scale_at, 4, lane, acc);
      free_stage = stage;
      stage = stage + kStage == ring + kDepth * kStage ? ring : stage + kStage;
      at += shares * 4 * record;
      ++since;
    }
  };
  // Before tokens that cp.async brings are read: they came with the chunk copies of kDepth steps ago, or are waited for.
  const auto arrived = [&]() {
    if (since < kDepth) cp_async_wait_all();
    __syncthreads();
    since = 0;
  };

  if constexpr (kMode == kDown) {
    const auto bytes = [&](const Part& v) { return static_cast<uint32_t>(v.blocks * record_bytes(v.slot.n, true)); };
    // As many parts at a time as fit.
    const auto pass_end = [&](int u) {
      uint32_t used = bytes(part_at(u));
      for (++u; u < u_end; ++u) {
        used += bytes(part_at(u));
        if (used > p.buffer) break;
      }
      return u;
    };
    const auto bring = [&](int from, int to_u, uint8_t* to) {
      for (int u = from; u < to_u; ++u) {
        const Part v = part_at(u);
        const uint8_t* src =
            p.act + few_act_at(v.slot.start, K) + static_cast<int64_t>(v.first * 4) * record_bytes(v.slot.n, true);
        const uint32_t n = bytes(v), dst = smem_u32(to);
        for (uint32_t i = threadIdx.x * 16; i < n; i += kThreads * 16) cp_async16(dst + i, src + i);
        to += n;
      }
    };
    grid_wait();
    int u0 = u_begin, u1 = u_begin < u_end ? pass_end(u_begin) : u_end, which = 0;
    bring(u0, u1, tokens);
    while (u0 < u_end) {
      arrived();
      uint32_t at = smem_u32(tokens + which * p.buffer);
      which ^= 1;
      const int u2 = u1 < u_end ? pass_end(u1) : u_end;
      bring(u1, u2, tokens + which * p.buffer);
      for (int u = u0; u < u1; ++u) {
        const Part v = part_at(u);
        e8_at = (v.slot.expert * p.rows + row0) * W.scale_pitch;
        multiply(v.first + share, v.first + (v.blocks + 3) / 4, v.first, v.slot.n, at);
        at += bytes(v);
        // Another expert has other tokens in the columns.
        if (apart && (u + 1 == u_end || (u + 1) % p.parts == 0)) put(v.slot.mask, v.slot.n);
      }
      u0 = u1;
      u1 = u2;
    }
  } else if (kMode == kLinear && p.x != nullptr) {
    // Few elements: every block converts its own, a piece of 8 after the other, all of them in flight at once.
    const int per = (min(end * 16, K / 8) - begin * 16), total = per * p.M;  // pieces
    uint4 v[kInline];
#pragma unroll
    for (int j = 0; j < kInline; ++j) {
      const int i = threadIdx.x + j * kThreads, t = p.M == 1 ? 0 : i / max(per, 1);
      if (i < total) v[j] = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * K) + begin * 16 + (i - t * per));
    }
    __syncthreads();  // s_top
#pragma unroll
    for (int j = 0; j < kInline; ++j) {
      const int i0 = (threadIdx.x & ~31) + j * kThreads;
      if (i0 >= total) break;
      const int i = i0 + lane, t = p.M == 1 ? 0 : i / per;
      const uint32_t m = i < total ? largest(v[j]) : 0u, m1 = max(m & 0xFFFFu, m >> 16);
      if (p.M == 1 || __all_sync(kAll, t == __shfl_sync(kAll, t, 0))) {
        const uint32_t most = __reduce_max_sync(kAll, m1);
        if (lane == 0) atomicMax(s_top + t, most);  // a maximum does not depend on the order
      } else if (i < total) {
        atomicMax(s_top + t, m1);
      }
    }
    __syncthreads();
    if (threadIdx.x < p.M) s_scale[threadIdx.x] = of_field(254u - factor_field(s_top[threadIdx.x] >> 7));
#pragma unroll
    for (int j = 0; j < kInline; ++j) {
      const int i = threadIdx.x + j * kThreads, t = p.M == 1 ? 0 : i / max(per, 1), k8 = i - t * per;
      if (i < total)
        store_f16<kBits>(tokens + ((k8 >> 2) * p.M + t) * 64, k8 & 3, to_f16(v[j], of_field(factor_field(s_top[t] >> 7))));
    }
    __syncthreads();
    multiply(begin + share, end, begin, p.M, smem_u32(tokens));
  } else {
    const int n = one.n;
    const int each = n <= 1 ? 8 : n <= 2 ? 4 : n <= 4 ? 2 : 1;  // warps to a token
    const auto bring = [&](int c0, int c1, uint8_t* to) {
      const int pieces = min(c1 * 16, K / 8) - c0 * 16;
      for (int t = warp / each; t < n; t += kWarps / each) {
        const uint8_t* src = p.t.rows + (static_cast<int64_t>(s_list[0][t]) * K + c0 * kChunk) * 2;
        const uint32_t dst = smem_u32(to) + t * 64;
        for (int i = warp % each * 32 + lane; i < pieces; i += each * 32)
          cp_async16(dst + (i >> 2) * n * 64 + (i & 3) * 16, src + i * 16);
      }
    };
    if constexpr (kMode == kLinear) {
      grid_wait();
      if (warp == 0 && lane < n) s_scale[lane] = __ldcg(p.t.scales + lane);
    }
    __syncthreads();  // s_list
    // The part's chunks are whole rounds of the shares, so a warp's next chunk carries over.
    int which = 0, c = begin + share;
    if (begin < end) bring(begin, min(begin + p.part, end), tokens);
    for (int c0 = begin; c0 < end; c0 += p.part) {
      const int c1 = min(c0 + p.part, end);
      arrived();
      const uint32_t at = smem_u32(tokens + which * p.buffer);
      which ^= 1;
      if (c1 < end) bring(c1, min(c1 + p.part, end), tokens + which * p.buffer);
      multiply(c, c1, c0, n, at);
      c += p.part;
    }
  }
  cp_async_wait_all();
  __syncthreads();

  // The sums of the warps' shares, then of the cluster's blocks.
  const int n = kMode == kUp ? one.n : p.M;
  if (!apart) {
    put(0, n);
    __syncthreads();
  }
  const auto block_sum = [&](int token, int row) {
    float v = 0.f;
    const float* from = sums + (row / kTileRows * p.M + token) * kRowPitch + row % kTileRows;
    for (int i = 0; i < shares; ++i) v += from[i * p.row_warps * p.M * kRowPitch];
    return v;
  };
  float* const part = reinterpret_cast<float*>(smem) + (apart ? 0 : kWarps * p.M * kRowPitch);
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
    const int groups = p.row_warps / 2, F = static_cast<int>(p.rows / 2), record = record_bytes(n, true);
    const float* weights = few_weights(p.plan) + one.start;
    uint8_t* to = p.act + few_act_at(one.start, F);
    for (int i = rank * kWarps + warp; i < n * groups; i += p.splits * kWarps) {
      const int token = i / groups, gi = i % groups;
      const int f = (block * groups + gi) * kTileRows;
      if (f >= F) continue;
      const float gate = total(token, gi * kTileRows + lane), up = total(token, (groups + gi) * kTileRows + lane);
      const float a = gate / (1.f + expf(-gate)) * up;
      uint32_t top = __float_as_uint(a) & 0x7FFFFFFFu;
      top = __reduce_max_sync(kAll, top);
      const uint32_t field = factor_field(top >> 23);
      uint8_t* r = to + f / 32 * record;
      reinterpret_cast<uint16_t*>(r + token * 64)[place_of<kBits>(lane)] =
          static_cast<uint16_t>(pack_f16x2(a * of_field(field), 0.f));
      if (lane == 0) *reinterpret_cast<float*>(r + n * 64 + token * 4) = of_field(254u - field) * weights[token];
    }
  } else {
    for (int i = rank * kThreads + threadIdx.x; i < n * R; i += p.splits * kThreads) {
      const int token = i / R, row = i % R;
      const int64_t at = static_cast<int64_t>(block) * R + row;
      if (at < p.rows)
        p.y[token * p.rows + at] = static_cast<uint16_t>(pack_bf16x2(total(token, row), 0.f) & 0xFFFFu);
    }
  }
  if (p.splits > 1) cluster.sync();  // a block's shared memory is read until then
}

// ---------------------------------------------------------------- launches

struct Shape {
  int row_warps, splits, part, parts, share;
  uint32_t buffer, sums_at, table_at, smem;
};

constexpr uint32_t kMostSmem = 227 * 1024 - 2048;

// How a product of `rows` rows (of one matrix) is cut.  matrices: how many lie behind each other along the contraction
// (kDown), copies: how many share the grid (kUp).
Shape shape_of(Mode mode, int bits, int M, int64_t rows, int K, int matrices, int copies, bool inline_tokens,
               int num_sms) {
  Shape s{};
  const uint32_t ring = bits == 4 ? kRing<4> : kRing<8>;
  s.row_warps = M <= 4 ? 1 : M <= 16 ? 2 : 4;
  if (mode == kUp && s.row_warps < 2) s.row_warps = 2;
  const int64_t blocks = (rows + s.row_warps * kTileRows - 1) / (s.row_warps * kTileRows) * copies;
  const int chunks = (K + kChunk - 1) / kChunk, shares = kWarps / s.row_warps;
  s.splits = 1;
  while (s.splits < 8 && blocks * s.splits < num_sms && static_cast<int64_t>(chunks) * matrices >= 2 * s.splits * shares)
    s.splits *= 2;
  const int record = record_bytes(M, mode == kDown);
  const uint32_t sums = mode == kDown && M > 1 ? kWarps * M * kRowPitch * 4 : 0;  // else over the stages
  const uint32_t fixed = ring + kSlack + sums + (mode == kDown ? matrices * sizeof(FewSlot) : 0);
  s.share = (chunks + s.splits - 1) / s.splits;
  if (inline_tokens) {
    s.part = s.share;
    s.buffer = static_cast<uint32_t>(s.share) * 4 * record;
    s.smem = fixed + s.buffer;
    return s;
  }
  // Two blocks an SM where that leaves room for some tokens.
  const auto room_of = [&](uint32_t smem) { return (smem - fixed) / 2 / 128 * 128; };
  uint32_t room = room_of(kMostSmem / 2 > fixed + 16 * 1024 ? kMostSmem / 2 : kMostSmem);
  if (static_cast<int>(room / record) / 4 < shares) room = room_of(kMostSmem);
  int part = static_cast<int>(room / record) / 4;  // chunks whose tokens fit
  if (mode == kDown) {
    if (part > 8) part = 8;
    if (part > chunks) part = chunks;
    s.parts = (chunks + part - 1) / part;
    const int64_t most = (static_cast<int64_t>(s.parts) * matrices + s.splits - 1) / s.splits;  // parts of a block
    const int64_t want = most * part * 4 * record;
    s.buffer = static_cast<uint32_t>(want < room ? (want + 127) / 128 * 128 : room);
  } else {
    if (part > s.share) part = s.share;
    if (part < s.share) part = part / shares * shares;  // whole rounds
    s.buffer = (static_cast<uint32_t>(part) * 4 * record + 127) / 128 * 128;
  }
  s.part = part;
  const uint32_t buffers = mode == kDown || part < s.share ? 2 : 1;
  s.sums_at = sums ? ring + buffers * s.buffer + kSlack : 0;
  s.table_at = ring + buffers * s.buffer + kSlack + sums;
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
  const Shape s = shape_of(kMode, bits, p.M, p.rows, p.m.K, matrices, copies, p.x != nullptr, num_sms);
  p.row_warps = s.row_warps;
  p.part = s.part;
  p.parts = s.parts;
  p.share = s.share;
  p.splits = s.splits;
  p.buffer = s.buffer;
  p.sums_at = s.sums_at;
  p.table_at = s.table_at;
  const int64_t blocks = (p.rows + s.row_warps * kTileRows - 1) / (s.row_warps * kTileRows);
  const dim3 grid(static_cast<unsigned>(blocks * s.splits), static_cast<unsigned>(copies));
  const bool overlap = kMode != kLinear || p.x == nullptr;
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
  p.y = a.y;
  if (a.M * a.K <= kMostInline) {
    p.x = a.x;
  } else {
    p.t = few_tokens_at(a.workspace, a.M, a.K);
    auto* kernel = a.bits == 4 ? few_tokens_kernel<4> : few_tokens_kernel<8>;
    kernel<<<static_cast<unsigned>(a.M), kThreads, 0, st>>>(a.x, static_cast<int>(a.K), p.t);
    if (const cudaError_t e = cudaGetLastError()) return e;
  }
  return launch_product<kLinear>(p, a.bits, 1, 1, a.num_sms, st);
}

size_t few_linear_workspace_bytes(int64_t M, int64_t K) { return M * K <= kMostInline ? 0 : few_tokens_bytes(M, K); }

size_t few_moe_workspace_bytes(int64_t M, int64_t, int64_t top_k, int64_t C, int64_t F) {
  return few_plan_bytes(M, top_k) + few_tokens_bytes(M, C) + few_act_at(M * top_k, F);
}

cudaError_t launch_few_moe(const FewMoeArgs& a, cudaStream_t st) {
  const int64_t E = a.route.E, M = a.route.M, k = a.route.top_k;
  const int active = static_cast<int>(E < M * k ? E : M * k);
  uint8_t* at = static_cast<uint8_t*>(a.workspace);
  FewPlan* plan = reinterpret_cast<FewPlan*>(at);
  const FewTokens tokens = few_tokens_at(at + few_plan_bytes(M, k), M, a.C);
  uint8_t* act = at + few_plan_bytes(M, k) + few_tokens_bytes(M, a.C);
  if (const cudaError_t e = launch_few_route(a, plan, tokens, st)) return e;
  Product up{};
  up.m = Matrix{a.w13, a.e13, E * 2 * a.F * (a.C / 32), static_cast<int>(a.C)};
  up.rows = 2 * a.F;
  up.M = static_cast<int>(M);
  up.t = tokens;
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
