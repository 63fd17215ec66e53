// Products of a few tokens with MX weights: a linear, and the two products of
// a mixture-of-experts layer.
//
// At most 32 tokens read every weight once, so the products are bound by the
// bytes of the weights, and what counts is that nothing is done to a weight
// between memory and the tensor core.  tcgen05.mma kind::mxf8f6f4.block_scale
// takes e2m1 and e4m3 codes and their E8M0 scales as they are, as its 128-row
// operand; the tokens are the narrow one (N), in e4m3 as well, as the sum of
// two or three parts (few_tokens.cuh) that are columns of their own.  (A
// version that turned weights into f16 for mma.sync took 55 instructions for
// 32 weights of 32 rows: 33 us for 32 tokens of 8192 x 5120 in 4 bits, 12.6
// here.)
//
// Measured, one call behind the other, of weights larger than the cache where
// they are: up of 8 experts 5120 -> 4096, 8 bits, 32 tokens 59 us (5.9 TB/s),
// their down product 40 us (4.3 TB/s).  A linear of 8192 x 16384 for 4 tokens
// 28 us in 8 bits (4.9 TB/s), 20 in 4 (3.5 TB/s); of 8192 x 5120 13 and 9; of
// 2048 x 2048, one token, 4.8.  What bounds them:
//   8 bits          memory: longer rows come at 6.6 TB/s, 0.97 of the copy
//                   bandwidth
//   4 bits          the way of a chunk, 0.4 us in each of two blocks an SM, as
//                   long as one of 8 bits takes from the cache: longer rows come
//                   at 4.8 TB/s.  Of the 20 us of 8192 x 16384, 19 remain without
//                   products, 19 without scales, 18 without both, 18 with the
//                   weights in the cache, 19 with codes left packed, and 18 with
//                   six stages of such codes in place of five.  Not the rows that
//                   TMA asks for (8 bits in boxes of 64 bytes a row take 3 %
//                   more), and half of those by cp.async, a fifth stage, or chunks
//                   asked for ahead into the cache change 2 % or cost some
//   short products  a start of about 4 us with the pipeline's first chunks, and,
//                   of a cluster, 1 to 2 us for blocks to meet and sum (3 for
//                   more than 16 tokens)
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "few.h"
#include "few_tokens.cuh"
#include "launch.h"

namespace fp8bw {
namespace {

using few::kAll;

// A block walks through runs: 128 rows of a matrix by a stretch of its
// contraction, in chunks of 128.
//
//   kLinear  one run of the one matrix                    y
//   kUp      64 rows of gate and the 64 of up that go with them, of an active
//            expert: one run, or, where there are many, whole ones of tiles
//            and experts in turn                          the activation, in five parts
//   kDown    128 rows of all active experts, one run behind the other; the sum
//            over each is drained from tensor memory, weighted and added to its
//            tokens in shared memory                      y
//
// The `splits` blocks of a cluster share the contraction, and their sums meet
// in distributed shared memory, in the order of the blocks.
//
// Warps 0-3  drain the accumulators (warp w: rows 32 w ..); a linear's one or
//            two tokens they bring into parts at first
// Warps 4-7  copy the weights' scales, by cp.async, and spread 4-bit codes
//            that TMA brings as they are in memory
// Warp  8    copies weights, by TMA
// Warp  9    copies tokens, by bulk copies
// Warp  10   brings the scales of a stage that has landed into tensor memory
// Warp  11   owns tensor memory and issues the products
//
// Weights and tokens stay off the load and store units: with cp.async those
// held a block back at 800 to 2000 cycles a chunk, of which 350 to 700 are what
// the memory takes.
enum Mode { kLinear, kUp, kDown };

constexpr int kRows = 128, kChunk = 128;
constexpr int kDrainWarps = 4, kScaleWarps = 4;
constexpr int kWeights = kDrainWarps + kScaleWarps, kTokens = kWeights + 1, kScaler = kTokens + 1, kIssuer = kScaler + 1;
constexpr int kThreads = (kIssuer + 1) * 32;

// A stage of shared memory: codes of 128 rows, 128 bytes each with 128-byte swizzling (4-bit codes of 16 weights in the first
// 8 bytes of 16, which is how the tensor core wants them); a record of tokens (few.h), where they are not in shared memory for
// good; the weights' scales, row r's four bytes as word (r % 32) * 4 + r / 32; and room for 4-bit codes to be spread.
constexpr uint32_t kCodes = kRows * 128, kScales = 512, kPacked = kRows * 64;

struct Matrix {
  const uint8_t* w;   // codes
  const uint8_t* e8;  // scales
  int64_t scale_end;  // bytes of e8
  int64_t rows;       // of one matrix; kUp: 2F
  int K;
};

// Stages: weight codes, tokens, their scales, packed codes.
struct Stages {
  int depth;        // how many
  uint32_t tokens;  // bytes of tokens
  uint32_t bytes;
};
__host__ __device__ inline Stages stages_of(int depth, uint32_t ring, uint32_t tokens, bool packed) {
  const uint32_t bytes = (kCodes + tokens + kScales + (packed ? kPacked : 0) + 1023) / 1024 * 1024;
  const int room = static_cast<int>(ring / bytes);
  return Stages{room < depth ? room : depth, tokens, bytes};
}

// Columns of tensor memory for a stage's scales: 4 for the weights', and 4 or 8 for up to 128 or 256 token rows.
__host__ __device__ constexpr int scale_columns_of(int rows) { return rows > 128 ? 16 : 8; }
// Columns of tensor memory behind the accumulators: the stages' scales, and no fewer than a load may read past an accumulator.
__host__ __device__ inline int tmem_scales(int of_stage, int depth) { return of_stage * depth > 16 ? of_stage * depth : 16; }

struct Product {
  Matrix m;
  int M, splits;
  int tiles;            // kUp, in turn: tiles of an expert; else 0
  bool late;            // the cluster's sums meet in the stages
  int slots;            // kDown: room for as many
  bool packed;          // 4-bit weights land as they are in memory, for whole chunks of 128 only TMA can spread them
  int columns;          // of an accumulator: token rows, a multiple of 16; kDown: by the plan
  Stages stages;        // kDown: of slots of M tokens; there are more where the plan's are smaller
  uint32_t ring;        // bytes of all stages
  uint32_t tmem;        // columns of tensor memory
  int share;            // kLinear, one or two tokens: most chunks of a block,
  uint32_t held_at;     // and where they are, behind the stages
  const uint16_t* x;    // kLinear, one or two tokens: bf16 [M, K]
  const uint8_t* t;     // otherwise records of tokens; kDown: of activations
  const FewPlan* plan;  // kUp, kDown
  int choices;          // of the plan
  uint8_t* act;         // kUp: records of activations
  uint16_t* y;          // bf16 [M, rows]
  int* status;
  uint64_t wait_ns;  // of a role, at most
};

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrives on `bar` once the thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Whether a wait came to its end for all lanes: they go on, or unwind, together.
__device__ __forceinline__ bool all_of(bool ok) { return __all_sync(kAll, ok); }

// A chunk of tokens that stay in shared memory, and the most of them: beside three stages of packed codes as much as two blocks
// an SM have room for.
constexpr uint32_t kHeld = 16 * 128;
constexpr int kMostHeld = 12;
constexpr int kMostDepth = 5;  // of 17 KB beside tokens that are held, from 19 KB on with tokens of their own, in kHalfSmem
struct Shared {
  // Of a stage: packed codes have landed, all of it has, its scales are in tensor memory, it has been read.
  uint64_t landed[kMostDepth], full[kMostDepth], ready[kMostDepth], empty[kMostDepth];
  uint64_t tokens;                       // a linear's tokens are in shared memory
  uint64_t sum_full[2], sum_empty[2];    // an accumulator is complete, has been drained
  uint64_t drain[2];
  uint32_t tmem;
  int abort;
  int issued[kScaleWarps + 2];  // where a wait expired: chunks that the warps of scales, weights and tokens have asked for
};

__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Barrier 1 is for the warps that use tensor memory, 2 for those that drain it.
template <int kBarrier, int kCount>
__device__ __forceinline__ void named_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(kBarrier), "n"(kCount) : "memory");
}

// The same, with a word on whether all may go on.
template <int kBarrier, int kCount>
__device__ __forceinline__ bool named_all(bool ok) {
  uint32_t all;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(all)
               : "r"(static_cast<uint32_t>(ok)), "n"(kBarrier), "n"(kCount)
               : "memory");
  return all != 0;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// x [M, K] in parts.
__global__ void __launch_bounds__(256) few_tokens_kernel(const uint16_t* x, int64_t K, uint8_t* t) {
  grid_wait();
  grid_release();  // after the wait: the product reads weights that kernels before this one may have written
  const int64_t pieces = K / 8;  // of 8 values, of a token
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + (threadIdx.x & ~31);
  if (i0 >= pieces) return;
  const int lane = threadIdx.x & 31, r = static_cast<int>(blockIdx.y) * kTokenParts;
  const int64_t i = i0 + lane < pieces ? i0 + lane : i0 + lane % 4;  // past the end the same four again
  const int64_t rows = gridDim.y * kTokenParts;
  few::split8(load_after(reinterpret_cast<const uint4*>(x + blockIdx.y * K) + i),
              [&](int part) { return few::code_at(t, rows, i * 8, r + part); },
              [&](int part) { return few::scale_at(t, rows, i * 8, r + part); });
}

// A stage of the ring, as each role walks through it: which, and the parity of its next completion.
struct Ring {
  int depth, s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int n) : depth(n) {}
  __device__ __forceinline__ void next() {
    if (++s == depth) s = 0, phase ^= 1;
  }
};

// A run of a block: rows of tile `block` of the matrix of slot `at`, chunks c .. c + n.
struct Run {
  FewSlot slot;
  int at, block, c, n;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_remote(float* mine, int rank, float v) {  // to the same place of another block
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x2(uint32_t taddr, uint32_t (&r)[2]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
}

// kUp: element `lane` of a block of 32 of the activation, of column `column` of the run's slot.
__device__ void activate(const Product& p, const Run& r, int column, int i, float gate, float up) {
  const int64_t F = p.m.rows / 2, f = static_cast<int64_t>(r.block) * (kRows / 2) + i * 32;
  if (f >= F) return;
  // gate * sigmoid(gate): far below 0 that is gate * exp(gate), which lasts where 1 + exp(-gate) is over fp32, below -88.7.
  const bool far = gate < -80.f;
  const float e = expf(far ? gate : -gate), silu = far ? gate * e : gate / (1.f + e);
  few::split1(silu * up, p.act + few_act_at(r.at, r.slot.start, few_chunks(F)), r.slot.n,
              f + (threadIdx.x & 31), column);
}

// Waits of the roles: for as long as the call says, 0 not at all (a self-test).
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, AbortFlag ab, const Product& p) {
  if (mbar_test_wait(bar, parity)) return true;
  if (p.wait_ns != 0) return mbar_wait(bar, parity, ab, p.status, p.wait_ns);
  *ab.flag = 1;
  atomicExch(p.status, kStatusTimeout);
  return false;
}

// After a wait of any role has expired, and all roles have come to their ends: copies that are under way land before the block
// ends, whose shared memory is another's then.  A barrier tells that a stage's copies have landed only once all have arrived at
// it, so those that had not come so far arrive for the others' last chunks, without copies of their own.  None is more than
// `depth` chunks ahead of another: it waited for a stage to be read, which takes all.  Bytes of a copy that has been asked for
// land in microseconds, and the limit is for those that never will.
__device__ void land_copies(Shared& sh, int warp, int lane, int depth, bool packed, bool held, int* status) {
  constexpr uint64_t kLimitNs = 10000000;
  const int me = warp - kDrainWarps;
  if (me < 0 || me > kScaleWarps + 1 || (me > kScaleWarps && held)) return;
  int most = 0;
  for (int i = 0; i < kScaleWarps + 2; ++i)
    if (!(i == kScaleWarps && packed) && !(i > kScaleWarps && held)) most = max(most, sh.issued[i]);
  uint64_t* bars = sh.full;
  if (me == kScaleWarps && packed) {
    bars = sh.landed, most = sh.issued[me];
  } else if (me < kScaleWarps || lane == 0) {
    for (int c = sh.issued[me]; c < most; ++c) mbar_arrive(&bars[c % depth]);
  }
  int none = 0;
  for (int c = max(0, most - depth); c < most; ++c) mbar_wait(&bars[c % depth], c / depth & 1, AbortFlag{&none}, status, kLimitNs);
}

template <Mode kMode, int kBits>
__global__ void __launch_bounds__(kThreads, 2)
    few_kernel(const __grid_constant__ CUtensorMap weights_map, const __grid_constant__ Product p) {
  constexpr int kParts = kMode == kDown ? kActParts : kTokenParts;
  constexpr int kRowBytes = 16 * kBits;  // of a chunk in memory
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool packed = kBits == 4 && p.packed, held = kMode == kLinear && p.x != nullptr, in_turn = kMode == kUp && p.tiles > 0;
  if (warp == kWeights && lane == 0) {
    tma_prefetch_desc(&weights_map);
    for (int s = 0; s < kMostDepth; ++s) {
      if (packed) mbar_init(&sh.landed[s], 1);
      mbar_init(&sh.full[s], kScaleWarps * 32 + !packed + !held);
      mbar_init(&sh.ready[s], 1);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.sum_full[b], 1);
      mbar_init(&sh.sum_empty[b], kDrainWarps);
    }
    mbar_init(&sh.drain[0], 1);
    mbar_init(&sh.drain[1], 1);
    mbar_init(&sh.tokens, kDrainWarps);
    sh.abort = 0;
    fence_mbar_init();
  }
  uint8_t* const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const uint32_t stage0 = smem_u32(smem);
  const int rank = blockIdx.x % p.splits;
  const int K = p.m.K, chunks = (K + kChunk - 1) / kChunk;
  // Sums [M][128]: over the stages, once those have been read; where there are more runs, behind them.  Then slots, and what the
  // cluster's other blocks send (or over the stages too, where two blocks an SM need the room, once all of the cluster's blocks
  // have read theirs).  A linear's tokens last.
  const bool many = kMode == kDown || in_turn;
  float* const sums = reinterpret_cast<float*>(many ? smem + p.ring : smem);
  float* const behind = reinterpret_cast<float*>(smem + p.ring) + (many ? p.M * kRows : 0);
  FewSlot* const table = reinterpret_cast<FewSlot*>(behind);
  float* const received = p.late ? reinterpret_cast<float*>(smem) + (many ? 0 : p.M * kRows) : behind + p.slots * 4;

  // What the plan says.  The plan is older than the kernel before this one, which waited for it before it let this one
  // start, so kDown reads it, and starts on the weights, while that kernel still runs.
  int slots = 1;
  Stages stages = p.stages;
  int columns = p.columns, scale_columns = scale_columns_of(1), accs = many ? 2 : 1;  // accumulators, and columns of one
  FewSlot one{0, 0, 0xffffffffu >> (32 - p.M), p.M};
  if constexpr (kMode == kUp) {
    grid_wait();
    grid_release();
    slots = few_header(p.plan).active;
    if (!in_turn) {
      one = few_slot(p.plan, p.choices, blockIdx.y);
      if (static_cast<int>(blockIdx.y) >= slots) return;  // with its whole cluster
    } else if (static_cast<int>(blockIdx.x) >= slots * p.tiles) {
      return;
    }
  } else if constexpr (kMode == kDown) {
    // Stages have room for the tokens that slots have, not for all of the batch's: 32 tokens of 8 experts, two each, take 4 or 5
    // stages of the room of 3.
    const FewPlan plan = few_header(p.plan);
    slots = plan.active;
    columns = (plan.most * kParts + 15) / 16 * 16;
    scale_columns = scale_columns_of(columns);
    stages = stages_of(kMostDepth, p.ring, columns * 128 + static_cast<uint32_t>(few_scale_bytes(columns)), packed);
    // Two accumulators, so that one is drained while the next run's products go to the other, where half of tensor memory, a
    // block's share, has room for them: up to 19 to 22 tokens of an expert.
    accs = 2 * columns + tmem_scales(scale_columns, stages.depth) <= static_cast<int>(p.tmem) ? 2 : 1;
  }
  const AbortFlag ab{&sh.abort};

  // The runs.  t0 .. t1: the block's chunks of all matrices' one behind the other; in turn: runs.
  // (A cluster has no more blocks than a matrix has chunks; of kDown's, which go by the most slots, some may have none.)
  const uint32_t all = (kMode == kDown ? slots : 1) * chunks;
  const int t0 = in_turn ? blockIdx.x : static_cast<int>(all * rank / p.splits);
  const int t1 = in_turn ? slots * p.tiles : static_cast<int>(all * (rank + 1) / p.splits);
  const auto run_at = [&](int t, bool from_plan) {
    Run r;
    if (in_turn) {
      r.at = t / p.tiles, r.block = t - r.at * p.tiles, r.c = 0, r.n = chunks;
    } else {
      r.at = kMode == kDown && slots > 1 ? t / chunks : 0;
      r.block = blockIdx.x / p.splits, r.c = t - r.at * chunks, r.n = min(chunks - r.c, t1 - t);
    }
    r.slot = !many ? one : from_plan ? few_slot(p.plan, p.choices, r.at) : table[r.at];
    return r;
  };
  const auto after = [&](int t, const Run& r) { return t + (in_turn ? static_cast<int>(gridDim.x) : r.n); };
  // A block's first row in a matrix (kUp: of each half), and its last valid row.
  const int tile = kMode == kUp ? kRows / 2 : kRows;
  const int64_t half = kMode == kUp ? p.m.rows / 2 : 0;  // from a row of gate to its row of up
  const auto row_of = [&](const Run& r) { return static_cast<int64_t>(r.block) * tile; };
  const auto last_of = [&](const Run& r) {
    return static_cast<int>(min((kMode == kUp ? half : p.m.rows) - row_of(r), static_cast<int64_t>(tile))) - 1;
  };
  const uint32_t tokens_at = kCodes, scales_at = kCodes + stages.tokens, packed_at = scales_at + kScales;
  // Rows of the tokens of a slot: kDown has those of its columns, the others every token's for every expert.
  const auto rows_of = [&](const FewSlot& s) { return (kMode == kDown ? s.n : p.M) * kParts; };
  const uint32_t held_codes = stage0 + p.ring + p.held_at, held_scales = held_codes + p.share * kHeld;
  const auto come_together = [&]() {
    __syncthreads();
    if (p.splits > 1 && !p.late) cluster_arrive();  // the others may write to this block's memory once it runs
  };

  if (warp >= kDrainWarps && warp < kWeights) {
    // ------------------------------------------------------------ scales of the weights
    come_together();
    if (held) grid_wait();
    // Of a chunk a thread copies the four bytes of row tid.
    const int tid = threadIdx.x - kDrainWarps * 32;
    const uint32_t scale_pitch = K / 32;
    const bool whole_words = K % kChunk == 0;  // a row's scale bytes are whole words
    const uint32_t scale_to = scales_at + (tid & 31) * 16 + (tid >> 5) * 4;
    // Spreads the packed codes: pieces of 16 bytes, tid % 4 of rows tid / 4 + 32 j, to twice 8 bytes each.
    const uint32_t spread_from = packed_at + tid * 16;
    const uint32_t spread_to = (tid >> 2) * 128 + (((tid & 3) * 2 ^ (tid >> 2 & 7)) << 4);

    // Where no word holds a row's four bytes: they come through registers, two chunks ahead.
    const auto scale_word = [&](int64_t s) {
      const int64_t word = s & ~int64_t{3};
      const uint32_t* at = reinterpret_cast<const uint32_t*>(p.m.e8 + word);
      uint32_t lo = 0, hi = 0;
      if (word + 8 <= p.m.scale_end) {
        lo = load_after(at), hi = load_after(at + 1);
      } else {  // the array's last bytes, one by one
#pragma unroll 1
        for (int i = 0; i < 8 && word + i < p.m.scale_end; ++i)
          (i < 4 ? lo : hi) |= static_cast<uint32_t>(p.m.e8[word + i]) << (i & 3) * 8;
      }
      return make_uint2(lo, hi);
    };

    Ring ring(stages.depth);
    bool refill = false, alive = true;
    int issued = 0;
#pragma unroll 1
    for (int t = t0; t < t1 && alive;) {
      const Run r = run_at(t, false);
      t = after(t, r);
      const int last = last_of(r);
      const int64_t row = row_of(r) + (kMode == kUp ? min(tid & 63, last) + (tid >= 64 ? half : 0) : min(tid, last));
      int64_t scale = (r.slot.expert * p.m.rows + row) * scale_pitch + r.c * 4;
      const uint32_t shift = (static_cast<uint32_t>(scale) & 3) * 8;
      uint2 words[2] = {};
      if (!whole_words) {
        words[0] = scale_word(scale);
        if (r.n > 1) words[1] = scale_word(scale + 4);
      }
#pragma unroll 1
      for (int i = 0; i < r.n; ++i) {
        if (refill && !all_of(wait_for(&sh.empty[ring.s], ring.phase ^ 1, ab, p))) {
          alive = false;
          break;
        }
        const uint32_t stage = stage0 + ring.s * stages.bytes;
        if (whole_words && !packed) {
          cp_async4(stage + scale_to, p.m.e8 + scale);
          cp_async_arrive(&sh.full[ring.s]);
        } else {
          uint32_t word;
          if (whole_words) {
            word = load_after(reinterpret_cast<const uint32_t*>(p.m.e8 + scale));
          } else {
            word = __funnelshift_r(words[0].x, words[0].y, shift);
            words[0] = words[1];
            if (i + 2 < r.n) words[1] = scale_word(scale + 8);
          }
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + scale_to), "r"(word) : "memory");
          if (packed) {
            if (!all_of(wait_for(&sh.landed[ring.s], ring.phase, ab, p))) {
              alive = false;
              break;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t v[4];
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                           : "r"(stage + spread_from + j * 2048));
              const uint32_t at = stage + spread_to + j * 4096;
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(v[0]), "r"(v[1]) : "memory");
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at ^ 16), "r"(v[2]), "r"(v[3]) : "memory");
            }
          }
          mbar_arrive(&sh.full[ring.s]);
        }
        scale += 4;
        ++issued;
        ring.next();
        refill |= ring.s == 0;
      }
    }
    cp_async_wait_all();
    if (lane == 0) sh.issued[warp - kDrainWarps] = issued;
    // The next call's first kernel may start: it waits for the end of this one before it reads or writes anything.  One token of
    // 8192 x 5120 9.6 -> 9.1 us; a linear behind a kernel of its own for the tokens gains nothing, 32 tokens 12.5 -> 13.3.
    if (kMode == kDown || held) grid_release();
  } else if (warp == kWeights) {
    // ------------------------------------------------------------ weights
    Ring ring(stages.depth);
    int t = t0, issued = 0;
    Run r{};
    int32_t row = 0;
    const auto begin_run = [&](bool from_plan) {
      r = run_at(t, from_plan);
      t = after(t, r);
      row = static_cast<int32_t>(r.slot.expert * p.m.rows + row_of(r));
    };
    const auto load = [&]() {
      const uint32_t stage = stage0 + ring.s * stages.bytes;
      uint64_t* bar = packed ? &sh.landed[ring.s] : &sh.full[ring.s];
      // Codes that TMA spreads out count as they are in memory.
      mbar_arrive_expect_tx(bar, kRows * kRowBytes);
      const uint32_t to = packed ? stage + packed_at : stage, second = to + (packed ? kPacked / 2 : kCodes / 2);
      const int x = r.c * (packed ? kChunk / 2 : kChunk);
      tile_load(to, &weights_map, x, row, bar);
      if (kMode == kUp) tile_load(second, &weights_map, x, row + static_cast<int32_t>(half), bar);
      ring.next();
      ++r.c, --r.n, ++issued;
    };
    // The first chunks before the others of the block have come together.
    if (lane == 0 && t < t1) {
      if (held) grid_wait();
      fence_proxy_async_global();  // codes that a kernel wrote may be read at once
      begin_run(true);
      while (r.n > 0 && issued < stages.depth) load();
    }
    __syncwarp();
    come_together();
    if (lane == 0) {
#pragma unroll 1
      while (r.n > 0 || t < t1) {
        if (r.n == 0) begin_run(false);
        if (issued >= stages.depth && !wait_for(&sh.empty[ring.s], ring.phase ^ 1, ab, p)) break;
        load();
      }
      sh.issued[kScaleWarps] = issued;
    }
    __syncwarp();
  } else if (warp == kTokens) {
    // ------------------------------------------------------------ tokens
    come_together();
    if (lane == 0 && !held) {
      if (kMode != kUp) grid_wait();
      fence_proxy_async_global();  // the kernel before wrote what the bulk copies read
      Ring ring(stages.depth);
      bool alive = true;
      int issued = 0;
#pragma unroll 1
      for (int t = t0; t < t1 && alive;) {
        const Run r = run_at(t, false);
        t = after(t, r);
        const uint32_t record = static_cast<uint32_t>(few_record(rows_of(r.slot)));
        const uint8_t* from =
            p.t + (kMode == kDown ? few_act_at(r.at, r.slot.start, chunks) : 0) + static_cast<int64_t>(r.c) * record;
#pragma unroll 1
        for (int i = 0; i < r.n; ++i, ++issued) {
          if (issued >= stages.depth && !wait_for(&sh.empty[ring.s], ring.phase ^ 1, ab, p)) {
            alive = false;
            break;
          }
          mbar_arrive_expect_tx(&sh.full[ring.s], record);
          bulk_load(stage0 + ring.s * stages.bytes + tokens_at, from, record, &sh.full[ring.s]);
          from += record;
          ring.next();
        }
      }
      sh.issued[kScaleWarps + 1] = issued;
    }
    __syncwarp();
  } else if (warp == kScaler) {
    // ------------------------------------------------------------ scales
    come_together();
    // cp.async wrote what the tensor core reads: the fence between the two, and the copies, stay off the thread that issues
    // the products (together 250 to 800 cycles a chunk).
    named_sync<1, (kDrainWarps + 2) * 32>();
    tc_fence_after();
    const uint32_t sf0 = __shfl_sync(kAll, sh.tmem, 0) + accs * columns;
    const uint64_t sa0 = sdesc_plain_128b_rows(stage0 + scales_at);
    const uint64_t sb0 = sdesc_plain_128b_rows(held ? held_scales : stage0 + tokens_at);
    const bool elected = elect_one();
    Ring ring(stages.depth);
    bool alive = !held || all_of(wait_for(&sh.tokens, 0, ab, p));
#pragma unroll 1
    for (int t = t0; t < t1 && alive;) {
      const Run r = run_at(t, false);
      t = after(t, r);
      const uint64_t token_scales = sb0 + (held ? 0 : rows_of(r.slot) * (128 >> 4));
      const bool two_blocks = rows_of(r.slot) > 128;
#pragma unroll 1
      for (int i = 0; i < r.n; ++i) {
        if (!all_of(wait_for(&sh.full[ring.s], ring.phase, ab, p))) {
          alive = false;
          break;
        }
        fence_proxy_async_smem();
        tc_fence_after();
        const uint64_t stage = static_cast<uint64_t>(ring.s * (stages.bytes >> 4));
        if (elected) {
          // The columns were last read by products that were complete before the stage was filled again.
          const uint32_t sf = sf0 + ring.s * scale_columns;
          const uint64_t sb = token_scales + (held ? static_cast<uint64_t>(i * (kScales >> 4)) : stage);
          tmem_cp_32x128b_warpx4(sf, sa0 + stage);
          tmem_cp_32x128b_warpx4(sf + 4, sb);
          if (kMode == kDown && two_blocks) tmem_cp_32x128b_warpx4(sf + 8, sb + (512 >> 4));
          mma_commit(&sh.ready[ring.s]);
        }
        __syncwarp();
        ring.next();
      }
    }
    if (elected) {  // nothing may be under way when tensor memory is given back
      mma_commit(&sh.drain[0]);
      int none = 0;
      mbar_wait(&sh.drain[0], 0, AbortFlag{&none}, p.status, 1000000ull);
    }
    __syncwarp();
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ products
    come_together();
    tmem_alloc(&sh.tmem, p.tmem);
    tmem_relinquish();
    tc_fence_before();
    named_sync<1, (kDrainWarps + 2) * 32>();
    tc_fence_after();
    // All lanes walk through the loop, so that what the products take stays in uniform registers; one issues them.
    const uint32_t tmem = __shfl_sync(kAll, sh.tmem, 0), sf0 = tmem + accs * columns;
    const uint64_t a0 = sdesc_kmajor_sw128(stage0), b0 = sdesc_kmajor_sw128(held ? held_codes : stage0 + tokens_at);
    const bool elected = elect_one();
    bool alive = true;
    Ring ring(stages.depth);
    Ring sum(accs);
    bool again = false;  // whether the accumulator has been used before
#pragma unroll 1
    for (int t = t0; t < t1 && alive;) {
      const Run r = run_at(t, false);
      t = after(t, r);
      const uint32_t acc = tmem + sum.s * columns;
      if (many && again && !all_of(wait_for(&sh.sum_empty[sum.s], sum.phase ^ 1, ab, p))) break;
      const uint32_t N = (__shfl_sync(kAll, rows_of(r.slot), 0) + 15) & ~15;
      const uint32_t kind = idesc_mx_e4m3(kRows, N, 0, 0) | (kBits == 4 ? 5u << 7 : 0u);  // A: e2m1
      int left = K / 32 - r.c * 4;  // blocks of 32
      uint32_t more = 0;            // whether there is something in the accumulator
#pragma unroll 1
      for (int i = 0; i < r.n; ++i, left -= 4) {
        if (!all_of(wait_for(&sh.ready[ring.s], ring.phase, ab, p))) {
          alive = false;
          break;
        }
        tc_fence_after();
        const uint64_t stage = static_cast<uint64_t>(ring.s * (stages.bytes >> 4));
        const uint32_t sfa = sf0 + ring.s * scale_columns, sfb = sfa + 4;
        const uint64_t a = a0 + stage, b = b0 + (held ? static_cast<uint64_t>(i * (kHeld >> 4)) : stage);
        if (elected) {
          mma_mx_e4m3(acc, a, b, kind, sfa, sfb, more);
          if (left > 1) mma_mx_e4m3_k<true>(acc, a + 2, b + 2, kind | idesc_mx_e4m3(0, 0, 1, 1), sfa, sfb);
          if (left > 2) mma_mx_e4m3_k<true>(acc, a + 4, b + 4, kind | idesc_mx_e4m3(0, 0, 2, 2), sfa, sfb);
          if (left > 3) mma_mx_e4m3_k<true>(acc, a + 6, b + 6, kind | idesc_mx_e4m3(0, 0, 3, 3), sfa, sfb);
          mma_commit(&sh.empty[ring.s]);
        }
        __syncwarp();
        more = 1;
        ring.next();
      }
      if (elected) mma_commit(&sh.sum_full[sum.s]);
      __syncwarp();
      sum.next();
      again |= sum.s == 0;
    }
    if (elected) {
      mma_commit(&sh.drain[1]);
      int none = 0;
      mbar_wait(&sh.drain[1], 0, AbortFlag{&none}, p.status, 1000000ull);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ sums
    if (many)
      for (int i = threadIdx.x; i < slots; i += kDrainWarps * 32) table[i] = few_slot(p.plan, p.choices, i);
    if (kMode == kDown)
      for (int i = threadIdx.x; i < p.M * kRows; i += kDrainWarps * 32) sums[i] = 0.f;
    come_together();
    if (held) {
      // One or two tokens: the block's share of them stays in shared memory, in tiles of 16 rows.
      grid_wait();
      const int pieces = (min(t1 * kChunk, K) - t0 * kChunk) / 8, work = pieces * p.M;  // of 8 values
#pragma unroll 1
      for (int i0 = warp * 32; i0 < work; i0 += kDrainWarps * 32) {
        const int i = i0 + lane < work ? i0 + lane : i0 + lane % 4;  // past the end the same four again
        const int token = i >= pieces, k = (i - token * pieces) * 8, r = token * kTokenParts, b = k & 127;
        uint8_t* codes = smem + (held_codes - stage0) + (k >> 7) * kHeld;
        uint8_t* scales = smem + (held_scales - stage0) + (k >> 7) * kScales;
        few::split8(
            load_after(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(token) * K + t0 * kChunk + k)),
            [&](int part) { return codes + (r + part) * 128 + (((b >> 4) ^ (r + part)) << 4) + (b & 15); },
            [&](int part) { return scales + (r + part) * 16 + (b >> 5); });
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tokens);
    }
    named_sync<1, (kDrainWarps + 2) * 32>();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const int row = threadIdx.x;  // warps 0-3
    const float* weights = kMode == kDown ? few_weights(p.plan) : nullptr;
    Ring sum(accs);
#pragma unroll 1
    for (int t = t0; t < t1; sum.next()) {
      const Run r = run_at(t, false);
      t = after(t, r);
      const FewSlot& s = r.slot;
      // Lane i has the weight of column i.
      const float weight =
          kMode == kDown && lane < s.n ? __uint_as_float(load_after(reinterpret_cast<const uint32_t*>(weights + s.start + lane))) : 0.f;
      bool landed = all_of(wait_for(&sh.sum_full[sum.s], sum.phase, ab, p));
      // Together: the sums of the run before have been read, and a warp that gave up would leave the others at a barrier.
      if (in_turn) landed = named_all<2, kDrainWarps * 32>(landed);
      if (!landed) break;
      tc_fence_after();
      const uint32_t acc = tmem + sum.s * columns + (static_cast<uint32_t>(warp * 32) << 16);
      uint32_t mask = s.mask;
      if constexpr (kMode == kDown) {
#pragma unroll 1
        for (int n0 = 0; n0 < s.n; n0 += 6) {  // twice three tokens' parts at a time, and a column that is not read
          uint32_t v[2][16];
          static_assert(3 * kActParts <= 16, "of a load");
          tmem_ld_32x32b_x16(acc + n0 * kParts, v[0]);
          if (n0 + 3 < s.n) tmem_ld_32x32b_x16(acc + (n0 + 3) * kParts, v[1]);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            if (n0 + i >= s.n) break;
            float f = 0.f;
#pragma unroll
            for (int q = kParts - 1; q >= 0; --q) f += __uint_as_float(v[i / 3][i % 3 * kParts + q]);
            sums[(__ffs(mask) - 1) * kRows + row] += f * __shfl_sync(kAll, weight, n0 + i);
            mask &= mask - 1;
          }
        }
      } else {
        // The tokens of the mask, four at a time (past the last one that one again).
#pragma unroll 1
        for (int n0 = 0; n0 < s.n; n0 += 4) {
          uint32_t v[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            tmem_ld_32x32b_x2(acc + (__ffs(mask) - 1) * kParts, v[i]);
            if (n0 + i + 1 < s.n) mask &= mask - 1;
          }
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n0 + i < s.n) sums[(n0 + i) * kRows + row] = __uint_as_float(v[i][0]) + __uint_as_float(v[i][1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sum_empty[sum.s]);
      if (in_turn) {
        named_sync<2, kDrainWarps * 32>();
        for (int i = warp; i < s.n * 2; i += kDrainWarps)
          activate(p, r, i >> 1, i & 1, sums[(i >> 1) * kRows + (i & 1) * 32 + lane],
                   sums[(i >> 1) * kRows + 64 + (i & 1) * 32 + lane]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*ab.flag) {  // raised by a wait, of which there are no more
    land_copies(sh, warp, lane, stages.depth, packed, held, p.status);
    __syncthreads();
  }
  if (warp == kIssuer) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, p.tmem);
  }
  if (in_turn) return;

  // The sums of the cluster's blocks.  Block r of them brings home items r, r + splits, ...: for each the others send theirs,
  // item i of block q to received[i / splits * splits + q].  An item: 32 rows of a token (kUp: of gate and of up).
  constexpr int kHalves = kMode == kUp ? 2 : 1, kItems = kRows / 32 / kHalves;  // of an item, of a token
  const int items = (kMode == kUp ? one.n : p.M) * kItems;
  const auto value_of = [&](int item, int h) {  // row `lane` of its half h
    return sums[item / kItems * kRows + item % kItems * 32 + h * 64 + lane];
  };
  if (p.splits > 1) {
    if (p.late) cluster_arrive();
    cluster_wait();
    for (int item = warp; item < items; item += kIssuer + 1) {
      const int home = item % p.splits;
      if (home == rank) continue;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        store_remote(received + ((item / p.splits * p.splits + rank) * kHalves + h) * 32 + lane, home, value_of(item, h));
    }
    cluster_arrive();
    cluster_wait();
  }
  Run r{one, static_cast<int>(blockIdx.y), static_cast<int>(blockIdx.x) / p.splits, 0, 0};
  for (int item = rank + warp * p.splits; item < items; item += (kIssuer + 1) * p.splits) {
    float v[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      v[h] = p.splits == 1 ? value_of(item, h) : 0.f;
      if (p.splits > 1)
        for (int q = 0; q < p.splits; ++q)
          v[h] += q == rank ? value_of(item, h) : received[((item / p.splits * p.splits + q) * kHalves + h) * 32 + lane];
    }
    const int token = item / kItems, row = item % kItems * 32 + lane;
    if constexpr (kMode == kUp) {
      activate(p, r, token, item % kItems, v[0], v[1]);
    } else {
      if (row <= last_of(r)) p.y[token * p.m.rows + row_of(r) + row] = static_cast<uint16_t>(pack_bf16x2(v[0], 0.f) & 0xFFFFu);
    }
  }
}

// ---------------------------------------------------------------- launches

// Shared memory of a block beside its fixed part, as one of two on an SM, which has 228 KB; each block takes 1 KB more than it
// asks for.
constexpr uint32_t kHalfSmem = 111 * 1024;
static_assert(sizeof(Shared) <= 1024, "of the kilobyte that this leaves");

// Blocks of clusters of `size` that run at once, two to an SM: shared memory decides.  Clusters stay within a part of the chip,
// whose SMs do not always come out even: of 304 places, 296 in clusters of four, 276 of six and 288 of eight.  The query goes by a
// kernel without tensor memory; of one that takes some it counts a block an SM, where two do run.
int places(int size) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = kHalfSmem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaFuncSetAttribute(few_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kHalfSmem)) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&clusters, few_tokens_kernel, &cfg) == cudaSuccess && clusters > 0)
    return clusters * size;
  (void)cudaGetLastError();
  return size;
}

// Blocks of a cluster, up to eight, for `tiles` row tiles over `chunks` chunks of contraction.  The cost in chunks' time of a
// block (0.185 us):
//   a block's own chunks, for each round of blocks, 1.3 times as long where it brings its tokens into parts itself or where rows
//   are not whole chunks; or what memory takes for all blocks' chunks, 118 (4 bits) or 60 (8) in that time for 128 blocks, 124 or
//   69 for 256; whichever is more, and some of the other;
//   the cluster's meeting and exchange (three blocks do not divide the parts of the chip), more for more than 16 tokens, whose
//   sums meet where the stages were, once all blocks have read theirs;
//   and blocks that share SMs.
// The numbers are fitted to 64 linears (1 to 32 tokens, 2048 x 2048 to 8192 x 16384) and six products of layers, each with every
// size of cluster.  Of those same products, none of others, the choice takes 0.6 % longer than the best on average, 17 % at most:
// that is where one block a tile gives under 128 blocks, to which the rates are only drawn out (8192 x 5120, 8 bits, 32 tokens:
// 18.2 us with one block a tile, as chosen, 16.7 with two, 16.2 with four).  By blocks of a cluster, us:
//   linear, 4 bits,  4 tokens, 2048 x 2048     1: 6.7    2: 6.8    4: 5.9 *  8: 7.5
//                              8192 x 5120     1: 11.2   2: 9.1 *  4: 10.2   8: 15.5 (more blocks than places)
//                              8192 x 16384    1: 31.7   2: 21.5   4: 20.1 * 8: 25.4
//                              1024 x 8192     1: 15.5   2: 11.4   4: 8.6    8: 7.5 *
//                   32 tokens, 4096 x 4096     1: 12.7   2: 11.8   4: 9.9 *  8: 12.7
//   up of two experts 5120 -> 4096, 4 bits     1: 28.0 * 2: 31.0   4: 35.9 (the whole layer, here and below)
//   down of 8 experts 4096 -> 5120, 8 bits     4: 103.2  5: 100.4  6: 99.2 * 8: 112.5
int splits_of(int64_t tiles, int64_t chunks, int bits, int tokens, bool slow, int num_sms, const int (&room)[8]) {
  const double exchange[8] = {0., 5.4, 11.8, 6.2, 6.9, 7.8, 9.3, 9.5};
  const double rates[2] = {bits == 4 ? 118. : 60., bits == 4 ? 124. : 69.};  // with 128 blocks, with 256
  int best = 1;
  double least = INFINITY;
  for (int s = 1; s <= 8 && s <= chunks; ++s) {
    const double blocks = static_cast<double>(tiles) * s, rounds = std::ceil(blocks / room[s - 1]);
    const double own = rounds * static_cast<double>((chunks + s - 1) / s) * (slow ? 1.3 : 1.);
    const double all = static_cast<double>(tiles) * chunks / (rates[0] + (rates[1] - rates[0]) * (std::min(blocks, 256.) - 128.) / 128.);
    const double cost = std::max(own, all) + 0.15 * std::min(own, all) + exchange[s - 1] + (s > 1 && tokens > 16 ? 7.3 : 0.) +
                        (blocks > num_sms ? 7.2 : 0.);
    if (cost < least) best = s, least = cost;
  }
  return best;
}

// The weights as TMA reads them, boxes of `box` rows by a chunk: e4m3 codes as bytes; e2m1 codes spread out, or, where rows are
// not whole chunks of 128 or not aligned to 32 bytes, which that takes, as bytes.
bool weights_map(CUtensorMap* map, const Matrix& m, int64_t rows, int bits, bool packed, uint32_t box) {
  typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const auto fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!fn) return false;
  const int64_t bytes = m.K / 8 * bits;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(packed ? bytes : m.K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(bytes)};
  const cuuint32_t boxes[2] = {packed ? kChunk / 2u : kChunk, box}, each[2] = {1, 1};
  return fn(map, bits == 8 || packed ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2,
            const_cast<uint8_t*>(m.w), dims, strides, boxes, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
            packed ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <Mode kMode, int kBits>
cudaError_t launch(const CUtensorMap& map, const Product& p, uint32_t smem, dim3 grid, cudaStream_t st) {
  auto* kernel = few_kernel<kMode, kBits>;
  static thread_local bool allowed[64] = {};  // by device
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev >= 64 || !allowed[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kHalfSmem));
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = true;
  }
  cudaLaunchAttribute attrs[2]{};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attrs;
  // The kernel starts under the one before and waits for it itself.
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (p.splits > 1) {
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = p.splits;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, map, p);
}

// How a product is divided: p's sizes, the grid and the shared memory of a block.  matrices: how many lie behind each other along
// the contraction (kDown), copies: how many share the grid (kUp).
template <Mode kMode, int kBits>
cudaError_t divide(Product& p, int matrices, int copies, int num_sms, dim3* grid, uint32_t* smem) {
  const int parts = kMode == kDown ? kActParts : kTokenParts;
  const int64_t rows = kMode == kUp ? p.m.rows / 2 : p.m.rows, tile = kMode == kUp ? kRows / 2 : kRows;
  const int64_t tiles = (rows + tile - 1) / tile;
  const int chunks = (p.m.K + kChunk - 1) / kChunk;
  p.columns = (p.M * parts + 15) / 16 * 16;
  p.packed = kBits == 4 && (p.m.K % kChunk != 0 || (reinterpret_cast<uintptr_t>(p.m.w) & 31) != 0);
  const uint32_t tokens = p.x != nullptr ? 0 : p.columns * 128 + static_cast<uint32_t>(few_scale_bytes(p.columns));
  const uint32_t stage = stages_of(0, 0, tokens, p.packed).bytes;
  // Enough runs for every block to have some: whole ones in turn, which leaves the stages no gaps (17 tokens over 64 experts 46.8
  // us, otherwise 50.5), where their sums leave room for two blocks of three stages an SM.
  const uint32_t sums = p.M * kRows * 4, slot = sizeof(FewSlot);
  const bool in_turn = kMode == kUp && tiles * copies >= 3 * num_sms && 1024 + 3 * stage + sums + copies * slot <= kHalfSmem;
  const bool many = kMode == kDown || in_turn;
  p.tiles = in_turn ? static_cast<int>(tiles) : 0;
  // Room to receive: whole rounds of items, a round a share of every block, which is under 7 items more than there are.
  const uint32_t received = (p.M * kRows + 7 * 64) * 4;
  p.late = p.M > 16;
  p.slots = many ? (kMode == kDown ? matrices : copies) : 0;
  const uint32_t behind = (p.late || in_turn ? 0 : received) +
                          (many ? sums + p.slots * slot : 0);
  if (in_turn) {
    p.splits = 1;
  } else {
    static thread_local int room[64][8] = {};  // by device
    int dev = 0, here[8] = {};
    if (const cudaError_t e = cudaGetDevice(&dev)) return e;
    int(&mine)[8] = dev < 64 ? room[dev] : here;
    if (mine[0] == 0)
      for (int i = 7; i >= 0; --i) mine[i] = places(i + 1);
    p.splits = splits_of(tiles * copies, static_cast<int64_t>(chunks) * matrices, kBits, p.M, p.x != nullptr || p.m.K % kChunk != 0,
                         num_sms, mine);
  }
  uint32_t beside = 1024 + behind;
  if (p.x != nullptr) {
    while (p.splits * kMostHeld < chunks) ++p.splits;  // at most eight, as held_tokens has it
    p.share = (chunks + p.splits - 1) / p.splits;
    p.held_at = (behind + 1023) / 1024 * 1024;
    beside = 1024 + p.held_at + p.share * (kHeld + kScales);
  }
  // Two blocks an SM, of five stages to three (a block before the next product's, or before the next call's, then has the
  // other's time to start: alone, with eight stages, a token of 8192 x 5120 took 13.9 us, so 9.6).  Five, where there is room,
  // took 28.7 us for a layer's step of one token and 30.9 for a linear of 65536 x 4096, four 29.4 and 31.9.  kDown takes what
  // there is and divides it by the plan.
  const auto fits = [&](int n) { return beside + n * stage <= kHalfSmem; };
  const int depth = kMode == kDown ? 1 : fits(5) ? 5 : fits(4) ? 4 : 3;
  p.ring = kMode == kDown ? (kHalfSmem - beside) / 1024 * 1024 : depth * stage;
  p.stages = Stages{depth, tokens, stage};
  if (beside + p.ring > kHalfSmem || p.ring < depth * stage) return cudaErrorInvalidConfiguration;
  // At most half of tensor memory, which two blocks an SM share: a block that had to wait for another's, which may wait for
  // this one's kernel to end, would wait for ever.
  const int columns = kMode == kDown ? 2 * p.columns + tmem_scales(scale_columns_of(p.columns), kMostDepth)
                                     : (many ? 2 : 1) * p.columns + tmem_scales(scale_columns_of(1), depth);
  p.tmem = 32;
  while (p.tmem < columns && p.tmem < 256) p.tmem *= 2;
  *grid = in_turn ? dim3(static_cast<unsigned>(2 * num_sms))
                  : dim3(static_cast<unsigned>(tiles * p.splits), static_cast<unsigned>(copies));
  *smem = beside + p.ring;
  return cudaSuccess;
}

template <Mode kMode, int kBits>
cudaError_t launch_sized(Product p, int64_t experts, int matrices, int copies, int num_sms, cudaStream_t st) {
  dim3 grid;
  uint32_t smem = 0;
  if (const cudaError_t e = divide<kMode, kBits>(p, matrices, copies, num_sms, &grid, &smem)) return e;
  CUtensorMap map{};
  const uint32_t box = kMode == kUp ? kRows / 2 : kRows;
  if (!weights_map(&map, p.m, experts * p.m.rows, kBits, p.packed, box)) return cudaErrorInvalidValue;
  return launch<kMode, kBits>(map, p, smem, grid, st);
}

// Launches a product, or, with a shape to fill, says how it would be divided.
template <Mode kMode>
cudaError_t launch_product(const Product& p, int bits, int64_t experts, int matrices, int copies, int num_sms, cudaStream_t st,
                           FewShape* shape) {
  // A runtime call binds the device's context to a thread that has made none yet; the driver's encoder does not.
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev)) return e;
  if (shape == nullptr)
    return bits == 4 ? launch_sized<kMode, 4>(p, experts, matrices, copies, num_sms, st)
                     : launch_sized<kMode, 8>(p, experts, matrices, copies, num_sms, st);
  Product q = p;
  dim3 grid;
  uint32_t smem = 0;
  if (const cudaError_t e = bits == 4 ? divide<kMode, 4>(q, matrices, copies, num_sms, &grid, &smem)
                                      : divide<kMode, 8>(q, matrices, copies, num_sms, &grid, &smem))
    return e;
  const int chunks = (q.m.K + kChunk - 1) / kChunk * (kMode == kDown ? matrices : 1);
  *shape = FewShape{q.splits, stages_of(kMode == kDown ? kMostDepth : q.stages.depth, q.ring, q.stages.tokens, q.packed).depth,
                    (chunks + q.splits - 1) / q.splits, q.tiles > 0, q.x != nullptr, q.packed};
  return cudaSuccess;
}

}  // namespace

// One or two tokens are brought into parts by the product itself, as long as a block's share of them fits beside the stages and
// no block follows another, with the tokens once more: 9.1 us for one token of 8192 x 5120 in 4 bits, 13.8 with the kernel in
// front; but 44 us for 65536 x 4096, 32 with it.  Eight tokens (8 bits) took 16.9 us so, 14.1 with it.
static bool held_tokens(int64_t M, int64_t N, int64_t K) {
  // Two blocks an SM in clusters of eight on a GB300.  The workspace's size goes by it, which a host without the device may ask
  // for; on another number of SMs the choice would be as right, and slower or faster.
  constexpr int64_t kPlaces = 288;
  const int64_t splits = (K + kMostHeld * kChunk - 1) / (kMostHeld * kChunk);
  return M <= 2 && splits <= 8 && (N + kRows - 1) / kRows * splits <= kPlaces;
}

size_t few_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) { return held_tokens(M, N, K) ? 0 : few_tokens_bytes(M, K); }

cudaError_t launch_few_linear(const FewLinearArgs& a, cudaStream_t st, FewShape* shape) {
  Product p{};
  p.m = Matrix{a.w, a.e8, a.N * (a.K / 32), a.N, static_cast<int>(a.K)};
  p.M = static_cast<int>(a.M);
  p.y = a.y;
  p.status = a.status;
  p.wait_ns = a.wait_ns;
  if (held_tokens(a.M, a.N, a.K)) {
    p.x = a.x;
  } else if (shape == nullptr) {
    uint8_t* tokens = static_cast<uint8_t*>(a.workspace);
    p.t = tokens;
    const dim3 grid(static_cast<unsigned>((a.K / 8 + 255) / 256), static_cast<unsigned>(a.M));
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (const cudaError_t e = cudaLaunchKernelEx(&cfg, few_tokens_kernel, a.x, a.K, tokens)) return e;
  }
  return launch_product<kLinear>(p, a.bits, 1, 1, 1, a.num_sms, st, shape);
}

namespace {

struct MoeScratch {
  FewPlan* plan;
  uint8_t *tokens, *act;
  int64_t bytes;
};
MoeScratch scratch_of(void* p, int64_t M, int64_t E, int64_t k, int64_t C, int64_t F) {
  uint8_t* at = static_cast<uint8_t*>(p);
  const int64_t tokens = few_plan_bytes(M, k), act = tokens + few_tokens_bytes(M, C);
  return MoeScratch{reinterpret_cast<FewPlan*>(at), at + tokens, at + act,
                    act + few_act_bytes(M * k, E < M * k ? E : M * k, F)};
}

}  // namespace

size_t few_moe_workspace_bytes(int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F) {
  return scratch_of(nullptr, M, E, top_k, C, F).bytes;
}

cudaError_t launch_few_moe(const FewMoeArgs& a, cudaStream_t st, FewShape* up_shape, FewShape* down_shape) {
  const int64_t E = a.route.E, M = a.route.M, k = a.route.top_k;
  const int active = static_cast<int>(E < M * k ? E : M * k);  // at most
  const MoeScratch s = scratch_of(a.workspace, M, E, k, a.C, a.F);
  if (up_shape == nullptr)
    if (const cudaError_t e = launch_few_route(a, s.plan, s.tokens, st)) return e;
  Product up{};
  up.m = Matrix{a.w13, a.e13, E * 2 * a.F * (a.C / 32), 2 * a.F, static_cast<int>(a.C)};
  up.M = static_cast<int>(M);
  up.t = s.tokens;
  up.plan = s.plan;
  up.choices = static_cast<int>(M * k);
  up.act = s.act;
  up.status = a.route.status;
  up.wait_ns = a.wait_ns;
  if (const cudaError_t e = launch_product<kUp>(up, a.bits, E, 1, active, a.num_sms, st, up_shape)) return e;
  Product down{};
  down.m = Matrix{a.w2, a.e2, E * a.C * (a.F / 32), a.C, static_cast<int>(a.F)};
  down.M = static_cast<int>(M);
  down.t = s.act;
  down.plan = s.plan;
  down.choices = static_cast<int>(M * k);
  down.y = a.y;
  down.status = a.route.status;
  down.wait_ns = a.wait_ns;
  return launch_product<kDown>(down, a.bits, E, active, 1, a.num_sms, st, down_shape);
}

}  // namespace fp8bw
