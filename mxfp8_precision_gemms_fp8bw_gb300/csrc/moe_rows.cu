// Rows of the experts: gathering tokens into them as MX codes, and summing
// them back into the tokens.
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "mx_tile.cuh"

namespace fp8bw {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

constexpr int kGatherWarps = 8;

// Where a block has its copies: two tiles of x, and of four tiles in turn the
// rows' tokens (-1: none) and weights, because the tokens are needed two
// tiles before the weights are done with; and two tiles of column codes on
// their way out.
template <bool kCol>
struct GatherSmem {
  uint4 x[2][128][16];
  alignas(kCol ? 1024 : 16) uint8_t qT[kCol ? 2 : 1][kCol ? 128 * 128 : 16];
  ScaleTile scales[2];
  int32_t token[4][16][8];  // row r at [r % 16][r / 16]: the eight that a thread copies are contiguous
  float weight[4][128];
};

__device__ __forceinline__ void cp_async_16(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}

// Column codes leave through shared memory by a tensor store of 128 rows x 128
// columns: straight from the lanes they are 32-byte pieces, and the requests
// for those, more than the bytes, were what the two-layout kernel waited for
// (7.1 million write requests for 170 MB, L1 to crossbar 58 % busy).  A
// column's 128 codes are a 128-byte line of shared memory under the 128-byte
// swizzle; lines are ordered by (column % 8, column / 8), which the tensor map
// undoes, so that the eight columns that lanes write together are lines with
// different swizzles and hit different banks.
__device__ __forceinline__ void put_column(uint8_t* cols, int rt, int ct, int j, uint2 codes) {
  const int line = j * 16 + ct / 8;
  *reinterpret_cast<uint2*>(cols + line * 128 + (((rt >> 4) ^ (line & 7)) << 4) + (rt & 8)) = codes;
}
__device__ __forceinline__ void store_columns(const CUtensorMap* map, const uint8_t* cols, int row, int group) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(map),
      "r"(smem_u32(cols)), "r"(row), "r"(group), "r"(0)
      : "memory");
}

// Blocks per SM: the rows alone leave room for three, the column codes on their
// way out for two.
constexpr int gather_ctas_per_sm(bool columns) { return columns ? 2 : 3; }

// MX codes of gathered rows, v_p = w_p * x[src_p / top_k], in both layouts.
//
// Blocks are persistent, two or three to an SM, and walk 128 x 128 tiles whose
// rows of x are on their way (cp.async, one 16-byte chunk at a time, zeros
// where there is no row) while the tile before is converted, and whose tokens
// were looked up one tile earlier still.  A thread takes its 8 x 8 part into
// registers (mx_tile.cuh) and reads nothing twice; 128 x 128 because the codes
// of a tile's rows and of its columns then fill whole 128-byte lines.  Without
// weights the maxima and products are taken on packed bf16 pairs.  With them
// the max of a row block is still the bf16 max, times |w| (rounding is
// monotonic, so the product of the max is the max of the products); a column
// block mixes weights and takes the max of the fp32 products.
//
// 8192 tokens x 2, 5120 columns: 54 us for both layouts (0.70 of the measured
// copy bandwidth, counting x once), 34 us for the rows alone (0.75), 60 us
// weighted.  No unit is full: leaving out the scale bytes, the column store,
// the copies or the row stores saves 4, 8, 8 and 4 us, and what is left, the
// conversion alone, takes 37.  Not persistent, with the loads straight into
// registers, and with the column codes stored by the lanes it took 70, 43 and
// 80; with 4 x 8 values per thread and twice the warps 72, 42 and 80; with a
// 256-byte bulk copy per row in place of the cp.async 67, 39 and 71.
//
// The tiles of one 128-column stripe come one after another: a token is
// gathered up to top_k times, and a stripe of x stays in L2 between them
// (with the columns fastest, 5120 of them and 8192 x 2 entries, x came from
// DRAM 1.9 times).
template <bool kWeighted, bool kCol>
__global__ void __launch_bounds__(kGatherWarps * 32, gather_ctas_per_sm(kCol))
    gather_quant_kernel(const __grid_constant__ CUtensorMap map, const uint16_t* __restrict__ x,
                        const float* __restrict__ weights, const int32_t* __restrict__ src_of, uint32_t entries, uint32_t top_k, int P, int C, int bands,
                        int tiles, uint8_t* __restrict__ q, uint8_t* __restrict__ e8, uint8_t* __restrict__ e8T,
                        int mode, int* status) {
  extern __shared__ uint8_t gather_smem[];
  GatherSmem<kCol>& sm = *reinterpret_cast<GatherSmem<kCol>*>(
      (reinterpret_cast<uintptr_t>(gather_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  const TileLane t = tile_lane();
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t round = mx_round_f32(mode);

  struct Tile {
    int stripe, band;  // band -1: behind the last tile
  };
  auto tile_at = [&](int n) {  // the block's n-th
    const uint32_t i = blockIdx.x + static_cast<uint32_t>(n) * gridDim.x;
    if (i >= static_cast<uint32_t>(tiles)) return Tile{0, -1};
    const uint32_t stripe = i / static_cast<uint32_t>(bands);
    return Tile{static_cast<int>(stripe), static_cast<int>(i - stripe * static_cast<uint32_t>(bands))};
  };
  // The entry of row `tid` of a tile, and its note in the tables of tile n.
  auto look_up = [&](Tile w) {
    const int64_t row = static_cast<int64_t>(w.band) * 128 + tid;
    return tid < 128 && w.band >= 0 && row < P ? static_cast<uint32_t>(src_of[row]) : 0xffffffffu;
  };
  auto note = [&](int n, uint32_t src) {
    if (tid >= 128) return;
    int32_t token = -1;
    float weight = 0.f;
    if (src < entries) {
      token = static_cast<int32_t>(src / top_k);
      if (kWeighted) weight = weights[src];
    } else if (src != 0xffffffffu) {
      atomicExch(status, kStatusShape);
    }
    sm.token[n & 3][tid & 15][tid >> 4] = token;
    if (kWeighted) sm.weight[n & 3][tid] = weight;
  };
  // Starts the copies of tile n: thread i has chunk i % 16 of rows i / 16 + 16 j.
  auto fetch = [&](int n, Tile w) {
    if (w.band >= 0) {
      const int chunk = tid & 15, r0 = tid >> 4;
      const int c = w.stripe * 128 + chunk * 8;
      const uint16_t* xc = x + (c < C ? c : 0);
      const int4 a = *reinterpret_cast<const int4*>(&sm.token[n & 3][r0][0]);
      const int4 b = *reinterpret_cast<const int4*>(&sm.token[n & 3][r0][4]);
      const int32_t token[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool live = token[j] >= 0 && c < C;
        cp_async_16(&sm.x[n & 1][r0 + 16 * j][chunk],
                    xc + static_cast<uint64_t>(live ? token[j] : 0) * static_cast<uint32_t>(C), live);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto finish = [&](int n, Tile w) {  // of tile n, once every thread has written its part
    if (kCol && tid == 0) store_columns(&map, sm.qT[n & 1], w.band * 128, w.stripe * 16);
    put_scales(sm.scales[n & 1].row, tid, static_cast<int64_t>(w.band) * 128, P, e8, w.stripe * 4, C / 32);
    if (kCol)
      put_scales(sm.scales[n & 1].col, tid - 128, static_cast<int64_t>(w.stripe) * 128, C, e8T, w.band * 4, P / 32);
  };

  Tile last{0, -1}, now = tile_at(0), next = tile_at(1);
  note(0, look_up(now));
  note(1, look_up(next));
  __syncthreads();
  fetch(0, now);
  int n = 0;
  for (; now.band >= 0; ++n) {
    // Tile n has landed, the column codes of tile n - 2 have left; everyone has left tile n - 1 and its buffers.
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (kCol && tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncthreads();
    fetch(n + 1, next);
    const Tile after = tile_at(n + 2);
    const uint32_t src = look_up(after);
    if (n > 0) finish(n - 1, last);

    const int rt = (warp >> 1) * 32 + t.rg * 8, ct = (warp & 1) * 64 + t.cg * 8;  // the thread's part of the tile
    const int c0 = now.stripe * 128 + ct;
    const int64_t r0 = static_cast<int64_t>(now.band) * 128 + rt;
    const bool live = r0 < P && c0 < C;  // P and C % 32 == 0: blocks are all in or all out
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sm.x[n & 1][rt + i][ct / 8];
    uint8_t* qrow = q + r0 * C + c0;
    uint8_t* cols = sm.qT[n & 1];

    uint32_t m[4];  // of rows 2 p and 2 p + 1
#pragma unroll
    for (int p = 0; p < 4; ++p) m[p] = block_absmax2<1>(fold2(absmax2_of8(v[2 * p]), absmax2_of8(v[2 * p + 1])));

    uint32_t cm[4];  // of columns 2 k and 2 k + 1
    if (!kWeighted && kCol) {  // before the conversions, which hide the shuffles
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        cm[k] = word_of(v[0], k);
#pragma unroll
        for (int i = 1; i < 8; ++i) cm[k] = absmax2(cm[k], word_of(v[i], k));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) cm[k] = block_absmax2<8>(cm[k]);
    }
    uint32_t rb[4], cb[4] = {};  // scale bytes of the thread's rows and columns, two to a word
    if (!kWeighted) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t e = mx_t2(m[p], round), mul = mx_mul2(e);
        st_codes8(qrow, codes8_row(v[2 * p], __byte_perm(mul, 0, 0x1010)), live);
        st_codes8(qrow + C, codes8_row(v[2 * p + 1], __byte_perm(mul, 0, 0x3232)), live);
        qrow += 2 * static_cast<int64_t>(C);
        rb[p] = mx_bytes2(e);
      }
      if (kCol) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // columns c0 + 2k and c0 + 2k + 1
          const uint32_t e = mx_t2(cm[k], round);
          const CodePair codes = codes8_cols(v, k, mx_mul2(e));
          put_column(cols, rt, ct, 2 * k, codes.lo);
          put_column(cols, rt, ct, 2 * k + 1, codes.hi);
          cb[k] = mx_bytes2(e);
        }
      }
    } else {
      // The products stay in registers between the two passes.
      float2 f[8][4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float wa = sm.weight[n & 3][rt + 2 * p], wb = sm.weight[n & 3][rt + 2 * p + 1];
        const uint32_t e = mx_clamp2(mx_raw2(fabsf(__uint_as_float(f32_bits_lo(m[p])) * wa),
                                             fabsf(__uint_as_float(f32_bits_hi(m[p])) * wb), round));
        const float2 mul = mx_mul2_f32(e);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[2 * p][k] = __fmul2_rn(bf16x2_to_f32(word_of(v[2 * p], k)), make_float2(wa, wa));
          f[2 * p + 1][k] = __fmul2_rn(bf16x2_to_f32(word_of(v[2 * p + 1], k)), make_float2(wb, wb));
        }
        st_codes8(qrow, codes8(f[2 * p], mul.x), live);
        st_codes8(qrow + C, codes8(f[2 * p + 1], mul.y), live);
        qrow += 2 * static_cast<int64_t>(C);
        rb[p] = mx_bytes2(e);
      }
      if (kCol) {
        uint32_t e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float lo = absmax3(absmax3(absmax3(f[0][k].x, f[1][k].x, f[2][k].x), f[3][k].x, f[4][k].x),
                                   absmax3(f[5][k].x, f[6][k].x, f[7][k].x), 0.f);
          const float hi = absmax3(absmax3(absmax3(f[0][k].y, f[1][k].y, f[2][k].y), f[3][k].y, f[4][k].y),
                                   absmax3(f[5][k].y, f[6][k].y, f[7][k].y), 0.f);
          e[k] = mx_raw2(lo, hi, round);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          e[k] = __vmaxu2(e[k], __shfl_xor_sync(kAll, e[k], 8));
          e[k] = mx_clamp2(__vmaxu2(e[k], __shfl_xor_sync(kAll, e[k], 16)));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 mul = mx_mul2_f32(e[k]);
          float2 p[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = __fmul2_rn(f[i][k], mul);
          const CodePair codes = pair_of_columns(p);
          put_column(cols, rt, ct, 2 * k, codes.lo);
          put_column(cols, rt, ct, 2 * k + 1, codes.hi);
          cb[k] = mx_bytes2(e[k]);
        }
      }
    }
    put_bytes(sm.scales[n & 1], rt, ct, rb, cb);
    if (kCol) fence_proxy_async_smem();  // the column codes, for the bulk store behind the barrier
    note(n + 2, src);
    last = now;
    now = next;
    next = after;
  }
  __syncthreads();
  finish(n - 1, last);
  if (kCol && tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ int64_t checked_row(const int32_t* row_of, int64_t i, int64_t P, int* status) {
  int64_t r = row_of[i];
  if (r < -1 || r >= P) {
    atomicExch(status, kStatusShape);
    r = -1;
  }
  return r;
}

// A warp per token and run of 1024 columns, lane l with four 16-byte chunks 32
// apart.  Lane j looks up entry j; the rows are then loaded two entries at a
// time before the first is used, and added in the order of j.  Bound by
// memory: each of a token's rows is read once (8192 x 2 rows of 5120: 43 us,
// 0.86 of the measured copy bandwidth; without the streaming stores 45, with
// two chunks and four rows ahead 50, with one chunk 54).
constexpr int kCombineChunks = 4, kCombineAhead = 2;

__global__ void __launch_bounds__(256)
    combine_kernel(const uint16_t* __restrict__ y, const float* __restrict__ weights,
                   const int32_t* __restrict__ row_of, const uint16_t* base, int64_t units, uint32_t runs, int chunks,
                   int top_k, int64_t P, uint16_t* out, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (unit >= units) return;
  const int64_t t = unit / runs;
  const int first = static_cast<int>(unit - t * runs) * 32 * kCombineChunks + lane;
  int64_t row = -1;
  float weight = 0.f;
  if (lane < top_k) {
    row = checked_row(row_of, t * top_k + lane, P, status);
    if (row >= 0) weight = weights != nullptr ? weights[t * top_k + lane] : 1.f;
  }
  const int mine = static_cast<int>(row);
  float2 acc[kCombineChunks][4];
#pragma unroll
  for (int u = 0; u < kCombineChunks; ++u) {
    const int c = first + 32 * u;
    uint4 b = make_uint4(0, 0, 0, 0);
    if (base != nullptr && c < chunks) b = reinterpret_cast<const uint4*>(base)[t * chunks + c];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[u][k] = bf16x2_to_f32(word_of(b, k));
  }
  for (int j0 = 0; j0 < top_k; j0 += kCombineAhead) {
    uint4 v[kCombineAhead][kCombineChunks];
    float w[kCombineAhead];
#pragma unroll
    for (int i = 0; i < kCombineAhead; ++i) {
      const int from = __shfl_sync(kAll, mine, j0 + i);  // lanes past top_k hold -1
      w[i] = __shfl_sync(kAll, weight, j0 + i);
#pragma unroll
      for (int u = 0; u < kCombineChunks; ++u) {
        const int c = first + 32 * u;
        v[i][u] = ld_once_v4(reinterpret_cast<const uint4*>(y) + (static_cast<int64_t>(max(from, 0)) * chunks + c),
                             from >= 0 && c < chunks);
      }
    }
#pragma unroll
    for (int i = 0; i < kCombineAhead; ++i)
#pragma unroll
      for (int u = 0; u < kCombineChunks; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          acc[u][k] = __ffma2_rn(bf16x2_to_f32(word_of(v[i][u], k)), make_float2(w[i], w[i]), acc[u][k]);
  }
#pragma unroll
  for (int u = 0; u < kCombineChunks; ++u) {
    const int c = first + 32 * u;
    if (c < chunks)
      __stcs(reinterpret_cast<uint4*>(out) + t * chunks + c,
             make_uint4(pack_bf16x2(acc[u][0].x, acc[u][0].y), pack_bf16x2(acc[u][1].x, acc[u][1].y),
                        pack_bf16x2(acc[u][2].x, acc[u][2].y), pack_bf16x2(acc[u][3].x, acc[u][3].y)));
  }
}

// A warp per entry.
__global__ void __launch_bounds__(256)
    combine_dweights_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y,
                            const int32_t* __restrict__ row_of, int64_t entries, int top_k, int64_t P, int64_t chunks,
                            float* __restrict__ dweights, int* status) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= entries) return;
  const int64_t r = checked_row(row_of, i, P, status);
  float acc = 0.f;
  if (r >= 0) {
    for (int64_t c = lane; c < chunks; c += 32) {
      const uint4 a = reinterpret_cast<const uint4*>(dout)[i / top_k * chunks + c];
      const uint4 b = reinterpret_cast<const uint4*>(y)[r * chunks + c];
      const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
      for (int k = 0; k < 4; ++k) {
        acc = fmaf(bf16lo_to_f32(u[k]), bf16lo_to_f32(v[k]), acc);
        acc = fmaf(bf16hi_to_f32(u[k]), bf16hi_to_f32(v[k]), acc);
      }
    }
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kAll, acc, o);
  }
  if (lane == 0) dweights[i] = acc;
}

}  // namespace

// qT [C][P] as (row, column / 8, column % 8), in boxes of 128 x 16 x 8.
static bool column_map(CUtensorMap* map, uint8_t* qT, int64_t C, int64_t P) {
  typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const auto fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(P), static_cast<cuuint64_t>(C / 8), 8};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(8 * P), static_cast<cuuint64_t>(P)};
  const cuuint32_t box[3] = {128, 16, 8}, each[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, qT, dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_moe_gather_quant(const MoeGatherArgs& a, cudaStream_t st) {
  const int64_t bands = (a.P + 127) / 128, tiles = bands * ((a.C + 127) / 128);
  if (tiles > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  auto go = [&](auto weighted, auto columns) {
    constexpr bool kWeighted = decltype(weighted)::value, kCol = decltype(columns)::value;
    const auto kernel = gather_quant_kernel<kWeighted, kCol>;
    constexpr int smem = sizeof(GatherSmem<kCol>) + 1024;  // for its alignment
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // Behind a runtime call, which binds the device's context to a thread that has made none yet (a backward
    // pass runs in one); the driver's encoder does not.
    CUtensorMap map{};
    if (kCol && !column_map(&map, a.qT, a.C, a.P)) return cudaErrorInvalidValue;
    const int64_t cap = static_cast<int64_t>(a.num_sms) * gather_ctas_per_sm(kCol);
    kernel<<<dim3(static_cast<unsigned>(tiles < cap ? tiles : cap)), kGatherWarps * 32, smem, st>>>(
        map, a.x, a.weights, a.src_of, static_cast<uint32_t>(a.M * a.top_k), static_cast<uint32_t>(a.top_k),
        static_cast<int>(a.P), static_cast<int>(a.C), static_cast<int>(bands), static_cast<int>(tiles), a.q, a.e8, a.e8T,
        a.mode, a.status);
    return cudaGetLastError();
  };
  const std::true_type yes;
  const std::false_type no;
  if (a.weights != nullptr) return a.qT != nullptr ? go(yes, yes) : go(yes, no);
  return a.qT != nullptr ? go(no, yes) : go(no, no);
}

cudaError_t launch_moe_combine(const MoeCombineArgs& a, cudaStream_t st) {
  const int64_t chunks = a.C / 8, runs = (chunks + 32 * kCombineChunks - 1) / (32 * kCombineChunks);
  const int64_t units = a.M * runs;
  if ((units + 7) / 8 > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  combine_kernel<<<dim3(static_cast<unsigned>((units + 7) / 8)), 256, 0, st>>>(
      a.y, a.weights, a.row_of, a.base, units, static_cast<uint32_t>(runs), static_cast<int>(chunks),
      static_cast<int>(a.top_k), a.P, a.out, a.status);
  return cudaGetLastError();
}

cudaError_t launch_moe_combine_dweights(const MoeCombineArgs& a, cudaStream_t st) {
  const int64_t entries = a.M * a.top_k;
  combine_dweights_kernel<<<dim3(static_cast<unsigned>((entries + 7) / 8)), 256, 0, st>>>(
      a.dout, a.y, a.row_of, entries, static_cast<int>(a.top_k), a.P, a.C / 8, a.dweights, a.status);
  return cudaGetLastError();
}

}  // namespace fp8bw
