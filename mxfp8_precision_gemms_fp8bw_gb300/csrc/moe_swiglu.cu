// The gated activation of an MXFP8 layer, held as MX codes, with its input
// kept in 8 bits, and its gradient from those 8 bits.
//
// Both kernels read each element once and write only codes (8.1 bytes per
// element of a forward, 8.2 backward).  The forward pass is bound by memory:
// 90 us for 16640 x 4096 (0.91 of the measured copy bandwidth), 168 us for
// 130048 x 1024 (0.95).  The backward pass has twice the results to convert,
// some forty instructions per element, and is bound by them as much as by
// memory: 115 us (0.71) and 216 us (0.75).
//
// A thread has 4 rows x 8 columns, a warp 32 x 32: lane 4 i + j has rows
// 4 i + [0, 4) and columns 8 j + [0, 8), so that a row block is four
// neighbouring lanes and a column block the eight lanes 4 apart.  (8 x 8 per
// thread, as in moe_rows.cu, needs twice the registers here, where two
// operands and one or two results are live at once.)  A block has 64 x 128.
#include "common.cuh"
#include "launch.h"
#include "mx_tile.cuh"

namespace fp8bw {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kRows = 64, kCols = 128, kThreads = 256;

// 1 / (1 + 2^(-x log2 e)) of two values.  The exponent's argument is rounded
// to fp32 before ex2, which costs up to |x log2 e| / 2 units of 2^-24 (29 at
// -30, 64 at -88) beside the few of ex2 and rcp: far below the 2^-4 of the
// codes that it goes into (with the argument in two parts the backward pass
// takes 121 and 227 us in place of 115 and 216).  rcp flushes what lies below
// 2^-126, so it gets a quarter of the sum (1 % of the backward pass): the
// result then reaches as far down as 1 + exp(-x) fits fp32, x >= -88.7, and is
// 0 beyond.  Exactly 1 far out on the other side, NaN for NaN.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  constexpr float kMinusLog2e = -1.4426950408889634f;
  const float2 quarter = make_float2(0.25f, 0.25f);
  const float2 t = __fmul2_rn(x, make_float2(kMinusLog2e, kMinusLog2e));
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = __ffma2_rn(e, quarter, quarter);
  float2 s;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
  return __fmul2_rn(s, quarter);
}

struct Lane {
  int rt, ct;  // first row and column of the thread in the block's tile
};
__device__ __forceinline__ Lane lane_of() {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  return Lane{(warp >> 2) * 32 + (lane >> 2) * 4, (warp & 3) * 32 + (lane & 3) * 8};
}

// Scale bytes of the tile, gathered to go out as words (see ScaleTile).
struct alignas(8) Scales {
  uint8_t row[4][kRows];  // [block][row]
  uint8_t col[2][kCols];  // [block][column]
};
// t's of the thread's four rows and eight columns, two to a word.
__device__ __forceinline__ void put_row_bytes(Scales& s, Lane l, uint32_t t01, uint32_t t23) {
  if ((l.ct & 31) == 0)
    *reinterpret_cast<uint32_t*>(&s.row[l.ct / 32][l.rt]) = __byte_perm(mx_bytes2(t01), mx_bytes2(t23), 0x6420);
}
__device__ __forceinline__ void put_col_bytes(Scales& s, Lane l, const uint32_t (&t)[4]) {
  if ((l.rt & 31) == 0)
    *reinterpret_cast<uint2*>(&s.col[l.rt / 32][l.ct]) =
        make_uint2(__byte_perm(mx_bytes2(t[0]), mx_bytes2(t[1]), 0x6420), __byte_perm(mx_bytes2(t[2]), mx_bytes2(t[3]), 0x6420));
}
// Row scales of the tile at rows r0, blocks b0 .. b0 + 3 of e8 [R][per_row], by threads 0 to 63.
__device__ __forceinline__ void flush_rows(const Scales& s, int64_t r0, int64_t R, uint8_t* __restrict__ e8,
                                           int64_t b0, int64_t b_end, int64_t per_row) {
  const int i = threadIdx.x;
  if (i >= kRows || r0 + i >= R) return;
  uint8_t* to = e8 + (r0 + i) * per_row + b0;
  if ((reinterpret_cast<uintptr_t>(to) & 3) == 0 && b0 + 4 <= b_end) {
    *reinterpret_cast<uint32_t*>(to) = s.row[0][i] | s.row[1][i] << 8 | s.row[2][i] << 16 | uint32_t{s.row[3][i]} << 24;
  } else {
    for (int b = 0; b < 4 && b0 + b < b_end; ++b) to[b] = s.row[b][i];
  }
}
// Column scales of the tile at columns c0, blocks b0 and b0 + 1 of e8T [C][per_col], by threads 128 to 255.
__device__ __forceinline__ void flush_cols(const Scales& s, int64_t c0, int64_t c_end, uint8_t* __restrict__ e8T,
                                           int64_t b0, int64_t per_col) {
  const int i = static_cast<int>(threadIdx.x) - 128;
  if (i < 0 || c0 + i >= c_end) return;
  uint8_t* to = e8T + (c0 + i) * per_col + b0;
  if ((per_col & 1) == 0) {
    *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(s.col[0][i] | s.col[1][i] << 8);
  } else {
    to[0] = s.col[0][i];
    if (b0 + 1 < per_col) to[1] = s.col[1][i];
  }
}

// max over a row block's lanes (xor 1, 2) or a column block's (xor 4, 8, 16)
// of two t's in a word: the exponent grows with the max.
__device__ __forceinline__ uint32_t row_max2(uint32_t t) {
  t = __vmaxu2(t, __shfl_xor_sync(kAll, t, 1));
  return __vmaxu2(t, __shfl_xor_sync(kAll, t, 2));
}
__device__ __forceinline__ uint32_t col_max2(uint32_t t) {
  t = __vmaxu2(t, __shfl_xor_sync(kAll, t, 4));
  t = __vmaxu2(t, __shfl_xor_sync(kAll, t, 8));
  return __vmaxu2(t, __shfl_xor_sync(kAll, t, 16));
}
// Both layouts of the thread's 4 x 8 values: q at (row, col) of a matrix with
// `ld` columns, qT transposed with R rows (qcol may be null).
__device__ __forceinline__ void quant_4x8(const float2 (&v)[4][4], Lane l, bool live, uint32_t round, uint8_t* qrow,
                                          int64_t ld, uint8_t* qcol, int64_t R, Scales& s) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m[i] = absmax3(absmax3(v[i][0].x, v[i][0].y, v[i][1].x), absmax3(v[i][1].y, v[i][2].x, v[i][2].y),
                   absmax3(v[i][3].x, v[i][3].y, 0.f));
  const uint32_t t[2] = {mx_clamp2(row_max2(mx_raw2(m[0], m[1], round))), mx_clamp2(row_max2(mx_raw2(m[2], m[3], round)))};
  uint32_t tc[4];
  if (qcol != nullptr) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      tc[k] = mx_raw2(absmax3(absmax3(v[0][k].x, v[1][k].x, v[2][k].x), v[3][k].x, 0.f),
                      absmax3(absmax3(v[0][k].y, v[1][k].y, v[2][k].y), v[3][k].y, 0.f), round);
#pragma unroll
    for (int k = 0; k < 4; ++k) tc[k] = mx_clamp2(col_max2(tc[k]));
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float2 mul = mx_mul2_f32(t[p]);
    st_codes8(qrow + 2 * p * ld, codes8(v[2 * p], mul.x), live);
    st_codes8(qrow + (2 * p + 1) * ld, codes8(v[2 * p + 1], mul.y), live);
  }
  put_row_bytes(s, l, t[0], t[1]);
  if (qcol == nullptr) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {  // two columns at a time, each with its own scale
    const float2 mul = mx_mul2_f32(tc[k]);
    const float2 a = __fmul2_rn(v[0][k], mul), b = __fmul2_rn(v[1][k], mul), c = __fmul2_rn(v[2][k], mul),
                 d = __fmul2_rn(v[3][k], mul);
    st_codes4(qcol, e4m3x4(a.x, b.x, c.x, d.x), live);
    st_codes4(qcol + R, e4m3x4(a.y, b.y, c.y, d.y), live);
    qcol += 2 * R;
  }
  put_col_bytes(s, l, tc);
}

// Rowwise codes of four rows of packed bf16.
__device__ __forceinline__ void keep_4x8(const uint4 (&v)[4], Lane l, bool live, uint32_t round, uint8_t* qrow,
                                         int64_t ld, Scales& s) {
  uint32_t t[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) t[p] = mx_t2(block_absmax2<1>(fold2(absmax2_of8(v[2 * p]), absmax2_of8(v[2 * p + 1]))), round);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    st_codes8(qrow + i * ld, codes8_row(v[i], __byte_perm(mx_mul2(t[i >> 1]), 0, (i & 1) ? 0x3232 : 0x1010)), live);
  put_row_bytes(s, l, t[0], t[1]);
}

__global__ void __launch_bounds__(kThreads)
    swiglu_kernel(const uint16_t* __restrict__ h, int64_t R, int64_t F, uint32_t stripes, uint8_t* __restrict__ aq,
                  uint8_t* __restrict__ ae, uint8_t* __restrict__ aqT, uint8_t* __restrict__ aeT,
                  uint8_t* __restrict__ hq, uint8_t* __restrict__ he, int mode) {
  __shared__ Scales sa, sg, su;
  const Lane l = lane_of();
  // Columns fastest: whole rows of h are read together (16640 x 4096: 94 us with the rows fastest, 90 so).
  const uint32_t band = blockIdx.x / stripes;
  const int64_t tr = static_cast<int64_t>(band) * kRows, tc = static_cast<int64_t>(blockIdx.x - band * stripes) * kCols;
  const int64_t r0 = tr + l.rt, c0 = tc + l.ct;
  const bool live = r0 < R && c0 < F;  // R and F % 32 == 0: blocks are all in or all out
  const uint32_t round = mx_round_f32(mode);
  uint4 g[4], u[4];
  const uint16_t* hp = h + (live ? r0 * 2 * F + c0 : 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = ld_once_v4(hp + i * 2 * F, live);
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = ld_once_v4(hp + i * 2 * F + F, live);
  if (hq != nullptr) {
    keep_4x8(g, l, live, round, hq + r0 * 2 * F + c0, 2 * F, sg);
    keep_4x8(u, l, live, round, hq + r0 * 2 * F + F + c0, 2 * F, su);
  }
  float2 a[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = bf16x2_to_f32(word_of(g[i], k)), y = bf16x2_to_f32(word_of(u[i], k));
      a[i][k] = __fmul2_rn(__fmul2_rn(x, sigmoid2(x)), y);
    }
  quant_4x8(a, l, live, round, aq + r0 * F + c0, F, aqT != nullptr ? aqT + c0 * R + r0 : nullptr, R, sa);
  __syncthreads();
  flush_rows(sa, tr, R, ae, tc / 32, F / 32, F / 32);
  if (hq != nullptr) {
    flush_rows(sg, tr, R, he, tc / 32, F / 32, F / 16);
    flush_rows(su, tr, R, he, F / 32 + tc / 32, F / 16, F / 16);
  }
  if (aqT != nullptr) flush_cols(sa, tc, F, aeT, tr / 32, R / 32);
}

// Eight values of codes times a scale.
__device__ __forceinline__ void decode8(uint2 c, float scale, float2 (&v)[4]) {
  const float2 s = make_float2(scale, scale);
  v[0] = __fmul2_rn(e4m3x2_to_f32(c.x & 0xFFFFu), s);
  v[1] = __fmul2_rn(e4m3x2_to_f32(c.x >> 16), s);
  v[2] = __fmul2_rn(e4m3x2_to_f32(c.y & 0xFFFFu), s);
  v[3] = __fmul2_rn(e4m3x2_to_f32(c.y >> 16), s);
}

// The backward pass keeps two results of 32 values a thread, so few warps fit
// (16 an SM), too few to wait for their own loads: blocks are persistent and
// copy the next tile's operands to shared memory (cp.async) while they convert
// the present one.  16-byte chunks are swizzled by the rows that one
// instruction reads together, 4 apart.
struct BwdSmem {
  uint4 gate[2][kRows][8];   // chunk c of row r at c ^ ((r / 4) % 4) * 2
  uint4 up[2][kRows][8];
  uint4 da[2][kRows][16];    // chunk c of row r at c ^ ((r / 4) % 2) * 4
  Scales sg[2], su[2];       // of the gradient
  uint8_t exps[2][8][kRows];  // of the operands: four blocks of gate, four of up
};
constexpr int kBwdCtasPerSm = 2;

__device__ __forceinline__ void copy16(void* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}

__global__ void __launch_bounds__(kThreads, kBwdCtasPerSm)
    swiglu_bwd_kernel(const uint16_t* __restrict__ da, const uint8_t* __restrict__ hq, const uint8_t* __restrict__ he,
                      int64_t R, int64_t F, uint32_t stripes, uint32_t tiles, uint8_t* __restrict__ dq,
                      uint8_t* __restrict__ de, uint8_t* __restrict__ dqT, uint8_t* __restrict__ deT, int mode) {
  extern __shared__ __align__(128) uint8_t bwd_smem[];
  BwdSmem& sm = *reinterpret_cast<BwdSmem*>(bwd_smem);
  const Lane l = lane_of();
  const uint32_t round = mx_round_f32(mode);
  const int tid = threadIdx.x;

  struct Origin {
    int64_t r, c;
  };
  auto origin = [&](uint32_t tile) {
    const uint32_t band = tile / stripes;
    return Origin{static_cast<int64_t>(band) * kRows, static_cast<int64_t>(tile - band * stripes) * kCols};
  };
  // The thread's chunks of a tile: rows tid / 8 + {0, 32} of gate and of up, rows tid / 16 + {0, 16, 32, 48} of da.
  const int hr = tid >> 3, hc = tid & 7, dr = tid >> 4, dc = tid & 15;
  const uint8_t* h0 = hq + hr * 2 * F + 16 * hc;
  const uint16_t* d0 = da + dr * F + 8 * dc;
  auto fetch = [&](int s, Origin o) {
    const bool whole = o.r + kRows <= R && o.c + kCols <= F;
    const uint8_t* hp = h0 + o.r * 2 * F + o.c;
    const uint16_t* dp = d0 + o.r * F + o.c;
    const int64_t h_rows = 64 * F, d_rows = 16 * F;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool live = whole || (o.r + hr + 32 * j < R && o.c + 16 * hc < F);
      const int chunk = hc ^ ((hr >> 2) & 3) << 1;
      copy16(&sm.gate[s][hr + 32 * j][chunk], live ? hp + j * h_rows : hq, live);
      copy16(&sm.up[s][hr + 32 * j][chunk], live ? hp + j * h_rows + F : hq, live);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool live = whole || (o.r + dr + 16 * j < R && o.c + 8 * dc < F);
      copy16(&sm.da[s][dr + 16 * j][dc ^ ((dr >> 2) & 1) << 2], live ? dp + j * d_rows : da, live);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Scale bytes of the operands: thread i < 128 has the four blocks of row i / 2 of gate (i even) or up.
  auto exps_of = [&](Origin o) {
    uint32_t e = 0;
    const int64_t r = o.r + (tid >> 1);
    if (tid < 128 && r < R) {
      const uint8_t* from = he + r * (F / 16) + (tid & 1) * (F / 32) + o.c / 32;
      if ((reinterpret_cast<uintptr_t>(from) & 3) == 0 && o.c + kCols <= F) {
        e = *reinterpret_cast<const uint32_t*>(from);
      } else {
        for (int b = 0; b < 4 && o.c + 32 * b < F; ++b) e |= uint32_t{from[b]} << 8 * b;
      }
    }
    return e;
  };
  auto note_exps = [&](int s, uint32_t e) {
    if (tid >= 128) return;
#pragma unroll
    for (int b = 0; b < 4; ++b) sm.exps[s][(tid & 1) * 4 + b][tid >> 1] = static_cast<uint8_t>(e >> 8 * b);
  };
  auto flush = [&](int s, Origin o) {
    flush_rows(sm.sg[s], o.r, R, de, o.c / 32, F / 32, F / 16);
    flush_rows(sm.su[s], o.r, R, de, F / 32 + o.c / 32, F / 16, F / 16);
    flush_cols(sm.sg[s], o.c, F, deT, o.r / 32, R / 32);
    flush_cols(sm.su[s], F + o.c, 2 * F, deT, o.r / 32, R / 32);
  };

  uint32_t tile = blockIdx.x;
  Origin now = origin(tile), last{};
  fetch(0, now);
  note_exps(0, exps_of(now));
  for (int n = 0;; ++n) {
    const int s = n & 1;
    const uint32_t ahead = tile + gridDim.x;
    const bool more = ahead < tiles;
    const Origin next = origin(more ? ahead : tile);
    // This tile has landed; everyone has left the one before and its buffers.
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    uint32_t exps = 0;
    if (more) {
      fetch(s ^ 1, next);
      exps = exps_of(next);
    }
    if (n > 0) flush(s ^ 1, last);

    const int64_t r0 = now.r + l.rt, c0 = now.c + l.ct;
    const bool live = r0 < R && c0 < F;
    const uint32_t ge = *reinterpret_cast<const uint32_t*>(&sm.exps[s][l.ct / 32][l.rt]);
    const uint32_t ue = *reinterpret_cast<const uint32_t*>(&sm.exps[s][4 + l.ct / 32][l.rt]);
    const int gu = (l.ct >> 4) ^ ((l.rt >> 2) & 3) << 1, dd = (l.ct >> 3) ^ ((l.rt >> 2) & 1) << 2;
    float2 dg[4][4], du[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 g[4], u[4];
      decode8(reinterpret_cast<const uint2*>(&sm.gate[s][l.rt + i][gu])[(l.ct >> 3) & 1], e8m0_value(ge >> 8 * i & 0xFF), g);
      decode8(reinterpret_cast<const uint2*>(&sm.up[s][l.rt + i][gu])[(l.ct >> 3) & 1], e8m0_value(ue >> 8 * i & 0xFF), u);
      const uint4 d = sm.da[s][l.rt + i][dd];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = bf16x2_to_f32(word_of(d, k));
        const float2 sig = sigmoid2(g[k]), one = make_float2(1.f, 1.f);
        const float2 p = __fmul2_rn(x, sig), rest = __fadd2_rn(one, make_float2(-sig.x, -sig.y));
        du[i][k] = __fmul2_rn(p, g[k]);
        dg[i][k] = __fmul2_rn(__fmul2_rn(p, u[k]), __ffma2_rn(g[k], rest, one));
      }
    }
    quant_4x8(du, l, live, round, dq + r0 * 2 * F + F + c0, 2 * F, dqT + (F + c0) * R + r0, R, sm.su[s]);
    quant_4x8(dg, l, live, round, dq + r0 * 2 * F + c0, 2 * F, dqT + c0 * R + r0, R, sm.sg[s]);
    if (more) note_exps(s ^ 1, exps);
    last = now;
    now = next;
    tile = ahead;
    if (!more) {
      __syncthreads();
      flush(s, last);
      return;
    }
  }
}

struct Tiles {
  int64_t stripes, count;
};
Tiles tiles_of(int64_t R, int64_t F) {
  const int64_t stripes = (F + kCols - 1) / kCols;
  return Tiles{stripes, stripes * ((R + kRows - 1) / kRows)};
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t st) {
  const Tiles t = tiles_of(a.R, a.F);
  if (t.count > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  swiglu_kernel<<<dim3(static_cast<unsigned>(t.count)), kThreads, 0, st>>>(
      a.h, a.R, a.F, static_cast<uint32_t>(t.stripes), a.aq, a.ae, a.aqT, a.aeT, a.hq, a.he, a.mode);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t st) {
  const Tiles t = tiles_of(a.R, a.F);
  if (t.count > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      cudaFuncSetAttribute(swiglu_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(BwdSmem));
  if (e != cudaSuccess) return e;
  const int64_t cap = static_cast<int64_t>(a.num_sms) * kBwdCtasPerSm;
  swiglu_bwd_kernel<<<dim3(static_cast<unsigned>(t.count < cap ? t.count : cap)), kThreads, sizeof(BwdSmem), st>>>(
      a.da, a.hq, a.he, a.R, a.F, static_cast<uint32_t>(t.stripes), static_cast<uint32_t>(t.count), a.dq, a.de, a.dqT,
      a.deT, a.mode);
  return cudaGetLastError();
}

}  // namespace fp8bw
