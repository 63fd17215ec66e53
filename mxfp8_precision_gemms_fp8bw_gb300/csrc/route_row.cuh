// A row of router logits in registers, for the kernels of moe_route.cu and
// moe_route_bwd.cu.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "route_math.cuh"

namespace fp8bw {
namespace {  // included by two units

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLowest = -3.4028234663852886e38f;

__device__ __forceinline__ float logit_at(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float logit_at(const uint16_t* p, int64_t i) { return __uint_as_float(uint32_t{p[i]} << 16); }
__device__ __forceinline__ void put_logit(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put_logit(uint16_t* p, int64_t i, float v) {
  p[i] = static_cast<uint16_t>(pack_bf16x2(v, 0.f) & 0xFFFFu);
}

// Keys as unsigned integers of the same order: 0 is a masked expert, below
// the lowest finite key (0x00800000), and NaN is above everything.
__device__ __forceinline__ uint32_t ordered(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t b = __float_as_uint(f + 0.f);  // -0 becomes +0
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
  if (u == 0xffffffffu) return __uint_as_float(0x7FFFFFFFu);
  return __uint_as_float((u >> 31) ? u & 0x7FFFFFFFu : ~u);
}

// A row belongs to L lanes (8, or 32 where a row is long), 32 / L rows to a
// warp, and lane l of the row holds experts v * L + l, v < V.  Everything but
// the reductions is then work of V registers per lane, which with L = 8 is
// shared by four rows; and the reductions are three shuffles.  (A whole warp
// per row, with warp-wide reductions, took 104 us for 127999 rows of 160
// experts, 4 of them chosen, against 41.)
template <int L, typename F>
__device__ __forceinline__ float lanes_reduce(float v, F&& f) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_reduce<L>(v, [](float a, float b) { return a + b; });
}

__host__ __device__ constexpr int pow2_from(int n) { return n <= 1 ? 1 : 2 * pow2_from((n + 1) / 2); }

// What the softmax scores of a row have in common.
struct RowScale {
  float top, total, inv;
  bool tiny;  // an exponential too small for the short division
};
// fl(e / total): one correction step of Markstein's division from the rounded
// reciprocal (route_math.cuh), and the plain division for the rows in which
// that could lose bits.
__device__ __forceinline__ float softmax_of(float e, const RowScale& r) {
  return r.tiny ? __fdiv_rn(e, r.total) : div_by(e, r.total, r.inv);
}
__device__ __forceinline__ float sigmoid_of(float x) { return __frcp_rn(1.f + expf(-x)); }  // rounded as 1 / (...)

// The scores of a row.  For the choice (kExact) quotients are correctly
// rounded, exponentials the library's, and the sum runs by halves (first over
// v, then over the lanes, zeros past the last expert), because the choice has
// to come out the same however the row is split.  A gradient takes the
// product with the reciprocal, an ulp off.
template <int L, int V, bool kExact>
__device__ __forceinline__ RowScale scores_of(const float (&x)[V], int score, float (&s)[V]) {
  RowScale r{};
  if (score != 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = sigmoid_of(x[v]);
    return r;
  }
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) top = fmaxf(top, x[v]);
  top = lanes_reduce<L>(top, [](float a, float b) { return fmaxf(a, b); });
  // A row of nothing but -inf gets exponentials 0 over a sum of 1: no scores.
  // NaN makes the sum NaN, and with it every score.
  r.top = top == -INFINITY ? 0.f : top;
  float part[V];
  uint32_t least = 0xffffffffu;  // bits of the smallest exponential that is not 0, less one
#pragma unroll
  for (int v = 0; v < V; ++v) {
    part[v] = s[v] = expf(x[v] - r.top);
    if (kExact) least = min(least, __float_as_uint(s[v]) - 1u);
  }
  if (kExact) r.tiny = __any_sync(kAll, least < __float_as_uint(kShortDivisionMin) - 1u);
  constexpr int kHalf = pow2_from(V) / 2;
#pragma unroll
  for (int h = kHalf; h > 0; h /= 2)
#pragma unroll
    for (int v = 0; v < h; ++v)
      if (v + h < V) part[v] += part[v + h];
  const float total = lanes_sum<L>(part[0]);
  r.total = total == 0.f ? 1.f : total;
  r.inv = __frcp_rn(r.total);
  if (!kExact) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] *= r.inv;
  } else if (r.tiny) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = __fdiv_rn(s[v], r.total);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = div_by(s[v], r.total, r.inv);
  }
  return r;
}
// The score of one logit of a row, the same bits.
__device__ __forceinline__ float score_at(float x, int score, const RowScale& r) {
  return score != 0 ? sigmoid_of(x) : softmax_of(expf(x - r.top), r);
}

struct RouteShape {
  int64_t M;
  int E, k, groups, kept, group_top, score, renorm;
  float scale;
};

constexpr int kRouteWarps = 4;

inline RouteShape shape_of(const MoeRouteArgs& a) {
  return RouteShape{a.M,
                    static_cast<int>(a.E),
                    static_cast<int>(a.top_k),
                    static_cast<int>(a.groups),
                    static_cast<int>(a.groups_kept),
                    static_cast<int>(a.group_top),
                    a.score,
                    a.renorm,
                    a.scale};
}

// Rows per block and the shared memory of one copy of them, padded so that
// rows start at different banks.
template <int L>
constexpr int kRouteRows = kRouteWarps * 32 / L;
template <int L>
size_t staged_bytes(int64_t E) {
  return kRouteRows<L> * (E | 8) * sizeof(uint32_t);
}

// Calls go(lanes per row, registers per lane) for E experts: the next of these
// widths.  A row holds up to a third more registers than it fills, 60 % more
// at 33 experts, and with a warp per row 78 % more at 257 and 88 % at 513
// (forward, 384 experts, 8 of them chosen, 127999 rows: 238 us).
template <typename Go>
cudaError_t for_experts(int64_t E, Go&& go) {
  using std::integral_constant;
  const integral_constant<int, 8> eight;
  const integral_constant<int, 32> all;
  if (E <= 8) return go(eight, integral_constant<int, 1>{});
  if (E <= 16) return go(eight, integral_constant<int, 2>{});
  if (E <= 32) return go(eight, integral_constant<int, 4>{});
  if (E <= 64) return go(eight, integral_constant<int, 8>{});
  if (E <= 96) return go(eight, integral_constant<int, 12>{});
  if (E <= 128) return go(eight, integral_constant<int, 16>{});
  if (E <= 160) return go(eight, integral_constant<int, 20>{});
  if (E <= 192) return go(eight, integral_constant<int, 24>{});
  if (E <= 256) return go(eight, integral_constant<int, 32>{});
  if (E <= 512) return go(all, integral_constant<int, 16>{});
  return go(all, integral_constant<int, 32>{});
}

}  // namespace
}  // namespace fp8bw
