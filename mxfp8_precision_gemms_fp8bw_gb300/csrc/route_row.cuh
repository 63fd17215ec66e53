// A row of router logits in registers, for the kernels of moe_route.cu,
// moe_route_bwd.cu and few_route.cu.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "route_math.cuh"

namespace fp8bw {
namespace {  // included by several units

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

// The choice of one row by its L lanes, from logits [.., E] to experts and
// weights [.., k].  mine: the row's place among those of the block; keys: E | 8
// words of shared memory for each of them, where there are groups.
template <typename T, int L, int V>
__device__ __forceinline__ void route_row(const T* __restrict__ logits, const float* __restrict__ bias, const RouteShape& p,
                                          int64_t row, bool live, int mine, uint32_t* staged,
                                          int32_t* __restrict__ experts, float* __restrict__ weights) {
  constexpr int kRowsPerWarp = 32 / L;
  const int l = threadIdx.x & (L - 1);  // the lane in its row
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
