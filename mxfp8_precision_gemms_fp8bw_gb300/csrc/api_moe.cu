// C ABI of libfp8bw, second part (declared in include/fp8bw_moe.h): argument
// validation and dispatch of the operators around the experts' products.
#include "api_common.h"
#include "fp8bw_moe.h"

using namespace fp8bw;

namespace {

// Entries and their padded rows are numbered in int32.
bool plan_dims_ok(int64_t M, int64_t E, int64_t top_k) {
  return choices_ok(M, E, top_k) && M * top_k <= kMaxDim - 32 * FP8BW_MOE_MAX_EXPERTS;
}

bool rows_dims_ok(int64_t M, int64_t top_k, int64_t P, int64_t C, int64_t c_mult) {
  return dim_ok(M, 1) && dim_ok(top_k, 1) && top_k <= FP8BW_MOE_MAX_TOP_K && M * top_k <= kMaxDim && dim_ok(P, 32) &&
         dim_ok(C, c_mult) && C <= (int64_t{1} << 22);
}

const char* kRowsShape =
    "%s: need 0 < M, 0 < top_k <= 32, M * top_k < 2^31, P a positive multiple of 32 and C a positive multiple of %d up "
    "to 2^22";

int route_common(const char* name, MoeRouteArgs& a, int logits_type, void* stream) {
  if (!choices_ok(a.M, a.E, a.top_k))
    return fail(FP8BW_ERR_SHAPE, "%s: need 0 < M, 0 < E <= 1024 and 0 < top_k <= min(E, 32); got M=%lld E=%lld top_k=%lld",
                name, (long long)a.M, (long long)a.E, (long long)a.top_k);
  if (!groups_ok(a.E, a.top_k, a.groups, a.groups_kept))
    return fail(FP8BW_ERR_SHAPE,
                "%s: groups (%lld) must be 1 to 32 and divide E, groups_kept (%lld) 1 to groups, and top_k at most the "
                "experts of the kept groups",
                name, (long long)a.groups, (long long)a.groups_kept);
  if (!all_aligned({a.logits, a.bias, a.experts, a.weights, a.dweights, a.experts_in, a.dlogits}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (logits_type != FP8BW_LOGITS_F32 && logits_type != FP8BW_LOGITS_BF16)
    return fail(FP8BW_ERR_ARG, "%s: logits_type %d is neither F32 (0) nor BF16 (1)", name, logits_type);
  if (a.score != FP8BW_SCORE_SOFTMAX && a.score != FP8BW_SCORE_SIGMOID)
    return fail(FP8BW_ERR_ARG, "%s: score %d is neither SOFTMAX (0) nor SIGMOID (1)", name, a.score);
  if (a.group_top != 1 && a.group_top != 2)
    return fail(FP8BW_ERR_ARG, "%s: group_top %lld is neither 1 nor 2", name, (long long)a.group_top);
  const int64_t n = a.M * a.E * (a.bf16 ? 2 : 4), c = a.M * a.top_k * 4;
  if (any_overlap({{a.experts, c}, {a.weights, c}, {a.dlogits, n}},
                  {{a.logits, n}, {a.bias, a.E * 4}, {a.dweights, c}, {a.experts_in, c}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: outputs overlap an input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  a.status = d->error_word;
  return launched(a.dlogits ? launch_moe_route_bwd(a, as_stream(stream)) : launch_moe_route(a, as_stream(stream)), name);
}

}  // namespace

// ============================================================ routing

FP8BW_API int fp8bw_moe_route(const void* logits, int logits_type, const float* bias, int64_t M, int64_t E,
                              int64_t top_k, int64_t groups, int64_t groups_kept, int64_t group_top, int score,
                              int renorm, float scale, int32_t* experts, float* weights, void* stream) {
  const char* name = "fp8bw_moe_route";
  if (!logits || !experts || !weights)
    return fail(FP8BW_ERR_NULL, "%s: logits, experts and weights must be non-NULL", name);
  MoeRouteArgs a{};
  a.logits = logits;
  a.bf16 = logits_type == FP8BW_LOGITS_BF16;
  a.bias = bias;
  a.M = M;
  a.E = E;
  a.top_k = top_k;
  a.groups = groups;
  a.groups_kept = groups_kept;
  a.group_top = group_top;
  a.score = score;
  a.renorm = renorm;
  a.scale = scale;
  a.experts = experts;
  a.weights = weights;
  return route_common(name, a, logits_type, stream);
}

FP8BW_API int fp8bw_moe_route_bwd(const float* dweights, const void* logits, int logits_type, const int32_t* experts,
                                  int64_t M, int64_t E, int64_t top_k, int score, int renorm, float scale,
                                  void* dlogits, void* stream) {
  const char* name = "fp8bw_moe_route_bwd";
  if (!dweights || !logits || !experts || !dlogits)
    return fail(FP8BW_ERR_NULL, "%s: dweights, logits, experts and dlogits must be non-NULL", name);
  MoeRouteArgs a{};
  a.logits = logits;
  a.bf16 = logits_type == FP8BW_LOGITS_BF16;
  a.M = M;
  a.E = E;
  a.top_k = top_k;
  a.groups = a.groups_kept = a.group_top = 1;
  a.score = score;
  a.renorm = renorm;
  a.scale = scale;
  a.dweights = dweights;
  a.experts_in = experts;
  a.dlogits = dlogits;
  return route_common(name, a, logits_type, stream);
}

// ============================================================ rows of the experts

FP8BW_API int64_t fp8bw_moe_plan_rows(int64_t M, int64_t E, int64_t top_k) {
  if (!plan_dims_ok(M, E, top_k)) return 0;
  const int64_t n = M * top_k, rows = (n + 31 * (E < n ? E : n)) / 32 * 32;
  return rows < 32 ? 32 : rows;
}

FP8BW_API size_t fp8bw_moe_plan_workspace_bytes(int64_t M, int64_t E, int64_t top_k) {
  return plan_dims_ok(M, E, top_k) ? moe_plan_workspace_bytes(M, E, top_k) : 0;
}

FP8BW_API int fp8bw_moe_plan(const int32_t* experts, int64_t M, int64_t E, int64_t top_k, int64_t P,
                             int32_t* group_end, int32_t* counts, int32_t* row_of, int32_t* src_of, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const char* name = "fp8bw_moe_plan";
  if (!experts || !group_end || !counts || !row_of || !src_of)
    return fail(FP8BW_ERR_NULL, "%s: experts, group_end, counts, row_of and src_of must be non-NULL", name);
  if (!plan_dims_ok(M, E, top_k))
    return fail(FP8BW_ERR_SHAPE,
                "%s: need 0 < M, 0 < E <= 1024, 0 < top_k <= min(E, 32) and M * top_k < 2^31 - 2^15; got M=%lld E=%lld "
                "top_k=%lld",
                name, (long long)M, (long long)E, (long long)top_k);
  if (!dim_ok(P, 32) || P < fp8bw_moe_plan_rows(M, E, top_k))
    return fail(FP8BW_ERR_SHAPE, "%s: P=%lld must be a multiple of 32 and at least fp8bw_moe_plan_rows = %lld", name,
                (long long)P, (long long)fp8bw_moe_plan_rows(M, E, top_k));
  if (!all_aligned({experts, group_end, counts, row_of, src_of, workspace}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  const size_t need = moe_plan_workspace_bytes(M, E, top_k);
  if (need > 0 && !workspace)
    return fail(FP8BW_ERR_NULL, "%s: these dims need a workspace of %zu bytes", name, need);
  if (workspace_bytes < need)
    return fail(FP8BW_ERR_ARG, "%s: workspace of %zu bytes is smaller than the %zu bytes these dims need", name,
                workspace_bytes, need);
  const int64_t n = M * top_k * 4;
  if (any_overlap({{group_end, E * 4}, {counts, E * 4}, {row_of, n}, {src_of, P * 4},
                   {workspace, static_cast<int64_t>(need)}},
                  {{experts, n}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: outputs overlap the input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  const MoePlanArgs a{experts, M, E, top_k, P, group_end, counts, row_of, src_of, workspace, d->error_word, d->num_sms};
  return launched(launch_moe_plan(a, as_stream(stream)), name);
}

FP8BW_API int mxfp8_moe_gather_quant(const fp8bw_bf16* x, const float* weights, const int32_t* src_of, int64_t M,
                                     int64_t top_k, int64_t P, int64_t C, uint8_t* q, uint8_t* e8, uint8_t* qT,
                                     uint8_t* e8T, int mode, void* stream) {
  const char* name = "mxfp8_moe_gather_quant";
  if (!x || !src_of || !q || !e8 || (qT == nullptr) != (e8T == nullptr))
    return fail(FP8BW_ERR_NULL, "%s: x, src_of, q and e8 must be non-NULL, qT and e8T both set or both NULL", name);
  if (!rows_dims_ok(M, top_k, P, C, 32)) return fail(FP8BW_ERR_SHAPE, kRowsShape, name, 32);
  if (!all_aligned({x, weights, src_of, q, e8, qT, e8T}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (!mode_ok(mode)) return fail(FP8BW_ERR_ARG, "%s: mode %d is neither RCEIL (0) nor FLOOR (1)", name, mode);
  const int64_t n = P * C;
  if (any_overlap({{q, n}, {e8, n / 32}, {qT, n}, {e8T, n / 32}},
                  {{x, M * C * 2}, {weights, M * top_k * 4}, {src_of, P * 4}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: outputs overlap an input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  const MoeGatherArgs a{x, weights, src_of, M, top_k, P, C, q, e8, qT, e8T, mode, d->error_word, d->num_sms};
  return launched(launch_moe_gather_quant(a, as_stream(stream)), name);
}

FP8BW_API int fp8bw_moe_combine(const fp8bw_bf16* y, const float* weights, const int32_t* row_of,
                                const fp8bw_bf16* base, int64_t M, int64_t top_k, int64_t P, int64_t C,
                                fp8bw_bf16* out, void* stream) {
  const char* name = "fp8bw_moe_combine";
  if (!y || !row_of || !out) return fail(FP8BW_ERR_NULL, "%s: y, row_of and out must be non-NULL", name);
  if (!rows_dims_ok(M, top_k, P, C, 8)) return fail(FP8BW_ERR_SHAPE, kRowsShape, name, 8);
  if (!all_aligned({y, weights, row_of, base, out}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  const int64_t n = M * C * 2;
  if (any_overlap({{out, n}}, {{y, P * C * 2}, {weights, M * top_k * 4}, {row_of, M * top_k * 4},
                               {base == out ? nullptr : base, n}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: out overlaps an input (only base may be out itself)", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  const MoeCombineArgs a{y, weights, row_of, base, M, top_k, P, C, out, nullptr, nullptr, d->error_word};
  return launched(launch_moe_combine(a, as_stream(stream)), name);
}

FP8BW_API int fp8bw_moe_combine_dweights(const fp8bw_bf16* dout, const fp8bw_bf16* y, const int32_t* row_of,
                                         int64_t M, int64_t top_k, int64_t P, int64_t C, float* dweights,
                                         void* stream) {
  const char* name = "fp8bw_moe_combine_dweights";
  if (!dout || !y || !row_of || !dweights)
    return fail(FP8BW_ERR_NULL, "%s: dout, y, row_of and dweights must be non-NULL", name);
  if (!rows_dims_ok(M, top_k, P, C, 8)) return fail(FP8BW_ERR_SHAPE, kRowsShape, name, 8);
  if (!all_aligned({dout, y, row_of, dweights}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (any_overlap({{dweights, M * top_k * 4}}, {{dout, M * C * 2}, {y, P * C * 2}, {row_of, M * top_k * 4}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: dweights overlaps an input", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  const MoeCombineArgs a{y, nullptr, row_of, nullptr, M, top_k, P, C, nullptr, dout, dweights, d->error_word};
  return launched(launch_moe_combine_dweights(a, as_stream(stream)), name);
}

// ============================================================ gated activation

static bool swiglu_dims_ok(int64_t R, int64_t F) { return dim_ok(R, 32) && dim_ok(F, 32) && F <= (int64_t{1} << 21); }

FP8BW_API int mxfp8_swiglu(const fp8bw_bf16* h, int64_t R, int64_t F, uint8_t* aq, uint8_t* ae, uint8_t* aqT,
                           uint8_t* aeT, uint8_t* hq, uint8_t* he, int mode, void* stream) {
  const char* name = "mxfp8_swiglu";
  if (!h || !aq || !ae || (aqT == nullptr) != (aeT == nullptr) || (hq == nullptr) != (he == nullptr))
    return fail(FP8BW_ERR_NULL, "%s: h, aq and ae must be non-NULL, aqT and aeT, and hq and he, both set or both NULL",
                name);
  if (!swiglu_dims_ok(R, F))
    return fail(FP8BW_ERR_SHAPE, "%s: R=%lld and F=%lld must be positive multiples of 32, F up to 2^21", name,
                (long long)R, (long long)F);
  if (!all_aligned({h, aq, ae, aqT, aeT, hq, he}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (!mode_ok(mode)) return fail(FP8BW_ERR_ARG, "%s: mode %d is neither RCEIL (0) nor FLOOR (1)", name, mode);
  const int64_t n = R * F;
  if (any_overlap({{aq, n}, {ae, n / 32}, {aqT, n}, {aeT, n / 32}, {hq, 2 * n}, {he, n / 16}}, {{h, 4 * n}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: outputs overlap the input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  return launched(launch_swiglu(SwigluArgs{h, R, F, aq, ae, aqT, aeT, hq, he, mode}, as_stream(stream)), name);
}

FP8BW_API int mxfp8_swiglu_bwd(const fp8bw_bf16* da, const uint8_t* hq, const uint8_t* he, int64_t R, int64_t F,
                               uint8_t* dq, uint8_t* de, uint8_t* dqT, uint8_t* deT, int mode, void* stream) {
  const char* name = "mxfp8_swiglu_bwd";
  if (!da || !hq || !he || !dq || !de || !dqT || !deT)
    return fail(FP8BW_ERR_NULL, "%s: every pointer must be non-NULL", name);
  if (!swiglu_dims_ok(R, F))
    return fail(FP8BW_ERR_SHAPE, "%s: R=%lld and F=%lld must be positive multiples of 32, F up to 2^21", name,
                (long long)R, (long long)F);
  if (!all_aligned({da, hq, he, dq, de, dqT, deT}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (!mode_ok(mode)) return fail(FP8BW_ERR_ARG, "%s: mode %d is neither RCEIL (0) nor FLOOR (1)", name, mode);
  const int64_t n = R * F;
  if (any_overlap({{dq, 2 * n}, {de, n / 16}, {dqT, 2 * n}, {deT, n / 16}}, {{da, 2 * n}, {hq, 2 * n}, {he, n / 16}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: outputs overlap an input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  return launched(launch_swiglu_bwd(SwigluBwdArgs{da, hq, he, R, F, dq, de, dqT, deT, mode, d->num_sms}, as_stream(stream)), name);
}
