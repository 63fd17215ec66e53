// C ABI of libfp8bw, third part (declared in include/fp8bw_few.h): argument
// validation and dispatch of the operators on MX weights for a few tokens.
#include "api_common.h"
#include "fp8bw_few.h"

using namespace fp8bw;

namespace {

constexpr int64_t kMaxWidth = int64_t{1} << 22;  // contraction lengths and rows of an expert

constexpr uint64_t kWaitNs = 2000000000;  // legitimate waits last microseconds

bool bits_ok(int bits) { return bits == 4 || bits == 8; }

void put_shape(const FewShape& s, int32_t* out) {
  const int32_t all[6] = {s.cluster, s.stages, s.chunks, s.in_turn, s.held, s.spread};
  for (int i = 0; i < 6; ++i) out[i] = all[i];
}

bool linear_dims_ok(int64_t M, int64_t N, int64_t K) {
  return dim_ok(M, 1) && M <= FP8BW_FEW_TOKENS && dim_ok(N, 1) && dim_ok(K, 32) && K <= kMaxWidth;
}

bool layer_dims_ok(int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F) {
  return M <= FP8BW_FEW_TOKENS && choices_ok(M, E, top_k) && dim_ok(C, 32) && dim_ok(F, 32) && C <= kMaxWidth &&
         F <= kMaxWidth && E * 2 * F <= kMaxDim && E * C <= kMaxDim;  // rows are numbered in int32
}

}  // namespace

FP8BW_API int mxfp4_quant_1x32_row(const fp8bw_bf16* w, int64_t R, int64_t C, uint8_t* q, uint8_t* e8, int mode,
                                   void* stream) {
  const char* name = "mxfp4_quant_1x32_row";
  if (!w || !q || !e8) return fail(FP8BW_ERR_NULL, "%s: w, q and e8 must be non-NULL", name);
  if (!dim_ok(R, 1) || !dim_ok(C, 32))
    return fail(FP8BW_ERR_SHAPE, "%s: need 0 < R < 2^31 and C a positive multiple of 32; got R=%lld C=%lld", name,
                (long long)R, (long long)C);
  if (!all_aligned({w, q, e8})) return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (!mode_ok(mode)) return fail(FP8BW_ERR_ARG, "%s: mode %d is neither RCEIL (0) nor FLOOR (1)", name, mode);
  const int64_t n = R * C;
  if (any_overlap({{q, n / 2}, {e8, n / 32}}, {{w, 2 * n}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: outputs overlap the input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  return launched(launch_mxfp4_quant_row(w, n, q, e8, mode, d->num_sms, as_stream(stream)), name);
}

FP8BW_API int mxfp4_to_mxfp8(const uint8_t* q4, int64_t R, int64_t C, uint8_t* q8, void* stream) {
  const char* name = "mxfp4_to_mxfp8";
  if (!q4 || !q8) return fail(FP8BW_ERR_NULL, "%s: q4 and q8 must be non-NULL", name);
  if (!dim_ok(R, 1) || !dim_ok(C, 32))
    return fail(FP8BW_ERR_SHAPE, "%s: need 0 < R < 2^31 and C a positive multiple of 32; got R=%lld C=%lld", name,
                (long long)R, (long long)C);
  if (!all_aligned({q4, q8})) return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (any_overlap({{q8, R * C}}, {{q4, R * C / 2}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: q8 overlaps q4", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  return launched(launch_mxfp4_to_mxfp8(q4, R * C, q8, d->num_sms, as_stream(stream)), name);
}

namespace {

int few_linear(const char* name, const fp8bw_bf16* x, const uint8_t* w, const uint8_t* e8, int bits, int64_t M, int64_t N, int64_t K,
               fp8bw_bf16* y, void* workspace, size_t workspace_bytes, uint64_t wait_ns, void* stream) {
  if (!x || !w || !e8 || !y) return fail(FP8BW_ERR_NULL, "%s: x, w, e8 and y must be non-NULL", name);
  if (!linear_dims_ok(M, N, K))
    return fail(FP8BW_ERR_SHAPE,
                "%s: need 0 < M <= 32, 0 < N < 2^31 and K a positive multiple of 32 up to 2^22; got M=%lld N=%lld "
                "K=%lld",
                name, (long long)M, (long long)N, (long long)K);
  if (!all_aligned({x, w, e8, y, workspace})) return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (!bits_ok(bits)) return fail(FP8BW_ERR_ARG, "%s: bits %d is neither 4 nor 8", name, bits);
  const size_t need = few_linear_workspace_bytes(M, N, K);
  if (need > 0 && !workspace)
    return fail(FP8BW_ERR_NULL, "%s: these dims need a workspace of %zu bytes", name, need);
  if (workspace_bytes < need)
    return fail(FP8BW_ERR_ARG, "%s: workspace of %zu bytes is smaller than the %zu bytes these dims need", name,
                workspace_bytes, need);
  if (any_overlap({{y, M * N * 2}, {need > 0 ? workspace : nullptr, static_cast<int64_t>(need)}},
                  {{x, M * K * 2}, {w, N * (K / 8) * bits}, {e8, N * (K / 32)}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: y or the workspace overlaps an input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  return launched(launch_few_linear(FewLinearArgs{x, w, e8, bits, M, N, K, y, workspace, d->error_word, d->num_sms, wait_ns},
                                    as_stream(stream)),
                  name);
}

int few_moe(const char* name, const fp8bw_bf16* x, const float* router, const float* bias, const uint8_t* w13, const uint8_t* e13,
            const uint8_t* w2, const uint8_t* e2, int bits, int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F, int64_t groups,
            int64_t groups_kept, int64_t group_top, int score, int renorm, float scale, fp8bw_bf16* y, void* workspace,
            size_t workspace_bytes, uint64_t wait_ns, void* stream) {
  if (!x || !router || !w13 || !e13 || !w2 || !e2 || !y || !workspace)
    return fail(FP8BW_ERR_NULL, "%s: every pointer but bias must be non-NULL", name);
  if (!layer_dims_ok(M, E, top_k, C, F))
    return fail(FP8BW_ERR_SHAPE,
                "%s: need 0 < M <= 32, 0 < E <= 1024, 0 < top_k <= min(E, 32), C and F positive multiples of 32 up to "
                "2^22, E * 2F and E * C under 2^31; got M=%lld E=%lld top_k=%lld C=%lld F=%lld",
                name, (long long)M, (long long)E, (long long)top_k, (long long)C, (long long)F);
  if (!groups_ok(E, top_k, groups, groups_kept))
    return fail(FP8BW_ERR_SHAPE,
                "%s: groups (%lld) must be 1 to 32 and divide E, groups_kept (%lld) 1 to groups, and top_k at most the "
                "experts of the kept groups",
                name, (long long)groups, (long long)groups_kept);
  if (!all_aligned({x, router, bias, w13, e13, w2, e2, y, workspace}))
    return fail(FP8BW_ERR_ALIGN, "%s: pointers must be 16-byte aligned", name);
  if (!bits_ok(bits)) return fail(FP8BW_ERR_ARG, "%s: bits %d is neither 4 nor 8", name, bits);
  if (score != FP8BW_SCORE_SOFTMAX && score != FP8BW_SCORE_SIGMOID)
    return fail(FP8BW_ERR_ARG, "%s: score %d is neither SOFTMAX (0) nor SIGMOID (1)", name, score);
  if (group_top != 1 && group_top != 2)
    return fail(FP8BW_ERR_ARG, "%s: group_top %lld is neither 1 nor 2", name, (long long)group_top);
  const size_t need = few_moe_workspace_bytes(M, E, top_k, C, F);
  if (workspace_bytes < need)
    return fail(FP8BW_ERR_ARG, "%s: workspace of %zu bytes is smaller than the %zu bytes these dims need", name,
                workspace_bytes, need);
  const int64_t n = E * F * (C / 32);  // blocks of w2; w13 has twice as many
  if (any_overlap({{y, M * C * 2}, {workspace, static_cast<int64_t>(need)}},
                  {{x, M * C * 2}, {router, E * C * 4}, {bias, E * 4}, {w13, n * 8 * bits}, {e13, 2 * n},
                   {w2, n * 4 * bits}, {e2, n}}))
    return fail(FP8BW_ERR_LAYOUT, "%s: y or the workspace overlaps an input or each other", name);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  FewMoeArgs a{};
  a.x = x;
  a.router = router;
  a.w13 = w13;
  a.e13 = e13;
  a.w2 = w2;
  a.e2 = e2;
  a.bits = bits;
  a.C = C;
  a.F = F;
  a.route.bias = bias;
  a.route.M = M;
  a.route.E = E;
  a.route.top_k = top_k;
  a.route.groups = groups;
  a.route.groups_kept = groups_kept;
  a.route.group_top = group_top;
  a.route.score = score;
  a.route.renorm = renorm;
  a.route.scale = scale;
  a.route.status = d->error_word;
  a.y = y;
  a.workspace = workspace;
  a.num_sms = d->num_sms;
  a.wait_ns = wait_ns;
  return launched(launch_few_moe(a, as_stream(stream)), name);
}

}  // namespace

FP8BW_API size_t mx_few_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return linear_dims_ok(M, N, K) ? few_linear_workspace_bytes(M, N, K) : 0;
}

FP8BW_API int mx_few_linear(const fp8bw_bf16* x, const uint8_t* w, const uint8_t* e8, int bits, int64_t M, int64_t N,
                            int64_t K, fp8bw_bf16* y, void* workspace, size_t workspace_bytes, void* stream) {
  return few_linear("mx_few_linear", x, w, e8, bits, M, N, K, y, workspace, workspace_bytes, kWaitNs, stream);
}

FP8BW_API size_t mx_few_moe_workspace_bytes(int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F) {
  return layer_dims_ok(M, E, top_k, C, F) ? few_moe_workspace_bytes(M, E, top_k, C, F) : 0;
}

FP8BW_API int mx_few_moe(const fp8bw_bf16* x, const float* router, const float* bias, const uint8_t* w13,
                         const uint8_t* e13, const uint8_t* w2, const uint8_t* e2, int bits, int64_t M, int64_t E,
                         int64_t top_k, int64_t C, int64_t F, int64_t groups, int64_t groups_kept, int64_t group_top,
                         int score, int renorm, float scale, fp8bw_bf16* y, void* workspace, size_t workspace_bytes,
                         void* stream) {
  return few_moe("mx_few_moe", x, router, bias, w13, e13, w2, e2, bits, M, E, top_k, C, F, groups, groups_kept, group_top, score, renorm,
                 scale, y, workspace, workspace_bytes, kWaitNs, stream);
}

FP8BW_API int fp8bw_selftest_few_linear(const fp8bw_bf16* x, const uint8_t* w, const uint8_t* e8, int bits, int64_t M, int64_t N,
                                        int64_t K, fp8bw_bf16* y, void* workspace, size_t workspace_bytes, uint32_t wait_ns,
                                        void* stream) {
  const char* name = "fp8bw_selftest_few_linear";
  if (wait_ns > kWaitNs) return fail(FP8BW_ERR_ARG, "%s: wait_ns=%u is over 2000000000", name, wait_ns);
  return few_linear(name, x, w, e8, bits, M, N, K, y, workspace, workspace_bytes, wait_ns, stream);
}

FP8BW_API int fp8bw_selftest_few_moe(const fp8bw_bf16* x, const float* router, const float* bias, const uint8_t* w13,
                                     const uint8_t* e13, const uint8_t* w2, const uint8_t* e2, int bits, int64_t M, int64_t E,
                                     int64_t top_k, int64_t C, int64_t F, int64_t groups, int64_t groups_kept, int64_t group_top,
                                     int score, int renorm, float scale, fp8bw_bf16* y, void* workspace, size_t workspace_bytes,
                                     uint32_t wait_ns, void* stream) {
  const char* name = "fp8bw_selftest_few_moe";
  if (wait_ns > kWaitNs) return fail(FP8BW_ERR_ARG, "%s: wait_ns=%u is over 2000000000", name, wait_ns);
  return few_moe(name, x, router, bias, w13, e13, w2, e2, bits, M, E, top_k, C, F, groups, groups_kept, group_top, score, renorm, scale,
                 y, workspace, workspace_bytes, wait_ns, stream);
}

FP8BW_API int mx_few_linear_shape(int64_t M, int64_t N, int64_t K, int bits, int32_t* product) {
  const char* name = "mx_few_linear_shape";
  if (!product) return fail(FP8BW_ERR_NULL, "%s: product must be non-NULL", name);
  if (!linear_dims_ok(M, N, K)) return fail(FP8BW_ERR_SHAPE, "%s: dims that mx_few_linear refuses", name);
  if (!bits_ok(bits)) return fail(FP8BW_ERR_ARG, "%s: bits %d is neither 4 nor 8", name, bits);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  FewLinearArgs a{};
  a.bits = bits;
  a.M = M;
  a.N = N;
  a.K = K;
  a.num_sms = d->num_sms;
  a.x = reinterpret_cast<const uint16_t*>(kMaxWidth);  // some address: nothing is read
  FewShape shape{};
  const int rc = launched(launch_few_linear(a, nullptr, &shape), name);
  put_shape(shape, product);
  return rc;
}

FP8BW_API int mx_few_moe_shape(int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F, int bits, int32_t* up, int32_t* down,
                               int32_t* slices) {
  const char* name = "mx_few_moe_shape";
  if (!up || !down || !slices) return fail(FP8BW_ERR_NULL, "%s: up, down and slices must be non-NULL", name);
  if (!layer_dims_ok(M, E, top_k, C, F)) return fail(FP8BW_ERR_SHAPE, "%s: dims that mx_few_moe refuses", name);
  if (!bits_ok(bits)) return fail(FP8BW_ERR_ARG, "%s: bits %d is neither 4 nor 8", name, bits);
  DeviceState* d;
  if (int rc = current_device(&d)) return rc;
  FewMoeArgs a{};
  a.bits = bits;
  a.C = C;
  a.F = F;
  a.route.M = M;
  a.route.E = E;
  a.route.top_k = top_k;
  a.num_sms = d->num_sms;
  FewShape of_up{}, of_down{};
  const int rc = launched(launch_few_moe(a, nullptr, &of_up, &of_down), name);
  put_shape(of_up, up);
  put_shape(of_down, down);
  *slices = few_route_slices(E, C);
  return rc;
}
