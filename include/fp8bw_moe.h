/*
 * fp8bw_moe.h -- C ABI of libfp8bw.so, second part: the operators around the
 * grouped GEMMs of an MXFP8 mixture-of-experts layer (fp8bw.h has the GEMMs
 * and the quantizers, and the conventions, status codes and MX modes that
 * hold here too).
 *
 * A layer of E experts runs, for M tokens of C features with k choices each:
 *
 *   fp8bw_moe_route            router logits       -> experts, weights
 *   fp8bw_moe_plan             experts             -> group_end, row_of, src_of
 *   mxfp8_moe_gather_quant     tokens              -> MX rows of the experts
 *   mxfp8_grouped_gemm (FWD)   MX rows, W1         -> h = [gate | up]
 *   mxfp8_swiglu               h                   -> MX rows of a, h in 8 bits
 *   mxfp8_grouped_gemm (FWD)   MX rows of a, W2    -> y
 *   fp8bw_moe_combine          y, weights          -> tokens
 *
 * and, backward, mxfp8_moe_gather_quant with the weights (the gradient of y),
 * fp8bw_moe_combine_dweights, mxfp8_swiglu_bwd, fp8bw_moe_combine without
 * weights (the gradient of the tokens) and fp8bw_moe_route_bwd, with the
 * DGRAD and WGRAD grouped GEMMs between them.
 *
 * Arguments are checked in the order of fp8bw.h.  Indices that the kernels
 * read from device memory (experts, row_of, src_of) are checked there: one
 * outside its range is skipped as if it were -1 and raises FP8BW_ERR_SHAPE
 * through fp8bw_sync_status.  No result depends on the order in which blocks
 * run: equal inputs give equal bits.
 */
#ifndef FP8BW_MOE_H
#define FP8BW_MOE_H

#include "fp8bw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Routing.
 * ------------------------------------------------------------------------- */

enum fp8bw_logits_type { FP8BW_LOGITS_F32 = 0, FP8BW_LOGITS_BF16 = 1 };
enum fp8bw_moe_score { FP8BW_SCORE_SOFTMAX = 0, FP8BW_SCORE_SIGMOID = 1 };

#define FP8BW_MOE_MAX_EXPERTS 1024
#define FP8BW_MOE_MAX_TOP_K 32
#define FP8BW_MOE_MAX_GROUPS 32

/* The top_k experts of each token and their weights, all in fp32:
 *   s_e   = softmax(logits)_e or 1 / (1 + exp(-logits_e))
 *   key_e = s_e + bias_e (s_e without a bias); an expert whose logit or bias
 *           is -inf is masked and never chosen.  The bias only chooses: it is
 *           not part of the weights and has no gradient.
 *   groups > 1: the experts form `groups` runs of E / groups.  A run's score
 *           is the sum of the group_top (1 or 2) largest keys of its unmasked
 *           experts, held at the lowest finite value where it is below that;
 *           only the experts of the groups_kept best runs remain.
 *   The top_k largest keys are chosen, largest first; of equal keys the
 *   lowest index is first, and so it is for runs.  A NaN key counts as larger
 *   than every number, so that it shows up in the weights.
 *   weights_j = scale * s_j / (sum of the chosen s + 1e-20) with renorm != 0,
 *               scale * s_j without.
 * Where fewer than top_k experts are left, the remaining entries are expert
 * -1 with weight 0; a token whose logits are all -inf gets nothing but those.
 * The softmax denominator is summed by halves (x[i] + x[i + n/2], and so on),
 * so the keys do not depend on how the kernel splits a row.
 *   logits  : fp32 or bf16 [M, E]      bias    : fp32 [E] or NULL
 *   experts : int32 [M, top_k]         weights : fp32 [M, top_k]
 * 1 <= E <= 1024, 1 <= top_k <= min(E, 32), groups <= 32 divides E, 1 <=
 * groups_kept <= groups, top_k <= groups_kept * E / groups. */
int fp8bw_moe_route(const void* logits, int logits_type, const float* bias, int64_t M, int64_t E, int64_t top_k,
                    int64_t groups, int64_t groups_kept, int64_t group_top, int score, int renorm, float scale,
                    int32_t* experts, float* weights, void* stream);

/* Gradient of the logits from that of the weights.  With D the sum of the
 * chosen s + 1e-20:
 *   ds_j = (scale * dw_j - sum_i scale * dw_i * s_i / D) / D   (renorm), or scale * dw_j
 *   dlogits_e = s_e * (ds_e - sum_i ds_i s_i)   (softmax; ds_e = 0 where e was not chosen)
 *   dlogits_e = s_e * (1 - s_e) * ds_e          (sigmoid)
 * The scores are computed again from the logits.  The chosen experts of a
 * token are distinct, as fp8bw_moe_route gives them.  Arguments as there;
 *   dweights : fp32 [M, top_k]   dlogits : [M, E] of the logits' type. */
int fp8bw_moe_route_bwd(const float* dweights, const void* logits, int logits_type, const int32_t* experts, int64_t M,
                        int64_t E, int64_t top_k, int score, int renorm, float scale, void* dlogits, void* stream);

/* ---------------------------------------------------------------------------
 * Rows of the experts.
 * ------------------------------------------------------------------------- */

/* Rows that hold any choice of M * top_k entries over E experts with every
 * group padded to whole 32-row blocks: M * top_k + 31 * min(E, M * top_k),
 * rounded down to a multiple of 32 and at least 32.  0 for invalid dims.
 * Host-only. */
int64_t fp8bw_moe_plan_rows(int64_t M, int64_t E, int64_t top_k);

/* Bytes of workspace fp8bw_moe_plan needs for these dims: 0 for few entries
 * (and for invalid dims).  Host-only. */
size_t fp8bw_moe_plan_workspace_bytes(int64_t M, int64_t E, int64_t top_k);

/* Sorts the entries (token t, choice j), numbered t * top_k + j, by expert.
 * Group e owns the rows [group_end[e - 1], group_end[e]); its entries take the
 * first of them in the order of their numbers, and the rest, up to the next
 * multiple of 32, are empty.  The last group also owns the empty rows up to P,
 * so that group_end[E - 1] = P, as the grouped GEMM wants, without the host
 * knowing the counts.  Entries of expert -1 get no row.
 *   experts   : int32 [M, top_k], each in [-1, E)
 *   group_end : int32 [E]   counts : int32 [E], entries per expert
 *   row_of    : int32 [M, top_k], the entry's row or -1
 *   src_of    : int32 [P], the row's entry or -1 (an empty row)
 * P: a multiple of 32, at least fp8bw_moe_plan_rows(M, E, top_k).
 * workspace: caller-owned DEVICE scratch of at least
 * fp8bw_moe_plan_workspace_bytes bytes, NULL where that is 0; concurrent calls
 * need one each. */
int fp8bw_moe_plan(const int32_t* experts, int64_t M, int64_t E, int64_t top_k, int64_t P, int32_t* group_end,
                   int32_t* counts, int32_t* row_of, int32_t* src_of, void* workspace, size_t workspace_bytes,
                   void* stream);

/* The MX quantizations of v[P, C] without writing v: with entry s = src_of[p],
 *   v_p = x[s / top_k]                                (weights NULL)
 *   v_p = fl32(weights[s] * x[s / top_k])             (weights given)
 *   v_p = 0                                           (s = -1)
 * Without weights these are the rows that the experts read; with the weights
 * and x the gradient of fp8bw_moe_combine's output, the gradient of its y.
 * The codes are those of the MX rule of fp8bw.h applied to v in fp32.  A NaN
 * becomes the e4m3 NaN; an infinity or a NaN takes its block's scale to the
 * largest one.
 *   x       : bf16 [M, C]              weights : fp32 [M, top_k] or NULL
 *   q       : e4m3 [P, C]              e8      : E8M0 [P][C/32]
 *   qT      : e4m3 [C, P]              e8T     : E8M0 [C][P/32]   (both or neither NULL)
 * P and C positive multiples of 32. */
int mxfp8_moe_gather_quant(const fp8bw_bf16* x, const float* weights, const int32_t* src_of, int64_t M, int64_t top_k,
                           int64_t P, int64_t C, uint8_t* q, uint8_t* e8, uint8_t* qT, uint8_t* e8T, int mode,
                           void* stream);

/* out[t] = base[t] + sum over j of weights[t, j] * y[row_of[t, j]], in fp32 in
 * the order of j, rounded once to bf16.  Entries without a row add nothing,
 * whatever their weight.  Without weights (NULL) each counts once: the
 * gradient of the tokens from that of the experts' rows.
 *   y    : bf16 [P, C]     weights : fp32 [M, top_k] or NULL
 *   base : bf16 [M, C] or NULL (may be out itself)     out : bf16 [M, C]
 * C a positive multiple of 8. */
int fp8bw_moe_combine(const fp8bw_bf16* y, const float* weights, const int32_t* row_of, const fp8bw_bf16* base,
                      int64_t M, int64_t top_k, int64_t P, int64_t C, fp8bw_bf16* out, void* stream);

/* dweights[t, j] = sum over c of dout[t, c] * y[row_of[t, j], c] in fp32, 0
 * where the entry has no row.  dout : bf16 [M, C]; dweights : fp32 [M, top_k];
 * other arguments as fp8bw_moe_combine. */
int fp8bw_moe_combine_dweights(const fp8bw_bf16* dout, const fp8bw_bf16* y, const int32_t* row_of, int64_t M,
                               int64_t top_k, int64_t P, int64_t C, float* dweights, void* stream);

/* ---------------------------------------------------------------------------
 * Gated activation with its input kept in 8 bits.
 * ------------------------------------------------------------------------- */

/* a = gate * sigmoid(gate) * up of h = [gate | up], in fp32, held as MX codes;
 * and h itself as rowwise MX codes, which are all that the backward pass needs
 * of it (33/32 bytes per element instead of the 2 of bf16).
 * Where 1 + exp(-gate) is over fp32 (gates below -88.7) the sigmoid is 0.
 *   h  : bf16 [R, 2F]
 *   aq : e4m3 [R, F]   ae : E8M0 [R][F/32]
 *   aqT: e4m3 [F, R]   aeT: E8M0 [F][R/32]    (both or neither NULL)
 *   hq : e4m3 [R, 2F]  he : E8M0 [R][2F/32]   (both or neither NULL)
 * R and F positive multiples of 32. */
int mxfp8_swiglu(const fp8bw_bf16* h, int64_t R, int64_t F, uint8_t* aq, uint8_t* ae, uint8_t* aqT, uint8_t* aeT,
                 uint8_t* hq, uint8_t* he, int mode, void* stream);

/* The gradient of h as MX codes, both layouts, from da and the kept codes.
 * With gate and up the values of hq, he and sig = sigmoid(gate), in fp32:
 *   d gate = da * up * sig * (1 + gate * (1 - sig)),   d up = da * gate * sig
 *   da : bf16 [R, F]
 *   dq : e4m3 [R, 2F]  de : E8M0 [R][2F/32]   dqT : e4m3 [2F, R]  deT : E8M0 [2F][R/32]
 * R and F positive multiples of 32. */
int mxfp8_swiglu_bwd(const fp8bw_bf16* da, const uint8_t* hq, const uint8_t* he, int64_t R, int64_t F, uint8_t* dq,
                     uint8_t* de, uint8_t* dqT, uint8_t* deT, int mode, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BW_MOE_H */
