/*
 * fp8bw_few.h -- C ABI of libfp8bw.so, third part: answering a few tokens with
 * weights held in MX codes, 4 or 8 bits (fp8bw.h has the conventions, status
 * codes and MX modes that hold here too, fp8bw_moe.h the routing).
 *
 * An MX weight matrix W[R, C] is its codes and E8M0 bytes e8[R][C/32]:
 *   W[r, c] = value(code[r, c]) * 2^(e8[r][c / 32] - 127)
 * with, for bits = 8, e4m3 codes [R, C] (as mxfp8_quant_1x32_row writes them),
 * and, for bits = 4, e2m1 codes [R, C/2], two to a byte, the lower nibble
 * first: bit 3 the sign, codes 0 to 7 the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4
 * and 6.  An E8M0 byte of 255 makes its block NaN.
 *
 * Products read a token as the sum of two MXFP8 numbers: that is the bf16 value
 * itself down to 2^-12 of the largest element of its block of 32, and off by at
 * most 2^-21 of that largest below that; weights are what their codes stand for, sums run in fp32, and the
 * result is rounded once to bf16.  (The grouped GEMM of fp8bw.h reads tokens
 * that are rounded to MXFP8 once.)  A token with an infinity or a NaN gives
 * NaN (of a layer whose bias leaves no expert, zeros as of any token).  No result
 * depends on the order in which blocks run.
 */
#ifndef FP8BW_FEW_H
#define FP8BW_FEW_H

#include "fp8bw.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FP8BW_FEW_TOKENS 32

/* MXFP4 codes of w, blocks of 32 along C: E is the smallest with
 * 6 * 2^E >= amax (FP8BW_MX_RCEIL), or floor(log2 amax) - 2 (FP8BW_MX_FLOOR),
 * clamped to [-127, 127]; codes are e2m1 of w * 2^-E, to the nearest, ties to
 * even, saturating at 6.  A block with an infinity or a NaN gets byte 255.
 *   w : bf16 [R, C]    q : e2m1 [R, C/2]    e8 : E8M0 [R][C/32]
 * C a positive multiple of 32. */
int mxfp4_quant_1x32_row(const fp8bw_bf16* w, int64_t R, int64_t C, uint8_t* q, uint8_t* e8, int mode, void* stream);

/* The same values as e4m3 codes, which with the same E8M0 bytes are an MXFP8
 * matrix: every e2m1 value is an e4m3 value.
 *   q4 : e2m1 [R, C/2]    q8 : e4m3 [R, C]      C a positive multiple of 32. */
int mxfp4_to_mxfp8(const uint8_t* q4, int64_t R, int64_t C, uint8_t* q8, void* stream);

/* Bytes of workspace mx_few_linear needs: 0 for one or two tokens and a matrix
 * that is not large, and for invalid dims.  Host-only. */
size_t mx_few_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* y = x W^T.
 *   x : bf16 [M, K]    w : codes of W[N, K]    e8 : E8M0 [N][K/32]    y : bf16 [M, N]
 * 1 <= M <= 32, N positive, K a positive multiple of 32, bits 4 or 8.
 * workspace: caller-owned DEVICE scratch of at least
 * mx_few_linear_workspace_bytes bytes, in any state, NULL where that is 0;
 * concurrent calls need one each. */
int mx_few_linear(const fp8bw_bf16* x, const uint8_t* w, const uint8_t* e8, int bits, int64_t M, int64_t N, int64_t K,
                  fp8bw_bf16* y, void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace mx_few_moe needs; 0 for invalid dims.  Host-only. */
size_t mx_few_moe_workspace_bytes(int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F);

/* A mixture-of-experts layer of gated feed-forward experts on M tokens:
 *   logits = x router^T (fp32);  experts e_j, weights w_j: fp8bw_moe_route's of them
 *   [gate; up] = W13[e_j] x;  a_j = gate * sigmoid(gate) * up;  y = sum_j w_j W2[e_j] a_j
 * A choice without an expert adds nothing.  h = [gate; up] stays fp32, and so
 * does the activation between the two products, down to 2^-12 of the largest
 * of its block of 32 (below that it is off by at most 2^-36 of that largest);
 * one that leaves fp32 gives NaN.
 *   x   : bf16 [M, C]           router : fp32 [E, C]      bias : fp32 [E] or NULL
 *   w13 : codes of [E, 2F, C]   e13    : E8M0 [E][2F][C/32]
 *   w2  : codes of [E, C, F]    e2     : E8M0 [E][C][F/32]     y : bf16 [M, C]
 * 1 <= M <= 32, C and F positive multiples of 32, bits 4 or 8, and the routing's arguments as in fp8bw_moe.h.
 * workspace: caller-owned DEVICE scratch of at least mx_few_moe_workspace_bytes bytes, in any state; concurrent calls
 * need one each. */
int mx_few_moe(const fp8bw_bf16* x, const float* router, const float* bias, const uint8_t* w13, const uint8_t* e13,
               const uint8_t* w2, const uint8_t* e2, int bits, int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F,
               int64_t groups, int64_t groups_kept, int64_t group_top, int score, int renorm, float scale, fp8bw_bf16* y,
               void* workspace, size_t workspace_bytes, void* stream);

/* How the two calls divide their products on the current device, for tests and
 * profiles (codes aligned to 32 bytes).  Of a product, six numbers: blocks of a
 * cluster, which share the contraction; stages of a block's pipeline, at least;
 * chunks of 128 of the contraction that a block walks through, at most (past its
 * stages it fills them again); and whether blocks take whole tiles in turn, hold
 * the tokens themselves, and have warps spread the 4-bit codes (0 or 1).  slices:
 * warps of a block that share the features of 16 experts in the router's logits. */
int mx_few_linear_shape(int64_t M, int64_t N, int64_t K, int bits, int32_t* product);
int mx_few_moe_shape(int64_t M, int64_t E, int64_t top_k, int64_t C, int64_t F, int bits, int32_t* up, int32_t* down,
                     int32_t* slices);

/* mx_few_linear and mx_few_moe whose kernels wait for no longer than wait_ns at
 * a time inside a block (0: not at all; 2,000,000,000 as the calls themselves
 * do).  Where that runs out the kernels give up, their copies land, FP8BW_ERR_TIMEOUT
 * is recorded in the error word and y means nothing: a test sees what becomes of
 * a wait that expires, without a fault.  The calls after it are not affected. */
int fp8bw_selftest_few_linear(const fp8bw_bf16* x, const uint8_t* w, const uint8_t* e8, int bits, int64_t M, int64_t N,
                              int64_t K, fp8bw_bf16* y, void* workspace, size_t workspace_bytes, uint32_t wait_ns,
                              void* stream);
int fp8bw_selftest_few_moe(const fp8bw_bf16* x, const float* router, const float* bias, const uint8_t* w13,
                           const uint8_t* e13, const uint8_t* w2, const uint8_t* e2, int bits, int64_t M, int64_t E,
                           int64_t top_k, int64_t C, int64_t F, int64_t groups, int64_t groups_kept, int64_t group_top,
                           int score, int renorm, float scale, fp8bw_bf16* y, void* workspace, size_t workspace_bytes,
                           uint32_t wait_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BW_FEW_H */
