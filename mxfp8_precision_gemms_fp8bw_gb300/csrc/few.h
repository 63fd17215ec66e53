// What the kernels of few.cu and few_route.cu share: the plan of a batch of a
// few tokens, in the workspace.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.h"

namespace fp8bw {

// An expert that some token chose.  Its tokens are the bits of `mask`, in
// ascending order the columns of its products; `start` is the number of
// choices of the experts before it.
struct alignas(16) FewSlot {
  int expert;
  int start;
  uint32_t mask;
  int n;
};

constexpr int kFewTokens = 32;

// The plan of a number of choices (M * top_k): this header, then each choice's weight by slot and column, then the
// slots.
struct alignas(16) FewPlan {
  int active;  // slots
};

__host__ __device__ inline int64_t few_weights_bytes(int64_t choices) { return (choices * 4 + 15) / 16 * 16; }
inline int64_t few_plan_bytes(int64_t M, int64_t top_k) {
  const int64_t n = M * top_k;
  return (static_cast<int64_t>(sizeof(FewPlan)) + few_weights_bytes(n) + n * static_cast<int64_t>(sizeof(FewSlot)) + 255) / 256 * 256;
}

__device__ __forceinline__ float* few_weights(const FewPlan* p) {
  return reinterpret_cast<float*>(const_cast<FewPlan*>(p) + 1);
}
__device__ __forceinline__ FewSlot* few_slots(const FewPlan* p, int choices) {
  return reinterpret_cast<FewSlot*>(reinterpret_cast<uint8_t*>(few_weights(p)) + few_weights_bytes(choices));
}
// Read past the first-level cache: the plan may be written by a kernel this one overlaps with the end of.
__device__ __forceinline__ int few_active(const FewPlan* p) { return __ldcg(&p->active); }
__device__ __forceinline__ FewSlot few_slot(const FewPlan* p, int choices, int i) {
  const int4 v = __ldcg(reinterpret_cast<const int4*>(few_slots(p, choices) + i));
  return FewSlot{v.x, v.y, static_cast<uint32_t>(v.z), v.w};
}

// Values as the products read them (few_tokens.cuh): for every row, `parts` rows of e4m3 codes and as many of E8M0 bytes,
// both padded to whole chunks of 128.  Tokens come in two parts, activations (a row for every choice, by slot and column) in
// three.
constexpr int kTokenParts = 2, kActParts = 3;
struct FewRows {
  uint8_t* codes;   // [rows * parts][pitch]
  uint8_t* scales;  // [rows * parts][pitch / 32]
  int64_t pitch;
};
__host__ __device__ inline int64_t few_pitch(int64_t K) { return (K + 127) / 128 * 128; }
inline int64_t few_rows_bytes(int64_t rows, int parts, int64_t K) {
  return (rows * parts * (few_pitch(K) / 32) * 33 + 255) / 256 * 256;
}
inline FewRows few_rows_at(void* p, int64_t rows, int parts, int64_t K) {
  uint8_t* at = static_cast<uint8_t*>(p);
  return FewRows{at, at + rows * parts * few_pitch(K), few_pitch(K)};
}

cudaError_t launch_few_route(const FewMoeArgs& a, FewPlan* plan, const FewRows& tokens, cudaStream_t st);

}  // namespace fp8bw
