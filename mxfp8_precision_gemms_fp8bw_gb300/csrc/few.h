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

// Where the activation's records of a slot begin: a record of n tokens is at most 80 n bytes.
__host__ __device__ inline int64_t few_act_at(int64_t start, int64_t F) { return start * 80 * (F / 32); }

// Tokens as the products read them: f16 [M, K] under a power of two for each token, the elements of each 32 in the order
// of few::place_of.
struct FewTokens {
  uint8_t* rows;
  float* scales;
};
inline int64_t few_tokens_bytes(int64_t M, int64_t K) { return (M * K * 2 + 255) / 256 * 256 + 256; }
inline FewTokens few_tokens_at(void* p, int64_t M, int64_t K) {
  uint8_t* at = static_cast<uint8_t*>(p);
  return FewTokens{at + 256, reinterpret_cast<float*>(at)};
}

cudaError_t launch_few_route(const FewMoeArgs& a, FewPlan* plan, const FewTokens& tokens, cudaStream_t st);

}  // namespace fp8bw
