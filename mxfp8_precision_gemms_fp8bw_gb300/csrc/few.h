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
  int most;    // tokens of a slot, at most
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
// Loads that stay behind a wait for the kernel before: the compiler moves none of these, as it may plain loads of what it
// takes for constant.
__device__ __forceinline__ uint32_t load_after(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_after(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 load_after(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ FewPlan few_header(const FewPlan* p) {
  const uint2 v = load_after(reinterpret_cast<const uint2*>(p));
  return FewPlan{static_cast<int>(v.x), static_cast<int>(v.y)};
}
__device__ __forceinline__ FewSlot few_slot(const FewPlan* p, int choices, int i) {
  const uint4 v = load_after(reinterpret_cast<const uint4*>(few_slots(p, choices) + i));
  return FewSlot{static_cast<int>(v.x), static_cast<int>(v.y), v.z, static_cast<int>(v.w)};
}

// Values as the products read them (few_tokens.cuh): a record for every chunk of 128 of the contraction, of `rows` rows of
// e4m3 codes, 128 bytes each and already in the order of 128-byte swizzling, and their scales in the layout of tcgen05.cp, 512
// bytes for 128 rows.  A stage of the products takes a record as it is.
// Tokens come in two parts, rows 2 t and 2 t + 1 of the batch's records; activations in five, rows 5 i .. of the records of an
// expert's slot, which has a record for every chunk.
constexpr int kTokenParts = 2, kActParts = 5;
__host__ __device__ constexpr int64_t few_scale_bytes(int64_t rows) { return (rows + 127) / 128 * 512; }
__host__ __device__ inline int64_t few_record(int64_t rows) { return rows * 128 + few_scale_bytes(rows); }
__host__ __device__ inline int64_t few_chunks(int64_t K) { return (K + 127) / 128; }
inline int64_t few_tokens_bytes(int64_t M, int64_t K) { return few_chunks(K) * few_record(M * kTokenParts); }
// Where the records of a slot begin that has `start` choices before it.
__host__ __device__ inline int64_t few_act_at(int64_t slot, int64_t start, int64_t chunks) {
  return chunks * (start * kActParts * 128 + slot * few_scale_bytes(kFewTokens * kActParts));
}
inline int64_t few_act_bytes(int64_t choices, int64_t slots, int64_t F) { return few_act_at(slots, choices, few_chunks(F)); }

cudaError_t launch_few_route(const FewMoeArgs& a, FewPlan* plan, uint8_t* tokens, cudaStream_t st);

}  // namespace fp8bw
