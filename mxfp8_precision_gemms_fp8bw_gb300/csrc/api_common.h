// What the files of the C ABI share: error codes and messages, the per-device
// state and the argument checks.  Defined in api.cu unless inline.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "fp8bw.h"
#include "fp8bw_moe.h"
#include "launch.h"

#define FP8BW_API extern "C" __attribute__((visibility("default")))

namespace fp8bw {

struct DeviceState {
  bool probed = false;
  bool supported = false;
  int num_sms = 0;
  int* error_word = nullptr;
  char why[160] = {0};
};

// Sets the calling thread's message and returns `code`; ok() clears it.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

// Checks (once per device) that the current device is compute capability
// 10.3 and resolves the address of its error word.
int current_device(DeviceState** out);

// The call's return code from its launch status.
int launched(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;

inline bool dim_ok(int64_t d, int64_t mult) { return d > 0 && d <= kMaxDim && d % mult == 0; }

inline bool overlaps(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

// A memory range of a call: outputs may overlap nothing.
struct Range {
  const void* p;
  int64_t bytes;
};

inline bool any_overlap(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range* a = outs.begin(); a != outs.end(); ++a) {
    if (a->p == nullptr) continue;
    for (const Range& b : ins)
      if (b.p != nullptr && overlaps(a->p, a->bytes, b.p, b.bytes)) return true;
    for (const Range* b = a + 1; b != outs.end(); ++b)
      if (b->p != nullptr && overlaps(a->p, a->bytes, b->p, b->bytes)) return true;
  }
  return false;
}

inline bool all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return false;
  return true;
}

inline bool mode_ok(int mode) { return mode == FP8BW_MX_RCEIL || mode == FP8BW_MX_FLOOR; }

inline bool choices_ok(int64_t M, int64_t E, int64_t top_k) {
  return dim_ok(M, 1) && dim_ok(E, 1) && E <= FP8BW_MOE_MAX_EXPERTS && dim_ok(top_k, 1) &&
         top_k <= FP8BW_MOE_MAX_TOP_K && top_k <= E;
}

inline bool groups_ok(int64_t E, int64_t top_k, int64_t groups, int64_t kept) {
  return groups >= 1 && groups <= FP8BW_MOE_MAX_GROUPS && E % groups == 0 && kept >= 1 && kept <= groups &&
         top_k <= kept * (E / groups);
}

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace fp8bw
