// What the files of the C ABI share: error codes and messages, the per-device
// state and the argument checks.  Defined in api.cu unless inline.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fp8bw.h"
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

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace fp8bw
