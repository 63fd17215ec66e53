// Division of the routing scores, shared by moe_route.cu and its check in
// tests/cuda/.
#pragma once

#include <cuda_runtime.h>

namespace fp8bw {

// fl32(a / b) for inv = fl32(1 / b): Markstein's correction step.  With q =
// RN(a * inv) within an ulp of the quotient, the remainder a - q * b is exact
// in one FMA and RN(q + remainder * inv) is the correctly rounded quotient.
// It needs a remainder that does not fall below the fp32 range: a zero or at
// least kShortDivisionMin in magnitude (the remainder is a multiple of 2^-48 a
// or so), with b in [1, 1024] as the sums of exponentials here are.  Checked
// against the IEEE division in tests/cuda/route_division.cu.
constexpr float kShortDivisionMin = 7.8886091e-31f;  // 2^-100

__device__ __forceinline__ float div_by(float a, float b, float inv) {
  const float q = __fmul_rn(a, inv);
  return __fmaf_rn(__fmaf_rn(-q, b, a), inv, q);
}

}  // namespace fp8bw
