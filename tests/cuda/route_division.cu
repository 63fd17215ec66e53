// Check that the short division of the routing scores (one Markstein
// correction from the rounded reciprocal) equals the IEEE division: every
// significand of the dividend against 24576 divisors -- the 4096 smallest and
// the 4096 largest significands and 16384 scattered ones -- at the smallest
// dividend it is used for and at 1, and over the divisors' exponents.  Prints
// "checked <pairs> mismatches <n>".
#include <cstdint>
#include <cstdio>

#include "route_math.cuh"

using namespace fp8bw;

constexpr unsigned kDivisors = 24576;

__global__ void check(unsigned long long* out) {
  const uint32_t i = blockIdx.x;
  uint32_t m = i < 4096 ? i : i < 8192 ? 0x7FFFFFu - (i - 4096) : (i * 2654435761u >> 7) & 0x7FFFFFu;
  const float b = __uint_as_float((127u + i % 10u) << 23 | m);  // in [1, 1024)
  const float inv = __frcp_rn(b);
  // exponents -100 (kShortDivisionMin up) and -1, by turns
  const uint32_t exponent = (i & 1) ? (127u - 100u) << 23 : 126u << 23;
  unsigned long long bad = 0;
  for (uint32_t a = threadIdx.x; a < 1u << 23; a += blockDim.x) {
    const float x = __uint_as_float(exponent | a);
    bad += __float_as_uint(div_by(x, b, inv)) != __float_as_uint(__fdiv_rn(x, b));
  }
  if (threadIdx.x == 0) bad += __float_as_uint(div_by(0.f, b, inv)) != 0u;
  atomicAdd(&out[0], bad);
}

int main() {
  unsigned long long* d = nullptr;
  if (cudaMalloc(&d, sizeof(unsigned long long)) != cudaSuccess) return 2;
  cudaMemset(d, 0, sizeof(unsigned long long));
  check<<<kDivisors, 256>>>(d);
  unsigned long long bad = 0;
  const cudaError_t e = cudaMemcpy(&bad, d, sizeof(bad), cudaMemcpyDeviceToHost);
  cudaFree(d);
  if (e != cudaSuccess) {
    printf("cuda error %s\n", cudaGetErrorString(e));
    return 3;
  }
  printf("checked %llu mismatches %llu\n", static_cast<unsigned long long>(kDivisors) << 23, bad);
  return bad == 0 ? 0 : 1;
}
