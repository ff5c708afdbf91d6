// decay.cuh -- powers of a head's decay g, shared by the kernels of decay attention.
#pragma once

#include <cstdint>

namespace delta {
namespace decay {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// g^e for a weight that is used once, from lg = log2 g (-inf for g = 0): relative
// error about 2^-22 and that of the exponent's product
__device__ __forceinline__ float power(float lg, int e) { return e <= 0 ? 1.f : ex2(lg * (float)e); }

// g^n as a factor of the state, chunk after chunk: S -> a S + b S.  Where it is near 1
// its rounding would add up over all chunks that a state remembers, so it is split into
// 1 and g^n - 1, whose rounding is as small as it is.
struct Keep {
  float a, b;
};
__device__ __forceinline__ Keep keep_of(float lg, int64_t n) {
  if (n <= 0) return {0.f, 1.f};
  const float x = lg * (float)n, k = exp2f(x);
  return k > 0.5f ? Keep{expm1f(0.6931471805599453f * x), 1.f} : Keep{k, 0.f};
}

}  // namespace decay
}  // namespace delta
