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

// g^n as a factor of the state, chunk after chunk, a + b.  Rounded to one float32 its
// error would add up over all chunks that a state remembers (3e-8 each, many where g is
// near 1); so what a chunk's factor leaves out is owed to the next.
struct Keep {
  float a, b;
};
__device__ __forceinline__ Keep keep_of(float lg, int64_t n) {
  if (n <= 0) return {1.f, 0.f};
  const float x = lg * (float)n, k = exp2f(x);
  if (k <= 0.5f) return {k, 0.f};
  const float m = expm1f(0.6931471805599453f * x), a = 1.f + m;  // (1 - a is exact)
  return {a, (1.f - a) + m};
}
// the factor of the next chunk
__device__ __forceinline__ float keep_now(const Keep &k, float &owed) {
  owed += k.b;
  const float now = k.a + owed;
  owed -= now - k.a;
  return now;
}

}  // namespace decay
}  // namespace delta
