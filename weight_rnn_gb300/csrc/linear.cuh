// linear.cuh -- the epilogue of the linear layer, shared by its kernels:
//
//   pre = acc * x_scale[m] * w_scale[n] + bias[n]      (scales: 8-bit operands)
//   out = act(pre) + residual
//
// and of the gated layer, whose w has a half of N rows for the gate g and one for u:
//
//   pre = (acc_g + bias[n], acc_u + bias[N + n]),   out = act(pre_g) pre_u
//
// in float32 throughout; pre and out are rounded once, when they are stored.
#pragma once

#include <cuda_bf16.h>

#include "kernels.h"

namespace delta {
namespace linear {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// the logistic function on two MUFU operations, relative error about 2^-21
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-1.4426950408889634f * x)); }

// the tanh form of GELU is x s(2 c (x + 0.044715 x^3)), c = sqrt(2 / pi)
constexpr float kGelu2c = 1.5957691216057308f, kGelu3 = 0.044715f;

__device__ __forceinline__ float activate(int act, float p) {
  if (act == kActSilu) return p * sigmoid(p);
  if (act == kActGelu) return p * sigmoid(kGelu2c * (p + kGelu3 * p * p * p));
  return p;
}
// its derivative
__device__ __forceinline__ float slope(int act, float p) {
  if (act == kActSilu) {
    const float s = sigmoid(p);
    return s * (1.f + p * (1.f - s));
  }
  if (act == kActGelu) {
    const float s = sigmoid(kGelu2c * (p + kGelu3 * p * p * p));
    // past 16, s (1 - s) is 0 in float32, but the square of a large p is not finite
    const float q = fminf(fmaxf(p, -16.f), 16.f);
    return s + q * s * (1.f - s) * kGelu2c * (1.f + 3.f * kGelu3 * q * q);
  }
  return 1.f;
}

// both, for one exponential
__device__ __forceinline__ void curve(int act, float p, float &value, float &der) {
  value = p, der = 1.f;
  if (act == kActSilu) {
    const float s = sigmoid(p);
    value = p * s, der = s * (1.f + p * (1.f - s));
  } else if (act == kActGelu) {
    const float s = sigmoid(kGelu2c * (p + kGelu3 * p * p * p));
    const float q = fminf(fmaxf(p, -16.f), 16.f);  // (as in slope)
    value = p * s, der = s + q * s * (1.f - s) * kGelu2c * (1.f + 3.f * kGelu3 * q * q);
  }
}

__device__ __forceinline__ float bias_at(const LinearArgs &a, int64_t n) {
  if (!a.bias) return 0.f;
  return a.bias_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.bias)[n])
                     : static_cast<const float *>(a.bias)[n];
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float &r) { r = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16 &r) { r = __float2bfloat16_rn(x); }

// one element, start to end
template <typename Out>
__device__ __forceinline__ void finish(const LinearArgs &a, int64_t m, int64_t n, float acc) {
  if (a.x_scale) acc *= a.x_scale[m] * a.w_scale[n];
  const float pre = acc + bias_at(a, n);
  if (a.pre) from_f(pre, static_cast<Out *>(a.pre)[m * a.N + n]);
  float o = activate(a.act, pre);
  if (a.residual) o += to_f(static_cast<const Out *>(a.residual)[m * a.ldr + n]);
  from_f(o, static_cast<Out *>(a.out)[m * a.N + n]);
}

// the same of the gated layer: the sums of both halves
template <typename Out>
__device__ __forceinline__ void finish_glu(const LinearArgs &a, int64_t m, int64_t n, float gate, float up) {
  gate += bias_at(a, n), up += bias_at(a, a.N + n);
  if (a.pre) {
    from_f(gate, static_cast<Out *>(a.pre)[m * 2 * a.N + n]);
    from_f(up, static_cast<Out *>(a.pre)[m * 2 * a.N + a.N + n]);
  }
  from_f(activate(a.act, gate) * up, static_cast<Out *>(a.out)[m * a.N + n]);
}

}  // namespace linear
}  // namespace delta
