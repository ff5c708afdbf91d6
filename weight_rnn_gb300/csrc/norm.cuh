// norm.cuh -- what the residual addition with a norm, root-mean-square (norm.cu, where
// the reasons stand) or layer norm (layernorm.cu), is built of: how rows are shared
// out, copied ahead, reduced and stored, and how the kernels are launched.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "chain.cuh"
#include "kernels.h"

namespace delta {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr int kMostThreads = 512;  // of a CTA
constexpr int kMostRing = 200 * 1024;  // bytes of a CTA's ring; the largest, float32 at D = 8189, takes 196704
// Threads an SM is compiled to hold.  More of them and fewer registers were
// slower but for the 8-bit output (32768 x 4096: 182 us for 192; 162 for 173).
constexpr int kSmThreads = 768, kQuantThreads = 1024;

// V elements: one 16-byte vector, a pair, or a single element
template <typename T, int V>
struct Pack {
  T v[V];
};
template <typename T, int V>
struct __align__(sizeof(T) * V) APack : Pack<T, V> {};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float &r) { r = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16 &r) { r = __float2bfloat16_rn(x); }

template <typename T, int V>
__device__ __forceinline__ void store_v(T *p, const float (&v)[V]) {
  APack<T, V> o;
#pragma unroll
  for (int i = 0; i < V; ++i) from_f(v[i], o.v[i]);
  *reinterpret_cast<APack<T, V> *>(p) = o;
}

// V values to e4m3, saturating, round to nearest even
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    struct __align__(V) { __nv_fp8x2_storage_t h[V / 2]; } o;
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      o.h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<decltype(o) *>(p) = o;
  }
}

// float32 pairs: one instruction for two elements.  The single-element path
// (V = 1) uses the plain forms.
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpk(uint64_t r, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a vector as pairs
template <typename T, int V>
__device__ __forceinline__ uint64_t pair_of(const Pack<T, V> &p, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = reinterpret_cast<const uint32_t *>(p.v)[i];
    return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  } else {
    return pk(p.v[2 * i], p.v[2 * i + 1]);
  }
}

// One row's reduction over its nt threads (a multiple of 32): warp shuffles,
// then the row's warps meet in `part`.  Every thread gets the same sum, taken
// in the same order.  `part` alternates between calls, so one barrier a call
// is enough.
template <bool kMax>
__device__ __forceinline__ float join(float a, float b) { return kMax ? fmaxf(a, b) : a + b; }
template <bool kMax>
__device__ __forceinline__ float row_reduce(float v, float *part, int nwarp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = join<kMax>(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (nwarp == 1) return v;  // the same for every row of the CTA
  const int w = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.y * 32 + w] = v;
  __syncthreads();
  v = part[threadIdx.y * 32];
  for (int i = 1; i < nwarp; ++i) v = join<kMax>(v, part[threadIdx.y * 32 + i]);
  return v;
}

// weights (or biases; 0 without) of this thread's elements, float32 in registers
template <int V, int kPer>
__device__ __forceinline__ void load_weight(const void *weight, bool w_bf16, int64_t D, float (&w)[kPer][V]) {
#pragma unroll
  for (int j = 0; j < kPer; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t d = ((int64_t)j * blockDim.x + threadIdx.x) * V + i;
      w[j][i] = d >= D || !weight ? 0.f
                : w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(weight)[d])
                         : static_cast<const float *>(weight)[d];
    }
}

// rows in a ring: three, or two where N tensors of the widest rows would pass a
// CTA's shared memory
__host__ __device__ constexpr int ring_rows(int N, int per, int V, int size) {
  return V * size == 16 ? (N * per >= 12 ? 2 : 3) : N == 3 && per == 16 && size == 4 ? 2 : 3;
}
// bytes that the pieces covering a row take, wherever it starts
__host__ __device__ constexpr int64_t cover(int64_t bytes) { return (bytes + 31) / 16 * 16; }

// One row of N tensors, kPer vectors a thread.  Whole vectors (16 bytes) are
// copied and read by the thread that uses them; single elements and pairs lie
// in a buffer that the row's threads share.
template <typename In, int V, int kPer, int N, int kT>
struct Rows {
  using Vec = APack<In, V>;
  static constexpr bool kOwn = V * sizeof(In) == 16;
  static constexpr int kStages = ring_rows(N, kPer, V, sizeof(In));
  const In *base[N];
  int64_t ld[N], rows, D;
  unsigned char *ring;  // own: [kStages][N][kPer][kT] vectors; else [kStages][N][rows a CTA][cover()] bytes
  const In *now[kOwn ? 1 : N];
  int slot = 0;

  // a shared buffer of tensor n, and where its row begins in it
  __device__ __forceinline__ unsigned char *buffer(int s, int n) const {
    return ring + ((s * N + n) * blockDim.y + threadIdx.y) * cover(D * sizeof(In));
  }
  __device__ __forceinline__ static void copy(void *to, const void *from, int bytes) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
  }
  __device__ __forceinline__ void fetch(int64_t row, int to) {
    if (row < rows) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (!base[n]) continue;
        const In *from = base[n] + row * ld[n];
        if constexpr (kOwn) {
          Vec *mine = reinterpret_cast<Vec *>(ring) + threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int64_t d = ((int64_t)j * blockDim.x + threadIdx.x) * V;
            if (d < D) copy(mine + ((to * N + n) * kPer + j) * kT, from + d, 16);
          }
        } else {
          const int head = (int)(reinterpret_cast<uintptr_t>(from) & 15);
          const int bytes = head + (int)(D * sizeof(In));
          const unsigned char *first = reinterpret_cast<const unsigned char *>(from) - head;
          unsigned char *buf = buffer(to, n);
          for (int c = threadIdx.x * 16; c < bytes; c += blockDim.x * 16)
            copy(buf + c, first + c, bytes - c < 16 ? bytes - c : 16);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void start(int64_t first, int64_t step) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(first + i * step, i);
  }
  // the row becomes readable, and a later one is asked for
  __device__ __forceinline__ void turn(int64_t row, int64_t step) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    if constexpr (!kOwn) {
      // of all the row's threads; and the last row's reads are over
      if (blockDim.x == 32)
        __syncwarp();
      else
        __syncthreads();
#pragma unroll
      for (int n = 0; n < N; ++n)
        now[n] = reinterpret_cast<const In *>(buffer(slot, n) + (reinterpret_cast<uintptr_t>(base[n] + row * ld[n]) & 15));
    }
    fetch(row + (kStages - 1) * step, slot == 0 ? kStages - 1 : slot - 1);
  }
  __device__ __forceinline__ void done() { slot = slot == kStages - 1 ? 0 : slot + 1; }
  __device__ __forceinline__ void finish() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
  __device__ __forceinline__ Vec get(int n, int j) const {
    if constexpr (kOwn) {
      const Vec *mine = reinterpret_cast<const Vec *>(ring) + threadIdx.y * blockDim.x + threadIdx.x;
      return mine[((slot * N + n) * kPer + j) * kT];
    } else {
      const int64_t d = ((int64_t)j * blockDim.x + threadIdx.x) * V;
      return *reinterpret_cast<const Vec *>(now[n] + (d < D ? d : 0));
    }
  }
};

// ------------------------------------------------------------------ launches
struct Plan {
  int V, per, nt, rpc;  // elements a vector, vectors a thread, threads a row, rows a CTA
  int64_t grid;
  int threads;          // of a CTA at most, which its ring is laid out for
  int smem;             // the ring
};

// One vector a thread while rows are few (latency), two where a row has more
// than a warp's worth and there are rows for every SM (fewer, longer-lived
// CTAs); more only where a row would not fit kMostThreads threads.  Of single
// elements as many as keep a row to few warps, one if it can be: then rows need
// no barrier.
Plan plan(int64_t rows, int64_t D, int vec, int wide, int tensors, int resident, bool many, bool narrow = false) {
  Plan q;
  const int size = 16 / vec;
  const bool aligned = wide == vec;
  q.V = wide;
  const int64_t n = (D + q.V - 1) / q.V;  // vectors a row
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (aligned)
    q.per = rows >= 2 * sms && n > 32 ? 2 : 1;
  else
    q.per = rows < 2 * sms ? (n <= 256 ? 1 : 4) : n <= 32 ? 1 : n <= 128 ? 4 : n <= 256 ? 8 : 16;
  if (q.V == 2 && q.per > 8) q.per = 8;
  while (n > (int64_t)q.per * kMostThreads) q.per *= 2;
  q.nt = (int)((n + q.per - 1) / q.per + 31) / 32 * 32;
  // rows of a few vectors: several to a warp, where the kernel can (layer norm)
  if (narrow && aligned && n <= 16) q.per = 1, q.nt = n <= 4 ? 4 : n <= 8 ? 8 : 16;
  q.rpc = q.nt >= 256 ? 1 : 256 / q.nt;
  const int64_t ctas = (rows + q.rpc - 1) / q.rpc;
  q.threads = q.nt * q.rpc <= 256 ? 256 : kMostThreads;
  q.smem = ring_rows(tensors, q.per, q.V, size) * tensors *
           (aligned ? q.per * q.threads * 16 : q.rpc * (int)cover(D * size));
  // (the backward's column sums take the ring's place: 4 bytes an element)
  if (q.smem < q.rpc * q.nt * q.per * q.V * 4) q.smem = q.rpc * q.nt * q.per * q.V * 4;
  // as many CTAs as an SM holds, by its resident threads and by rings; with
  // `many`, 8 to 16 an SM where each still has a dozen rows: CTAs that come
  // later even out what the memory gives each (32768 x 4096 bfloat16 forward
  // 161 us, 6.7 TB/s, for 182 with the resident ones alone; the backward, which
  // ends in a row of sums per CTA, 195 for 173)
  int fit = resident / q.threads;
  if (fit > kMostRing / q.smem) fit = kMostRing / q.smem;
  int64_t cap = (int64_t)sms * (fit > 1 ? fit : 1);
  if (many && ctas / 12 >= 8 * sms) cap = ctas / 12 < 16 * sms ? ctas / 12 : 16 * sms;
  q.grid = ctas < cap ? ctas : cap;
  return q;
}

// the instance for a plan: up to 4 (float32) or 2 (bfloat16) vectors of 16
// bytes a thread, up to 8 pairs, or up to 16 single elements, which covers kNormMaxD
template <typename In, template <typename, int, int> class F, typename... X>
cudaError_t dispatch(const Plan &q, X &&...x) {
  constexpr int V = 16 / sizeof(In);
  if constexpr (sizeof(In) == 2)
    if (q.V == 2) switch (q.per) {
        case 1: return F<In, 2, 1>::run(x...);
        case 4: return F<In, 2, 4>::run(x...);
        case 8: return F<In, 2, 8>::run(x...);
        default: return cudaErrorInvalidConfiguration;
      }
  if (q.V == 1) switch (q.per) {
      case 1: return F<In, 1, 1>::run(x...);
      case 4: return F<In, 1, 4>::run(x...);
      case 8: return F<In, 1, 8>::run(x...);
      case 16: return F<In, 1, 16>::run(x...);
    }
  else switch (q.per) {
      case 1: return F<In, V, 1>::run(x...);
      case 2: return F<In, V, 2>::run(x...);
      case 4:
        if constexpr (V == 4) return F<In, V, 4>::run(x...);
    }
  return cudaErrorInvalidConfiguration;
}

template <typename K, typename A>
cudaError_t go(K kern, const A &a, const Plan &q, cudaStream_t s) {
  if (q.smem > kMostRing) return cudaErrorInvalidConfiguration;
  if (q.smem > 48 * 1024 - 4096) {  // more than the default only after asking
    // (the limit belongs to the kernel, not to the call: every thread of the
    // program sets the same one)
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRing);
    if (e != cudaSuccess) return e;
  }
  return chain_launch(kern, dim3((unsigned)q.grid), dim3(q.nt, q.rpc), q.smem, 1, true, s, a);
}

// whole vectors, pairs, or single elements, by what every row's start allows
template <typename In>
int fwd_width(const NormArgs &a) {
  constexpr int V = 16 / sizeof(In);
  const auto ok = [&](int n) {
    const auto at = [&](const void *p) { return reinterpret_cast<uintptr_t>(p) % (n * sizeof(In)) == 0; };
    return a.D % n == 0 && a.ldx % n == 0 && (!a.residual || a.ldr % n == 0) && at(a.x) && at(a.residual);
  };
  return ok(V) ? V : V == 8 && ok(2) ? 2 : 1;
}
template <typename In>
Plan bwd_plan(const NormBwdArgs &a, int resident, bool narrow = false) {
  constexpr int V = 16 / sizeof(In);
  return plan(a.rows, a.D, V, a.D % V == 0 ? V : V == 8 && a.D % 2 == 0 ? 2 : 1, 3, resident, false, narrow);
}

}  // namespace
}  // namespace delta
