// norm.cu -- the residual addition with the root-mean-square norm:
//
//   t = x + r,   rstd = (mean_d t_d^2 + eps)^{-1/2},   y = t rstd w
//
// t goes out in the input type (the residual stream), y in the input type or
// in e4m3 with one float32 scale a row (scale = max |y| / 448, q = y / scale).
// The norm is taken of the float32 sum, before that is rounded for the stream.
// Gradient, with t^ = t rstd:
//
//   dx = rstd (w dy - t^ mean_d(w dy t^)) + dsum,   dw = sum over rows of dy t^
//
// HBM-bound: two tensors in and two out (8 bytes an element in bfloat16, 7
// with an 8-bit y; backward three in, one out).  A row has `nt` threads of
// kPer 16-byte vectors.  The CTAs walk the rows, so that the weight is read
// once a CTA and the backward keeps its column sums in registers; each thread
// copies its own vectors of the next row or two into its own places of a
// ring in shared memory, asynchronously, which keeps the memory busy during
// the reductions without a barrier or a register.  The column sums meet in a
// second kernel in CTA order, so the result does not depend on scheduling.
// Rows whose width, strides or addresses are not multiples of 16 bytes are
// copied as the 16-byte pieces that cover them, by all threads of the row, and
// read from there one element at a time (4096 x 4097 bfloat16: element loads
// into registers took 124 us forward and 520 backward), or two where bfloat16
// rows lie on 4-byte addresses (4672 x 3514: 32 us forward for 63).
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

// weights of this thread's elements, float32 in registers
template <int V, int kPer>
__device__ __forceinline__ void load_weight(const void *weight, bool w_bf16, int64_t D, float (&w)[kPer][V]) {
#pragma unroll
  for (int j = 0; j < kPer; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t d = ((int64_t)j * blockDim.x + threadIdx.x) * V + i;
      w[j][i] = d >= D ? 0.f
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

// ------------------------------------------------------------------ forward
// blockDim (nt, rows a CTA); a thread's vectors are nt apart
template <typename In, int V, int kPer, int kT, bool kQuant>
__global__ void __launch_bounds__(kT, V *kPer <= 16 ? (kQuant ? kQuantThreads : kSmThreads) / kT : 1) norm_fwd_kernel(NormArgs p) {
  __shared__ float part[2][8 * 32];  // at most 8 rows a CTA, 16 warps a row
  extern __shared__ __align__(16) unsigned char ring[];
  const int nwarp = blockDim.x >> 5;
  float w[kPer][V];
  chain_wait();
  load_weight<V, kPer>(p.weight, p.w_bf16, p.D, w);
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  Rows<In, V, kPer, 2, kT> in;
  in.base[0] = static_cast<const In *>(p.x); in.base[1] = static_cast<const In *>(p.residual);
  in.ld[0] = p.ldx; in.ld[1] = p.ldr; in.rows = p.rows; in.D = p.D;
  in.ring = ring;
  in.start(first, step);
  int buf = 0;
  // every row of the CTA takes part in the barriers until the last is done
  for (int64_t row = first; row - threadIdx.y < p.rows; row += step, buf ^= 1) {
    in.turn(row, step);
    float t[kPer][V], ss = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool on = row < p.rows && ((int64_t)j * blockDim.x + threadIdx.x) * V < p.D;
      const APack<In, V> xv = in.get(0, j), rv = in.get(1, j);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        t[j][i] = on ? to_f(xv.v[i]) + (p.residual ? to_f(rv.v[i]) : 0.f) : 0.f;
        ss = fmaf(t[j][i], t[j][i], ss);
      }
    }
    in.done();
    ss = row_reduce<false>(ss, part[kQuant ? 0 : buf], nwarp);
    const float rstd = rsqrtf(ss / (float)p.D + p.eps);
    float inv = 1.f;
    if constexpr (kQuant) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, fabsf(t[j][i] * rstd * w[j][i]));
      top = row_reduce<true>(top, part[1], nwarp);
      // a row of zeros, or of values too small for a float32 scale: scale 1
      float scale = top / kE4m3Max;
      if (scale < 1.1754944e-38f) scale = 1.f;
      inv = 1.f / scale;
      if (row < p.rows && threadIdx.x == 0) p.scale[row] = scale;
    }
    if (row < p.rows) {
      if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int64_t d = ((int64_t)j * blockDim.x + threadIdx.x) * V;
        if (d >= p.D) continue;
        if (p.sum) store_v<In, V>(static_cast<In *>(p.sum) + row * p.D + d, t[j]);
#pragma unroll
        for (int i = 0; i < V; ++i) t[j][i] = t[j][i] * rstd * w[j][i] * inv;
        if constexpr (kQuant)
          store_e4m3<V>(static_cast<uint8_t *>(p.y) + row * p.D + d, t[j]);
        else
          store_v<In, V>(static_cast<In *>(p.y) + row * p.D + d, t[j]);
      }
    }
  }
  in.finish();
}

// ----------------------------------------------------------------- backward
// The row is read from its ring twice, before and after the reduction, rather
// than held: that is what lets two CTAs of 512 threads share an SM.
template <typename In, int V, int kPer, int kT>
__global__ void __launch_bounds__(kT, V *kPer <= 16 ? kSmThreads / kT : 1) norm_bwd_kernel(NormBwdArgs p) {
  __shared__ float part[2][8 * 32];
  extern __shared__ __align__(16) unsigned char ring[];
  const int nwarp = blockDim.x >> 5;
  chain_next();
  chain_wait();
  float w[kPer][V], dw[kPer][V];
  load_weight<V, kPer>(p.weight, p.w_bf16, p.D, w);
#pragma unroll
  for (int j = 0; j < kPer; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  Rows<In, V, kPer, 3, kT> in;
  in.base[0] = static_cast<const In *>(p.dy); in.base[1] = static_cast<const In *>(p.sum);
  in.base[2] = static_cast<const In *>(p.dsum);
  in.ld[0] = in.ld[1] = in.ld[2] = in.D = p.D; in.rows = p.rows;
  in.ring = ring;
  in.start(first, step);
  float ahead = first < p.rows ? p.rstd[first] : 0.f;
  int buf = 0;
  for (int64_t row = first; row - threadIdx.y < p.rows; row += step, buf ^= 1) {
    in.turn(row, step);
    const float rstd = ahead;
    if (row + step < p.rows) ahead = p.rstd[row + step];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const APack<In, V> gv = in.get(0, j), tv = in.get(1, j);
      if (row < p.rows && ((int64_t)j * blockDim.x + threadIdx.x) * V < p.D) {
        if constexpr (V > 1) {
          uint64_t sum = pk(0.f, 0.f);
          const uint64_t rr = pk(rstd, rstd);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const uint64_t t = mul2(pair_of(tv, i), rr), y = pair_of(gv, i);
            unpk(fma2(y, t, pk(dw[j][2 * i], dw[j][2 * i + 1])), dw[j][2 * i], dw[j][2 * i + 1]);
            sum = fma2(mul2(y, pk(w[j][2 * i], w[j][2 * i + 1])), t, sum);
          }
          float a, b;
          unpk(sum, a, b);
          dot += a + b;
        } else {
          const float t = to_f(tv.v[0]) * rstd, y = to_f(gv.v[0]);
          dw[j][0] = fmaf(y, t, dw[j][0]);
          dot = fmaf(y * w[j][0], t, dot);
        }
      }
    }
    dot = row_reduce<false>(dot, part[buf], nwarp) / (float)p.D;
    if (row < p.rows) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int64_t d = ((int64_t)j * blockDim.x + threadIdx.x) * V;
        if (d >= p.D) continue;
        const APack<In, V> gv = in.get(0, j), tv = in.get(1, j), sv = in.get(2, j);
        float g[V];
        // rstd (w dy - t^ dot) + dsum, with t^ = sum * rstd
        const float c = -rstd * rstd * dot;
        if constexpr (V > 1) {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const uint64_t wy = mul2(pair_of(gv, i), pk(w[j][2 * i], w[j][2 * i + 1]));
            const uint64_t low = p.dsum ? pair_of(sv, i) : pk(0.f, 0.f);
            unpk(fma2(wy, pk(rstd, rstd), fma2(pair_of(tv, i), pk(c, c), low)), g[2 * i], g[2 * i + 1]);
          }
        } else {
          g[0] = fmaf(rstd, to_f(gv.v[0]) * w[j][0], fmaf(to_f(tv.v[0]), c, p.dsum ? to_f(sv.v[0]) : 0.f));
        }
        store_v<In, V>(static_cast<In *>(p.dx) + row * p.D + d, g);
      }
    }
    in.done();
  }
  in.finish();
  // the CTA's rows of threads meet in order, where the ring was
  float *sums = reinterpret_cast<float *>(ring);
  const int width = blockDim.x * kPer * V;
  if (blockDim.y > 1) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) sums[threadIdx.y * width + (j * blockDim.x + threadIdx.x) * V + i] = dw[j][i];
    __syncthreads();
    if (threadIdx.y > 0) return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int d = (j * blockDim.x + threadIdx.x) * V + i;
      float s = dw[j][i];
      for (int y = 1; y < blockDim.y; ++y) s += sums[y * width + d];
      if (d < p.D) p.partial[(int64_t)blockIdx.x * p.D + d] = s;
    }
}

// dw[d] = sum of n partial rows: C columns a CTA, every R-th row to a thread,
// then a warp a column over the R sums.  Few columns take 8 at a time (a sector
// of each row), so that there are CTAs; many take 32 (4096 x 8192: 53 us with
// the gradients before it, 57 with 8).
template <int C>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *partial, float *dw, int64_t n, int64_t D) {
  constexpr int R = 1024 / C;
  __shared__ float s[R][C + 1];
  const int64_t d = (int64_t)blockIdx.x * C + threadIdx.x;
  float v = 0.f;
  chain_wait();
  // (no chain_next(): the next gradient's CTAs, whose rows are dealt out evenly,
  // would crowd on the SMs that are free early; 94 -> 108 us)
  if (d < D)
    for (int64_t i = threadIdx.y; i < n; i += R) v += partial[i * D + d];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  const int warp = (threadIdx.y * C + threadIdx.x) / 32, lane = (threadIdx.y * C + threadIdx.x) % 32;
  if (warp >= C) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < R; k += 32) v += s[lane + k][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t c = (int64_t)blockIdx.x * C + warp;
  if (lane == 0 && c < D) dw[c] = v;
}

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
Plan plan(int64_t rows, int64_t D, int vec, int wide, int tensors, int resident, bool many) {
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

template <typename In, int V, int kPer>
struct FwdOne {
  static cudaError_t run(const NormArgs &a, const Plan &q, cudaStream_t s) {
    if (q.threads == 256)
      return a.scale ? go(norm_fwd_kernel<In, V, kPer, 256, true>, a, q, s)
                     : go(norm_fwd_kernel<In, V, kPer, 256, false>, a, q, s);
    return a.scale ? go(norm_fwd_kernel<In, V, kPer, kMostThreads, true>, a, q, s)
                   : go(norm_fwd_kernel<In, V, kPer, kMostThreads, false>, a, q, s);
  }
};
template <typename In, int V, int kPer>
struct BwdOne {
  static cudaError_t run(const NormBwdArgs &a, const Plan &q, cudaStream_t s) {
    return q.threads == 256 ? go(norm_bwd_kernel<In, V, kPer, 256>, a, q, s)
                            : go(norm_bwd_kernel<In, V, kPer, kMostThreads>, a, q, s);
  }
};

template <typename In>
cudaError_t fwd_all(const NormArgs &a, cudaStream_t s) {
  constexpr int V = 16 / sizeof(In);
  // whole vectors, pairs, or single elements, by what every row's start allows
  const auto ok = [&](int n) {
    const auto at = [&](const void *p) { return reinterpret_cast<uintptr_t>(p) % (n * sizeof(In)) == 0; };
    return a.D % n == 0 && a.ldx % n == 0 && (!a.residual || a.ldr % n == 0) && at(a.x) && at(a.residual);
  };
  const Plan q = plan(a.rows, a.D, V, ok(V) ? V : V == 8 && ok(2) ? 2 : 1, 2, a.scale ? kQuantThreads : kSmThreads, true);
  return dispatch<In, FwdOne>(q, a, q, s);
}

template <typename In>
Plan bwd_plan(const NormBwdArgs &a) {
  constexpr int V = 16 / sizeof(In);
  return plan(a.rows, a.D, V, a.D % V == 0 ? V : V == 8 && a.D % 2 == 0 ? 2 : 1, 3, kSmThreads, false);
}
template <typename In>
cudaError_t bwd_all(const NormBwdArgs &a, cudaStream_t s) {
  const Plan q = bwd_plan<In>(a);
  cudaError_t e = q.grid > 0 ? dispatch<In, BwdOne>(q, a, q, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  return launch_column_sum(a.partial, a.dweight, q.grid, a.D, s);
}

}  // namespace

cudaError_t launch_column_sum(const float *partial, float *out, int64_t n, int64_t D, cudaStream_t s) {
  return D < 1024 ? chain_launch(column_sum_kernel<8>, dim3((unsigned)((D + 7) / 8)), dim3(8, 128), 0, 1, true, s,
                                 partial, out, n, D)
                  : chain_launch(column_sum_kernel<32>, dim3((unsigned)((D + 31) / 32)), dim3(32, 32), 0, 1, true, s,
                                 partial, out, n, D);
}

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s) {
  return a.bf16 ? fwd_all<__nv_bfloat16>(a, s) : fwd_all<float>(a, s);
}

int64_t norm_bwd_ctas(const NormBwdArgs &a) {
  const Plan q = a.bf16 ? bwd_plan<__nv_bfloat16>(a) : bwd_plan<float>(a);
  return q.grid;
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t s) {
  return a.bf16 ? bwd_all<__nv_bfloat16>(a, s) : bwd_all<float>(a, s);
}

}  // namespace delta
