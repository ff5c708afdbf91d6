// layernorm.cu -- the residual addition with layer norm:
//
//   t = x + r,   mean = mean_d t,   rstd = (mean_d (t - mean)^2 + eps)^{-1/2},
//   y = (t - mean) rstd w + b
//
// and its gradient, with t^ = (t - mean) rstd:
//
//   dx = rstd (w dy - mean_d(w dy) - t^ mean_d(w dy t^)) + dsum,
//   dw = sum over rows of dy t^,   db = sum over rows of dy
//
// Rows are shared out and copied ahead as in norm.cu, and the bound is the same, HBM.
// A row stays in registers between its sums and its output, so that the data is read
// once.  Its variance is that of the differences, of parts: each warp takes the squares
// about its own mean, and with n_w, m_w and M_w of the warps' elements, means and
// squares,
//
//   sum (t - mean)^2 = sum_w M_w + n_w (m_w - mean)^2,
//
// nothing of which cancels, at one barrier a row.  Sums behind means are of elements over
// D's power of two: the same roundings, and a row of finite elements has a finite mean.
// (A second barrier for the squares about the row's mean, and single elements in place of
// pairs: 32768 x 4096 bfloat16 198 us.)  32768 x 4096 bfloat16 takes 164 us, 6.5 TB/s (163
// without the scaling); one row of 4096 3.2, a launch.
#include "norm.cuh"

namespace delta {
namespace {

// V elements of a lane as pairs, or one
template <int V>
struct Lane {
  static constexpr int kN = V / 2;
  uint64_t v[kN];
  template <typename T>
  __device__ __forceinline__ static Lane of(const Pack<T, V> &p) {
    Lane r;
#pragma unroll
    for (int i = 0; i < kN; ++i) r.v[i] = pair_of(p, i);
    return r;
  }
  __device__ __forceinline__ static Lane all(float x) {
    Lane r;
#pragma unroll
    for (int i = 0; i < kN; ++i) r.v[i] = pk(x, x);
    return r;
  }
  __device__ __forceinline__ Lane operator+(const Lane &o) const {
    Lane r;
#pragma unroll
    for (int i = 0; i < kN; ++i) asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v[i]) : "l"(v[i]), "l"(o.v[i]));
    return r;
  }
  __device__ __forceinline__ Lane operator*(const Lane &o) const {
    Lane r;
#pragma unroll
    for (int i = 0; i < kN; ++i) r.v[i] = mul2(v[i], o.v[i]);
    return r;
  }
  // this * o + c
  __device__ __forceinline__ Lane fma(const Lane &o, const Lane &c) const {
    Lane r;
#pragma unroll
    for (int i = 0; i < kN; ++i) r.v[i] = fma2(v[i], o.v[i], c.v[i]);
    return r;
  }
  __device__ __forceinline__ float sum() const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float a, b;
      unpk(v[i], a, b);
      s += a + b;
    }
    return s;
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) unpk(v[i], f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ static Lane from(const float (&f)[V]) {
    Lane r;
#pragma unroll
    for (int i = 0; i < kN; ++i) r.v[i] = pk(f[2 * i], f[2 * i + 1]);
    return r;
  }
};
template <>
struct Lane<1> {
  float v;
  template <typename T>
  __device__ __forceinline__ static Lane of(const Pack<T, 1> &p) { return {to_f(p.v[0])}; }
  __device__ __forceinline__ static Lane all(float x) { return {x}; }
  __device__ __forceinline__ Lane operator+(const Lane &o) const { return {v + o.v}; }
  __device__ __forceinline__ Lane operator*(const Lane &o) const { return {v * o.v}; }
  __device__ __forceinline__ Lane fma(const Lane &o, const Lane &c) const { return {fmaf(v, o.v, c.v)}; }
  __device__ __forceinline__ float sum() const { return v; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = v; }
  __device__ __forceinline__ static Lane from(const float (&f)[1]) { return {f[0]}; }
};

template <int V, int kPer>
__device__ __forceinline__ void load_lanes(const void *weight, bool bf16, int64_t D, Lane<V> (&w)[kPer]) {
  float f[kPer][V];
  load_weight<V, kPer>(weight, bf16, D, f);
#pragma unroll
  for (int j = 0; j < kPer; ++j) w[j] = Lane<V>::from(f[j]);
}
template <typename T, int V>
__device__ __forceinline__ void store_lane(T *p, const Lane<V> &v) {
  float f[V];
  v.get(f);
  store_v<T, V>(p, f);
}

// the least power of two that is no less than D: its logarithm
__device__ __forceinline__ int log2_up(int D) { return 32 - __clz(D - 1); }
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

// A row whose squares pass float32's range has rstd 0; its differences may be infinite,
// and are left out.
__device__ __forceinline__ float mean_used(float mean, float rstd) { return rstd == 0.f ? 0.f : mean; }

// over the lanes of a row in this warp: all of them, or 4, 8 or 16 where rows are narrow
__device__ __forceinline__ float row_sum(float v) {
  if (blockDim.x < 32) {
    for (int o = blockDim.x / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void row_sum(float &a, float &b) {  // (both at a time)
  if (blockDim.x < 32) {
    for (int o = blockDim.x / 2; o > 0; o >>= 1)
      a += __shfl_xor_sync(0xffffffffu, a, o), b += __shfl_xor_sync(0xffffffffu, b, o);
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o), b += __shfl_xor_sync(0xffffffffu, b, o);
}
template <int kFrom>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = kFrom; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------ forward
template <typename In, int V, int kPer, int kT>
__global__ void __launch_bounds__(kT, V *kPer <= 16 ? kSmThreads / kT : 1) layernorm_fwd_kernel(NormArgs p) {
  __shared__ float4 part[2][8 * 16];  // at most 8 rows a CTA, 16 warps a row
  extern __shared__ __align__(16) unsigned char ring[];
  const int nwarp = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Lane<V> w[kPer], b[kPer];
  chain_wait();
  load_lanes<V, kPer>(p.weight, p.w_bf16, p.D, w);
  load_lanes<V, kPer>(p.bias, p.b_bf16, p.D, b);
  int own = 0;  // elements of a row that this warp has
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int left = (int)p.D - (j * (int)blockDim.x + warp * 32) * V;
    own += left < 0 ? 0 : left < 32 * V ? left : 32 * V;
  }
  const int up = log2_up((int)p.D);
  const float down = power_of_two(-up), sum_of_ones = (float)p.D * down;
  const float n_w = (float)own, inv_w = own ? 1.f / n_w * power_of_two(up) : 0.f;
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
    Lane<V> t[kPer], acc = Lane<V>::all(0.f);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      t[j] = Lane<V>::all(0.f);
      if (row < p.rows && (int64_t)(j * blockDim.x + threadIdx.x) * V < p.D) {
        t[j] = Lane<V>::of(in.get(0, j));
        if (p.residual) t[j] = t[j] + Lane<V>::of(in.get(1, j));
        acc = t[j].fma(Lane<V>::all(down), acc);
      }
    }
    in.done();
    float s = row_sum(acc.sum());
    float m_w = s * inv_w;
    acc = Lane<V>::all(0.f);
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if ((int64_t)(j * blockDim.x + threadIdx.x) * V < p.D) {
        const Lane<V> c = t[j] + Lane<V>::all(-m_w);
        acc = c.fma(c, acc);
      }
    float q = row_sum(acc.sum()), mean = m_w;
    if (nwarp > 1) {
      if (lane == 0) part[buf][threadIdx.y * 16 + warp] = make_float4(s, q, m_w, n_w);
      __syncthreads();
      // 16 lanes take a warp's part each
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if ((lane & 15) < nwarp) a = part[buf][threadIdx.y * 16 + (lane & 15)];
      mean = lanes_sum<8>(a.x) / sum_of_ones;
      q = lanes_sum<8>(fmaf(a.w * (a.z - mean), a.z - mean, a.y));
    }
    const float rstd = rsqrtf(q / (float)p.D + p.eps);
    if (row < p.rows) {
      if (threadIdx.x == 0) {
        if (p.rstd) p.rstd[row] = rstd;
        if (p.mean) p.mean[row] = mean;
      }
      const Lane<V> away = Lane<V>::all(-mean_used(mean, rstd));
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int64_t d = (int64_t)(j * blockDim.x + threadIdx.x) * V;
        if (d >= p.D) continue;
        if (p.sum) store_lane<In, V>(static_cast<In *>(p.sum) + row * p.D + d, t[j]);
        const Lane<V> c = (t[j] + away) * Lane<V>::all(rstd);
        store_lane<In, V>(static_cast<In *>(p.y) + row * p.D + d, c.fma(w[j], b[j]));
      }
    }
  }
  in.finish();
}

// ----------------------------------------------------------------- backward
// Two dot products a row and two column sums, which go out side by side, [CTA][2 D].
// w dy and t^ stay in registers between the dots and dx: 512 threads an SM, at up to
// 128 registers.  32768 x 2048 bfloat16 takes 95 us, 5.6 TB/s, 5 of them in the kernel
// that adds the CTAs' column sums up.  (w dy and t^ read from the ring a second time, at
// 80 registers: 152 us.)  With one vector of a row a thread, 768 (rows of up to 32
// vectors; a million of 128 elements 205 -> 180 us, 1024 threads 202; wider rows take two
// a thread, 32768 x 2048 with one 111 us).
template <typename In, int V, int kPer>
constexpr int bwd_threads() { return kPer == 1 && V * sizeof(In) == 16 ? 768 : 512; }

template <typename In, int V, int kPer, int kT>
__global__ void __launch_bounds__(kT, V *kPer <= 16 ? bwd_threads<In, V, kPer>() / kT : 1)
    layernorm_bwd_kernel(NormBwdArgs p) {
  __shared__ float2 part[2][8 * 16];
  extern __shared__ __align__(16) unsigned char ring[];
  const int nwarp = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  chain_next();
  chain_wait();
  Lane<V> w[kPer], dw[kPer], db[kPer];
  load_lanes<V, kPer>(p.weight, p.w_bf16, p.D, w);
#pragma unroll
  for (int j = 0; j < kPer; ++j) dw[j] = db[j] = Lane<V>::all(0.f);
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  Rows<In, V, kPer, 3, kT> in;
  in.base[0] = static_cast<const In *>(p.dy); in.base[1] = static_cast<const In *>(p.sum);
  in.base[2] = static_cast<const In *>(p.dsum);
  in.ld[0] = in.ld[1] = in.ld[2] = in.D = p.D; in.rows = p.rows;
  in.ring = ring;
  in.start(first, step);
  float ahead = first < p.rows ? p.rstd[first] : 0.f, ahead_m = first < p.rows ? p.mean[first] : 0.f;
  int buf = 0;
  for (int64_t row = first; row - threadIdx.y < p.rows; row += step, buf ^= 1) {
    in.turn(row, step);
    const float rstd = ahead, mean = mean_used(ahead_m, rstd);
    if (row + step < p.rows) ahead = p.rstd[row + step], ahead_m = p.mean[row + step];
    Lane<V> wy[kPer], t[kPer], s2 = Lane<V>::all(0.f), d2 = Lane<V>::all(0.f);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      wy[j] = t[j] = Lane<V>::all(0.f);
      if (row < p.rows && (int64_t)(j * blockDim.x + threadIdx.x) * V < p.D) {
        // (the difference first: a product of the mean would cancel)
        t[j] = (Lane<V>::of(in.get(1, j)) + Lane<V>::all(-mean)) * Lane<V>::all(rstd);
        const Lane<V> y = Lane<V>::of(in.get(0, j));
        dw[j] = y.fma(t[j], dw[j]);
        db[j] = db[j] + y;
        wy[j] = y * w[j];
        s2 = s2 + wy[j];
        d2 = wy[j].fma(t[j], d2);
      }
    }
    float sum = s2.sum(), dot = d2.sum();
    row_sum(sum, dot);
    if (nwarp > 1) {
      if (lane == 0) part[buf][threadIdx.y * 16 + warp] = make_float2(sum, dot);
      __syncthreads();
      float2 a = make_float2(0.f, 0.f);
      if ((lane & 15) < nwarp) a = part[buf][threadIdx.y * 16 + (lane & 15)];
      sum = lanes_sum<8>(a.x), dot = lanes_sum<8>(a.y);
    }
    const Lane<V> ms = Lane<V>::all(-sum / (float)p.D), md = Lane<V>::all(-dot / (float)p.D), r = Lane<V>::all(rstd);
    if (row < p.rows) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int64_t d = (int64_t)(j * blockDim.x + threadIdx.x) * V;
        if (d >= p.D) continue;
        Lane<V> g = t[j].fma(md, wy[j] + ms);
        g = p.dsum ? g.fma(r, Lane<V>::of(in.get(2, j))) : g * r;
        store_lane<In, V>(static_cast<In *>(p.dx) + row * p.D + d, g);
      }
    }
    in.done();
  }
  in.finish();
  // the CTA's rows of threads meet in order, where the ring was, one sum after the other
  float *sums = reinterpret_cast<float *>(ring);
  const int width = blockDim.x * kPer * V;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float s[kPer][V];
#pragma unroll
    for (int j = 0; j < kPer; ++j) (which ? db[j] : dw[j]).get(s[j]);
    if (blockDim.y > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) sums[threadIdx.y * width + (j * blockDim.x + threadIdx.x) * V + i] = s[j][i];
      __syncthreads();
    }
    if (threadIdx.y == 0) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int d = (j * blockDim.x + threadIdx.x) * V + i;
          for (int y = 1; y < blockDim.y; ++y) s[j][i] += sums[y * width + d];
          if (d < p.D) p.partial[((int64_t)blockIdx.x * 2 + which) * p.D + d] = s[j][i];
        }
    }
  }
}

template <typename In, int V, int kPer>
struct FwdOne {
  static cudaError_t run(const NormArgs &a, const Plan &q, cudaStream_t s) {
    return q.threads == 256 ? go(layernorm_fwd_kernel<In, V, kPer, 256>, a, q, s)
                            : go(layernorm_fwd_kernel<In, V, kPer, kMostThreads>, a, q, s);
  }
};
template <typename In, int V, int kPer>
struct BwdOne {
  static cudaError_t run(const NormBwdArgs &a, const Plan &q, cudaStream_t s) {
    return q.threads == 256 ? go(layernorm_bwd_kernel<In, V, kPer, 256>, a, q, s)
                            : go(layernorm_bwd_kernel<In, V, kPer, kMostThreads>, a, q, s);
  }
};

template <typename In>
cudaError_t fwd_all(const NormArgs &a, cudaStream_t s) {
  const Plan q = plan(a.rows, a.D, 16 / sizeof(In), fwd_width<In>(a), 2, kSmThreads, true, true);
  return dispatch<In, FwdOne>(q, a, q, s);
}
template <typename In>
Plan plan_of(const NormBwdArgs &a) {
  constexpr int V = 16 / sizeof(In);
  const bool one = a.D % V == 0 && a.D <= 32 * V;  // (as plan() has it)
  return bwd_plan<In>(a, one ? bwd_threads<In, V, 1>() : bwd_threads<In, V, 2>(), true);
}
template <typename In>
cudaError_t bwd_all(const NormBwdArgs &a, cudaStream_t s) {
  const Plan q = plan_of<In>(a);
  const cudaError_t e = q.grid > 0 ? dispatch<In, BwdOne>(q, a, q, s) : cudaSuccess;
  return e != cudaSuccess ? e : launch_column_sum(a.partial, a.dweight, a.dbias, a.D, q.grid, 2 * a.D, s);
}

}  // namespace

cudaError_t launch_layernorm_fwd(const NormArgs &a, cudaStream_t s) {
  return a.bf16 ? fwd_all<__nv_bfloat16>(a, s) : fwd_all<float>(a, s);
}
int64_t layernorm_bwd_ctas(const NormBwdArgs &a) {
  return (a.bf16 ? plan_of<__nv_bfloat16>(a) : plan_of<float>(a)).grid;
}
cudaError_t launch_layernorm_bwd(const NormBwdArgs &a, cudaStream_t s) {
  return a.bf16 ? bwd_all<__nv_bfloat16>(a, s) : bwd_all<float>(a, s);
}

}  // namespace delta
