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
#include "norm.cuh"

namespace delta {
namespace {

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

// dw[d] = sum of n partial rows (db from the first `first` columns on): C columns a CTA, every R-th row to a thread,
// then a warp a column over the R sums.  Few columns take 8 at a time (a sector
// of each row), so that there are CTAs; many take 32 (4096 x 8192: 53 us with
// the gradients before it, 57 with 8).
template <int C>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *partial, float *dw, float *db, int64_t first,
                                                          int64_t n, int64_t D) {
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
  if (lane == 0 && c < D) *(c < first ? dw + c : db + (c - first)) = v;
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
  const Plan q = plan(a.rows, a.D, 16 / sizeof(In), fwd_width<In>(a), 2, a.scale ? kQuantThreads : kSmThreads, true);
  return dispatch<In, FwdOne>(q, a, q, s);
}

template <typename In>
cudaError_t bwd_all(const NormBwdArgs &a, cudaStream_t s) {
  const Plan q = bwd_plan<In>(a, kSmThreads);
  cudaError_t e = q.grid > 0 ? dispatch<In, BwdOne>(q, a, q, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  return launch_column_sum(a.partial, a.dweight, q.grid, a.D, s);
}

}  // namespace

cudaError_t launch_column_sum(const float *partial, float *out, float *rest, int64_t first, int64_t n, int64_t D,
                              cudaStream_t s) {
  return D < 1024 ? chain_launch(column_sum_kernel<8>, dim3((unsigned)((D + 7) / 8)), dim3(8, 128), 0, 1, true, s,
                                 partial, out, rest, first, n, D)
                  : chain_launch(column_sum_kernel<32>, dim3((unsigned)((D + 31) / 32)), dim3(32, 32), 0, 1, true, s,
                                 partial, out, rest, first, n, D);
}
cudaError_t launch_column_sum(const float *partial, float *out, int64_t n, int64_t D, cudaStream_t s) {
  return launch_column_sum(partial, out, nullptr, D, n, D, s);
}

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s) {
  return a.bf16 ? fwd_all<__nv_bfloat16>(a, s) : fwd_all<float>(a, s);
}

int64_t norm_bwd_ctas(const NormBwdArgs &a) {
  const Plan q = a.bf16 ? bwd_plan<__nv_bfloat16>(a, kSmThreads) : bwd_plan<float>(a, kSmThreads);
  return q.grid;
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t s) {
  return a.bf16 ? bwd_all<__nv_bfloat16>(a, s) : bwd_all<float>(a, s);
}

}  // namespace delta
