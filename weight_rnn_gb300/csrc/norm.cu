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
      return a.scale ? go(norm_fwd_kernel<In, V, kPer, 256, true, false>, a, q, s)
                     : go(norm_fwd_kernel<In, V, kPer, 256, false, false>, a, q, s);
    return a.scale ? go(norm_fwd_kernel<In, V, kPer, kMostThreads, true, false>, a, q, s)
                   : go(norm_fwd_kernel<In, V, kPer, kMostThreads, false, false>, a, q, s);
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
  const Plan q = bwd_plan<In>(a);
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
  const Plan q = a.bf16 ? bwd_plan<__nv_bfloat16>(a) : bwd_plan<float>(a);
  return q.grid;
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t s) {
  return a.bf16 ? bwd_all<__nv_bfloat16>(a, s) : bwd_all<float>(a, s);
}

}  // namespace delta
