// layernorm.cu -- the residual addition with layer norm:
//
//   t = x + r,   mean = mean_d t,   rstd = (mean_d (t - mean)^2 + eps)^{-1/2},
//   y = (t - mean) rstd w + b
//
// on the kernels of norm.cuh (norm.cu has how a row is shared out and why).  The
// row stays in registers between its two sums, so the variance is that of the
// differences and the data is read once.  Gradient, with t^ = (t - mean) rstd:
//
//   dx = rstd (w dy - mean_d(w dy) - t^ mean_d(w dy t^)) + dsum,
//   dw = sum over rows of dy t^,   db = sum over rows of dy
//
// HBM-bound like the root-mean-square norm.
#include "norm.cuh"

namespace delta {
namespace {

template <typename In, int V, int kPer>
struct FwdOne {
  static cudaError_t run(const NormArgs &a, const Plan &q, cudaStream_t s) {
    return q.threads == 256 ? go(norm_fwd_kernel<In, V, kPer, 256, false, true>, a, q, s)
                            : go(norm_fwd_kernel<In, V, kPer, kMostThreads, false, true>, a, q, s);
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
  const Plan q = plan(a.rows, a.D, 16 / sizeof(In), fwd_width<In>(a), 2, kSmThreads, true);
  return dispatch<In, FwdOne>(q, a, q, s);
}
template <typename In>
cudaError_t bwd_all(const NormBwdArgs &a, cudaStream_t s) {
  const Plan q = bwd_plan<In>(a);
  const cudaError_t e = q.grid > 0 ? dispatch<In, BwdOne>(q, a, q, s) : cudaSuccess;
  return e != cudaSuccess ? e : launch_column_sum(a.partial, a.dweight, a.dbias, a.D, q.grid, 2 * a.D, s);
}

}  // namespace

cudaError_t launch_layernorm_fwd(const NormArgs &a, cudaStream_t s) {
  return a.bf16 ? fwd_all<__nv_bfloat16>(a, s) : fwd_all<float>(a, s);
}
int64_t layernorm_bwd_ctas(const NormBwdArgs &a) {
  return (a.bf16 ? bwd_plan<__nv_bfloat16>(a) : bwd_plan<float>(a)).grid;
}
cudaError_t launch_layernorm_bwd(const NormBwdArgs &a, cudaStream_t s) {
  return a.bf16 ? bwd_all<__nv_bfloat16>(a, s) : bwd_all<float>(a, s);
}

}  // namespace delta
