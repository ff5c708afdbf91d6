// kernels.h -- internal launch interface between the C-ABI layer (api.cu)
// and the CUDA kernels.  Not installed; callers use include/delta.h.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace delta {

// Arguments of one forward call after validation.  Sizes are widened to
// 64 bits; `L` is the extended sequence length n_h * T.
struct FwdArgs {
  const void *q, *k, *v;
  const float *beta, *g, *h0;
  void *out;
  float *hT;
  int64_t B, H, T, L;
  int dk, dv, n_h, chunk;
  bool bf16;
  // channel-wise gate [B, T, H, dk] (KDA), instead of g; nullptr: none
  const float *alpha = nullptr;
};

struct StepArgs {
  const void *q, *k, *v;
  const float *beta, *g;
  float *state;
  void *out;
  int64_t B, H;
  int dk, dv, n_h;
  bool bf16;
  // channel-wise gate [B, H, dk] (KDA), instead of g; nullptr: none
  const float *alpha = nullptr;
  // input prologue applied in the kernel: -1 none (q, k, beta as given);
  // 0: q, k -> SiLU -> L2 norm, beta -> sigmoid; 1: the same, beta -> 2 sigmoid
  int beta_map = -1;
};

// The input prologue as one pass over raw inputs: rows of dk elements
// (rows_q query rows, then rows_k key rows) -> SiLU -> L2 norm, written to
// q_out / k_out in the input dtype; n_beta betas -> sigmoid (beta_map 0) or
// 2 sigmoid (beta_map 1), float32.
struct PrologueArgs {
  const void *q, *k;
  const float *beta;
  void *q_out, *k_out;
  float *beta_out;
  int64_t rows_q, rows_k, n_beta;
  int dk, beta_map;
  bool bf16;
};
cudaError_t launch_prologue(const PrologueArgs &a, cudaStream_t s);

// Gradients of the forward (float32, CUDA cores): inputs as FwdArgs plus the
// loss gradients dout (dtype) and dhT (float32, or nullptr); outputs, all
// float32: gq [B,T,H,dk], gk [B,L,H,dk], gv [B,L,H,dv], gbeta [B,L,H], gg
// [B,T,H] (when g is set) and gh0 [B,H,dk,dv] (or nullptr).  scratch holds
// bwd_scratch_floats() floats (block-start states), scratch2 `second` floats
// (the states inside one block), scratch3 `third` floats (the per-column-group
// partial sums of gq, gk, gbeta and gg; none when one group covers dv).
struct BwdArgs {
  const void *q, *k, *v, *dout;
  const float *beta, *g, *h0, *dhT;
  float *gq, *gk, *gv, *gbeta, *gg, *gh0;
  float *scratch, *scratch2, *scratch3;
  int64_t B, H, T;
  int dk, dv, n_h;
  bool bf16;
};
int64_t bwd_scratch_floats(const BwdArgs &a, int64_t *second, int64_t *third);
int64_t bwd_ctas(const BwdArgs &a);  // the grid of the backward kernel
cudaError_t launch_bwd(const BwdArgs &a, cudaStream_t s);

// Generic chunked forward on CUDA cores, float32 arithmetic, any supported
// shape.  Returns the launch error (cudaSuccess if enqueued).
cudaError_t launch_chunk_generic(const FwdArgs &a, cudaStream_t s);

// Tensor-core chunked forward (tcgen05 + TMEM + TMA) for bf16 I/O with
// dk = dv = 128 and chunk = 64: the state pass, given the T tiles the UT pass
// (launch_ut) wrote to t_mat.  Returns cudaErrorNotSupported when the shape
// is outside that set.
cudaError_t launch_chunk_tc(const FwdArgs &a, const void *t_mat, cudaStream_t s);
bool chunk_tc_supports(const FwdArgs &a);
// kernels one tensor-core forward launches (UT pass + state pass)
constexpr int kChunkTcKernels = 2;

// The intra-chunk UT transform T = (I + A)^{-1} diag(beta) of every chunk,
// bf16 [B*H*NT][64][64] row-major (tensor cores; bf16 keys, dk = 128,
// chunk = 64).  t_mat must hold ut_workspace_bytes(a) bytes, 16-byte aligned.
bool ut_supports(const FwdArgs &a);
int64_t ut_workspace_bytes(const FwdArgs &a);
cudaError_t launch_ut(const FwdArgs &a, void *t_mat, cudaStream_t s);

// Read and clear the word the tensor-core kernels set when one of their
// bounded waits gives up (0 = no error).  Synchronises the device.
cudaError_t read_and_clear_tc_error(unsigned int *word);
cudaError_t read_and_clear_ut_error(unsigned int *word);

// One warp waits, at most `polls` tries, on a barrier that nothing completes,
// then records its giving up in the same device error word.
cudaError_t launch_wait_selftest(unsigned int polls, cudaStream_t s);

// hT <- h0 (or 0) for an empty sequence (T == 0).
cudaError_t launch_state_passthrough(const FwdArgs &a, cudaStream_t s);

// One decode step, state updated in place.
cudaError_t launch_step(const StepArgs &a, cudaStream_t s);

// Effective rank of each of the BH state matrices [dk][dv] (float32) into
// erank[BH]; one block per matrix with erank_smem_bytes of shared memory.
int64_t erank_smem_bytes(int dk, int dv);
cudaError_t launch_erank(const float *state, float *erank, int64_t BH, int dk, int dv,
                         cudaStream_t s);

// The attention map of the fully parallel form for N <= 64 steps (n_h = 1):
// q, k [B][N][H][dk] (bf16 or float32), beta, g [B][N][H], attn [B][H][N][N].
cudaError_t launch_attention_map(const void *q, const void *k, const float *beta, const float *g,
                                 float *attn, int64_t B, int64_t H, int N, int dk, bool bf16,
                                 cudaStream_t s);

// The gated linear recurrence (scan.cu).  x, gate: element strides of the batch
// row (sb) and the step (st), channels contiguous; everything else contiguous.
// gate is float32 in the linear form, in x's type in the sigmoid form.
constexpr int kScanBlock = 64;  // steps between two saved states
struct ScanArgs {
  const void *x, *gate;
  const float *h0;       // nullptr: 0
  const int *lengths;    // [B], clamped to [0, T]; nullptr: T
  void *out;
  float *hT, *states;    // states [B][ceil(T / kScanBlock)][D] or nullptr
  int64_t B, T, D, x_sb, x_st, g_sb, g_st;
  bool bf16, sigmoid;
};
struct ScanBwdArgs : ScanArgs {  // states is read; out, hT and h0 are unused
  const void *dout;
  const float *dhT;      // nullptr: 0
  void *dx, *dgate;
  float *dh0;            // or nullptr
};
cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s);
cudaError_t launch_scan_bwd(const ScanBwdArgs &a, cudaStream_t s);
// one token: h0 is the state before and hT the state after (the same memory)
cudaError_t launch_scan_step(const ScanArgs &a, cudaStream_t s);
cudaError_t launch_exchange_selftest(unsigned int polls, cudaStream_t s);
cudaError_t read_and_clear_scan_error(unsigned int *word);
// hT <- h0 (or 0): a sequence without steps
cudaError_t launch_scan_passthrough(const float *h0, float *hT, int64_t n, cudaStream_t s);

// Residual addition and RMS norm (norm.cu), rows of D elements.  Row strides
// ld* in elements; weight is float32 or, with w_bf16, bfloat16.
struct NormArgs {
  const void *x, *residual;  // residual nullptr: the sum is x and is not written
  const void *weight;
  void *y;                   // input type, or e4m3 with scale set
  void *sum;                 // [rows][D] contiguous
  float *rstd, *scale;       // [rows]; nullptr: not written
  int64_t rows, D, ldx, ldr;
  float eps;
  bool bf16, w_bf16;
};
struct NormBwdArgs {
  const void *dy, *sum, *weight, *dsum;  // dsum nullptr: 0
  const float *rstd;
  void *dx;
  float *dweight, *partial;  // partial [norm_bwd_ctas()][D]
  int64_t rows, D;
  bool bf16, w_bf16;
};
constexpr int kNormMaxD = 8192;
cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t s);
int64_t norm_bwd_ctas(const NormBwdArgs &a);
cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t s);

// The linear layer (linear.cu, linear_tc.cu): out = act(x w^T + bias) +
// residual, x [M][K], w [N][K], out and pre [M][N] contiguous.  kind: the type
// of x and w; out, pre and residual are float32 for float32 operands, else
// bfloat16.  e4m3 operands come with a scale per row of x and of w.
enum LinearKind { kLinF32, kLinBf16, kLinE4m3 };
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2;
struct LinearArgs {
  const void *x, *w, *bias, *residual;  // bias, residual: nullptr for none
  const float *x_scale, *w_scale;
  void *out, *pre;                      // pre: nullptr if not wanted
  int64_t M, N, K, ldx, ldw, ldr;
  int act;
  LinearKind kind;
  bool bias_bf16;
};
// A matrix product of two operands for the tensor-core kernel, D[M][N] = sum_k
// A(m, k) B(n, k).  *_mn: the operand lies with m (or n) contiguous and k as
// the row (ld apart), else with k contiguous.  Base addresses and ld in bytes
// are multiples of 16.
struct GemmArgs {
  const void *a, *b;
  int64_t lda, ldb, K;
  bool a_mn, b_mn;
  LinearArgs epi;  // M, N, out and the epilogue
  bool dependent;  // follows a kernel of the same call
};
cudaError_t launch_gemm_tc(const GemmArgs &g, cudaStream_t s);
// about how long it takes
double gemm_tc_us(int64_t M, int64_t N, int64_t K, bool f8);
cudaError_t read_and_clear_linear_error(unsigned int *word);
// streams the weight once for every 16 rows of x: for M <= kLinSmallM once
constexpr int kLinSmallM = 16;
cudaError_t launch_linear_small(const LinearArgs &a, cudaStream_t s);
// about how long it takes
double linear_small_us(int64_t M, int64_t N, int64_t K, bool f8, bool whole);
// all gradients of a small bfloat16 layer (those whose pointers are set), in one
// launch without scratch
constexpr double kSmallBwdUs = 14;
bool small_bwd_fits(int64_t M, int64_t N, int64_t K);
cudaError_t launch_small_bwd(const void *x, const void *w, const void *dout, const void *pre, void *dx, void *dw,
                             float *dbias, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw, int act,
                             cudaStream_t s);
// float32 on the CUDA cores, operands with any strides (elements)
cudaError_t launch_gemm_f32(const LinearArgs &epi, const float *a, int64_t am, int64_t ak, const float *b,
                            int64_t bn, int64_t bk, int64_t K, cudaStream_t s);
// rows x cols elements of `size` bytes into rows of ldp elements
cudaError_t launch_pack(const void *src, void *dst, int64_t rows, int64_t cols, int64_t ld, int64_t ldp,
                        int size, bool dependent, cudaStream_t s);
// dpre = dout * act'(pre) in rows of ldp elements where dpre is set, and dbias = its column sums in float32 where dbias is set
struct DpreArgs {
  const void *dout, *pre;
  void *dpre;
  float *dbias, *partial;  // partial [dpre_parts()][N]
  int64_t M, N, ldp;
  int act;
  bool bf16;
};
int64_t dpre_parts(const DpreArgs &a);
cudaError_t launch_dpre(const DpreArgs &a, cudaStream_t s);
// out[c] = sum over n partial rows (norm.cu)
cudaError_t launch_column_sum(const float *partial, float *out, int64_t n, int64_t D, cudaStream_t s);

}  // namespace delta
