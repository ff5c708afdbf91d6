// block_api.cu -- the C ABI of the operators that stand around the token
// mixers in a block (scan, norm, linear): argument checks, scratch and launches, with
// the conventions of api.cu: nothing is synchronised, errors are returned
// before anything is enqueued.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/delta.h"
#include "api_common.h"
#include "block_common.h"
#include "kernels.h"

namespace {

using namespace delta::api;

// bytes from the first to the last element of a [B][T][D] view
int64_t view_bytes(int64_t B, int64_t T, int64_t D, int64_t sb, int64_t st, int64_t e) {
  return ((B - 1) * sb + (T - 1) * st + D) * e;
}

int scan_sizes(int B, int T, int D, int64_t x_sb, int64_t x_st, int64_t g_sb, int64_t g_st,
               delta_dtype dtype, delta_scan_form form, delta::ScanArgs &a) {
  if (B < 0 || T < 0 || D < 0) return fail(DELTA_ERR_INVALID, "negative size B=%d T=%d D=%d", B, T, D);
  int st;
  if ((st = check_dtype(dtype)) != DELTA_OK) return st;
  if (form != DELTA_SCAN_LINEAR && form != DELTA_SCAN_SIGMOID)
    return fail(DELTA_ERR_INVALID, "unknown scan form %d", (int)form);
  a.B = B; a.T = T; a.D = D;
  // the stride of an axis with one entry is never used
  a.x_sb = B > 1 ? x_sb : 0; a.x_st = T > 1 ? x_st : 0;
  a.g_sb = B > 1 ? g_sb : 0; a.g_st = T > 1 ? g_st : 0;
  a.bf16 = dtype == DELTA_BF16;
  a.sigmoid = form == DELTA_SCAN_SIGMOID;
  if ((int64_t)B * T >= kMaxElems / (D > 0 ? D : 1))
    return fail(DELTA_ERR_UNSUPPORTED, "B*T*D too large");
  for (const int64_t s : {a.x_sb, a.x_st, a.g_sb, a.g_st})
    if (s < 0 || s >= kMaxElems) return fail(DELTA_ERR_INVALID, "stride %lld out of range", (long long)s);
  if ((B > 1 && a.x_sb >= kMaxElems / B) || (T > 1 && a.x_st >= kMaxElems / T) ||
      (B > 1 && a.g_sb >= kMaxElems / B) || (T > 1 && a.g_st >= kMaxElems / T))
    return fail(DELTA_ERR_UNSUPPORTED, "strides too large");
  // a CTA, or for a few rows a cluster of at most 16, per row and 32 channels
  if ((int64_t)B * ((D + 31) / 32) >= (int64_t(1) << 31) / 8)
    return fail(DELTA_ERR_UNSUPPORTED, "B*D=%lld too large", (long long)B * D);
  return DELTA_OK;
}

int scan_pointers(const delta::ScanArgs &a, delta_dtype dtype) {
  if (!a.x || !a.gate) return fail(DELTA_ERR_INVALID, "x and gate must be non-NULL");
  const int64_t e = esize(dtype), ge = a.sigmoid ? e : 4;
  if (!aligned_to(a.x, e) || !aligned_to(a.gate, ge) || !aligned_to(a.lengths, 4))
    return fail(DELTA_ERR_ALIGN, "x, gate and lengths must be aligned to their elements");
  return DELTA_OK;
}

Span span_x(const delta::ScanArgs &a, delta_dtype dt) {
  return {"x", range(a.x, view_bytes(a.B, a.T, a.D, a.x_sb, a.x_st, esize(dt)))};
}
Span span_gate(const delta::ScanArgs &a, delta_dtype dt) {
  return {"gate", range(a.gate, view_bytes(a.B, a.T, a.D, a.g_sb, a.g_st, a.sigmoid ? esize(dt) : 4))};
}

int norm_sizes(int64_t rows, int D, int64_t ldx, int64_t ldr, float eps, delta_dtype dtype,
               delta_dtype wdtype) {
  if (rows < 0 || D < 0) return fail(DELTA_ERR_INVALID, "negative size rows=%lld D=%d", (long long)rows, D);
  int st;
  if ((st = check_dtype(dtype)) != DELTA_OK || (st = check_dtype(wdtype)) != DELTA_OK) return st;
  if (!(eps > 0.f)) return fail(DELTA_ERR_INVALID, "eps=%g must be positive", (double)eps);
  if (D > delta::kNormMaxD)
    return fail(DELTA_ERR_UNSUPPORTED, "D=%d: the norm is built for D <= %d", D, delta::kNormMaxD);
  if (rows >= kMaxElems / (D > 0 ? D : 1)) return fail(DELTA_ERR_UNSUPPORTED, "rows*D too large");
  if (rows > 1 && (ldx < D || ldr < D || ldx >= kMaxElems / rows || ldr >= kMaxElems / rows))
    return fail(DELTA_ERR_INVALID, "row strides %lld, %lld must be at least D=%d", (long long)ldx,
                (long long)ldr, D);
  return DELTA_OK;
}

enum class Norm { kRms, kRmsQuant, kLayer };

int run_norm_fwd(Norm kind, const void *x, const void *residual, const void *weight, const void *bias, void *y,
                 float *scale, void *sum_out, float *mean, float *rstd, int64_t rows, int D, int64_t ldx, int64_t ldr,
                 float eps, delta_dtype dtype, delta_dtype wdtype, delta_dtype bdtype, struct CUstream_st *stream) {
  const bool quant = kind == Norm::kRmsQuant;
  int st;
  if ((st = norm_sizes(rows, D, ldx, residual ? ldr : D, eps, dtype, wdtype)) != DELTA_OK) return st;
  if ((st = check_dtype(bdtype)) != DELTA_OK) return st;
  if (rows == 0 || D == 0) return DELTA_OK;
  if (!x || !weight || !y || (quant && !scale))
    return fail(DELTA_ERR_INVALID, "x, weight, the output and its scales must be non-NULL");
  if (sum_out && !residual) return fail(DELTA_ERR_INVALID, "sum_out without a residual: the sum is x");
  const int64_t e = esize(dtype), we = esize(wdtype);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(weight, we) || !aligned_to(bias, esize(bdtype)))
    return fail(DELTA_ERR_ALIGN, "x, residual and the weights must be aligned to their elements");
  if (!aligned16(y) || !aligned16(sum_out) || !aligned16(mean) || !aligned16(rstd) || !aligned16(scale))
    return fail(DELTA_ERR_ALIGN, "every output must be 16-byte aligned");
  const Span xs = {"x", range(x, ((rows - 1) * ldx + D) * e)};
  const Span rs = {"residual", range(residual, ((rows - 1) * ldr + D) * e)};
  const Span ws = {"weight", range(weight, D * we)};
  const Span ys = {"y", range(y, rows * D * (quant ? 1 : e))};
  const Span ss = {"sum_out", range(sum_out, rows * D * e)};
  const Span ds = {"rstd", range(rstd, rows * 4)}, cs = {"y_scale", range(scale, rows * 4)};
  const Span bs = {"bias", range(bias, D * esize(bdtype))}, ms = {"mean", range(mean, rows * 4)};
  if ((st = check_overlap({ys, ds, cs, ms}, {xs, rs, ws, bs})) != DELTA_OK) return st;
  if ((st = check_overlap({ss}, {ws, bs, ys, ds, cs, ms})) != DELTA_OK) return st;
  // the residual stream may be updated in place: the same rows, or none
  const struct {
    Span span;
    int64_t ld;
  } inputs[] = {{xs, ldx}, {rs, ldr}};
  for (const auto &in : inputs) {
    const bool same = in.span.r.lo == ss.r.lo && (rows == 1 || in.ld == D);
    if (overlap(ss.r, in.span.r) && !same)
      return fail(DELTA_ERR_INVALID, "sum_out partly overlaps %s", in.span.name);
  }
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  delta::NormArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.sum = sum_out; a.rstd = rstd;
  a.scale = quant ? scale : nullptr;
  a.bias = bias; a.b_bf16 = bdtype == DELTA_BF16; a.mean = mean;
  a.rows = rows; a.D = D; a.ldx = rows > 1 ? ldx : 0; a.ldr = rows > 1 ? ldr : 0;
  a.eps = eps; a.bf16 = dtype == DELTA_BF16; a.w_bf16 = wdtype == DELTA_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = kind == Norm::kLayer ? delta::launch_layernorm_fwd(a, s) : delta::launch_norm_fwd(a, s);
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "norm kernel launch");
}

int run_norm_bwd(Norm kind, const void *dy, const void *sum, const void *weight, const float *mean, const float *rstd,
                 const void *dsum, void *dx, float *dweight, float *dbias, int64_t rows, int D, delta_dtype dtype,
                 delta_dtype wdtype, struct CUstream_st *stream) {
  const bool layer = kind == Norm::kLayer;
  int st;
  if ((st = norm_sizes(rows, D, D, D, 1.f, dtype, wdtype)) != DELTA_OK) return st;
  if (D == 0) return DELTA_OK;
  if (!dweight || !weight || (layer && !dbias))
    return fail(DELTA_ERR_INVALID, "weight and the gradients must be non-NULL");
  if (rows > 0 && (!dy || !sum || !rstd || !dx || (layer && !mean)))
    return fail(DELTA_ERR_INVALID, "dy, sum, the rows' statistics and dx must be non-NULL");
  const int64_t e = esize(dtype), we = esize(wdtype);
  if (!aligned16(dy) || !aligned16(sum) || !aligned16(dsum) || !aligned16(dx) || !aligned16(mean) || !aligned16(rstd) ||
      !aligned16(dweight) || !aligned16(dbias) || !aligned_to(weight, we))
    return fail(DELTA_ERR_ALIGN, "every pointer must be 16-byte aligned (weight: to its elements)");
  const Span ys = {"dy", range(dy, rows * D * e)}, ss = {"sum", range(sum, rows * D * e)};
  const Span gs = {"dsum", range(dsum, rows * D * e)}, ws = {"weight", range(weight, D * we)};
  const Span rs = {"rstd", range(rstd, rows * 4)}, ms = {"mean", range(mean, rows * 4)};
  const Span xs = {"dx", range(dx, rows * D * e)}, dws = {"dweight", range(dweight, (int64_t)D * 4)};
  const Span dbs = {"dbias", range(dbias, (int64_t)D * 4)};
  if ((st = check_overlap({xs, dws, dbs}, {ss, ws, rs, ms})) != DELTA_OK) return st;
  if ((st = check_overlap({dws, dbs}, {ys, gs})) != DELTA_OK) return st;
  for (const Span &in : {ys, gs})  // dx may take dy's or dsum's place
    if (overlap(xs.r, in.r) && xs.r.lo != in.r.lo)
      return fail(DELTA_ERR_INVALID, "dx partly overlaps %s", in.name);
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  delta::NormBwdArgs a{};
  a.dy = dy; a.sum = sum; a.weight = weight; a.mean = mean; a.rstd = rstd; a.dsum = dsum; a.dx = dx;
  a.dweight = dweight; a.dbias = dbias;
  a.rows = rows; a.D = D; a.bf16 = dtype == DELTA_BF16; a.w_bf16 = wdtype == DELTA_BF16;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t n = layer ? delta::layernorm_bwd_ctas(a) * 2 * D : delta::norm_bwd_ctas(a) * D;
  Scratch scr(s);
  scr.want(n * 4);
  cudaError_t err = scr.take();
  if (err != cudaSuccess) return cuda_fail(err, "scratch allocation");
  a.partial = static_cast<float *>(scr.cut(n * 4));
  err = layer ? delta::launch_layernorm_bwd(a, s) : delta::launch_norm_bwd(a, s);
  const cudaError_t ef = scr.release();
  if (err != cudaSuccess) return cuda_fail(err, "norm backward launch");
  return ef == cudaSuccess ? DELTA_OK : cuda_fail(ef, "scratch release");
}

int linear_sizes(int M, int N, int K, int64_t ldx, int64_t ldw, int64_t ldr, delta_act act) {
  if (M < 0 || N < 0 || K < 0) return fail(DELTA_ERR_INVALID, "negative size M=%d N=%d K=%d", M, N, K);
  if (act != DELTA_ACT_NONE && act != DELTA_ACT_SILU && act != DELTA_ACT_GELU)
    return fail(DELTA_ERR_INVALID, "unknown activation %d", (int)act);
  if (K == 0) return fail(DELTA_ERR_INVALID, "K must be positive");
  if ((M > 1 && (ldx < K || ldr < N)) || (N > 1 && ldw < K))
    return fail(DELTA_ERR_INVALID, "row strides ldx=%lld ldw=%lld ldr=%lld must cover a row", (long long)ldx,
                (long long)ldw, (long long)ldr);
  const int64_t most = int64_t(1) << 31;
  if (ldx >= most || ldw >= most || ldr >= most) return fail(DELTA_ERR_UNSUPPORTED, "row stride too large");
  return DELTA_OK;
}

// an operand of the tensor-core product: usable as it lies, or to be packed
// into rows that are multiples of 16 bytes
struct Operand {
  const void *p;
  int64_t rows, cols, ld;
  int size;
  bool whole() const { return aligned16(p) && ld * size % 16 == 0; }
  int64_t ldp() const { return up(cols, 128 / size); }  // whole lines: a copied box row touches one
  int64_t bytes() const { return rows * ldp() * size; }
  // after: a kernel of this call has been launched
  cudaError_t pack(Scratch &scr, bool &after, cudaStream_t s) {
    if (whole()) return cudaSuccess;
    void *to = scr.cut(bytes());
    const cudaError_t e = delta::launch_pack(p, to, rows, cols, ld, ldp(), size, after, s);
    after = true;
    p = to;
    ld = ldp();
    return e;
  }
};
Operand operand(const void *p, int64_t rows, int64_t cols, int64_t ld, int size) {
  return Operand{p, rows, cols, rows > 1 ? ld : up(cols, 16 / size), size};
}

constexpr double kPackUs = 6.0;  // scratch and two more kernels

cudaError_t linear_forward(const delta::LinearArgs &a, cudaStream_t s) {
  if (a.kind == delta::kLinF32)
    return delta::launch_gemm_f32(a, static_cast<const float *>(a.x), a.ldx, 1, static_cast<const float *>(a.w),
                                  a.ldw, 1, a.K, s);
  if (a.M <= delta::kLinSmallM) return delta::launch_linear_small(a, s);
  const int size = a.kind == delta::kLinE4m3 ? 1 : 2;
  Operand x = operand(a.x, a.M, a.K, a.ldx, size), w = operand(a.w, a.N, a.K, a.ldw, size);
  // Small products take the streaming kernel too, with a pass over w for every
  // 16 rows, where that is shorter than filling the tensor cores' pipeline (M64
  // N2048 K512 in 4.2 us for 5.2, M128 N2048 K512 in 6.7 for 5.3), or than
  // packing operands first, two launches and scratch more (M93 N133 K473 in 4.0
  // for 17).
  const bool f8 = size == 1, pack = !x.whole() || !w.whole();
  if (delta::linear_small_us(a.M, a.N, a.K, f8, !pack) < delta::gemm_tc_us(a.M, a.N, a.K, f8) + (pack ? kPackUs : 0.0))
    return delta::launch_linear_small(a, s);
  Scratch scr(s);
  if (!x.whole()) scr.want(x.bytes());
  if (!w.whole()) scr.want(w.bytes());
  cudaError_t err = scr.take();
  if (err != cudaSuccess) return err;
  bool after = false;
  err = x.pack(scr, after, s);
  if (err == cudaSuccess) err = w.pack(scr, after, s);
  if (err == cudaSuccess) err = delta::launch_gemm_tc({x.p, w.p, x.ld, w.ld, a.K, false, false, a, after}, s);
  const cudaError_t ef = scr.release();
  return err != cudaSuccess ? err : ef;
}

int run_linear(const void *x, const void *w, const float *x_scale, const float *w_scale, const void *bias,
               const void *residual, void *out, void *pre, int M, int N, int K, int64_t ldx, int64_t ldw,
               int64_t ldr, delta_act act, delta::LinearKind kind, delta_dtype bdtype,
               struct CUstream_st *stream) {
  int st;
  if ((st = linear_sizes(M, N, K, ldx, ldw, residual ? ldr : N, act)) != DELTA_OK) return st;
  if ((st = check_dtype(bdtype)) != DELTA_OK) return st;
  if (M == 0 || N == 0) return DELTA_OK;
  if (!x || !w || !out) return fail(DELTA_ERR_INVALID, "x, w and out must be non-NULL");
  const bool quant = kind == delta::kLinE4m3;
  if (quant && (!x_scale || !w_scale)) return fail(DELTA_ERR_INVALID, "the scales must be non-NULL");
  const int64_t e = kind == delta::kLinF32 ? 4 : quant ? 1 : 2, oe = kind == delta::kLinF32 ? 4 : 2;
  if (!aligned_to(x, e) || !aligned_to(w, e) || !aligned_to(residual, oe) || !aligned_to(bias, esize(bdtype)) ||
      !aligned_to(x_scale, 4) || !aligned_to(w_scale, 4))
    return fail(DELTA_ERR_ALIGN, "every input must be aligned to its elements");
  if (!aligned16(out) || !aligned16(pre)) return fail(DELTA_ERR_ALIGN, "out and pre must be 16-byte aligned");
  if (M <= 1) ldx = K, ldr = N;
  if (N <= 1) ldw = K;
  const int64_t m = M, n = N, k = K;
  const Span rs = {"residual", range(residual, ((m - 1) * ldr + n) * oe)};
  const Span os = {"out", range(out, m * n * oe)}, ps = {"pre", range(pre, m * n * oe)};
  if ((st = check_overlap({os, ps}, {Span{"x", range(x, ((m - 1) * ldx + k) * e)},
                                     Span{"w", range(w, ((n - 1) * ldw + k) * e)},
                                     Span{"bias", range(bias, n * esize(bdtype))},
                                     Span{"x_scale", range(x_scale, m * 4)},
                                     Span{"w_scale", range(w_scale, n * 4)}})) != DELTA_OK)
    return st;
  if ((st = check_overlap({ps}, {rs})) != DELTA_OK) return st;
  if (overlap(os.r, rs.r) && !(os.r.lo == rs.r.lo && ldr == n))
    return fail(DELTA_ERR_INVALID, "out partly overlaps residual");
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  delta::LinearArgs a{};
  a.x = x; a.w = w; a.bias = bias; a.residual = residual; a.x_scale = x_scale; a.w_scale = w_scale;
  a.out = out; a.pre = pre; a.M = m; a.N = n; a.K = k; a.ldx = ldx; a.ldw = ldw; a.ldr = ldr;
  a.act = (int)act; a.kind = kind; a.bias_bf16 = bdtype == DELTA_BF16;
  const cudaError_t err = linear_forward(a, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "linear layer");
}

// Gradients of a float32 or bfloat16 layer.  dpre = dout act'(pre) is formed
// once, in the operands' type: for bfloat16 a rounding of at most 2^-8 of each
// term of dx and dw.  That is chosen: at 2048^3 dx and dw are off by 2.35e-3 of
// their norm, 1.66e-3 of it by the rounding of the outputs themselves; to carry
// what dpre loses as a second operand would give that 1.66e-3, and double the
// products, 87 of the 110 us at M4096 N4096 K2048.  Layers that take one launch
// (small_bwd_fits) form dpre in registers on the CUDA cores, where rounding it
// would only cost, so they have the smaller error; a layer's sizes alone decide.
// dbias sums the unrounded terms.  glu: the gated layer, whose w has N rows in two
// halves; dpre has N columns and dout half as many.
cudaError_t linear_backward(const void *x, const void *w, const void *dout, const void *pre, void *dx, void *dw,
                            float *dbias, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw, int act,
                            bool bf16, bool glu, cudaStream_t s) {
  const int64_t e = bf16 ? 2 : 4;
  cudaError_t err = cudaSuccess;
  if (M == 0 || N == 0) {  // empty sums
    if (dw && N > 0) err = cudaMemsetAsync(dw, 0, (size_t)(N * K * e), s);
    if (err == cudaSuccess && dbias && N > 0) err = cudaMemsetAsync(dbias, 0, (size_t)N * 4, s);
    if (err == cudaSuccess && dx && M > 0) err = cudaMemsetAsync(dx, 0, (size_t)(M * K * e), s);
    return err;
  }
  if (bf16 && delta::small_bwd_fits(M, N, K))
    return delta::launch_small_bwd(x, w, dout, pre, dx, dw, dbias, M, N, K, ldx, ldw, act, glu, s);
  const bool form = (dx || dw) && (glu || act != delta::kActNone || (bf16 && N % 8 != 0));
  delta::DpreArgs d{};
  d.dout = dout; d.pre = pre; d.dbias = dbias; d.M = M; d.N = glu ? N / 2 : N; d.act = act; d.bf16 = bf16; d.glu = glu;
  d.ldp = form && bf16 ? up(N, 64) : N;
  Operand ox = operand(x, M, K, ldx, (int)e), ow = operand(w, N, K, ldw, (int)e);
  const bool packx = bf16 && dw && !ox.whole(), packw = bf16 && dx && !ow.whole();
  Scratch scr(s);
  if (form) scr.want(M * d.ldp * e), d.dpre = const_cast<void *>(dout);  // (a stand-in: aligned, set below)
  const int64_t parts = dbias ? delta::dpre_parts(d) : 0;
  if (dbias) scr.want(parts * N * 4);
  if (packx) scr.want(ox.bytes());
  if (packw) scr.want(ow.bytes());
  if ((err = scr.take()) != cudaSuccess) return err;
  d.dpre = form ? scr.cut(M * d.ldp * e) : nullptr;
  if (dbias) d.partial = static_cast<float *>(scr.cut(parts * N * 4));
  bool after = form || dbias;
  if (after) err = delta::launch_dpre(d, s);
  if (err == cudaSuccess && packx) err = ox.pack(scr, after, s);
  if (err == cudaSuccess && packw) err = ow.pack(scr, after, s);
  const void *g = form ? d.dpre : dout;
  delta::LinearArgs p{};
  p.kind = bf16 ? delta::kLinBf16 : delta::kLinF32;
  delta::LinearArgs px = p, pw = p;  // of dx, of dw
  px.out = dx, px.M = M, px.N = K, pw.out = dw, pw.M = N, pw.N = K;
  const delta::GemmArgs to_x = {g, ow.p, d.ldp, ow.ld, N, false, true, px, after};
  delta::GemmArgs to_w = {g, ox.p, d.ldp, ox.ld, M, true, true, pw, after};
  if (err == cudaSuccess && bf16 && dx && dw && delta::gradients_fit(to_x, to_w)) {
    err = delta::launch_gradients_tc(to_x, to_w, s);
    const cudaError_t ef = scr.release();
    return err != cudaSuccess ? err : ef;
  }
  if (err == cudaSuccess && dx)
    err = bf16 ? delta::launch_gemm_tc(to_x, s)
               : delta::launch_gemm_f32(px, static_cast<const float *>(g), d.ldp, 1, static_cast<const float *>(w), 1,
                                        ldw, N, s);
  to_w.dependent = after || dx;
  if (err == cudaSuccess && dw)
    err = bf16 ? delta::launch_gemm_tc(to_w, s)
               : delta::launch_gemm_f32(pw, static_cast<const float *>(g), 1, d.ldp, static_cast<const float *>(x), 1,
                                        ldx, M, s);
  const cudaError_t ef = scr.release();
  return err != cudaSuccess ? err : ef;
}

// The gated layer; a.N columns of the output, w [2 N][K], pre [M][2 N].
cudaError_t glu_forward(const delta::LinearArgs &a, cudaStream_t s) {
  Scratch scr(s);
  cudaError_t err;
  if (a.kind == delta::kLinF32) {
    delta::LinearArgs g = a;
    g.N = 2 * a.N, g.act = delta::kActNone, g.out = a.pre, g.pre = nullptr;
    if (!a.pre) {
      scr.want(a.M * g.N * 4);
      if ((err = scr.take()) != cudaSuccess) return err;
      g.out = scr.cut(a.M * g.N * 4);
    }
    err = delta::launch_gemm_f32(g, static_cast<const float *>(a.x), a.ldx, 1, static_cast<const float *>(a.w), a.ldw, 1,
                                 a.K, s);
    if (err == cudaSuccess)
      err = delta::launch_glu_act(static_cast<const float *>(g.out), static_cast<float *>(a.out), a.M, a.N, a.act, s);
  } else {
    Operand x = operand(a.x, a.M, a.K, a.ldx, 2), w = operand(a.w, 2 * a.N, a.K, a.ldw, 2);
    const bool pack = !x.whole() || !w.whole();
    // few rows and small products stream w, as in linear_forward
    if (a.M <= delta::kLinSmallM || delta::linear_small_us(a.M, 2 * a.N, a.K, false, !pack) <
                                        delta::gemm_tc_us(a.M, 2 * a.N, a.K, false) + (pack ? kPackUs : 0.0))
      return delta::launch_glu_small(a, s);
    if (!x.whole()) scr.want(x.bytes());
    if (!w.whole()) scr.want(w.bytes());
    if ((err = scr.take()) != cudaSuccess) return err;
    bool after = false;
    err = x.pack(scr, after, s);
    if (err == cudaSuccess) err = w.pack(scr, after, s);
    if (err == cudaSuccess) err = delta::launch_glu_tc({x.p, w.p, x.ld, w.ld, a.K, false, false, a, after}, s);
  }
  const cudaError_t ef = scr.release();
  return err != cudaSuccess ? err : ef;
}

int glu_sizes(int M, int N, int K, int64_t ldx, int64_t ldw, delta_act act, delta_dtype dtype) {
  const int st = check_dtype(dtype);
  if (st != DELTA_OK) return st;
  if (N >= (1 << 30)) return fail(DELTA_ERR_UNSUPPORTED, "N=%d: two halves of it must be below 2^31", N);
  return linear_sizes(M, 2 * N, K, ldx, ldw, 2 * (int64_t)N, act);
}

}  // namespace

extern "C" {

int delta_scan_fwd(const void *x, const void *gate, const float *h0, const int *lengths, void *out,
                   float *hT, float *states, int B, int T, int D, int64_t x_sb, int64_t x_st,
                   int64_t g_sb, int64_t g_st, delta_dtype dtype, delta_scan_form form,
                   struct CUstream_st *stream) {
  delta::ScanArgs a{};
  int st;
  if ((st = scan_sizes(B, T, D, x_sb, x_st, g_sb, g_st, dtype, form, a)) != DELTA_OK) return st;
  if (a.B * a.D == 0) return DELTA_OK;
  a.x = x; a.gate = gate; a.h0 = h0; a.lengths = lengths; a.out = out; a.hT = hT; a.states = states;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned16(h0) || !aligned16(out) || !aligned16(hT) || !aligned16(states))
    return fail(DELTA_ERR_ALIGN, "h0, out, hT and states must be 16-byte aligned");
  const int64_t n = a.B * a.D;
  const Span hs = {"h0", range(h0, n * 4)}, ts = {"hT", range(hT, n * 4)};
  if (hT != h0 && overlap(ts.r, hs.r)) return fail(DELTA_ERR_INVALID, "hT partly overlaps h0");
  if (T == 0) {
    if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
    const cudaError_t err = delta::launch_scan_passthrough(h0, hT, n, s);
    return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "state passthrough");
  }
  if ((st = scan_pointers(a, dtype)) != DELTA_OK) return st;
  if (!out) return fail(DELTA_ERR_INVALID, "out must be non-NULL");
  const Span xs = span_x(a, dtype), gs = span_gate(a, dtype), ls = {"lengths", range(lengths, B * 4)};
  const Span os = {"out", range(out, n * T * esize(dtype))};
  const Span ss = {"states", range(states, n * ((T + delta::kScanBlock - 1) / delta::kScanBlock) * 4)};
  if ((st = check_overlap({os, ss}, {xs, gs, ls, hs})) != DELTA_OK) return st;
  if ((st = check_overlap({ts}, {xs, gs, ls, os, ss})) != DELTA_OK) return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  const cudaError_t err = delta::launch_scan_fwd(a, s);
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "scan kernel launch");
}

int delta_scan_step(const void *x, const void *gate, float *state, void *out, int B, int D, int64_t x_sb,
                    int64_t g_sb, delta_dtype dtype, delta_scan_form form, struct CUstream_st *stream) {
  delta::ScanArgs a{};
  int st;
  if ((st = scan_sizes(B, 1, D, x_sb, 0, g_sb, 0, dtype, form, a)) != DELTA_OK) return st;
  if (a.B * a.D == 0) return DELTA_OK;
  a.x = x; a.gate = gate; a.h0 = state; a.hT = state; a.out = out;
  if ((st = scan_pointers(a, dtype)) != DELTA_OK) return st;
  if (!state || !out) return fail(DELTA_ERR_INVALID, "state and out must be non-NULL");
  if (!aligned16(state) || !aligned16(out)) return fail(DELTA_ERR_ALIGN, "state and out must be 16-byte aligned");
  const int64_t n = a.B * a.D;
  if ((st = check_overlap({Span{"out", range(out, n * esize(dtype))}, Span{"state", range(state, n * 4)}},
                          {span_x(a, dtype), span_gate(a, dtype)})) != DELTA_OK)
    return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  const cudaError_t err = delta::launch_scan_step(a, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "scan step launch");
}

int delta_scan_bwd(const void *x, const void *gate, const float *states, const int *lengths,
                   const void *dout, const float *dhT, void *dx, void *dgate, float *dh0, int B, int T,
                   int D, int64_t x_sb, int64_t x_st, int64_t g_sb, int64_t g_st, delta_dtype dtype,
                   delta_scan_form form, struct CUstream_st *stream) {
  delta::ScanBwdArgs a{};
  int st;
  if ((st = scan_sizes(B, T, D, x_sb, x_st, g_sb, g_st, dtype, form, a)) != DELTA_OK) return st;
  if (a.B * a.D == 0) return DELTA_OK;
  a.x = x; a.gate = gate; a.states = const_cast<float *>(states); a.lengths = lengths;
  a.dout = dout; a.dhT = dhT; a.dx = dx; a.dgate = dgate; a.dh0 = dh0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned16(states) || !aligned16(dout) || !aligned16(dhT) || !aligned16(dx) || !aligned16(dgate) ||
      !aligned16(dh0))
    return fail(DELTA_ERR_ALIGN, "states, dout, dhT and the gradients must be 16-byte aligned");
  const int64_t n = a.B * a.D;
  const Span hs = {"dhT", range(dhT, n * 4)}, zs = {"dh0", range(dh0, n * 4)};
  if (dh0 != dhT && overlap(zs.r, hs.r)) return fail(DELTA_ERR_INVALID, "dh0 partly overlaps dhT");
  if (T == 0) {
    if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
    const cudaError_t err = delta::launch_scan_passthrough(dhT, dh0, n, s);
    return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "state passthrough");
  }
  if ((st = scan_pointers(a, dtype)) != DELTA_OK) return st;
  if (!states || !dout || !dx || !dgate)
    return fail(DELTA_ERR_INVALID, "states, dout, dx and dgate must be non-NULL");
  const int64_t e = esize(dtype);
  const Span xs = span_x(a, dtype), gs = span_gate(a, dtype), ls = {"lengths", range(lengths, B * 4)};
  const Span ss = {"states", range(states, n * ((T + delta::kScanBlock - 1) / delta::kScanBlock) * 4)};
  const Span os = {"dout", range(dout, n * T * e)};
  const Span dxs = {"dx", range(dx, n * T * e)}, dgs = {"dgate", range(dgate, n * T * (a.sigmoid ? e : 4))};
  if ((st = check_overlap({dxs, dgs}, {xs, gs, ls, ss, os, hs})) != DELTA_OK) return st;
  if ((st = check_overlap({zs}, {xs, gs, ls, ss, os, dxs, dgs})) != DELTA_OK) return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  const cudaError_t err = delta::launch_scan_bwd(a, s);
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "scan backward launch");
}

int delta_add_rmsnorm_fwd(const void *x, const void *residual, const void *weight, void *y, void *sum_out,
                          float *rstd, int64_t rows, int D, int64_t ldx, int64_t ldr, float eps,
                          delta_dtype dtype, delta_dtype wdtype, struct CUstream_st *stream) {
  return run_norm_fwd(Norm::kRms, x, residual, weight, nullptr, y, nullptr, sum_out, nullptr, rstd, rows, D, ldx, ldr,
                      eps, dtype, wdtype, wdtype, stream);
}

int delta_add_rmsnorm_quant(const void *x, const void *residual, const void *weight, void *y, float *y_scale,
                            void *sum_out, int64_t rows, int D, int64_t ldx, int64_t ldr, float eps,
                            delta_dtype dtype, delta_dtype wdtype, struct CUstream_st *stream) {
  return run_norm_fwd(Norm::kRmsQuant, x, residual, weight, nullptr, y, y_scale, sum_out, nullptr, nullptr, rows, D, ldx,
                      ldr, eps, dtype, wdtype, wdtype, stream);
}

int delta_add_layernorm_fwd(const void *x, const void *residual, const void *weight, const void *bias, void *y,
                            void *sum_out, float *mean, float *rstd, int64_t rows, int D, int64_t ldx, int64_t ldr,
                            float eps, delta_dtype dtype, delta_dtype wdtype, delta_dtype bdtype,
                            struct CUstream_st *stream) {
  return run_norm_fwd(Norm::kLayer, x, residual, weight, bias, y, nullptr, sum_out, mean, rstd, rows, D, ldx, ldr, eps,
                      dtype, wdtype, bdtype, stream);
}

int delta_add_rmsnorm_bwd(const void *dy, const void *sum, const void *weight, const float *rstd,
                          const void *dsum, void *dx, float *dweight, int64_t rows, int D,
                          delta_dtype dtype, delta_dtype wdtype, struct CUstream_st *stream) {
  return run_norm_bwd(Norm::kRms, dy, sum, weight, nullptr, rstd, dsum, dx, dweight, nullptr, rows, D, dtype, wdtype,
                      stream);
}

int delta_add_layernorm_bwd(const void *dy, const void *sum, const void *weight, const float *mean, const float *rstd,
                            const void *dsum, void *dx, float *dweight, float *dbias, int64_t rows, int D,
                            delta_dtype dtype, delta_dtype wdtype, struct CUstream_st *stream) {
  return run_norm_bwd(Norm::kLayer, dy, sum, weight, mean, rstd, dsum, dx, dweight, dbias, rows, D, dtype, wdtype,
                      stream);
}

int delta_linear_fwd(const void *x, const void *w, const void *bias, const void *residual, void *out, void *pre,
                     int M, int N, int K, int64_t ldx, int64_t ldw, int64_t ldr, delta_act act,
                     delta_dtype dtype, delta_dtype bdtype, struct CUstream_st *stream) {
  const int st = check_dtype(dtype);
  if (st != DELTA_OK) return st;
  return run_linear(x, w, nullptr, nullptr, bias, residual, out, pre, M, N, K, ldx, ldw, ldr, act,
                    dtype == DELTA_BF16 ? delta::kLinBf16 : delta::kLinF32, bdtype, stream);
}

int delta_linear_quant(const void *x, const float *x_scale, const void *w, const float *w_scale,
                       const void *bias, const void *residual, void *out, int M, int N, int K, int64_t ldx,
                       int64_t ldw, int64_t ldr, delta_act act, delta_dtype bdtype, struct CUstream_st *stream) {
  return run_linear(x, w, x_scale, w_scale, bias, residual, out, nullptr, M, N, K, ldx, ldw, ldr, act,
                    delta::kLinE4m3, bdtype, stream);
}

int delta_linear_bwd(const void *x, const void *w, const void *dout, const void *pre, void *dx, void *dw,
                     float *dbias, int M, int N, int K, int64_t ldx, int64_t ldw, delta_act act,
                     delta_dtype dtype, struct CUstream_st *stream) {
  int st;
  if ((st = check_dtype(dtype)) != DELTA_OK) return st;
  if ((st = linear_sizes(M, N, K, ldx, ldw, N, act)) != DELTA_OK) return st;
  if (!dx && !dw && !dbias) return DELTA_OK;
  const int64_t e = esize(dtype), m = M, n = N, k = K;
  if (M <= 1) ldx = K;
  if (N <= 1) ldw = K;
  if (!aligned16(dout) || !aligned16(pre) || !aligned16(dx) || !aligned16(dw) || !aligned16(dbias))
    return fail(DELTA_ERR_ALIGN, "dout, pre and the gradients must be 16-byte aligned");
  if (!aligned_to(x, e) || !aligned_to(w, e)) return fail(DELTA_ERR_ALIGN, "x and w must be aligned to their elements");
  if (M > 0 && N > 0) {
    if (!dout || (dw && !x) || (dx && !w)) return fail(DELTA_ERR_INVALID, "x, w and dout must be non-NULL");
    if (act != DELTA_ACT_NONE && !pre) return fail(DELTA_ERR_INVALID, "an activation's gradient needs pre");
  }
  if ((st = check_overlap({Span{"dx", range(dx, m * k * e)}, Span{"dw", range(dw, n * k * e)},
                           Span{"dbias", range(dbias, n * 4)}},
                          {Span{"x", range(x, m > 0 ? ((m - 1) * ldx + k) * e : 0)},
                           Span{"w", range(w, n > 0 ? ((n - 1) * ldw + k) * e : 0)},
                           Span{"dout", range(dout, m * n * e)}, Span{"pre", range(pre, m * n * e)}})) != DELTA_OK)
    return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  const cudaError_t err = linear_backward(x, w, dout, act == DELTA_ACT_NONE ? nullptr : pre, dx, dw, dbias, m, n, k,
                                          ldx, ldw, (int)act, dtype == DELTA_BF16, false,
                                          reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "linear layer's gradients");
}

int delta_glu_fwd(const void *x, const void *w, const void *bias, void *out, void *pre, int M, int N, int K,
                  int64_t ldx, int64_t ldw, delta_act act, delta_dtype dtype, delta_dtype bdtype,
                  struct CUstream_st *stream) {
  int st;
  if ((st = glu_sizes(M, N, K, ldx, ldw, act, dtype)) != DELTA_OK) return st;
  if ((st = check_dtype(bdtype)) != DELTA_OK) return st;
  if (M == 0 || N == 0) return DELTA_OK;
  if (!x || !w || !out) return fail(DELTA_ERR_INVALID, "x, w and out must be non-NULL");
  const int64_t e = esize(dtype), m = M, n = N, k = K;
  if (!aligned_to(x, e) || !aligned_to(w, e) || !aligned_to(bias, esize(bdtype)))
    return fail(DELTA_ERR_ALIGN, "every input must be aligned to its elements");
  if (!aligned16(out) || !aligned16(pre)) return fail(DELTA_ERR_ALIGN, "out and pre must be 16-byte aligned");
  if (M == 1) ldx = K;
  if ((st = check_overlap({Span{"out", range(out, m * n * e)}, Span{"pre", range(pre, 2 * m * n * e)}},
                          {Span{"x", range(x, ((m - 1) * ldx + k) * e)}, Span{"w", range(w, ((2 * n - 1) * ldw + k) * e)},
                           Span{"bias", range(bias, 2 * n * esize(bdtype))}})) != DELTA_OK)
    return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  delta::LinearArgs a{};
  a.x = x; a.w = w; a.bias = bias; a.out = out; a.pre = pre; a.M = m; a.N = n; a.K = k; a.ldx = ldx; a.ldw = ldw;
  a.act = (int)act; a.kind = dtype == DELTA_BF16 ? delta::kLinBf16 : delta::kLinF32; a.bias_bf16 = bdtype == DELTA_BF16;
  const cudaError_t err = glu_forward(a, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "gated layer");
}

int delta_glu_bwd(const void *x, const void *w, const void *dout, const void *pre, void *dx, void *dw, float *dbias,
                  int M, int N, int K, int64_t ldx, int64_t ldw, delta_act act, delta_dtype dtype,
                  struct CUstream_st *stream) {
  int st;
  if ((st = glu_sizes(M, N, K, ldx, ldw, act, dtype)) != DELTA_OK) return st;
  if (!dx && !dw && !dbias) return DELTA_OK;
  const int64_t e = esize(dtype), m = M, n = N, k = K;
  if (M <= 1) ldx = K;
  if (!aligned16(dout) || !aligned16(pre) || !aligned16(dx) || !aligned16(dw) || !aligned16(dbias))
    return fail(DELTA_ERR_ALIGN, "dout, pre and the gradients must be 16-byte aligned");
  if (!aligned_to(x, e) || !aligned_to(w, e)) return fail(DELTA_ERR_ALIGN, "x and w must be aligned to their elements");
  if (M > 0 && N > 0 && (!dout || !pre || (dw && !x) || (dx && !w)))
    return fail(DELTA_ERR_INVALID, "x, w, dout and pre must be non-NULL");
  if ((st = check_overlap({Span{"dx", range(dx, m * k * e)}, Span{"dw", range(dw, 2 * n * k * e)},
                           Span{"dbias", range(dbias, 2 * n * 4)}},
                          {Span{"x", range(x, m > 0 ? ((m - 1) * ldx + k) * e : 0)},
                           Span{"w", range(w, n > 0 ? ((2 * n - 1) * ldw + k) * e : 0)},
                           Span{"dout", range(dout, m * n * e)}, Span{"pre", range(pre, 2 * m * n * e)}})) != DELTA_OK)
    return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  const cudaError_t err = linear_backward(x, w, dout, pre, dx, dw, dbias, m, 2 * n, k, ldx, ldw, (int)act,
                                          dtype == DELTA_BF16, true, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "gated layer's gradients");
}

}  // extern "C"
