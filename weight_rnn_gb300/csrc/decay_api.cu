// decay_api.cu -- the C ABI of linear attention with a decay for each head:
// argument checks, how the time axis is cut, scratch and launches.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/delta.h"
#include "api_common.h"
#include "block_common.h"
#include "kernels.h"

namespace {

using namespace delta::api;
using delta::DecayArgs;
using delta::DecayPass;

int sizes(int B, int T, int H, int dk, int dv, delta_dtype dtype) {
  if (B < 0 || T < 0 || H < 0) return fail(DELTA_ERR_INVALID, "negative size B=%d T=%d H=%d", B, T, H);
  const int st = check_dtype(dtype);
  if (st != DELTA_OK) return st;
  if (dk < 1 || dv < 1 || dk > delta::kDecayMaxD || dv > delta::kDecayMaxD)
    return fail(DELTA_ERR_UNSUPPORTED, "dk=%d and dv=%d must be in [1, %d]", dk, dv, delta::kDecayMaxD);
  if ((int64_t)B * T >= kMaxElems / 512 / (H > 0 ? H : 1) || (int64_t)B * H >= (int64_t(1) << 24))
    return fail(DELTA_ERR_UNSUPPORTED, "B*T*H too large");
  return DELTA_OK;
}

// strides of [n0][n1][n2][d] (of [n0][n2][d] with two), those of axes with one
// entry set to 0; the bytes from the first to the last element
int view(const char *name, const int64_t *st, const int64_t *n, int axes, int64_t d, int64_t e, int64_t *to,
         int64_t &bytes) {
  int64_t last = d;
  for (int i = 0; i < axes; ++i) {
    to[i] = n[i] > 1 ? st[i] : 0;
    if (to[i] < 0 || (n[i] > 1 && to[i] >= kMaxElems / n[i]))
      return fail(DELTA_ERR_INVALID, "a stride of %s, %lld, is out of range", name, (long long)st[i]);
    last += (n[i] - 1) * to[i];
  }
  bytes = last * e;
  return DELTA_OK;
}

int check_inputs(const void *q, const void *k, const void *v, const float *decay, const int *lengths, int64_t e) {
  if (!q || !k || !v || !decay) return fail(DELTA_ERR_INVALID, "q, k, v and decay must be non-NULL");
  if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(decay, 4) || !aligned_to(lengths, 4))
    return fail(DELTA_ERR_ALIGN, "q, k, v, decay and lengths must be aligned to their elements");
  return DELTA_OK;
}

int sm_count() {
  int dev = 0, n = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// Into how many segments the time axis is cut.  On the tensor cores 128 tokens take a CTA
// about 2.4 us with all products and 1.7 with those of the states alone, an item's start
// and end 6 us, and CTAs share the work evenly where there is more than a round of it,
// but for rows with lengths.  In float32 they take 20 and 5 us at 64 channels, 36 and 11
// at 128, two CTAs an SM (one above that), in whole rounds.  A cut adds the pass for the
// states, their way through memory, and two launches.
int segments(const DecayArgs &a, int64_t state_passes, bool tc) {
  const int64_t chunks = (a.T + delta::kDecayChunk - 1) / delta::kDecayChunk;
  const int width = tc ? 128 : 64;
  int dk = 1;
  for (int i = 0; i < a.passes; ++i) dk = dk > a.pass[i].dk ? dk : a.pass[i].dk;
  const double two = dk > 128 ? 0.5 : 1.0;
  const double whole = tc ? 2.4 : (4.0 + 0.25 * dk) * two, part = tc ? 1.7 : (0.3 + 0.08 * dk) * two;
  const int64_t slots = (int64_t)sm_count() * (tc || dk > 128 ? 1 : 2);
  int64_t items = 0, bytes = 0;
  for (int i = 0; i < a.passes; ++i) items += a.B * a.H * ((a.pass[i].dv + width - 1) / width);
  bytes = state_passes * a.B * a.H * a.pass[0].dk * a.pass[0].dv * 4;
  const int64_t state_items = state_passes * a.B * a.H * ((a.pass[0].dv + width - 1) / width);
  const auto up_div = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  const auto rounds = [&](int64_t n) {
    return tc && !a.lengths && n > slots ? (double)n / (double)slots : (double)up_div(n, slots);
  };
  const auto ends = [&](int64_t n) { return 6.0 * (double)up_div(n, slots); };
  int best = 1;
  double least = 1e30;
  for (int64_t n = 1; n <= chunks && n <= 256; ++n) {
    const int64_t each = up_div(chunks, n);
    if (up_div(chunks, each) != n) continue;  // every segment has tokens
    if (n > 1 && bytes * n > (int64_t(1) << 30)) break;
    double us = rounds(items * n) * (double)each * whole + ends(items * n);
    if (n > 1) {
      // (n - 1 segments have states that count; as such an estimate they cut B1 T8192 H32
      // into five on the tensor cores, 103 us for 86)
      const int64_t m = state_items * (tc ? n : n - 1);
      us += rounds(m) * (double)each * part + ends(m) + 5.0 + (double)(bytes * n) * 4 / 5e6;
    }
    if (us < 0.97 * least) least = us, best = (int)n;
  }
  return best;
}

// The passes of one call; states: passes that give every segment its first state,
// where the time axis is cut, and into which of `a`'s passes they go.
struct Start {
  DecayPass pass;        // k, v and the state's layout; init is the row's first state
  int into[2], count;
};
cudaError_t run(DecayArgs &a, const Start *starts, int count, cudaStream_t s) {
  const bool tc = delta::decay_tc_fits(a);
  a.nseg = segments(a, count, tc);
  const int64_t chunks = (a.T + delta::kDecayChunk - 1) / delta::kDecayChunk;
  a.seg = (chunks + a.nseg - 1) / a.nseg * delta::kDecayChunk;
  const bool cut = a.nseg > 1;
  const int64_t n = (int64_t)starts[0].pass.dk * starts[0].pass.dv, bytes = cut ? a.B * a.H * a.nseg * n * 4 : 0;
  DecayArgs st = a;
  st.passes = count;
  for (int i = 0; i < count; ++i) st.pass[i] = starts[i].pass;
  const int64_t handed = tc ? delta::decay_tc_scratch(a) : 0, handed_st = tc && cut ? delta::decay_tc_scratch(st) : 0;
  Scratch scr(s);
  for (int i = 0; cut && i < count; ++i) scr.want(bytes);
  scr.want(handed);
  scr.want(handed_st);
  cudaError_t err = scr.take();
  if (err != cudaSuccess) return err;
  if (cut) {
    for (int i = 0; i < count; ++i) {
      st.pass[i].final = static_cast<float *>(scr.cut(bytes));
      for (int j = 0; j < starts[i].count; ++j) a.pass[starts[i].into[j]].init = st.pass[i].final;
    }
    st.handed = handed_st ? scr.cut(handed_st) : nullptr;
    err = tc ? delta::launch_decay_tc(st, true, s) : delta::launch_decay_states(st, s);
    for (int i = 0; err == cudaSuccess && i < count; ++i)
      err = delta::launch_decay_join(st.pass[i].final, starts[i].pass.init, a, starts[i].pass.reverse, n, s);
    a.joined = true;
  }
  a.handed = handed ? scr.cut(handed) : nullptr;
  if (err == cudaSuccess) err = tc ? delta::launch_decay_tc(a, false, s) : delta::launch_decay(a, s);
  const cudaError_t ef = scr.release();
  return err != cudaSuccess ? err : ef;
}

DecayPass roles(const void *q, const int64_t *qs, const void *k, const int64_t *ks, const void *v, const int64_t *vs,
                int dk, int dv) {
  DecayPass p{};
  p.q = q; p.k = k; p.v = v;
  for (int i = 0; i < 3; ++i) p.qs[i] = qs[i], p.ks[i] = ks[i], p.vs[i] = vs[i];
  p.dk = dk; p.dv = dv;
  p.os = p.kvs = 1.f;
  return p;
}

}  // namespace

extern "C" {

int delta_decay_fwd(const void *q, const void *k, const void *v, const float *decay, const float *h0,
                    const int *lengths, void *out, float *hT, int B, int T, int H, int dk, int dv,
                    const int64_t *strides, float scale, delta_dtype dtype, struct CUstream_st *stream) {
  int st;
  if ((st = sizes(B, T, H, dk, dv, dtype)) != DELTA_OK) return st;
  if (B == 0 || H == 0) return DELTA_OK;
  if (!strides) return fail(DELTA_ERR_INVALID, "strides must be non-NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned16(h0) || !aligned16(out) || !aligned16(hT))
    return fail(DELTA_ERR_ALIGN, "h0, out and hT must be 16-byte aligned");
  const int64_t e = esize(dtype), bh = (int64_t)B * H, n = bh * dk * dv;
  const Span hs = {"h0", range(h0, n * 4)}, ts = {"hT", range(hT, n * 4)};
  if (hT != h0 && overlap(ts.r, hs.r)) return fail(DELTA_ERR_INVALID, "hT partly overlaps h0");
  if (T == 0) {
    if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
    const cudaError_t err = hT ? delta::launch_scan_passthrough(h0, hT, n, s) : cudaSuccess;
    return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "state passthrough");
  }
  if ((st = check_inputs(q, k, v, decay, lengths, e)) != DELTA_OK) return st;
  if (!out) return fail(DELTA_ERR_INVALID, "out must be non-NULL");
  const int64_t axes[3] = {B, T, H};
  int64_t qs[3], ks[3], vs[3], qb, kb, vb;
  if ((st = view("q", strides, axes, 3, dk, e, qs, qb)) != DELTA_OK) return st;
  if ((st = view("k", strides + 3, axes, 3, dk, e, ks, kb)) != DELTA_OK) return st;
  if ((st = view("v", strides + 6, axes, 3, dv, e, vs, vb)) != DELTA_OK) return st;
  const Span is[] = {{"q", range(q, qb)}, {"k", range(k, kb)}, {"v", range(v, vb)},
                     {"decay", range(decay, (int64_t)H * 4)}, {"lengths", range(lengths, (int64_t)B * 4)}};
  const Span os = {"out", range(out, bh * T * dv * e)};
  if ((st = check_overlap({os, ts}, is)) != DELTA_OK) return st;
  if ((st = check_overlap({os}, {hs})) != DELTA_OK) return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  DecayArgs a{};
  a.passes = 1; a.decay = decay; a.lengths = lengths; a.B = B; a.T = T; a.H = H; a.bf16 = dtype == DELTA_BF16;
  DecayPass &p = a.pass[0] = roles(q, qs, k, ks, v, vs, dk, dv);
  p.init = h0; p.final = hT; p.out = out; p.os = scale;
  const Start from = {p, {0}, 1};
  const cudaError_t err = run(a, &from, 1, s);
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "decay attention forward");
}

int delta_decay_step(const void *q, const void *k, const void *v, const float *decay, float *state, void *out, int B,
                     int H, int dk, int dv, const int64_t *strides, float scale, delta_dtype dtype,
                     struct CUstream_st *stream) {
  int st;
  if ((st = sizes(B, 1, H, dk, dv, dtype)) != DELTA_OK) return st;
  if (B == 0 || H == 0) return DELTA_OK;
  if (!strides) return fail(DELTA_ERR_INVALID, "strides must be non-NULL");
  const int64_t e = esize(dtype), bh = (int64_t)B * H;
  if ((st = check_inputs(q, k, v, decay, nullptr, e)) != DELTA_OK) return st;
  if (!state || !out) return fail(DELTA_ERR_INVALID, "state and out must be non-NULL");
  if (!aligned16(state) || !aligned16(out)) return fail(DELTA_ERR_ALIGN, "state and out must be 16-byte aligned");
  delta::DecayStepArgs a{};
  const int64_t axes[2] = {B, H};
  int64_t qb, kb, vb;
  if ((st = view("q", strides, axes, 2, dk, e, a.qs, qb)) != DELTA_OK) return st;
  if ((st = view("k", strides + 2, axes, 2, dk, e, a.ks, kb)) != DELTA_OK) return st;
  if ((st = view("v", strides + 4, axes, 2, dv, e, a.vs, vb)) != DELTA_OK) return st;
  if ((st = check_overlap({Span{"out", range(out, bh * dv * e)}, Span{"state", range(state, bh * dk * dv * 4)}},
                          {Span{"q", range(q, qb)}, Span{"k", range(k, kb)}, Span{"v", range(v, vb)},
                           Span{"decay", range(decay, (int64_t)H * 4)}})) != DELTA_OK)
    return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  a.q = q; a.k = k; a.v = v; a.decay = decay; a.state = state; a.out = out; a.B = B; a.H = H;
  a.dk = dk; a.dv = dv; a.scale = scale; a.bf16 = dtype == DELTA_BF16;
  const cudaError_t err = delta::launch_decay_step(a, reinterpret_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "decay attention step");
}

int delta_decay_bwd(const void *q, const void *k, const void *v, const float *decay, const float *h0,
                    const int *lengths, const void *dout, const float *dhT, void *dq, void *dk_out, void *dv_out,
                    float *dh0, int B, int T, int H, int dk, int dv, const int64_t *strides, float scale,
                    delta_dtype dtype, struct CUstream_st *stream) {
  int st;
  if ((st = sizes(B, T, H, dk, dv, dtype)) != DELTA_OK) return st;
  if (B == 0 || H == 0) return DELTA_OK;
  if (!strides) return fail(DELTA_ERR_INVALID, "strides must be non-NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned16(h0) || !aligned16(dout) || !aligned16(dhT) || !aligned16(dq) || !aligned16(dk_out) ||
      !aligned16(dv_out) || !aligned16(dh0))
    return fail(DELTA_ERR_ALIGN, "h0, dout, dhT and the gradients must be 16-byte aligned");
  const int64_t e = esize(dtype), bh = (int64_t)B * H, n = bh * dk * dv;
  const Span hs = {"h0", range(h0, n * 4)}, ts = {"dhT", range(dhT, n * 4)}, zs = {"dh0", range(dh0, n * 4)};
  if (T == 0) {
    if (dh0 != dhT && overlap(zs.r, ts.r)) return fail(DELTA_ERR_INVALID, "dh0 partly overlaps dhT");
    if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
    const cudaError_t err = dh0 ? delta::launch_scan_passthrough(dhT, dh0, n, s) : cudaSuccess;
    return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "state passthrough");
  }
  if ((st = check_inputs(q, k, v, decay, lengths, e)) != DELTA_OK) return st;
  if (!dout || !dq || !dk_out || !dv_out) return fail(DELTA_ERR_INVALID, "dout, dq, dk and dv must be non-NULL");
  const int64_t axes[3] = {B, T, H};
  int64_t qs[3], ks[3], vs[3], qb, kb, vb;
  if ((st = view("q", strides, axes, 3, dk, e, qs, qb)) != DELTA_OK) return st;
  if ((st = view("k", strides + 3, axes, 3, dk, e, ks, kb)) != DELTA_OK) return st;
  if ((st = view("v", strides + 6, axes, 3, dv, e, vs, vb)) != DELTA_OK) return st;
  const int64_t wide = (int64_t)H * dv, os[3] = {T * wide, wide, dv};
  if ((st = check_overlap({Span{"dq", range(dq, bh * T * dk * e)}, Span{"dk", range(dk_out, bh * T * dk * e)},
                           Span{"dv", range(dv_out, bh * T * dv * e)}, zs},
                          {Span{"q", range(q, qb)}, Span{"k", range(k, kb)}, Span{"v", range(v, vb)}, hs, ts,
                           Span{"dout", range(dout, bh * T * dv * e)}, Span{"decay", range(decay, (int64_t)H * 4)},
                           Span{"lengths", range(lengths, (int64_t)B * 4)}})) != DELTA_OK)
    return st;
  if (take_injection()) return fail(DELTA_ERR_CUDA, "injected failure (delta_inject_failure)");
  DecayArgs a{};
  a.passes = 3; a.decay = decay; a.lengths = lengths; a.B = B; a.T = T; a.H = H; a.bf16 = dtype == DELTA_BF16;
  // dq_t = scale S_t dout_t: the forward with dout as the query of the transposed states
  DecayPass &pq = a.pass[0] = roles(dout, os, v, vs, k, ks, dv, dk);
  pq.out = dq; pq.init = h0; pq.init_t = true; pq.os = scale;
  // dv_t = R_t^T k_t, dk_t = R_t v_t with R_t = scale q_t dout_t^T + g R_{t+1}
  DecayPass &pv = a.pass[1] = roles(k, ks, q, qs, dout, os, dk, dv);
  pv.out = dv_out; pv.init = dhT; pv.final = dh0; pv.reverse = true; pv.kvs = scale;
  DecayPass &pk = a.pass[2] = roles(v, vs, dout, os, q, qs, dv, dk);
  pk.out = dk_out; pk.init = dhT; pk.init_t = true; pk.reverse = true; pk.kvs = scale;
  // the states S once, transposed where they are read; the states R once for both
  Start from[2] = {{roles(nullptr, qs, k, ks, v, vs, dk, dv), {0}, 1}, {pv, {1, 2}, 2}};
  from[0].pass.init = h0;
  const cudaError_t err = run(a, from, 2, s);
  return err == cudaSuccess ? DELTA_OK : cuda_fail(err, "decay attention backward");
}

}  // extern "C"
