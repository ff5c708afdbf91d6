// decay.cu -- linear attention with a decay g for each head, outside the tensor
// cores: the step of one token, the pass over the time axis for float32 and for
// layouts that the tensor-core kernel does not take, and the joining of segments.
//
//   S_t = g S_{t-1} + k_t v_t^T,   out_t = scale S_t^T q_t
//
// A pass goes by chunks.  With n tokens from t0 on, S the state before them and
// p, j places in the chunk,
//
//   P_pj = (q_p . k_j) g^(p-j)  (j <= p),   out_p = P v + g^(p+1) q_p S,
//   S   <- g^n S + sum_j g^(n-1-j) k_j v_j^T.
//
// In reverse the roles of earlier and later change, and the state that a chunk
// takes over has been decayed into it already:
//
//   P_pj = (q_p . k_j) g^(j-p)  (j >= p),   out_p = P v + g^(n-1-p) q_p Y,
//   Y   <- g^n Y + sum_j g^(j+1) k_j v_j^T.
//
// Powers of g are 2^(e log2 g) with a whole e; no quotient of powers is formed, so
// any g in [0, 1] is safe.
#include <cuda_bf16.h>

#include "chain.cuh"
#include "kernels.h"

namespace delta {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float &r) { r = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16 &r) { r = __float2bfloat16_rn(x); }

// g^e from lg = log2 g (-inf for g = 0)
__device__ __forceinline__ float power(float lg, int64_t e) { return e <= 0 ? 1.f : exp2f(lg * (float)e); }

int sm_count() {
  int dev = 0, n = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// ------------------------------------------------------------------ one token
// HBM-bound: the state is read and written once.  A CTA has a head's state, or 32
// of its columns where there are few heads; a thread keeps V neighbouring columns
// of every RG-th row, kAhead rows asked for at a time, and the rows' partial
// outputs meet in shared memory in a fixed order.
constexpr int kStepThreads = 256;

template <typename In, int V>
__global__ void __launch_bounds__(kStepThreads, 4) decay_step_kernel(DecayStepArgs p, int slab) {
  constexpr int kAhead = 8;
  __shared__ float sq[kDecayMaxD], sk[kDecayMaxD];
  __shared__ __align__(16) float part[kStepThreads * V];
  struct __align__(4 * V) Vec { float v[V]; };
  const int slabs = (p.dv + slab - 1) / slab;
  const int64_t bh = blockIdx.x / slabs, b = bh / p.H, h = bh % p.H;
  const int c0 = (int)(blockIdx.x % slabs) * slab, cols = min(slab, p.dv - c0);
  const int nv = (cols + V - 1) / V, groups = kStepThreads / nv;
  const int g = threadIdx.x / nv, c = threadIdx.x % nv * V;
  const bool on = g < groups;
  chain_wait();
  float *state = p.state + bh * p.dk * p.dv + c0 + c;
  Vec s[kAhead];
  const auto ask = [&](int d0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int d = d0 + i * groups;
      if (on && d < p.dk) {
        const float *at = state + (int64_t)d * p.dv;
        if constexpr (V == 4)
          *reinterpret_cast<float4 *>(&s[i]) = __ldcs(reinterpret_cast<const float4 *>(at));
        else
          s[i].v[0] = __ldcs(at);
      }
    }
  };
  ask(g);
  const In *q = static_cast<const In *>(p.q) + b * p.qs[0] + h * p.qs[1];
  const In *k = static_cast<const In *>(p.k) + b * p.ks[0] + h * p.ks[1];
  for (int i = threadIdx.x; i < p.dk; i += kStepThreads) sq[i] = to_f(q[i]), sk[i] = to_f(k[i]);
  Vec v;
#pragma unroll
  for (int i = 0; i < V; ++i) v.v[i] = on ? to_f(static_cast<const In *>(p.v)[b * p.vs[0] + h * p.vs[1] + c0 + c + i]) : 0.f;
  const float decay = p.decay[h];
  __syncthreads();
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int d0 = g; on && d0 < p.dk; d0 += kAhead * groups) {
    if (d0 != g) ask(d0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int d = d0 + i * groups;
      if (d >= p.dk) continue;
      float *at = state + (int64_t)d * p.dv;
      const float qd = sq[d], kd = sk[d];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[i].v[j] = fmaf(kd, v.v[j], decay * s[i].v[j]);
        o[j] = fmaf(qd, s[i].v[j], o[j]);
      }
      if constexpr (V == 4)
        __stcs(reinterpret_cast<float4 *>(at), *reinterpret_cast<const float4 *>(&s[i]));
      else
        __stcs(at, s[i].v[0]);
    }
  }
  if (on) {
#pragma unroll
    for (int j = 0; j < V; ++j) part[(g * nv) * V + c + j] = o[j];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < cols; i += kStepThreads) {
    float a = 0.f;
    for (int r = 0; r < groups; ++r) a += part[r * nv * V + i];
    from_f(p.scale * a, static_cast<In *>(p.out)[bh * p.dv + c0 + i]);
  }
}

template <typename In>
cudaError_t step_all(const DecayStepArgs &a, cudaStream_t s) {
  const int64_t bh = a.B * a.H;
  const bool vec = a.dv % 4 == 0;
  // whole heads where they fill the GPU (each CTA's bytes are one piece then)
  const int slab = bh >= 2 * sm_count() ? a.dv : 32;
  const int64_t grid = bh * ((a.dv + slab - 1) / slab);
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  return chain_launch(vec ? decay_step_kernel<In, 4> : decay_step_kernel<In, 1>, dim3((unsigned)grid),
                      dim3(kStepThreads), 0, 1, true, s, a, slab);
}

// ----------------------------------------------------- the pass on CUDA cores
// A correctness path in float32: a CTA has a segment of a head and 64 value
// columns, the state [dk][64] in shared memory, chunks of 32 tokens.
constexpr int kC = 32, kCols = 64, kThreads = 256;

__host__ __device__ constexpr int generic_floats(int dk, bool states) {
  return dk * kCols + kC * kCols + (states ? 1 : 2) * kC * (dk | 1) + kC * (kC + 1);
}

template <typename In, bool kStates>
__global__ void __launch_bounds__(kThreads) decay_generic_kernel(const __grid_constant__ DecayArgs a, int groups) {
  extern __shared__ __align__(16) float smem[];
  int64_t i = blockIdx.x;
  const DecayPass &p = a.pass[i % a.passes];
  i /= a.passes;
  const int sg = (int)(i % a.nseg);
  i /= a.nseg;
  const int c0 = (int)(i % groups) * kCols;
  const int64_t bh = i / groups, b = bh / a.H, h = bh % a.H;
  if (c0 >= p.dv) return;
  const int dk = p.dk, cols = min(kCols, p.dv - c0), ldk = dk | 1;
  // (vectors of four are read from S and sv, which come first)
  float *S = smem, *sv = S + dk * kCols, *sk = sv + kC * kCols, *sp = sk + kC * ldk, *sq = sp + kC * (kC + 1);
  const int tid = threadIdx.x, row = tid / 8, c8 = tid % 8 * 8;
  chain_wait();
  const float lg = log2f(a.decay[h]);
  int64_t len = a.lengths ? a.lengths[b] : a.T;
  len = len < 0 ? 0 : len > a.T ? a.T : len;
  const int64_t t_lo = sg * a.seg, t_hi = min(t_lo + a.seg, a.T);
  const int64_t t_end = min(t_hi, len);  // tokens [t_lo, t_end) count
  const int64_t state_at = kStates || a.nseg > 1 ? bh * a.nseg + sg : bh;
  for (int e = tid; e < dk * kCols; e += kThreads) {
    const int d = e / kCols, c = e % kCols;
    float x = 0.f;
    if (!kStates && p.init && c < cols)
      x = p.init[state_at * dk * p.dv + (p.init_t ? (int64_t)(c0 + c) * dk + d : (int64_t)d * p.dv + c0 + c)];
    S[e] = x;
  }
  const int64_t chunks = t_end > t_lo ? (t_end - t_lo + kC - 1) / kC : 0;
  for (int64_t ci = 0; ci < chunks; ++ci) {
    const int64_t t0 = t_lo + (p.reverse ? chunks - 1 - ci : ci) * kC;
    const int n = (int)min((int64_t)kC, t_end - t0);
    __syncthreads();
    for (int e = tid; e < kC * dk; e += kThreads) {
      const int r = e / dk, d = e % dk;
      sk[r * ldk + d] = r < n ? to_f(static_cast<const In *>(p.k)[b * p.ks[0] + (t0 + r) * p.ks[1] + h * p.ks[2] + d]) : 0.f;
      if (!kStates)
        sq[r * ldk + d] = r < n ? to_f(static_cast<const In *>(p.q)[b * p.qs[0] + (t0 + r) * p.qs[1] + h * p.qs[2] + d]) : 0.f;
    }
    for (int e = tid; e < kC * kCols; e += kThreads) {
      const int r = e / kCols, c = e % kCols;
      sv[e] = r < n && c < cols
                  ? p.kvs * to_f(static_cast<const In *>(p.v)[b * p.vs[0] + (t0 + r) * p.vs[1] + h * p.vs[2] + c0 + c])
                  : 0.f;
    }
    __syncthreads();
    if constexpr (!kStates) {
      {  // P: a row and four columns a thread
        const int j0 = tid % 8 * 4;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int d = 0; d < dk; ++d) {
          const float qd = sq[row * ldk + d];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = fmaf(qd, sk[(j0 + j) * ldk + d], x[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int apart = p.reverse ? j0 + j - row : row - j0 - j;
          sp[row * (kC + 1) + j0 + j] = apart < 0 ? 0.f : x[j] * power(lg, apart);
        }
      }
      __syncthreads();
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int d = 0; d < dk; ++d) {
        const float qd = sq[row * ldk + d];
        const float4 x = *reinterpret_cast<const float4 *>(S + d * kCols + c8);
        const float4 y = *reinterpret_cast<const float4 *>(S + d * kCols + c8 + 4);
        o[0] = fmaf(qd, x.x, o[0]), o[1] = fmaf(qd, x.y, o[1]), o[2] = fmaf(qd, x.z, o[2]), o[3] = fmaf(qd, x.w, o[3]);
        o[4] = fmaf(qd, y.x, o[4]), o[5] = fmaf(qd, y.y, o[5]), o[6] = fmaf(qd, y.z, o[6]), o[7] = fmaf(qd, y.w, o[7]);
      }
      const float gam = power(lg, p.reverse ? n - 1 - row : row + 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= gam;
      for (int r = 0; r < kC; ++r) {
        const float w = sp[row * (kC + 1) + r];
        const float4 x = *reinterpret_cast<const float4 *>(sv + r * kCols + c8);
        const float4 y = *reinterpret_cast<const float4 *>(sv + r * kCols + c8 + 4);
        o[0] = fmaf(w, x.x, o[0]), o[1] = fmaf(w, x.y, o[1]), o[2] = fmaf(w, x.z, o[2]), o[3] = fmaf(w, x.w, o[3]);
        o[4] = fmaf(w, y.x, o[4]), o[5] = fmaf(w, y.y, o[5]), o[6] = fmaf(w, y.z, o[6]), o[7] = fmaf(w, y.w, o[7]);
      }
      if (row < n) {
        In *out = static_cast<In *>(p.out) + ((b * a.T + t0 + row) * a.H + h) * p.dv + c0 + c8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c8 + j < cols) from_f(p.os * o[j], out[j]);
      }
      __syncthreads();  // the state has been read
    }
    for (int r = row; r < kC; r += kThreads / 8) {  // keys decayed to the chunk's end (in reverse, past its start)
      const float w = power(lg, p.reverse ? r + 1 : n - 1 - r);
      for (int d = tid % 8; d < dk; d += 8) sk[r * ldk + d] *= w;
    }
    __syncthreads();
    const float keep = power(lg, n);
    for (int d = row; d < dk; d += kThreads / 8) {
      float4 x = *reinterpret_cast<float4 *>(S + d * kCols + c8), y = *reinterpret_cast<float4 *>(S + d * kCols + c8 + 4);
      x.x *= keep, x.y *= keep, x.z *= keep, x.w *= keep, y.x *= keep, y.y *= keep, y.z *= keep, y.w *= keep;
      for (int r = 0; r < kC; ++r) {
        const float w = sk[r * ldk + d];
        const float4 u = *reinterpret_cast<const float4 *>(sv + r * kCols + c8);
        const float4 v = *reinterpret_cast<const float4 *>(sv + r * kCols + c8 + 4);
        x.x = fmaf(w, u.x, x.x), x.y = fmaf(w, u.y, x.y), x.z = fmaf(w, u.z, x.z), x.w = fmaf(w, u.w, x.w);
        y.x = fmaf(w, v.x, y.x), y.y = fmaf(w, v.y, y.y), y.z = fmaf(w, v.z, y.z), y.w = fmaf(w, v.w, y.w);
      }
      *reinterpret_cast<float4 *>(S + d * kCols + c8) = x;
      *reinterpret_cast<float4 *>(S + d * kCols + c8 + 4) = y;
    }
  }
  __syncthreads();
  if (kStates || (p.final && sg == (p.reverse ? 0 : a.nseg - 1))) {
    float *to = p.final + (kStates ? state_at : bh) * dk * p.dv;
    for (int e = tid; e < dk * kCols; e += kThreads) {
      const int d = e / kCols, c = e % kCols;
      if (c < cols) to[(int64_t)d * p.dv + c0 + c] = S[e];
    }
  }
  if constexpr (!kStates) {  // tokens past the row's end
    const int64_t t0 = max(t_lo, t_end);
    for (int64_t e = tid; e < (t_hi - t0) * cols; e += kThreads)
      from_f(0.f, static_cast<In *>(p.out)[((b * a.T + t0 + e / cols) * a.H + h) * p.dv + c0 + e % cols]);
  }
}

template <typename In, bool kStates>
cudaError_t generic(const DecayArgs &a, cudaStream_t s) {
  int dk = 1, dv = 1;
  for (int i = 0; i < a.passes; ++i) dk = max(dk, a.pass[i].dk), dv = max(dv, a.pass[i].dv);
  const int groups = (dv + kCols - 1) / kCols;
  const int64_t grid = a.B * a.H * groups * a.nseg * a.passes;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  auto kern = decay_generic_kernel<In, kStates>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             generic_floats(kDecayMaxD, kStates) * 4);
  if (e != cudaSuccess) return e;
  return chain_launch(kern, dim3((unsigned)grid), dim3(kThreads), generic_floats(dk, kStates) * 4, 1, true, s, a, groups);
}

// -------------------------------------------------------------------- joining
// V neighbouring elements a thread; the segments' states are asked for kAhead at a time.
template <int V>
__global__ void __launch_bounds__(256) decay_join_kernel(float *states, const float *init, const float *decay,
                                                         const int *lengths, int64_t T, int H, int64_t seg, int nseg,
                                                         bool reverse, int64_t n, int blocks) {
  struct __align__(4 * V) Vec { float v[V]; };
  constexpr int kAhead = 8;
  const int bh = (int)(blockIdx.x / (unsigned)blocks);
  const int64_t e = ((int64_t)(blockIdx.x % (unsigned)blocks) * 256 + threadIdx.x) * V;
  chain_wait();
  if (e >= n) return;
  int64_t len = lengths ? lengths[bh / H] : T;
  len = len < 0 ? 0 : len > T ? T : len;
  const float lg = log2f(decay[bh % H]), whole = power(lg, seg);
  Vec carry = {};
  if (init) carry = *reinterpret_cast<const Vec *>(init + bh * n + e);
  float *at = states + (int64_t)bh * nseg * n + e;
  for (int i0 = 0; i0 < nseg; i0 += kAhead) {
    Vec own[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < nseg) own[i] = *reinterpret_cast<const Vec *>(at + (reverse ? nseg - 1 - i0 - i : i0 + i) * n);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= nseg) break;
      const int sg = reverse ? nseg - 1 - i0 - i : i0 + i;
      const int64_t have = len - sg * seg;  // tokens of the row from the segment's first on
      const float keep = have >= seg ? whole : power(lg, have);
      *reinterpret_cast<Vec *>(at + sg * n) = carry;
#pragma unroll
      for (int j = 0; j < V; ++j) carry.v[j] = fmaf(keep, carry.v[j], own[i].v[j]);
    }
  }
}

}  // namespace

cudaError_t launch_decay_step(const DecayStepArgs &a, cudaStream_t s) {
  return a.bf16 ? step_all<__nv_bfloat16>(a, s) : step_all<float>(a, s);
}

cudaError_t launch_decay_states(const DecayArgs &a, cudaStream_t s) {
  return a.bf16 ? generic<__nv_bfloat16, true>(a, s) : generic<float, true>(a, s);
}

cudaError_t launch_decay(const DecayArgs &a, cudaStream_t s) {
  return a.bf16 ? generic<__nv_bfloat16, false>(a, s) : generic<float, false>(a, s);
}

cudaError_t launch_decay_join(float *states, const float *init, const DecayArgs &a, bool reverse, int64_t n,
                              cudaStream_t s) {
  const int V = n % 4 == 0 ? 4 : 1;  // (init and states are whole 16-byte pieces)
  const int64_t blocks = (n / V + 255) / 256, grid = blocks * a.B * a.H;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  return chain_launch(V == 4 ? decay_join_kernel<4> : decay_join_kernel<1>, dim3((unsigned)grid), dim3(256), 0, 1, true, s,
                      states, init, a.decay, a.lengths, a.T, (int)a.H, a.seg, a.nseg, reverse, n, (int)blocks);
}

}  // namespace delta
