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
#include "decay.cuh"
#include "kernels.h"

namespace delta {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float &r) { r = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16 &r) { r = __float2bfloat16_rn(x); }

using namespace decay;

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
// In float32: a CTA has a segment of a head and 64 value columns, in chunks of 32
// tokens.  Its state is in registers, 4 x 4 elements a thread for every 64 key channels,
// with a copy in shared memory that the outputs read; two CTAs share an SM up to 128
// channels.  Operands are read from shared memory four at a time: 32 products for 6
// reads in the outputs, 16 for 2 in the state.  The next chunk's elements are asked for
// before this one's products.
constexpr int kC = 32, kCols = 64, kThreads = 256;
constexpr int kPre = 4;  // vectors of a row asked for ahead, of 8 lanes: 128 channels

struct Floats {  // shared memory
  int ld;        // of a row of q and k: whole vectors, one more against bank conflicts
  __host__ __device__ explicit Floats(int dk) : ld((dk + 3) / 4 * 4 + 4) {}
  __host__ __device__ int rows() const { return (ld - 4 + 63) / 64 * 64; }  // of the state
  __host__ __device__ int total(bool states) const {
    return rows() * kCols + 2 * kC * kCols + (states ? kC * ld : 2 * kC * ld + kC * (kC + 4));
  }
};

__device__ __forceinline__ float4 scaled(const float4 &a, float f) { return make_float4(a.x * f, a.y * f, a.z * f, a.w * f); }
__device__ __forceinline__ void axpy(float (&o)[4], float f, const float4 &x) {
  o[0] = fmaf(f, x.x, o[0]), o[1] = fmaf(f, x.y, o[1]), o[2] = fmaf(f, x.z, o[2]), o[3] = fmaf(f, x.w, o[3]);
}

// four elements of a row from column c on, zeros past its end; kVec: whole vectors
template <typename In, bool kVec>
__device__ __forceinline__ float4 load4(const In *row, int c, int width) {
  if (c >= width) return make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (kVec) {
    if constexpr (sizeof(In) == 4) {
      return *reinterpret_cast<const float4 *>(row + c);
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(row + c);
      return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                         __uint_as_float(u.y & 0xFFFF0000u));
    }
  } else {
    return make_float4(to_f(row[c]), c + 1 < width ? to_f(row[c + 1]) : 0.f, c + 2 < width ? to_f(row[c + 2]) : 0.f,
                       c + 3 < width ? to_f(row[c + 3]) : 0.f);
  }
}

// kMost: blocks of 64 key channels, 2 or 4
template <typename In, int kMost, bool kStates, bool kVec>
__global__ void __launch_bounds__(kThreads, kMost == 2 ? 2 : 1) decay_generic_kernel(const __grid_constant__ DecayArgs a, int groups) {
  extern __shared__ __align__(16) float smem[];
  uint32_t item = blockIdx.x;
  const DecayPass &p = a.pass[item % (uint32_t)a.passes];
  item /= (uint32_t)a.passes;
  const int sg = (int)(item % (uint32_t)a.nseg);
  item /= (uint32_t)a.nseg;
  const int c0 = (int)(item % (uint32_t)groups) * kCols;
  const int64_t bh = item / (uint32_t)groups, b = bh / a.H, h = bh % a.H;
  if (c0 >= p.dv) return;
  const int dk = p.dk, cols = min(kCols, p.dv - c0);
  const Floats f(dk);
  const int ld = f.ld, srows = f.rows();
  float *S = smem, *sv = S + srows * kCols, *sw = sv + kC * kCols, *sk = sw + kC * kCols, *sq = sk + kC * ld, *sp = sq + kC * ld;
  const int tid = threadIdx.x, r16 = tid / 16, c16 = tid % 16;  // a thread's places in products
  const int row = tid / 8, l8 = tid % 8;                         // and in copies
  chain_wait();
  const float lg = log2f(a.decay[h]);
  int64_t len = a.lengths ? a.lengths[b] : a.T;
  len = len < 0 ? 0 : len > a.T ? a.T : len;
  const int64_t t_lo = sg * a.seg, t_hi = min(t_lo + a.seg, a.T);
  const int64_t t_end = min(t_hi, len);  // tokens [t_lo, t_end) count
  const int64_t state_at = kStates || a.nseg > 1 ? bh * a.nseg + sg : bh;
  float st[kMost][4][4];  // state rows 64 i + 4 r16 .. + 3, columns 4 c16 .. + 3
#pragma unroll
  for (int i = 0; i < kMost; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int d = 64 * i + 4 * r16 + x, c = 4 * c16 + y;
        st[i][x][y] = 0.f;
        if (!kStates && p.init && d < dk && c < cols)
          st[i][x][y] = p.init[state_at * dk * p.dv + (p.init_t ? (int64_t)(c0 + c) * dk + d : (int64_t)d * p.dv + c0 + c)];
      }
  const int64_t chunks = t_end > t_lo ? (t_end - t_lo + kC - 1) / kC : 0;
  const auto start_of = [&](int64_t ci) { return t_lo + (p.reverse ? chunks - 1 - ci : ci) * kC; };
  const In *krow = static_cast<const In *>(p.k) + b * p.ks[0] + h * p.ks[2];
  const In *qrow = kStates ? nullptr : static_cast<const In *>(p.q) + b * p.qs[0] + h * p.qs[2];
  const In *vrow = static_cast<const In *>(p.v) + b * p.vs[0] + h * p.vs[2] + c0;
  float4 nk[kPre], nq[kStates ? 1 : kPre], nv[2];
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto ask = [&](int64_t ci) {
    const int64_t t = start_of(ci) + row;
    const bool on = t < t_end;
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      const int c = (l8 + 8 * i) * 4;
      nk[i] = on ? load4<In, kVec>(krow + t * p.ks[1], c, dk) : zero;
      if constexpr (!kStates) nq[i] = on ? load4<In, kVec>(qrow + t * p.qs[1], c, dk) : zero;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) nv[i] = on ? load4<In, kVec>(vrow + t * p.vs[1], (l8 + 8 * i) * 4, cols) : zero;
  };
  Keep keep = {0.f, 0.f};  // of a chunk of `kept` tokens
  float owed = 0.f;
  int kept = -1;
  if (chunks > 0) ask(0);
  for (int64_t ci = 0; ci < chunks; ++ci) {
    const int64_t t0 = start_of(ci);
    const int n = (int)min((int64_t)kC, t_end - t0);
    if (n != kept) keep = keep_of(lg, n), kept = n;
    const float now = keep_now(keep, owed);
    __syncthreads();  // what the last chunk read may be written
    {
      const float w = p.kvs * power(lg, p.reverse ? row + 1 : n - 1 - row);  // to the chunk's end, or past its start
#pragma unroll
      for (int i = 0; i < kPre; ++i) {
        const int c = (l8 + 8 * i) * 4;
        if (c < ld - 4) {
          *reinterpret_cast<float4 *>(sk + row * ld + c) = nk[i];
          if constexpr (!kStates) *reinterpret_cast<float4 *>(sq + row * ld + c) = nq[i];
        }
      }
      for (int c = (l8 + 8 * kPre) * 4; kMost > 2 && c < ld - 4; c += 32) {
        const bool on = row < n;
        *reinterpret_cast<float4 *>(sk + row * ld + c) = on ? load4<In, kVec>(krow + (t0 + row) * p.ks[1], c, dk) : zero;
        if constexpr (!kStates)
          *reinterpret_cast<float4 *>(sq + row * ld + c) = on ? load4<In, kVec>(qrow + (t0 + row) * p.qs[1], c, dk) : zero;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = (l8 + 8 * i) * 4;
        if constexpr (!kStates) *reinterpret_cast<float4 *>(sv + row * kCols + c) = scaled(nv[i], p.kvs);
        *reinterpret_cast<float4 *>(sw + row * kCols + c) = row < n ? scaled(nv[i], w) : zero;
      }
    }
    if constexpr (!kStates) {
#pragma unroll
      for (int i = 0; i < kMost; ++i)
        if (64 * i < srows)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<float4 *>(S + (64 * i + 4 * r16 + x) * kCols + 4 * c16) =
                make_float4(st[i][x][0], st[i][x][1], st[i][x][2], st[i][x][3]);
    }
    __syncthreads();
    if (ci + 1 < chunks) ask(ci + 1);
    if constexpr (!kStates) {
      // P: rows r16 and r16 + 16, columns c16 and c16 + 16
      float s[2][2] = {};
#pragma unroll 1
      for (int d = 0; d < ld - 4; d += 4) {
        float4 q[2], k[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          q[x] = *reinterpret_cast<const float4 *>(sq + (r16 + 16 * x) * ld + d);
          k[x] = *reinterpret_cast<const float4 *>(sk + (c16 + 16 * x) * ld + d);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            s[x][y] = fmaf(q[x].w, k[y].w, fmaf(q[x].z, k[y].z, fmaf(q[x].y, k[y].y, fmaf(q[x].x, k[y].x, s[x][y]))));
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int i = r16 + 16 * x, j = c16 + 16 * y, apart = p.reverse ? j - i : i - j;
          sp[i * (kC + 4) + j] = apart < 0 ? 0.f : s[x][y] * power(lg, apart);
        }
      // O: rows r16 and r16 + 16, columns 4 c16 ..; the state's part first, then its factor
      float o[2][4] = {};
#pragma unroll 1
      for (int d = 0; d < ld - 4; d += 4) {
        float4 q[2], x[4];
#pragma unroll
        for (int y = 0; y < 2; ++y) q[y] = *reinterpret_cast<const float4 *>(sq + (r16 + 16 * y) * ld + d);
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = *reinterpret_cast<const float4 *>(S + (d + y) * kCols + 4 * c16);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          axpy(o[y], q[y].x, x[0]), axpy(o[y], q[y].y, x[1]), axpy(o[y], q[y].z, x[2]), axpy(o[y], q[y].w, x[3]);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = r16 + 16 * y;
        const float c = power(lg, p.reverse ? n - 1 - i : i + 1);
#pragma unroll
        for (int x = 0; x < 4; ++x) o[y][x] *= c;
      }
      __syncthreads();  // P is there
#pragma unroll 2
      for (int r = 0; r < kC; r += 4) {
        float4 w[2], x[4];
#pragma unroll
        for (int y = 0; y < 2; ++y) w[y] = *reinterpret_cast<const float4 *>(sp + (r16 + 16 * y) * (kC + 4) + r);
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = *reinterpret_cast<const float4 *>(sv + (r + y) * kCols + 4 * c16);
#pragma unroll
        for (int y = 0; y < 2; ++y)
          axpy(o[y], w[y].x, x[0]), axpy(o[y], w[y].y, x[1]), axpy(o[y], w[y].z, x[2]), axpy(o[y], w[y].w, x[3]);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = r16 + 16 * y;
        if (i >= n) continue;
        In *out = static_cast<In *>(p.out) + ((b * a.T + t0 + i) * a.H + h) * p.dv + c0 + 4 * c16;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (4 * c16 + x < cols) from_f(p.os * o[y][x], out[x]);
      }
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      if (64 * i >= srows) break;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) st[i][x][y] *= now;
      // (channels past the last vector of k lie in the next row: of no state that counts)
      const int d = min(64 * i + 4 * r16, ld - 4);
#pragma unroll 4
      for (int r = 0; r < kC; ++r) {
        const float4 k = *reinterpret_cast<const float4 *>(sk + r * ld + d);
        const float4 v = *reinterpret_cast<const float4 *>(sw + r * kCols + 4 * c16);
        axpy(st[i][0], k.x, v), axpy(st[i][1], k.y, v), axpy(st[i][2], k.z, v), axpy(st[i][3], k.w, v);
      }
    }
  }
  if (kStates || (p.final && sg == (p.reverse ? 0 : a.nseg - 1))) {
    float *to = p.final + (kStates ? state_at : bh) * dk * p.dv;
#pragma unroll
    for (int i = 0; i < kMost; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int d = 64 * i + 4 * r16 + x, c = 4 * c16 + y;
          if (d < dk && c < cols) to[(int64_t)d * p.dv + c0 + c] = st[i][x][y];
        }
  }
  if constexpr (!kStates) {  // tokens past the row's end
    for (int64_t t = max(t_lo, t_end) + row; t < t_hi; t += kThreads / 8)
      for (int c = l8; c < cols; c += 8)
        from_f(0.f, static_cast<In *>(p.out)[((b * a.T + t) * a.H + h) * p.dv + c0 + c]);
  }
}

template <typename In, bool kStates>
cudaError_t generic(const DecayArgs &a, cudaStream_t s) {
  int dk = 1, dv = 1;
  bool vec = true;  // rows in whole vectors of four
  const int64_t n[3] = {a.B, a.T, a.H};
  const auto whole = [&](const void *q, const int64_t (&st)[3]) {
    bool ok = reinterpret_cast<uintptr_t>(q) % (4 * sizeof(In)) == 0;
    for (int i = 0; i < 3; ++i) ok = ok && (n[i] <= 1 || st[i] % 4 == 0);
    return ok;
  };
  for (int i = 0; i < a.passes; ++i) {
    const DecayPass &p = a.pass[i];
    dk = max(dk, p.dk), dv = max(dv, p.dv);
    vec = vec && p.dk % 4 == 0 && p.dv % 4 == 0 && whole(p.k, p.ks) && whole(p.v, p.vs) && (kStates || whole(p.q, p.qs));
  }
  const int groups = (dv + kCols - 1) / kCols;
  const int64_t grid = a.B * a.H * groups * a.nseg * a.passes;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  auto kern = dk <= 128 ? (vec ? decay_generic_kernel<In, 2, kStates, true> : decay_generic_kernel<In, 2, kStates, false>)
                        : (vec ? decay_generic_kernel<In, 4, kStates, true> : decay_generic_kernel<In, 4, kStates, false>);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             Floats(kDecayMaxD).total(kStates) * 4);
  if (e != cudaSuccess) return e;
  return chain_launch(kern, dim3((unsigned)grid), dim3(kThreads), Floats(dk).total(kStates) * 4, 1, true, s, a, groups);
}

// -------------------------------------------------------------------- joining
// V neighbouring elements a thread; the segments' states are asked for kAhead at a time.
template <int V>
__global__ void __launch_bounds__(256) decay_join_kernel(float *states, const float *init, const float *decay,
                                                         const int *lengths, int64_t T, int H, int64_t seg, int nseg,
                                                         bool reverse, int64_t n, int blocks) {
  struct __align__(4 * V) Vec { float v[V]; };
  constexpr int kAhead = 16;
  const int bh = (int)(blockIdx.x / (unsigned)blocks);
  const int64_t e = ((int64_t)(blockIdx.x % (unsigned)blocks) * 256 + threadIdx.x) * V;
  chain_wait();
  chain_next();  // (the pass that follows sets itself up meanwhile)
  if (e >= n) return;
  int64_t len = lengths ? lengths[bh / H] : T;
  len = len < 0 ? 0 : len > T ? T : len;
  const float lg = log2f(decay[bh % H]);
  const Keep whole = keep_of(lg, seg);
  float owed = 0.f;
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
      const float keep = keep_now(have >= seg ? whole : keep_of(lg, have), owed);
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
