// decay.cu -- linear attention with a decay g for each head: the step of one token,
// the pass over the time axis in float32, also for bfloat16 layouts that decay_tc.cu's
// kernel does not take, and the joining of segments.
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
// HBM-bound: the state is read and written once (256 sequences of 32 heads, d 128:
// 156 us, 6.9 TB/s; one sequence 2.5, a launch).  A CTA has a head's state, or 32
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

// -------------------------------------------------------- the pass in float32
// A CTA has a segment of a head and 64 value columns, in chunks of 32 tokens.  The
// products run on the warp-level matrix instructions, which take tf32: each factor is
// x = hi + lo, hi rounded to 11 bits and lo what that leaves, and a product is hi hi +
// hi lo + lo hi, which leaves out 2^-22 of a term at most.  The instructions' own sums
// are cut off, not rounded, so the small products have sums of their own, and no sum
// stays there for more than a chunk: the state is kept in float32 beside them,
// transposed, in the layout of their results, with a copy in shared memory that the
// outputs read.  (B7 T1021 H5 dk64 dv96 with errors of 3.7e-7: 61 us; on the float32
// units 96, of plain float32's 2e-7.)  The order of channels and tokens within a product
// is free, and such that a lane's factors are neighbours in shared memory.  The next
// chunk's elements are asked for before this one's products.
//
// Bound by the matrix instructions, a little: 576 a warp and 128 tokens at dk 64, 8
// cycles each on a quarter of an SM, take half of the time, and the rest are the three
// barriers of a chunk, which two CTAs an SM hide in part.
constexpr int kC = 32, kCols = 64, kThreads = 256;
constexpr int kLdV = kCols + 8, kLdP = kC + 4;  // of a row of v, of P

struct Floats {  // shared memory
  int ld, lds;   // of a row of q and k, of a row (a value column) of the state
  __host__ __device__ explicit Floats(int dk) : ld((dk + 15) / 16 * 16 + 8), lds((dk + 7) / 8 * 8 + 4) {}
  __host__ __device__ int total(bool states) const {
    return kC * kLdV + kC * ld + (states ? 32 : kC * ld + kC * kLdV + kCols * lds + kC * kLdP);
  }
};

// x = hi + lo, of which the instructions read the upper 19 bits each
template <int kN>
struct Parts {
  uint32_t hi[kN], lo[kN];
  __device__ __forceinline__ void set(int i, float x) {
    hi[i] = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    lo[i] = __float_as_uint(x - __uint_as_float(hi[i]));
  }
};
// Lane 4 g + t has, of A (16 x 8), (g, t), (g + 8, t), (g, t + 4), (g + 8, t + 4), of B
// (8 x 8) (t, g), (t + 4, g), of D (16 x 8) (g, 2 t), (g, 2 t + 1), (g + 8, 2 t), (g + 8, 2 t + 1).
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
struct Sum {
  float big[4] = {}, small[4] = {};
  __device__ __forceinline__ float operator[](int i) const { return big[i] + small[i]; }
};
// the three products of several sums in turn, so that none waits for its own last one
template <int kN>
__device__ __forceinline__ void add(Sum (&s)[kN], const Parts<4> &a, const Parts<2> (&b)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i)
    mma_tf32(s[i].small, a.lo, b[i].hi);
#pragma unroll
  for (int i = 0; i < kN; ++i)
    mma_tf32(s[i].big, a.hi, b[i].hi);
#pragma unroll
  for (int i = 0; i < kN; ++i)
    mma_tf32(s[i].small, a.hi, b[i].lo);
}
__device__ __forceinline__ Parts<2> pair_of(float x, float y) {
  Parts<2> b;
  b.set(0, x), b.set(1, y);
  return b;
}
__device__ __forceinline__ Parts<4> quad_of(float x, float y, float z, float w) {
  Parts<4> a;
  a.set(0, x), a.set(1, y), a.set(2, z), a.set(3, w);
  return a;
}
__device__ __forceinline__ float2 two_at(const float *p) { return *reinterpret_cast<const float2 *>(p); }

__device__ __forceinline__ float4 scaled(const float4 &a, float f) { return make_float4(a.x * f, a.y * f, a.z * f, a.w * f); }

// four neighbouring elements, zeros past the row's `live` ones; kVec: whole vectors
template <typename In, bool kVec>
__device__ __forceinline__ float4 load4(const In *row, int live) {
  if (live <= 0) return make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (kVec) {
    if constexpr (sizeof(In) == 4) {
      return *reinterpret_cast<const float4 *>(row);
    } else {
      const uint2 u = *reinterpret_cast<const uint2 *>(row);
      return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                         __uint_as_float(u.y & 0xFFFF0000u));
    }
  } else {
    return make_float4(to_f(row[0]), live > 1 ? to_f(row[1]) : 0.f, live > 2 ? to_f(row[2]) : 0.f,
                       live > 3 ? to_f(row[3]) : 0.f);
  }
}

// and back; live: columns to the row's end
template <typename In, bool kVec>
__device__ __forceinline__ void store4(In *to, const float4 &x, int live) {
  const float v[4] = {x.x, x.y, x.z, x.w};
  if constexpr (kVec) {
    struct __align__(4 * sizeof(In)) Vec { In v[4]; } w;
#pragma unroll
    for (int i = 0; i < 4; ++i) from_f(v[i], w.v[i]);
    if (live > 0) *reinterpret_cast<Vec *>(to) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < live) from_f(v[i], to[i]);
  }
}

// kMost: blocks of 64 key channels, 1, 2 or 4
template <typename In, int kMost, bool kStates, bool kVec>
__global__ void __launch_bounds__(kThreads, kMost <= 2 ? 2 : 1) decay_generic_kernel(const __grid_constant__ DecayArgs a, int groups) {
  constexpr int kPre = kMost == 1 ? 2 : 4;  // vectors of a row asked for ahead, of 8 lanes: up to 128 channels
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
  const int ld = f.ld, lds = f.lds;
  float *sw = smem, *sk = sw + kC * kLdV, *sq = sk + kC * ld, *sv = sq + kC * ld, *S = sv + kC * kLdV, *sp = S + kCols * lds;
  const int tid = threadIdx.x, row = tid / 8, l8 = tid % 8;  // a thread's place in copies
  const int warp = tid / 32, g = tid % 32 / 4, t = tid % 4;  // and in products:
  const int m0 = warp % 2 * 16, n0 = warp / 2;               // 16 tokens, 8 of P's columns, 16 of O's
  const int s0 = warp % 4 * 16, d0 = warp / 4 * 32;          // 16 value columns and 32 channels, every 64, of the state
  if (kStates || !a.joined) chain_wait();
  const float lg = log2f(a.decay[h]);
  int64_t len = a.lengths ? a.lengths[b] : a.T;
  len = len < 0 ? 0 : len > a.T ? a.T : len;
  const int64_t t_lo = sg * a.seg, t_hi = min(t_lo + a.seg, a.T);
  const int64_t t_end = min(t_hi, len);  // tokens [t_lo, t_end) count
  const int64_t state_at = kStates || a.nseg > 1 ? bh * a.nseg + sg : bh;
  const bool unread = kStates && sg == (p.reverse ? 0 : a.nseg - 1);  // no segment begins with its state
  const int64_t chunks = t_end > t_lo && !unread ? (t_end - t_lo + kC - 1) / kC : 0;
  const int64_t from = t_lo + (p.reverse && chunks > 0 ? chunks - 1 : 0) * kC, hop = p.reverse ? -kC : kC;
  // this thread's rows, of the chunk that is asked for
  const In *krow = static_cast<const In *>(p.k) + b * p.ks[0] + h * p.ks[2] + (from + row) * p.ks[1] + l8 * 4;
  const In *qrow = kStates ? nullptr : static_cast<const In *>(p.q) + b * p.qs[0] + h * p.qs[2] + (from + row) * p.qs[1] + l8 * 4;
  const In *vrow = static_cast<const In *>(p.v) + b * p.vs[0] + h * p.vs[2] + (from + row) * p.vs[1] + c0 + l8 * 4;
  const int64_t khop = hop * p.ks[1], qhop = hop * p.qs[1], vhop = hop * p.vs[1];
  const bool reverse = p.reverse;
  const float kvs = p.kvs, os = p.os;
  int left = (int)(t_end - from);  // tokens from the chunk's first on
  In *out = kStates ? nullptr : static_cast<In *>(p.out) + ((b * a.T + from + m0 + g) * a.H + h) * p.dv + c0 + 16 * n0 + 4 * t;
  const int64_t out8 = (int64_t)8 * a.H * p.dv;  // eight tokens on
  float4 nk[kPre], nq[kStates ? 1 : kPre], nv[2];
  const auto ask = [&](bool on) {
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      const int live = on ? dk - l8 * 4 - 32 * i : 0;
      nk[i] = load4<In, kVec>(krow + 32 * i, live);
      if constexpr (!kStates) nq[i] = load4<In, kVec>(qrow + 32 * i, live);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) nv[i] = load4<In, kVec>(vrow + 32 * i, on ? cols - l8 * 4 - 32 * i : 0);
  };
  Keep keep = {0.f, 0.f};  // of a chunk of `kept` tokens
  float owed = 0.f;
  int kept = -1;
  ask(chunks > 0 && row < left);
  if (!kStates && a.joined) chain_wait();  // (all but the joined states was there before)
  // st[i][x][y]: channel 64 i + d0 + 8 t + 4 (y % 2) + x, value column s0 + 2 g + y / 2
  float st[kMost][4][4];
#pragma unroll
  for (int i = 0; i < kMost; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int d = 64 * i + d0 + 8 * t + 4 * (y % 2) + x, c = s0 + 2 * g + y / 2;
        st[i][x][y] = 0.f;
        if (!kStates && p.init && d < dk && c < cols)
          st[i][x][y] = p.init[state_at * dk * p.dv + (p.init_t ? (int64_t)(c0 + c) * dk + d : (int64_t)d * p.dv + c0 + c)];
      }
  for (int64_t ci = 0; ci < chunks; ++ci) {
    const int n = min(kC, left);
    if (n != kept) keep = keep_of(lg, n), kept = n;
    const float now = keep_now(keep, owed);
    __syncthreads();  // what the last chunk read may be written
    {
      const float w = row < n ? kvs * power(lg, reverse ? row + 1 : n - 1 - row) : 0.f;  // to the chunk's end, or past its start
#pragma unroll
      for (int i = 0; i < kPre; ++i) {
        const int c = (l8 + 8 * i) * 4;
        if (c < ld - 8) {
          *reinterpret_cast<float4 *>(sk + row * ld + c) = nk[i];
          if constexpr (!kStates) *reinterpret_cast<float4 *>(sq + row * ld + c) = nq[i];
        }
      }
      for (int c = (l8 + 8 * kPre) * 4; kMost > 2 && c < ld - 8; c += 32) {
        const int live = row < n ? dk - c : 0;
        *reinterpret_cast<float4 *>(sk + row * ld + c) = load4<In, kVec>(krow + c - l8 * 4, live);
        if constexpr (!kStates) *reinterpret_cast<float4 *>(sq + row * ld + c) = load4<In, kVec>(qrow + c - l8 * 4, live);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = (l8 + 8 * i) * 4;
        if constexpr (!kStates) *reinterpret_cast<float4 *>(sv + row * kLdV + c) = scaled(nv[i], kvs);
        *reinterpret_cast<float4 *>(sw + row * kLdV + c) = scaled(nv[i], w);
      }
    }
    if constexpr (!kStates) {
#pragma unroll
      for (int i = 0; i < kMost; ++i)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int d = 64 * i + d0 + 8 * t + 4 * (y % 2);
          if (d < lds - 4)
            *reinterpret_cast<float4 *>(S + (s0 + 2 * g + y / 2) * lds + d) =
                make_float4(st[i][0][y], st[i][1][y], st[i][2][y], st[i][3][y]);
        }
    }
    __syncthreads();
    left -= (int)hop;
    krow += khop, vrow += vhop;
    if constexpr (!kStates) qrow += qhop;
    if (ci + 1 < chunks) ask(row < left);
    if constexpr (!kStates) {
      // G, and the state's part of O: column 2 x + e of 16 is e of the product's x
      const bool none = reverse ? 8 * n0 + 7 < m0 : 8 * n0 > m0 + 15;  // all of it is masked
      Sum o[3], out2[2];  // O's two, and G
      {
        const float *qa = sq + (m0 + g) * ld + 2 * t, *ka = sk + (8 * n0 + g) * ld + 2 * t;
        const float *sa = S + (16 * n0 + 2 * g) * lds + 2 * t;
#pragma unroll kMost == 1 ? 1 : 2
        for (int d = 0; d < lds - 4; d += 8) {
          const float2 x = two_at(qa + d), y = two_at(qa + 8 * ld + d), k = two_at(ka + d);
          const float2 u = two_at(sa + d), w = two_at(sa + lds + d);
          const Parts<4> q = quad_of(x.x, y.x, x.y, y.y);
          add(o, q, {pair_of(u.x, u.y), pair_of(w.x, w.y), pair_of(k.x, k.y)});
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = m0 + g + 8 * y, j = 8 * n0 + 2 * t, apart = reverse ? j - i : i - j;
        if (!none)
          *reinterpret_cast<float2 *>(sp + i * kLdP + j) =
              make_float2(apart < 0 ? 0.f : o[2][2 * y] * power(lg, apart),
                          apart < (reverse ? -1 : 1) ? 0.f : o[2][2 * y + 1] * power(lg, apart + (reverse ? 1 : -1)));
        const float c = power(lg, reverse ? n - 1 - i : i + 1);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 2 * y; e < 2 * y + 2; ++e) out2[x].big[e] = o[x][e] * c;
      }
      // the four warps of these 16 tokens have their part of P
      asm volatile("bar.sync %0, 128;" ::"r"(1 + warp % 2) : "memory");
      {
        const float *pa = sp + (m0 + g) * kLdP + t, *va = sv + t * kLdV + 16 * n0 + 2 * g;
        const int first = reverse ? m0 : 0, end = reverse ? kC : m0 + 16;
#pragma unroll 2
        for (int r = first; r < end; r += 8) {
          const Parts<4> w = quad_of(pa[r], pa[8 * kLdP + r], pa[r + 4], pa[8 * kLdP + r + 4]);
          const float2 x = two_at(va + r * kLdV), y = two_at(va + (r + 4) * kLdV);
          add(out2, w, {pair_of(x.x, y.x), pair_of(x.y, y.y)});
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = m0 + g + 8 * y, c = 16 * n0 + 4 * t;
        if (i >= n) continue;
        const float4 r = scaled(make_float4(out2[0][2 * y], out2[1][2 * y], out2[0][2 * y + 1], out2[1][2 * y + 1]), os);
        store4<In, kVec>(out + y * out8, r, cols - c);
      }
      out += reverse ? -4 * out8 : 4 * out8;
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
      const int d = 64 * i + d0;
      if (d >= dk) break;
      Sum sum[4];
      // (channels past the last vector of k lie in the next row: of no state that counts)
      const float *va = sw + t * kLdV + s0 + 2 * g, *ka = sk + t * ld + d + 4 * g;
#pragma unroll 1
      for (int r = 0; r < kC; r += 8) {
        const float2 x = two_at(va + r * kLdV), y = two_at(va + (r + 4) * kLdV);
        const float4 k = *reinterpret_cast<const float4 *>(ka + r * ld);
        const float4 l = *reinterpret_cast<const float4 *>(ka + (r + 4) * ld);
        const Parts<4> v = quad_of(x.x, x.y, y.x, y.y);
        add(sum, v, {pair_of(k.x, l.x), pair_of(k.y, l.y), pair_of(k.z, l.z), pair_of(k.w, l.w)});
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) st[i][x][y] = fmaf(now, st[i][x][y], sum[x][y]);
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
          const int d = 64 * i + d0 + 8 * t + 4 * (y % 2) + x, c = s0 + 2 * g + y / 2;
          if (d < dk && c < cols) to[(int64_t)d * p.dv + c0 + c] = st[i][x][y];
        }
  }
  if constexpr (!kStates) {  // tokens past the row's end
    for (int64_t at = max(t_lo, t_end) + row; at < t_hi; at += kThreads / 8)
      for (int c = l8; c < cols; c += 8)
        from_f(0.f, static_cast<In *>(p.out)[((b * a.T + at) * a.H + h) * p.dv + c0 + c]);
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
  auto kern = dk <= 64    ? (vec ? decay_generic_kernel<In, 1, kStates, true> : decay_generic_kernel<In, 1, kStates, false>)
              : dk <= 128 ? (vec ? decay_generic_kernel<In, 2, kStates, true> : decay_generic_kernel<In, 2, kStates, false>)
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
