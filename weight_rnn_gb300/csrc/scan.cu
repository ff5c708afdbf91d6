// scan.cu -- the gated linear recurrence, one state per channel:
//
//   h_t = a_t h_{t-1} + u_t x_t,   out_t = h_t
//
// linear form: a_t = gate_t (float32), u_t = 1, and a_t = 0 drops the past
// whatever it holds (an infinite or NaN state does not cross a reset).
// Sigmoid form: a_t = 1 / (1 + e), u_t = e / (1 + e) with e = exp(-f_t), so
// that neither loses digits when the other is close to 1.
//
// Reverse: with c_T = dhT,  dh_t = dout_t + c_t  and  c_{t-1} = a_t dh_t;
// dx_t = u_t dh_t, dgate_t = dh_t h_{t-1} (linear) or
// dh_t a_t (u_t h_{t-1} - u_t x_t) (sigmoid), dh0 = c_0.
//
// Both directions are bound by HBM: every element is read once and written
// once.  A recurrence step is the affine map h -> a h + b, and maps compose:
// (A, B) after (A', B') is (A A', A B' + B).  So a tile of 32 VEC channels is
// cut into sub-chunks of consecutive steps, one per warp, lane = VEC channels:
//   1. each warp takes its steps from its own ring in shared memory, filled
//      a tile ahead by asynchronous copies, and composes its map;
//   2. the maps meet in shared memory (one barrier), and every warp folds
//      them in time order onto the state carried from the last tile, which
//      gives the state at its own start and, redundantly in every warp, the
//      state carried to the next tile;
//   3. each warp runs the recurrence again from its start and writes out.
// Where the (batch row, channel strip) pairs alone do not fill the GPU, a
// cluster of `cs` CTAs takes cs neighbouring tiles at a time and exchanges one
// map per CTA through distributed shared memory, by asynchronous stores that
// count on the receiver's mbarrier (a cluster-wide barrier would release, that
// is wait for, every output store: it took a third of the cycles).  The fold
// order is the time order, so results do not depend on scheduling.  All maps and states are
// float32; two channels of a lane go through packed float32 pairs.
//
// A map stands for its steps only while its decay A and offsets B are float32
// numbers, and a product of decays can leave float32's range where no state does.
// In the linear form a warp's product is therefore taken with subnormals flushed:
// one that has left the normal range at any point ends as 0, Inf or NaN, and is
// then looked at again (look, settle):
//   a reset among the steps: A is 0, and 0 in a warp's map means that;
//   decays of at most 1: A is kept as a subnormal, never 0, which carries Inf and
//     NaN on and is off by less than 2^-145, nothing next to states up to 2^16;
//   else, where |A| passes 2^24 (B's rounding then hides a state that B all but
//     cancels), and where B is not finite: A is NaN, the map is not used.
// A warp whose map is one of these looks at its own state, which is what the map
// was applied to.  A cluster's maps are joined and sent unchecked; their CTA checks
// them while they are on their way (misjoined, misused).  Sigmoid decays are at
// most 1 and drop nothing, so there only a state that became NaN is suspect (Inf
// times a product that is 0).  Where a map did not hold, every CTA of the row goes
// through those channels again at its end, step by step (redo): 130 to 290 ns a step,
// which data in range never takes.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "chain.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace delta {
namespace {

__device__ unsigned int g_scan_error = 0;

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kFwdSteps = 16;            // steps per warp and tile
constexpr int kBwdSteps = 8;             // (the reverse holds twice the values per step)
static_assert(kScanBlock % kFwdSteps == 0 && kScanBlock == kWarps * kBwdSteps,
              "states are saved at a warp's start, and taken at a reverse tile's");
constexpr int kMaxCluster = 16;          // (8 is the portable size, 16 the opt-in)
// Tiles in a warp's ring.  With three (where they fit) B4 T8192 D4096 took
// 137 us instead of 127, and a reverse ring of the linear form kept a second
// CTA off the SM (732 us instead of 423 at B1 T65536 D2048).
constexpr int kStages = 2;

// VEC neighbouring elements as they lie in memory
template <typename T, int VEC>
struct Raw;
template <> struct Raw<float, 1> { using type = float; };
template <> struct Raw<float, 2> { using type = float2; };
template <> struct Raw<__nv_bfloat16, 1> { using type = unsigned short; };
template <> struct Raw<__nv_bfloat16, 2> { using type = unsigned int; };

__device__ __forceinline__ void widen(float r, float (&v)[1]) { v[0] = r; }
__device__ __forceinline__ void widen(float2 r, float (&v)[2]) { v[0] = r.x; v[1] = r.y; }
__device__ __forceinline__ void widen(unsigned short r, float (&v)[1]) {
  v[0] = __uint_as_float((unsigned)r << 16);
}
__device__ __forceinline__ void widen(unsigned int r, float (&v)[2]) {
  v[0] = __uint_as_float(r << 16);
  v[1] = __uint_as_float(r & 0xFFFF0000u);
}
// the one rounding of an output, to nearest even
__device__ __forceinline__ void narrow(const float (&v)[1], float &r) { r = v[0]; }
__device__ __forceinline__ void narrow(const float (&v)[2], float2 &r) { r = make_float2(v[0], v[1]); }
__device__ __forceinline__ void narrow(const float (&v)[1], unsigned short &r) {
  r = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
}
__device__ __forceinline__ void narrow(const float (&v)[2], unsigned int &r) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
  r = *reinterpret_cast<const unsigned int *>(&h);
}

template <typename T, int VEC>
__device__ __forceinline__ typename Raw<T, VEC>::type load(const T *p) {
  return __ldcs(reinterpret_cast<const typename Raw<T, VEC>::type *>(p));
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T *p, const float (&v)[VEC]) {
  typename Raw<T, VEC>::type r;
  narrow(v, r);
  __stcs(reinterpret_cast<typename Raw<T, VEC>::type *>(p), r);
}

// float32 pairs: one instruction for both channels
__device__ __forceinline__ uint64_t pk(const float (&v)[2]) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v[0]), "f"(v[1]));
  return r;
}
__device__ __forceinline__ void unpk(uint64_t r, float (&v)[2]) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(r));
}
template <int VEC>
__device__ __forceinline__ void vfma(const float (&a)[VEC], const float (&b)[VEC], const float (&c)[VEC],
                                     float (&d)[VEC]) {
  if constexpr (VEC == 2) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)), "l"(pk(c)));
    unpk(r, d);
  } else {
    d[0] = fmaf(a[0], b[0], c[0]);
  }
}
template <int VEC>
__device__ __forceinline__ void vmul(const float (&a)[VEC], const float (&b)[VEC], float (&d)[VEC]) {
  if constexpr (VEC == 2) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
    unpk(r, d);
  } else {
    d[0] = __fmul_rn(a[0], b[0]);  // (not to be fused: the same bits on every path, as for pairs)
  }
}
// the same with subnormal factors and results as 0
template <int VEC>
__device__ __forceinline__ void vmul_ftz(const float (&a)[VEC], const float (&b)[VEC], float (&d)[VEC]) {
  if constexpr (VEC == 2) {
    uint64_t r;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
    unpk(r, d);
  } else {
    asm("mul.rn.ftz.f32 %0, %1, %2;" : "=f"(d[0]) : "f"(a[0]), "f"(b[0]));
  }
}
template <int VEC>
__device__ __forceinline__ void vadd(const float (&a)[VEC], const float (&b)[VEC], float (&d)[VEC]) {
  if constexpr (VEC == 2) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a)), "l"(pk(b)));
    unpk(r, d);
  } else {
    d[0] = __fadd_rn(a[0], b[0]);
  }
}

// d = a h + b, the step map; with kDrop a = 0 drops h whatever it holds.  The
// selects that this takes are half of the linear form's instructions, so a warp
// uses them for its steps only where a reset is among them.
template <bool kDrop, int VEC>
__device__ __forceinline__ void affine(const float (&a)[VEC], const float (&h)[VEC], const float (&b)[VEC],
                                       float (&d)[VEC]) {
  if constexpr (!kDrop) {
    vfma(a, h, b, d);
  } else {
    float r[VEC];
    vfma(a, h, b, r);
#pragma unroll
    for (int i = 0; i < VEC; ++i) d[i] = a[i] == 0.f ? b[i] : r[i];
  }
}
// d = a h, likewise
template <bool kDrop, int VEC>
__device__ __forceinline__ void decay(const float (&a)[VEC], const float (&h)[VEC], float (&d)[VEC]) {
  float r[VEC];
  vmul(a, h, r);
#pragma unroll
  for (int i = 0; i < VEC; ++i) d[i] = kDrop && a[i] == 0.f ? 0.f : r[i];
}

// a and u from the gate.  Sigmoid: e = 2^min(-f log2 e, 126) stays finite, so
// that u = e / (1 + e) is 1 at f = -inf; taking 2^-126 off a then makes it
// exactly 0 there, and changes no a above 2^-102.  The MUFU operations are
// good to about 2^-22 and 2^-23.
template <bool kSig, int VEC>
__device__ __forceinline__ void gates(const float (&g)[VEC], float (&a)[VEC], float (&u)[VEC]) {
  if constexpr (kSig) {
    float e[VEC], l[VEC], one[VEC], low[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      l[i] = -1.4426950408889634f;
      one[i] = 1.f;
      low[i] = -1.1754943508222875e-38f;
    }
    vmul(g, l, e);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      asm("min.NaN.f32 %0, %1, %2;" : "=f"(e[i]) : "f"(e[i]), "f"(126.f));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(e[i]));
    }
    vadd(e, one, a);
#pragma unroll
    for (int i = 0; i < VEC; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a[i]) : "f"(a[i]));
    vmul(e, a, u);
    vadd(a, low, a);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = g[i], u[i] = 1.f;
  }
}

__device__ __forceinline__ int64_t row_length(const int *lengths, int64_t b, int64_t T) {
  if (!lengths) return T;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// ---------------------------------------------------------- the warps' rings
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A strip's row (32 VEC channels) in a ring.  kWide: rows are whole 16-byte
// pieces.  Else the pieces that cover a row are copied, wherever it starts (in
// memory before a tensor's first element lies the rest of its 16 bytes), and
// its elements begin `head` bytes in.
template <typename T, int VEC, bool kWide>
struct Strip {
  static constexpr int kBytes = 32 * VEC * (int)sizeof(T);
  static constexpr int kPieces = kBytes / 16 + (kWide ? 0 : 1);
  static constexpr int kPitch = kPieces * 16;

  // S rows into `to`, by one warp.  Rows from n on and channels past `left`
  // are not read.
  template <int S>
  __device__ __forceinline__ static void fetch(unsigned char *to, const T *row, int64_t stride, int64_t n,
                                               int64_t left, int lane) {
    const int have = left < 32 * VEC ? (int)left * (int)sizeof(T) : kBytes;
#pragma unroll
    for (int k = 0; k < (S * kPieces + 31) / 32; ++k) {
      const int i = k * 32 + lane, s = i / kPieces, c = i % kPieces * 16;
      const uint32_t d = (uint32_t)__cvta_generic_to_shared(to + s * kPitch + c);
      if constexpr (kWide) {
        const bool in = s < n && c < have;  // what is not there becomes zeros
        const T *from = row + (in ? s * stride + c / (int)sizeof(T) : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(from), "r"(in ? 16 : 0) : "memory");
      } else {
        const unsigned char *from = reinterpret_cast<const unsigned char *>(row + s * stride);
        const int head = (int)(reinterpret_cast<uintptr_t>(from) & 15), bytes = have + head - c;
        if (s < n && s < S && bytes > 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(from + c - head),
                       "r"(bytes < 16 ? bytes : 16)
                       : "memory");
      }
    }
  }
  // a lane's channels of row s, of a group whose row 0 is at `row`
  __device__ __forceinline__ static void read(const unsigned char *at, const T *row, int64_t stride, int s, int lane,
                                              float (&v)[VEC]) {
    int off = s * kPitch + lane * VEC * (int)sizeof(T);
    if constexpr (!kWide)
      off += ((uint32_t)reinterpret_cast<uintptr_t>(row) + (uint32_t)s * (uint32_t)stride * (uint32_t)sizeof(T)) & 15;
    widen(*reinterpret_cast<const typename Raw<T, VEC>::type *>(at + off), v);
  }
};

// one warp's map (or a CTA's): decays and offsets of a lane's channels
template <int VEC, int kOffsets>
struct Map {
  float a[VEC], b[kOffsets][VEC];
};

constexpr float kNormal = 1.1754943508222875e-38f;  // 2^-126
constexpr float kLeast = 1.401298464324817e-45f;    // 2^-149, the smallest subnormal
constexpr float kLooseState = 65536.f;              // the largest state that a subnormal decay is used on
constexpr float kMostGrowth = 16777216.f;           // 2^24
// A warp's decay that needs no look.  Eight such make a CTA's at most 2^8, and one
// that falls to 0 on the way has lost no more than 2^-126 of a state of 2^16.
constexpr float kPlain = 2.f;
__device__ __forceinline__ float infinity() { return __int_as_float(0x7f800000); }
__device__ __forceinline__ float unusable() { return __int_as_float(0x7fffffff); }
__device__ __forceinline__ bool subnormal(float v) { return v != 0.f && fabsf(v) < kNormal; }

// whether a map of the linear form needs no second look: its decays are normal
// numbers of at most 2, or 0 by a reset
template <int VEC, int kOffsets>
__device__ __forceinline__ bool plain(const Map<VEC, kOffsets> &m, const bool (&reset)[VEC]) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < VEC; ++i) ok &= (m.a[i] != 0.f || reset[i]) && fabsf(m.a[i]) <= kPlain;
  return ok;
}

// The map of a warp's n steps in the linear form again, step(s, a, x, d) giving
// them (in the reverse d too).  For what a reset alone does not explain: a rolled
// loop, so that it takes little of the instruction cache.
struct Settled {
  bool drop;     // a reset is among the steps of any lane
  bool strange;  // some map has to be checked against the state that it is applied to
  bool loose;    // some decay is neither 0 nor a normal number of at most 2
};
template <int S, int VEC, int kOffsets, typename F>
__device__ __forceinline__ Settled settle(Map<VEC, kOffsets> &m, int64_t n, bool live, F &&step) {
  float p[VEC], top[VEC], a[VEC], x[VEC], d[VEC];
  bool reset[VEC], any = false, strange = false, loose = false;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    p[i] = 1.f, top[i] = 0.f, reset[i] = false;
#pragma unroll
    for (int o = 0; o < kOffsets; ++o) m.b[o][i] = 0.f;
  }
#pragma unroll 1
  for (int s = 0; s < S && s < n; ++s) {
    step(s, a, x, d);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const bool z = a[i] == 0.f;
      reset[i] |= z;
      p[i] = __fmul_rn(p[i], a[i]);
      top[i] = fmaxf(top[i], fabsf(a[i]));
      m.b[0][i] = z || s == 0 ? x[i] : fmaf(a[i], m.b[0][i], x[i]);
    }
  }
  if constexpr (kOffsets == 2) {
#pragma unroll 1
    for (int s = n < S ? (int)n - 1 : S - 1; s >= 0; --s) {
      step(s, a, x, d);
#pragma unroll
      for (int i = 0; i < VEC; ++i) m.b[1][i] = a[i] == 0.f ? 0.f : __fmul_rn(a[i], __fadd_rn(d[i], m.b[1][i]));
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    bool whole = true;
#pragma unroll
    for (int o = 0; o < kOffsets; ++o) whole &= fabsf(m.b[o][i]) < infinity();
    if (reset[i])
      m.a[i] = 0.f;
    else if (m.a[i] == 0.f && top[i] <= 1.f && whole)
      m.a[i] = p[i] != 0.f ? p[i] : copysignf(kLeast, p[i]);
    else if (!(m.a[i] != 0.f && fabsf(m.a[i]) <= kMostGrowth && whole))
      m.a[i] = unusable();
    any |= reset[i];
    strange |= m.a[i] != m.a[i] || subnormal(m.a[i]);
    loose |= !whole || !(fabsf(m.a[i]) <= kPlain) || subnormal(m.a[i]);
  }
  return {__any_sync(0xffffffffu, any && live) != 0, __any_sync(0xffffffffu, strange && live) != 0,
          __any_sync(0xffffffffu, loose && live) != 0};
}

// The CTA's warps have stored their maps.  Returns whether those of any warp are
// loose, where that is asked for.
template <bool kAsk>
__device__ __forceinline__ bool meet(bool loose) {
  if constexpr (kAsk) return __syncthreads_or(loose);
  __syncthreads();
  return false;
}

// A map as its product of decays came out, looked at again if need be: restart()
// takes the offsets again with resets, step() is for settle.
template <int S, int VEC, int kOffsets, typename R, typename F>
__device__ __forceinline__ Settled look(const float (&a)[S][VEC], Map<VEC, kOffsets> &m, int64_t n, bool live,
                                        R &&restart, F &&step) {
  bool reset[VEC] = {};
  if (!__any_sync(0xffffffffu, live && !plain(m, reset))) return {false, false, false};
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
#pragma unroll
    for (int s = 0; s < S; ++s) reset[i] |= a[s][i] == 0.f;
    m.a[i] = reset[i] ? 0.f : m.a[i];
  }
  restart();
  if (!__any_sync(0xffffffffu, live && !plain(m, reset))) return {true, false, false};
  return settle<S>(m, n, live, step);
}

template <int VEC>
struct Steps {
  const float (&a)[VEC], (&b)[VEC];
};
// m after k: the same care for two maps, with m's offset as k's state
__device__ __forceinline__ void join(float &a, float &b, float ka, float kb) {
  if (ka == 0.f) {
    a = 0.f, b = kb;
    return;
  }
  float p = __fmul_rn(ka, a);
  const float sum = fmaf(ka, b, kb);
  if (a != 0.f) {
    if (p == 0.f) p = copysignf(kLeast, p);
    if ((subnormal(a) && fabsf(ka) > 1.f) || (subnormal(ka) && fabsf(a) > 1.f)) p = unusable();
    if (!(fabsf(p) <= kMostGrowth && fabsf(sum) < infinity())) p = unusable();
  }
  if (subnormal(ka) && fabsf(b) > kLooseState) p = unusable();
  a = p, b = sum;
}

// A CTA's map from those of its warps: decays and offsets by at(w), in the order
// of w.  It is sent as it comes out: checks before the send took 5 % of a launch
// in clusters, since every other CTA waits for them.
template <bool kSig, int VEC, typename At>
__device__ __forceinline__ void join_warps(Map<VEC, 1> &m, At &&at) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) m.a[i] = at(0).a[i], m.b[0][i] = at(0).b[i];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const Steps<VEC> k = at(w);
    affine<!kSig>(k.a, m.b[0], k.b, m.b[0]);
    vmul(m.a, k.a, m.a);
  }
}
// whether that map does not hold, if the decays of some warp are loose
template <int VEC>
__device__ __noinline__ bool misjoined(const float *a, const float *b, int pitch) {
  bool bad = false;
#pragma unroll 1
  for (int i = 0; i < VEC; ++i) {
    float ma = a[i], mb = b[i];
#pragma unroll 1
    for (int w = 1; w < kWarps; ++w) join(ma, mb, a[w * pitch + i], b[w * pitch + i]);
    bad |= ma != ma;
  }
  return bad;
}
// Whether it does not hold for the state h that it is applied to: its decay is
// subnormal, or 0 by the product alone, and h large or no number.
template <int VEC>
__device__ __noinline__ bool misused(const float *a, int pitch, float h0, float h1) {
  bool bad = false;
#pragma unroll 1
  for (int i = 0; i < VEC; ++i) {
    const float h = i == 0 ? h0 : h1;
    bool reset = false;
    float p = 1.f;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      reset |= a[w * pitch + i] == 0.f;
      p = __fmul_rn(p, a[w * pitch + i]);
    }
    // (a subnormal carries Inf and NaN on by itself)
    if (!reset && fabsf(p) < kNormal && !(fabsf(h) <= kLooseState) && (p == 0.f || fabsf(h) < infinity())) bad = true;
  }
  return bad;
}
template <int VEC>
__device__ __forceinline__ bool below_normal(const float (&a)[VEC]) {
  bool u = false;
#pragma unroll
  for (int i = 0; i < VEC; ++i) u |= fabsf(a[i]) < kNormal;
  return u;
}
template <int VEC>
__device__ __forceinline__ bool beyond(const float (&h)[VEC]) {
  bool u = false;
#pragma unroll
  for (int i = 0; i < VEC; ++i) u |= !(fabsf(h[i]) <= kLooseState);
  return u;
}
// whether a map does not hold for a state
template <int VEC>
__device__ __forceinline__ bool unsafe(const float (&a)[VEC], const float (&h)[VEC]) {
  bool u = false;
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    u |= a[i] != a[i] || (subnormal(a[i]) && fabsf(h[i]) > kLooseState && fabsf(h[i]) < infinity());
  return u;
}
template <int VEC>
__device__ __forceinline__ bool not_numbers(const float (&h)[VEC]) {
  bool n = false;
#pragma unroll
  for (int i = 0; i < VEC; ++i) n |= h[i] != h[i];
  return n;
}
// The exchange of one map per CTA in a cluster.  Two buffers: a CTA sends
// round r + 2 only after it has every map of round r + 1, which its peers send
// after they have read round r.  Waits are bounded.  One that runs out sets the
// error word; its warp sends no more, its CTA's other waits end too, and the
// kernel runs to its end, where every CTA meets the others (agree) and one that
// has given up leaves late, when what was on its way to it has landed.
struct Exchange {
  uint64_t bar[2];
  volatile int dead;

  __device__ __forceinline__ void init() {
    sm100::mbar_init(&bar[0], 1);
    sm100::mbar_init(&bar[1], 1);
    dead = 0;
    sm100::fence_mbar_init();
  }
  template <int VEC>
  __device__ __forceinline__ void send(int buf, const Map<VEC, 1> *slot, uint32_t to, const Map<VEC, 1> &m) {
    const uint32_t at = sm100::map_cluster(slot, to), b = sm100::map_cluster(&bar[buf], to);
    if constexpr (VEC == 2)
      asm volatile(
          "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
          "f"(m.a[0]), "f"(m.a[1]), "f"(m.b[0][0]), "f"(m.b[0][1]), "r"(b)
          : "memory");
    else
      asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                   "f"(m.a[0]), "f"(m.b[0][0]), "r"(b)
                   : "memory");
  }
  __device__ __forceinline__ void expect(int buf, uint32_t bytes) { sm100::mbar_arrive_expect_tx(&bar[buf], bytes); }
  __device__ __forceinline__ bool wait(int buf, uint32_t parity, uint32_t limit = 1u << 22) {
    for (uint32_t i = 0; i < limit; ++i) {
      if (sm100::mbar_try_wait(&bar[buf], parity)) return true;
      if (dead) return false;
    }
    dead = 1;
    atomicExch(&g_scan_error, 1u);
    return false;
  }
  // after the closing barrier
  __device__ __forceinline__ void leave() {
    if (dead) {
      for (int i = 0; i < 200; ++i) __nanosleep(1000);
    }
  }
};

// One channel's steps t .. t + kWalk - 1 as they lie in memory; those at or past
// n become steps that change nothing.
constexpr int kWalk = 16;
template <typename In, typename Gate, bool kSig>
__device__ __forceinline__ void walk(const In *x, int64_t xs, const Gate *g, int64_t gs, int64_t t, int64_t n,
                                     float (&a)[kWalk], float (&u)[kWalk], float (&ux)[kWalk]) {
  float xv[kWalk][1], gv[kWalk][1];
#pragma unroll
  for (int j = 0; j < kWalk; ++j) {
    xv[j][0] = gv[j][0] = 0.f;
    if (t + j < n) {
      widen(load<In, 1>(x + (t + j) * xs), xv[j]);
      widen(load<Gate, 1>(g + (t + j) * gs), gv[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kWalk; ++j) {
    float a1[1], u1[1], ux1[1];
    gates<kSig>(gv[j], a1, u1);
    vmul(u1, xv[j], ux1);
    a[j] = t + j < n ? a1[0] : 1.f;
    u[j] = t + j < n ? u1[0] : 0.f;
    ux[j] = t + j < n ? ux1[0] : 0.f;
  }
}
template <bool kSig>
__device__ __forceinline__ float one_step(float a, float h, float ux) {
  return !kSig && a == 0.f ? ux : fmaf(a, h, ux);
}

// Tells every CTA of the cluster which lanes want to go through their channels
// again.  All stores of the row come before those that replace them, and no CTA
// leaves while another may reach into it.  (Plain stores of one value: with an
// atomic in the kernel its loop takes a tenth longer.)
template <bool kCluster>
__device__ __forceinline__ void agree(int *flag, bool again, int cs) {
  if constexpr (kCluster) {
    if (again) {
      for (int q = 0; q < cs; ++q)
        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(sm100::map_cluster(flag, q)), "r"(1) : "memory");
    }
    __syncwarp();
    sm100::cluster_sync();
  } else {
    if (again) *flag = 1;
    __syncthreads();
  }
}

// A channel's whole row, step by step: x, g, out and states at its first step,
// states null where they are not wanted.  What lies in this CTA's tiles is
// stored.  Returns the last state.
template <typename In, typename Gate, bool kSig>
__device__ __noinline__ float redo_fwd(const In *x, int64_t xs, const Gate *g, int64_t gs, In *out, float *states,
                                       int64_t D, int64_t T, int64_t len, int rank, int cs, float h) {
  constexpr int kTile = kWarps * kFwdSteps;
  for (int64_t t = 0; t < T; t += kWalk) {
    const bool mine = t / kTile % cs == rank;
    if (mine && states && t % kScanBlock == 0) states[t / kScanBlock * D] = h;
    if (t >= len) continue;
    float a[kWalk], u[kWalk], ux[kWalk];
    walk<In, Gate, kSig>(x, xs, g, gs, t, len, a, u, ux);
#pragma unroll
    for (int j = 0; j < kWalk; ++j) {
      if (t + j >= len) break;
      h = one_step<kSig>(a[j], h, ux[j]);
      const float v[1] = {h};
      if (mine) store<In, 1>(out + (t + j) * D, v);
    }
  }
  return h;
}

// ------------------------------------------------------------------ forward
template <typename In, bool kSig, int VEC, bool kWide, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_fwd_kernel(ScanArgs p, int cs, int64_t strips) {
  using Gate = typename std::conditional<kSig, In, float>::type;
  using X = Strip<In, VEC, kWide>;
  using G = Strip<Gate, VEC, kWide>;
  constexpr int S = kFwdSteps, kTile = kWarps * S, kRow = 32 * VEC;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ __align__(16) Map<VEC, 1> s_map[2][kWarps][32];
  __shared__ int s_again[32];  // a lane's channels are gone through again
  __shared__ float s_first[32 * VEC];  // h0, which hT may overwrite
  __shared__ Exchange ex;
  // behind the ring: the maps of the cluster's CTAs, [2][cs][32]
  auto *s_cta = reinterpret_cast<Map<VEC, 1> *>(ring + kStages * kTile * (X::kPitch + G::kPitch));
  const auto cta = [&](int buf, int r) { return s_cta + (buf * cs + r) * 32; };
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // the same for all lanes, also to the compiler
  const int rank = kCluster ? (int)(blockIdx.x % cs) : 0;
  chain_wait();
  const int64_t id = kCluster ? blockIdx.x / cs : blockIdx.x;
  const int64_t b = id / strips, first = (id % strips) * kRow, c0 = first + lane * VEC;
  const bool live = c0 < p.D;
  const int64_t len = row_length(p.lengths, b, p.T), left = p.D - first;
  const int64_t tiles = (p.T + kTile - 1) / kTile, saved = (p.T + kScanBlock - 1) / kScanBlock;
  const In *x = static_cast<const In *>(p.x) + b * p.x_sb + first;
  const Gate *g = static_cast<const Gate *>(p.gate) + b * p.g_sb + first;
  In *out = static_cast<In *>(p.out) + b * p.T * p.D + c0;
  unsigned char *rx = ring + warp * kStages * S * X::kPitch;
  unsigned char *rg = ring + kWarps * kStages * S * X::kPitch + warp * kStages * S * G::kPitch;

  auto fetch = [&](int64_t tile, int slot) {
    const int64_t t0 = tile * kTile + warp * S, n = len - t0;
    if (n > 0) {
      X::template fetch<S>(rx + slot * S * X::kPitch, x + t0 * p.x_st, p.x_st, n, left, lane);
      G::template fetch<S>(rg + slot * S * G::kPitch, g + t0 * p.g_st, p.g_st, n, left, lane);
    }
    ring_commit();
  };

  float carry[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) carry[i] = live && p.h0 ? p.h0[b * p.D + c0 + i] : 0.f;
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) s_first[lane * VEC + i] = carry[i];
  }
  if (threadIdx.x < 32) s_again[threadIdx.x] = 0;
  bool alive = true;   // the exchange goes on
  bool again = false;  // the maps do not hold for this lane's channels

  const int64_t rounds = (tiles + cs - 1) / cs;
  // every CTA of the cluster runs before any writes into its shared memory
  if (kCluster) {
    if (threadIdx.x == 0) ex.init();
    cg::this_cluster().barrier_arrive();
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(rank + (int64_t)i * cs, i);
  if (kCluster) cg::this_cluster().barrier_wait();
  int slot = 0;
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t tile = it * cs + rank, t0 = tile * kTile + warp * S;
    const int64_t n = len - t0;  // steps that count, if below S
    const int buf = (int)(it & 1);
    ring_wait<kStages - 2>();
    __syncwarp();
    fetch(tile + (int64_t)(kStages - 1) * cs, slot == 0 ? kStages - 1 : slot - 1);
    float a[S][VEC], u[S][VEC];  // u: the whole input term
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float xv[VEC], gv[VEC];
      X::read(rx + slot * S * X::kPitch, x + t0 * p.x_st, p.x_st, s, lane, xv);
      G::read(rg + slot * S * G::kPitch, g + t0 * p.g_st, p.g_st, s, lane, gv);
      gates<kSig>(gv, a[s], u[s]);
      vmul(u[s], xv, u[s]);
    }
    const int now = slot;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    if (n < S) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          a[s][i] = s < n ? a[s][i] : 1.f;
          u[s][i] = s < n ? u[s][i] : 0.f;
        }
    }
    Settled map{};
    {
      Map<VEC, 1> m;
#pragma unroll
      for (int i = 0; i < VEC; ++i) m.a[i] = a[0][i], m.b[0][i] = u[0][i];
#pragma unroll
      for (int s = 1; s < S; ++s) {
        affine<false>(a[s], m.b[0], u[s], m.b[0]);
        kSig ? vmul(m.a, a[s], m.a) : vmul_ftz(m.a, a[s], m.a);
      }
      if constexpr (!kSig)
        map = look(
            a, m, n, live,
            [&] {
#pragma unroll
              for (int i = 0; i < VEC; ++i) m.b[0][i] = u[0][i];
#pragma unroll
              for (int s = 1; s < S; ++s) affine<true>(a[s], m.b[0], u[s], m.b[0]);
            },
            [&](int s, float (&av)[VEC], float (&xv)[VEC], float (&)[VEC]) {
              X::read(rx + now * S * X::kPitch, x + t0 * p.x_st, p.x_st, s, lane, xv);
              G::read(rg + now * S * G::kPitch, g + t0 * p.g_st, p.g_st, s, lane, av);
            });
      s_map[buf][warp][lane] = m;
    }
    const bool loose = meet<kCluster && !kSig>(map.loose);
    float h[VEC], start[VEC];
    if (kCluster) {
      // one map per CTA to every CTA of the cluster: warp w serves CTAs w and w + 8
      if (threadIdx.x == 0) ex.expect(buf, cs * 32 * sizeof(Map<VEC, 1>));
      bool small = false;  // a decay that may not hold for every state
      if (warp < cs) {
        Map<VEC, 1> m;
        join_warps<kSig>(m, [&](int w) {
          const Map<VEC, 1> &k = s_map[buf][w][lane];
          return Steps<VEC>{k.a, k.b[0]};
        });
        for (int to = warp; alive && to < cs; to += kWarps) ex.send(buf, cta(buf, rank) + lane, to, m);
        if (!kSig) small = below_normal(m.a);
        if (!kSig && loose) {
          const Map<VEC, 1> &k = s_map[buf][0][lane];
          again |= not_numbers(m.a) || misjoined<VEC>(k.a, k.b[0], 32 * sizeof(k) / sizeof(float));
        }
      }
      alive &= ex.wait(buf, (uint32_t)(it >> 1) & 1);
#pragma unroll
      for (int i = 0; i < VEC; ++i) h[i] = carry[i];
      for (int r = 0; r < cs; ++r) {
        const Map<VEC, 1> k = cta(buf, r)[lane];
        if (r == rank) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) h[i] = carry[i];
        }
        affine<!kSig>(k.a, carry, k.b[0], carry);
      }
      if (small && beyond(h)) {
        const Map<VEC, 1> &k = s_map[buf][0][lane];
        again |= misused<VEC>(k.a, 32 * sizeof(k) / sizeof(float), h[0], h[VEC - 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) h[i] = carry[i];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) start[i] = h[i];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const Map<VEC, 1> k = s_map[buf][w][lane];
      affine<!kSig>(k.a, h, k.b[0], h);
      if (w + 1 == warp) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) start[i] = h[i];
      }
    }
    if (map.strange) again |= unsafe(s_map[buf][warp][lane].a, start);
    if (kSig) again |= not_numbers(start);
    if (!kCluster) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) carry[i] = h[i];
    }
    if (p.states && t0 % kScanBlock == 0 && t0 < p.T && live)
      store<float, VEC>(p.states + (b * saved + t0 / kScanBlock) * p.D + c0, start);
    if (live) {
      In *o = out + t0 * p.D;
      if (n >= S && !map.drop) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          affine<false>(a[s], start, u[s], start);
          store<In, VEC>(o, start);
          o += p.D;
        }
      } else {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float v[VEC];
          affine<!kSig>(a[s], start, u[s], start);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[i] = s < n ? start[i] : 0.f;
          if (t0 + s < p.T) store<In, VEC>(o, v);
          o += p.D;
        }
      }
    }
  }
  ring_wait<0>();
  if (kSig) again |= not_numbers(carry);
  agree<kCluster>(s_again + lane, again && live, cs);
  if (kCluster) ex.leave();
  if (warp == 0 && s_again[lane]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      carry[i] = redo_fwd<In, Gate, kSig>(x + lane * VEC + i, p.x_st, g + lane * VEC + i, p.g_st, out + i,
                                          p.states ? p.states + b * saved * p.D + c0 + i : nullptr, p.D, p.T, len,
                                          rank, cs, s_first[lane * VEC + i]);
  }
  if (p.hT && rank == 0 && warp == 0 && live) store<float, VEC>(p.hT + b * p.D + c0, carry);
}

// ----------------------------------------------------------------- backward
// The same tiles in reverse time order.  The states before each step are run
// again from the state saved at the tile's start (the forward's states, kept
// in float32, so no rounded output enters the gradients); the gradients are
// the reversed recurrence, whose maps compose from the last step to the first.

// A channel's whole row in reverse, step by step, likewise; dout and the
// gradients are D apart.  A tile's states are run again from its saved one and
// held in `before`, `pitch` apart.  Returns the gradient of the first state.
template <typename In, typename Gate, bool kSig>
__device__ __noinline__ float redo_bwd(const In *x, int64_t xs, const Gate *g, int64_t gs, const In *dout, In *dx,
                                       Gate *dg, const float *states, int64_t D, int64_t T, int64_t len, int rank,
                                       int cs, float grad, float *before, int pitch) {
  const int64_t tiles = (T + kScanBlock - 1) / kScanBlock;
  for (int64_t tile = (len + kScanBlock - 1) / kScanBlock - 1; tile >= 0; --tile) {
    const int64_t t0 = tile * kScanBlock;
    const bool mine = (tiles - 1 - tile) % cs == rank;
    float a[kWalk], u[kWalk], ux[kWalk], d[kWalk];
    if (mine) {
      float h = states[tile * D];
      for (int s = 0; s < kScanBlock; s += kWalk) {
        walk<In, Gate, kSig>(x, xs, g, gs, t0 + s, len, a, u, ux);
#pragma unroll
        for (int j = 0; j < kWalk; ++j) {
          before[(s + j) * pitch] = h;
          h = one_step<kSig>(a[j], h, ux[j]);
        }
      }
    }
    for (int s = kScanBlock - kWalk; s >= 0; s -= kWalk) {
      if (t0 + s >= len) continue;
      walk<In, Gate, kSig>(x, xs, g, gs, t0 + s, len, a, u, ux);
#pragma unroll
      for (int j = 0; j < kWalk; ++j) {
        float v[1] = {0.f};
        if (t0 + s + j < len) widen(load<In, 1>(dout + (t0 + s + j) * D), v);
        d[j] = v[0];
      }
#pragma unroll
      for (int j = kWalk - 1; j >= 0; --j) {
        const int64_t t = t0 + s + j;
        if (t >= len) continue;
        const float dh = __fadd_rn(d[j], grad);
        if (mine) {
          const float h = before[(s + j) * pitch];
          const float vx[1] = {__fmul_rn(u[j], dh)};
          const float vg[1] = {__fmul_rn(kSig ? __fmul_rn(a[j], fmaf(u[j], h, -ux[j])) : h, dh)};
          store<In, 1>(dx + t * D, vx);
          store<Gate, 1>(dg + t * D, vg);
        }
        grad = !kSig && a[j] == 0.f ? 0.f : __fmul_rn(a[j], dh);
      }
    }
  }
  return grad;
}

template <typename In, bool kSig, int VEC, bool kWide, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_bwd_kernel(ScanBwdArgs p, int cs, int64_t strips) {
  using Gate = typename std::conditional<kSig, In, float>::type;
  using X = Strip<In, VEC, kWide>;
  using G = Strip<Gate, VEC, kWide>;
  constexpr int S = kBwdSteps, kTile = kWarps * S, kRow = 32 * VEC;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ __align__(16) Map<VEC, 2> s_map[2][kWarps][32];  // offsets: forward, reverse
  __shared__ int s_again[32];  // a lane's channels are gone through again
  __shared__ float s_last[32 * VEC];  // dhT, which dh0 may overwrite
  __shared__ Exchange ex;
  // behind the ring: the maps of the cluster's CTAs, [2][cs][32]
  auto *s_cta = reinterpret_cast<Map<VEC, 1> *>(ring + kStages * kTile * (2 * X::kPitch + G::kPitch));
  const auto cta = [&](int buf, int r) { return s_cta + (buf * cs + r) * 32; };
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int rank = kCluster ? (int)(blockIdx.x % cs) : 0;
  chain_wait();
  const int64_t id = kCluster ? blockIdx.x / cs : blockIdx.x;
  const int64_t b = id / strips, first = (id % strips) * kRow, c0 = first + lane * VEC;
  const bool live = c0 < p.D;
  const int64_t len = row_length(p.lengths, b, p.T), left = p.D - first;
  const int64_t tiles = (p.T + kTile - 1) / kTile;
  const In *x = static_cast<const In *>(p.x) + b * p.x_sb + first;
  const Gate *g = static_cast<const Gate *>(p.gate) + b * p.g_sb + first;
  const In *dout = static_cast<const In *>(p.dout) + b * p.T * p.D + first;
  In *dx = static_cast<In *>(p.dx) + b * p.T * p.D + c0;
  Gate *dg = static_cast<Gate *>(p.dgate) + b * p.T * p.D + c0;
  unsigned char *rx = ring + warp * 2 * kStages * S * X::kPitch, *rd = rx + kStages * S * X::kPitch;
  unsigned char *rg = ring + 2 * kWarps * kStages * S * X::kPitch + warp * kStages * S * G::kPitch;

  float ahead[VEC];  // the saved state of the next tile
#pragma unroll
  for (int i = 0; i < VEC; ++i) ahead[i] = 0.f;
  auto fetch = [&](int64_t tile, int slot) {  // a tile below 0 is not there
    const int64_t t0 = tile * kTile + warp * S, n = tile < 0 ? 0 : len - t0;
    if (n > 0) {
      X::template fetch<S>(rx + slot * S * X::kPitch, x + t0 * p.x_st, p.x_st, n, left, lane);
      X::template fetch<S>(rd + slot * S * X::kPitch, dout + t0 * p.D, p.D, n, left, lane);
      G::template fetch<S>(rg + slot * S * G::kPitch, g + t0 * p.g_st, p.g_st, n, left, lane);
    }
    ring_commit();
  };
  auto fetch_state = [&](int64_t tile) {
    if (tile >= 0 && live) widen(load<float, VEC>(p.states + (b * tiles + tile) * p.D + c0), ahead);
  };

  float carry[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) carry[i] = live && p.dhT ? p.dhT[b * p.D + c0 + i] : 0.f;
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) s_last[lane * VEC + i] = carry[i];
  }
  if (threadIdx.x < 32) s_again[threadIdx.x] = 0;
  bool alive = true;   // the exchange goes on
  bool again = false;

  const int64_t rounds = (tiles + cs - 1) / cs;
  if (kCluster) {
    if (threadIdx.x == 0) ex.init();
    cg::this_cluster().barrier_arrive();
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(tiles - 1 - rank - (int64_t)i * cs, i);
  fetch_state(tiles - 1 - rank);
  if (kCluster) cg::this_cluster().barrier_wait();
  int slot = 0;
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t tile = tiles - 1 - (it * cs + rank), t0 = tile * kTile + warp * S;
    const int64_t n = tile < 0 ? 0 : len - t0;
    const int buf = (int)(it & 1);
    ring_wait<kStages - 2>();
    __syncwarp();
    fetch(tile - (int64_t)(kStages - 1) * cs, slot == 0 ? kStages - 1 : slot - 1);
    float a[S][VEC], u[S][VEC], ux[S][VEC], d[S][VEC], h[VEC];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float xv[VEC], gv[VEC];
      X::read(rx + slot * S * X::kPitch, x + t0 * p.x_st, p.x_st, s, lane, xv);
      G::read(rg + slot * S * G::kPitch, g + t0 * p.g_st, p.g_st, s, lane, gv);
      X::read(rd + slot * S * X::kPitch, dout + t0 * p.D, p.D, s, lane, d[s]);
      gates<kSig>(gv, a[s], u[s]);
      vmul(u[s], xv, ux[s]);
    }
    const int now = slot;
    slot = slot == kStages - 1 ? 0 : slot + 1;
    if (n < S) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          a[s][i] = s < n ? a[s][i] : 1.f;
          u[s][i] = s < n ? u[s][i] : 0.f;
          ux[s][i] = s < n ? ux[s][i] : 0.f;
          d[s][i] = s < n ? d[s][i] : 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = ahead[i];
    if (it + 1 < rounds) fetch_state(tile - cs);
    Settled map{};
    {
      Map<VEC, 2> m;
#pragma unroll
      for (int i = 0; i < VEC; ++i) m.a[i] = a[0][i];
#pragma unroll
      for (int s = 1; s < S; ++s) kSig ? vmul(m.a, a[s], m.a) : vmul_ftz(m.a, a[s], m.a);
      const auto offsets = [&](auto with) {
        constexpr bool kDrop = decltype(with)::value;
#pragma unroll
        for (int i = 0; i < VEC; ++i) m.b[0][i] = ux[0][i];
#pragma unroll
        for (int s = 1; s < S; ++s) affine<kDrop>(a[s], m.b[0], ux[s], m.b[0]);
        decay<kDrop>(a[S - 1], d[S - 1], m.b[1]);
#pragma unroll
        for (int s = S - 2; s >= 0; --s) {
          vadd(d[s], m.b[1], m.b[1]);
          decay<kDrop>(a[s], m.b[1], m.b[1]);
        }
      };
      offsets(std::false_type{});
      if constexpr (!kSig)
        map = look(
            a, m, n, live, [&] { offsets(std::true_type{}); },
            [&](int s, float (&av)[VEC], float (&xv)[VEC], float (&dv)[VEC]) {
              X::read(rx + now * S * X::kPitch, x + t0 * p.x_st, p.x_st, s, lane, xv);
              G::read(rg + now * S * G::kPitch, g + t0 * p.g_st, p.g_st, s, lane, av);
              X::read(rd + now * S * X::kPitch, dout + t0 * p.D, p.D, s, lane, dv);
            });
      s_map[buf][warp][lane] = m;
    }
    const bool loose = meet<kCluster && !kSig>(map.loose);
    float r[VEC], c[VEC];
    if (kCluster) {
      if (threadIdx.x == 0) ex.expect(buf, cs * 32 * sizeof(Map<VEC, 1>));
      bool small = false;  // a decay that may not hold for every state
      if (warp < cs) {
        Map<VEC, 1> m;
        join_warps<kSig>(m, [&](int w) {
          const Map<VEC, 2> &k = s_map[buf][kWarps - 1 - w][lane];
          return Steps<VEC>{k.a, k.b[1]};
        });
        for (int to = warp; alive && to < cs; to += kWarps) ex.send(buf, cta(buf, rank) + lane, to, m);
        if (!kSig) small = below_normal(m.a);
        if (!kSig && loose) {
          const Map<VEC, 2> &k = s_map[buf][kWarps - 1][lane];
          again |= not_numbers(m.a) || misjoined<VEC>(k.a, k.b[1], -32 * (int)(sizeof(k) / sizeof(float)));
        }
      }
      alive &= ex.wait(buf, (uint32_t)(it >> 1) & 1);
#pragma unroll
      for (int i = 0; i < VEC; ++i) r[i] = carry[i];
      for (int k = 0; k < cs; ++k) {
        const Map<VEC, 1> q = cta(buf, k)[lane];
        if (k == rank) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) r[i] = carry[i];
        }
        affine<!kSig>(q.a, carry, q.b[0], carry);
      }
      if (small && beyond(r)) {
        const Map<VEC, 2> &k = s_map[buf][kWarps - 1][lane];
        again |= misused<VEC>(k.a, -32 * (int)(sizeof(k) / sizeof(float)), r[0], r[VEC - 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) r[i] = carry[i];
    }
    // the state at this warp's start, over the warps before it
    for (int w = 0; w < warp; ++w) {
      const Map<VEC, 2> k = s_map[buf][w][lane];
      affine<!kSig>(k.a, h, k.b[0], h);
    }
    // the gradient that arrives at its end, over the warps after it
#pragma unroll
    for (int i = 0; i < VEC; ++i) c[i] = r[i];
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      const Map<VEC, 2> k = s_map[buf][w][lane];
      affine<!kSig>(k.a, r, k.b[1], r);
      if (w - 1 == warp) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) c[i] = r[i];
      }
    }
    if (map.strange) again |= unsafe(s_map[buf][warp][lane].a, h) || unsafe(s_map[buf][warp][lane].a, c);
    if (kSig) again |= not_numbers(h) || not_numbers(c);
    if (!kCluster) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) carry[i] = r[i];
    }
    const auto finish = [&](auto with) {
      constexpr bool kDrop = decltype(with)::value;
      // the state before each step takes the place of its input term: sigmoid
      // keeps a (u h_{t-1} - u x), linear keeps h_{t-1}
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float before[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) before[i] = h[i];
        affine<kDrop>(a[s], before, ux[s], h);
        if constexpr (kSig) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) ux[s][i] = -ux[s][i];
          vfma(u[s], before, ux[s], ux[s]);
          vmul(a[s], ux[s], ux[s]);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) ux[s][i] = before[i];
        }
      }
      if (live && tile >= 0) {
        In *ox = dx + (t0 + S - 1) * p.D;
        Gate *og = dg + (t0 + S - 1) * p.D;
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
          float dh[VEC], vx[VEC], vg[VEC];
          vadd(d[s], c, dh);
          decay<kDrop>(a[s], dh, c);
          vmul(u[s], dh, vx);
          vmul(ux[s], dh, vg);
          if (n < S) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              vx[i] = s < n ? vx[i] : 0.f;
              vg[i] = s < n ? vg[i] : 0.f;
            }
          }
          if (n >= S || t0 + s < p.T) {
            store<In, VEC>(ox, vx);
            store<Gate, VEC>(og, vg);
          }
          ox -= p.D;
          og -= p.D;
        }
      }
    };
    if (!kSig && map.drop)
      finish(std::true_type{});
    else
      finish(std::false_type{});
  }
  ring_wait<0>();
  if (kSig) again |= not_numbers(carry);
  agree<kCluster>(s_again + lane, again && live, cs);
  if (kCluster) ex.leave();
  if (warp == 0 && s_again[lane]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      carry[i] = redo_bwd<In, Gate, kSig>(x + lane * VEC + i, p.x_st, g + lane * VEC + i, p.g_st,
                                          dout + lane * VEC + i, dx + i, dg + i, p.states + b * tiles * p.D + c0 + i,
                                          p.D, p.T, len, rank, cs, s_last[lane * VEC + i],
                                          reinterpret_cast<float *>(ring) + lane * VEC + i, kRow);
  }
  if (p.dh0 && rank == 0 && warp == 0 && live) store<float, VEC>(p.dh0 + b * p.D + c0, carry);
}

// --------------------------------------------------------------------- step
// One token: the state is read, updated in place and written, elementwise.
template <typename In, bool kSig, int VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs p, int64_t n) {
  using Gate = typename std::conditional<kSig, In, float>::type;
  const int64_t i0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  chain_wait();
  if (i0 >= n) return;
  const int64_t b = i0 / p.D, c = i0 - b * p.D;
  float xv[VEC], gv[VEC], hv[VEC], a[VEC], u[VEC];
  widen(load<In, VEC>(static_cast<const In *>(p.x) + b * p.x_sb + c), xv);
  widen(load<Gate, VEC>(static_cast<const Gate *>(p.gate) + b * p.g_sb + c), gv);
  widen(load<float, VEC>(p.h0 + i0), hv);
  gates<kSig>(gv, a, u);
  vmul(u, xv, u);
  affine<!kSig>(a, hv, u, hv);
  store<float, VEC>(p.hT + i0, hv);
  store<In, VEC>(static_cast<In *>(p.out) + i0, hv);
}

// The exchange of two CTAs of which one never sends: the other gives up.
__global__ void __launch_bounds__(32) exchange_selftest_kernel(uint32_t polls) {
  __shared__ __align__(16) Map<1, 1> s_cta[2][32];
  __shared__ int s_flag[32];
  __shared__ Exchange ex;
  const int lane = threadIdx.x, rank = (int)cg::this_cluster().block_rank();
  if (lane == 0) ex.init();
  s_flag[lane] = 0;
  cg::this_cluster().sync();
  if (rank == 0) {
    if (lane == 0) ex.expect(0, sizeof(s_cta));
    for (int to = 0; to < 2; ++to) ex.send(0, &s_cta[0][lane], to, Map<1, 1>{{1.f}, {{0.f}}});
    ex.wait(0, 0, polls);
  }
  agree<true>(s_flag + lane, false, 2);
  ex.leave();
}

// ------------------------------------------------------------------ launches
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;
  return n;
}

// the strides and addresses of x and gate allow pieces of nx and ng elements
bool pieces(const ScanArgs &a, int nx, int ng) {
  const int64_t ex = a.bf16 ? 2 : 4, eg = a.sigmoid ? ex : 4;
  const auto ok = [](const void *q, int64_t n) { return reinterpret_cast<uintptr_t>(q) % (uintptr_t)n == 0; };
  return a.D % nx == 0 && a.D % ng == 0 && a.x_sb % nx == 0 && a.x_st % nx == 0 && a.g_sb % ng == 0 &&
         a.g_st % ng == 0 && ok(a.x, nx * ex) && ok(a.gate, ng * eg);
}
// Two channels a lane (bfloat16; a row of a strip is 128 bytes either way) need
// even offsets everywhere; rows of whole 16-byte pieces are wide.
bool pairs(const ScanArgs &a) { return pieces(a, 2, 2); }
bool wide(const ScanArgs &a) { return pieces(a, a.bf16 ? 8 : 4, a.bf16 && a.sigmoid ? 8 : 4); }

// CTAs of a cluster along the time axis: as many as keep all CTAs resident at
// once (two an SM), and as there are tiles.  Past that a second wave costs more
// than the shorter CTAs give: 256 rows of 8192 steps take 137 us alone and 155
// to 205 in clusters of 2 to 8.
int cluster_size(int64_t rows, int64_t tiles) {
  const int64_t fit = 2 * (int64_t)sm_count();
  int cs = 1;
  while (cs < 8 && rows * cs * 2 <= fit && cs < tiles) cs *= 2;
  // 16 only for so few rows that its CTAs have SMs of their own: 1 x 30000 x 64
  // takes 34 us for 60, but 1 x 65536 x 512 (8 rows) 131 for 122
  if (cs == 8 && rows <= 7 && tiles > 8) cs = kMaxCluster;
  return cs;
}

// most: what the largest cluster takes.  The limit belongs to the kernel, not to
// the call, so every thread of the program sets the same one.
template <typename K, typename A>
cudaError_t launch(K kern, const A &p, int64_t rows, int64_t strips, int cs, int smem, int most, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  if (cs > 8 && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return e;
  return chain_launch(kern, dim3((unsigned)(rows * cs)), dim3(kWarps * 32), smem, cs, true, s, p, cs, strips);
}

template <typename In, bool kSig, int VEC, bool kWide>
cudaError_t launch_fwd(const ScanArgs &a, cudaStream_t s) {
  const int64_t strips = (a.D + 32 * VEC - 1) / (32 * VEC), rows = a.B * strips;
  const int cs = cluster_size(rows, (a.T + kWarps * kFwdSteps - 1) / (kWarps * kFwdSteps));
  using Gate = typename std::conditional<kSig, In, float>::type;
  constexpr int tile = kWarps * kFwdSteps * (Strip<In, VEC, kWide>::kPitch + Strip<Gate, VEC, kWide>::kPitch);
  constexpr int maps = 2 * 32 * (int)sizeof(Map<VEC, 1>);  // for each CTA of a cluster
  const int smem = kStages * tile + (cs > 1 ? cs * maps : 0);
  return cs > 1 ? launch(scan_fwd_kernel<In, kSig, VEC, kWide, true>, a, rows, strips, cs, smem,
                         kStages * tile + kMaxCluster * maps, s)
                : launch(scan_fwd_kernel<In, kSig, VEC, kWide, false>, a, rows, strips, cs, smem, kStages * tile, s);
}
template <typename In, bool kSig, int VEC, bool kWide>
cudaError_t launch_bwd(const ScanBwdArgs &a, cudaStream_t s) {
  const int64_t strips = (a.D + 32 * VEC - 1) / (32 * VEC), rows = a.B * strips;
  const int cs = cluster_size(rows, (a.T + kWarps * kBwdSteps - 1) / (kWarps * kBwdSteps));
  using Gate = typename std::conditional<kSig, In, float>::type;
  constexpr int tile = kWarps * kBwdSteps * (2 * Strip<In, VEC, kWide>::kPitch + Strip<Gate, VEC, kWide>::kPitch);
  constexpr int maps = 2 * 32 * (int)sizeof(Map<VEC, 1>);  // for each CTA of a cluster
  const int smem = kStages * tile + (cs > 1 ? cs * maps : 0);
  return cs > 1 ? launch(scan_bwd_kernel<In, kSig, VEC, kWide, true>, a, rows, strips, cs, smem,
                         kStages * tile + kMaxCluster * maps, s)
                : launch(scan_bwd_kernel<In, kSig, VEC, kWide, false>, a, rows, strips, cs, smem, kStages * tile, s);
}
template <typename In, bool kSig, int VEC>
cudaError_t launch_one(const ScanArgs &a, cudaStream_t s) {
  const int64_t n = a.B * a.D, blocks = (n / VEC + 255) / 256;
  return chain_launch(scan_step_kernel<In, kSig, VEC>, dim3((unsigned)blocks), dim3(256), 0, 1, true, s, a, n);
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s) {
  const bool v2 = pairs(a), w = wide(a);
  if (a.bf16) {
    if (a.sigmoid)
      return w ? launch_fwd<__nv_bfloat16, true, 2, true>(a, s)
           : v2 ? launch_fwd<__nv_bfloat16, true, 2, false>(a, s)
                : launch_fwd<__nv_bfloat16, true, 1, false>(a, s);
    return w ? launch_fwd<__nv_bfloat16, false, 2, true>(a, s)
         : v2 ? launch_fwd<__nv_bfloat16, false, 2, false>(a, s)
              : launch_fwd<__nv_bfloat16, false, 1, false>(a, s);
  }
  if (a.sigmoid)
    return w ? launch_fwd<float, true, 1, true>(a, s) : launch_fwd<float, true, 1, false>(a, s);
  return w ? launch_fwd<float, false, 1, true>(a, s) : launch_fwd<float, false, 1, false>(a, s);
}

cudaError_t launch_scan_bwd(const ScanBwdArgs &a, cudaStream_t s) {
  const bool v2 = pairs(a), w = wide(a);
  if (a.bf16) {
    if (a.sigmoid)
      return w ? launch_bwd<__nv_bfloat16, true, 2, true>(a, s)
           : v2 ? launch_bwd<__nv_bfloat16, true, 2, false>(a, s)
                : launch_bwd<__nv_bfloat16, true, 1, false>(a, s);
    return w ? launch_bwd<__nv_bfloat16, false, 2, true>(a, s)
         : v2 ? launch_bwd<__nv_bfloat16, false, 2, false>(a, s)
              : launch_bwd<__nv_bfloat16, false, 1, false>(a, s);
  }
  if (a.sigmoid)
    return w ? launch_bwd<float, true, 1, true>(a, s) : launch_bwd<float, true, 1, false>(a, s);
  return w ? launch_bwd<float, false, 1, true>(a, s) : launch_bwd<float, false, 1, false>(a, s);
}

cudaError_t launch_scan_step(const ScanArgs &a, cudaStream_t s) {
  const bool v2 = pairs(a);
  if (a.bf16) {
    if (a.sigmoid) return v2 ? launch_one<__nv_bfloat16, true, 2>(a, s) : launch_one<__nv_bfloat16, true, 1>(a, s);
    return v2 ? launch_one<__nv_bfloat16, false, 2>(a, s) : launch_one<__nv_bfloat16, false, 1>(a, s);
  }
  if (a.sigmoid) return v2 ? launch_one<float, true, 2>(a, s) : launch_one<float, true, 1>(a, s);
  return v2 ? launch_one<float, false, 2>(a, s) : launch_one<float, false, 1>(a, s);
}

cudaError_t launch_exchange_selftest(unsigned int polls, cudaStream_t s) {
  return chain_launch(exchange_selftest_kernel, dim3(2), dim3(32), 0, 2, false, s, polls);
}

cudaError_t read_and_clear_scan_error(unsigned int *word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_scan_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_scan_error, &zero, sizeof(unsigned int));
}

cudaError_t launch_scan_passthrough(const float *h0, float *hT, int64_t n, cudaStream_t s) {
  if (!hT || hT == h0) return cudaSuccess;
  return h0 ? cudaMemcpyAsync(hT, h0, (size_t)n * 4, cudaMemcpyDeviceToDevice, s)
            : cudaMemsetAsync(hT, 0, (size_t)n * 4, s);
}

}  // namespace delta
