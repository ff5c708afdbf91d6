// scan.cu -- the gated linear recurrence, one state per channel:
//
//   h_t = a_t h_{t-1} + u_t x_t,   out_t = h_t
//
// linear form: a_t = gate_t (float32), u_t = 1; sigmoid form: a_t = sigma(f_t)
// and u_t = 1 - a_t = sigma(-f_t), taken from the same exponential so that
// neither loses digits when the other is close to 1.  a_t = 0 drops the past
// whatever it holds (an infinite or NaN state does not cross a reset).
//
// Reverse: with c_T = dhT,  dh_t = dout_t + c_t  and  c_{t-1} = a_t dh_t;
// dx_t = u_t dh_t, dgate_t = dh_t h_{t-1} (linear) or
// dh_t a_t (u_t h_{t-1} - u_t x_t) (sigmoid), dh0 = c_0.
//
// Both directions are bound by HBM: every element is read once and written
// once, about 20 operations each.  A recurrence step is the affine map
// h -> a h + b, and maps compose: (A, B) after (A', B') is (A A', A B' + B).
// So a tile of kTile = 64 steps of 32 VEC channels is cut into kWarps
// sub-chunks of kSteps steps, one per warp, lane = VEC channels:
//   1. each warp loads its steps into registers and composes its own map;
//   2. the maps meet in shared memory (one barrier), and every warp folds
//      them in time order onto the state carried from the last tile, which
//      gives the state at its own start and, redundantly in every warp, the
//      state carried to the next tile;
//   3. each warp runs the recurrence again from its start and writes out.
// The next tile's loads are issued before step 1's arithmetic.  Where the
// (batch row, channel strip) pairs alone do not fill the GPU, a cluster of
// `cs` CTAs takes cs neighbouring tiles at a time and exchanges one map per
// CTA through distributed shared memory; the fold order is the time order, so
// results do not depend on scheduling.  All maps and states are float32.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "kernels.h"

namespace delta {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kSteps = 8;                // steps per warp and tile
constexpr int kTile = kWarps * kSteps;   // steps between two saved states
static_assert(kTile == kScanBlock, "a saved state per tile");
constexpr int kMaxCluster = 8;           // the portable cluster size

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

// a and u of one element.  Sigmoid: with t = e^-|f| and r = 1 / (1 + t), the
// larger of the pair is r and the smaller t r.
template <bool kSig>
__device__ __forceinline__ void gates(float g, float &a, float &u) {
  if (kSig) {
    const float t = __expf(-fabsf(g));
    const float r = __fdividef(1.f, 1.f + t);
    const float q = t * r;
    a = g < 0.f ? q : r;  // NaN: both are NaN
    u = g < 0.f ? r : q;
  } else {
    a = g;
    u = 1.f;
  }
}

// a h + b; a = 0 drops h
__device__ __forceinline__ float affine(float a, float h, float b) {
  return a == 0.f ? b : fmaf(a, h, b);
}

__device__ __forceinline__ int64_t row_length(const int *lengths, int64_t b, int64_t T) {
  if (!lengths) return T;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// ------------------------------------------------------------------ forward
template <typename In, bool kSig, int VEC, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_fwd_kernel(ScanArgs p, int cs, int64_t strips) {
  using Gate = typename std::conditional<kSig, In, float>::type;
  __shared__ float s_map[2][kWarps][2][VEC][32];
  __shared__ float s_cta[kCluster ? 2 : 1][kCluster ? kMaxCluster : 1][2][VEC][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kCluster ? (int)(blockIdx.x % cs) : 0;
  const int64_t id = kCluster ? blockIdx.x / cs : blockIdx.x;
  const int64_t b = id / strips, c0 = (id % strips) * (32 * VEC) + lane * VEC;
  const bool live = c0 < p.D;
  const int64_t len = row_length(p.lengths, b, p.T);
  const int64_t tiles = (p.T + kTile - 1) / kTile;
  const In *x = static_cast<const In *>(p.x) + b * p.x_sb + c0;
  const Gate *g = static_cast<const Gate *>(p.gate) + b * p.g_sb + c0;
  In *out = static_cast<In *>(p.out) + b * p.T * p.D + c0;

  typename Raw<In, VEC>::type xr[kSteps];
  typename Raw<Gate, VEC>::type gr[kSteps];
  auto fetch = [&](int64_t tile) {
    const int64_t t0 = tile * kTile + warp * kSteps;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (live && t0 + s < len) {
        xr[s] = load<In, VEC>(x + (t0 + s) * p.x_st);
        gr[s] = load<Gate, VEC>(g + (t0 + s) * p.g_st);
      }
  };

  float carry[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) carry[i] = live && p.h0 ? p.h0[b * p.D + c0 + i] : 0.f;

  const int64_t rounds = (tiles + cs - 1) / cs;
  // every CTA of the cluster runs before any writes into its shared memory
  if (kCluster) cg::this_cluster().barrier_arrive();
  fetch(rank);
  if (kCluster) cg::this_cluster().barrier_wait();
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t tile = it * cs + rank, t0 = tile * kTile + warp * kSteps;
    const int buf = (int)(it & 1);
    float a[kSteps][VEC], u[kSteps][VEC];  // u: the whole input term
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (live && t0 + s < len) {
        float xv[VEC], gv[VEC];
        widen(xr[s], xv);
        widen(gr[s], gv);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          gates<kSig>(gv[i], a[s][i], u[s][i]);
          u[s][i] *= xv[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[s][i] = 1.f, u[s][i] = 0.f;
      }
    }
    if (it + 1 < rounds) fetch(tile + cs);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float A = 1.f, B = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        B = affine(a[s][i], B, u[s][i]);
        A *= a[s][i];
      }
      s_map[buf][warp][0][i][lane] = A;
      s_map[buf][warp][1][i][lane] = B;
    }
    __syncthreads();
    if (kCluster) {
      // one map per CTA to every CTA of the cluster: warp w serves CTA w.  The
      // buffer written now was last read before the previous round's barrier.
      cg::cluster_group cluster = cg::this_cluster();
      if (warp < cs) {
        float *to = cluster.map_shared_rank(&s_cta[buf][rank][0][0][0], warp);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float A = 1.f, B = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float aw = s_map[buf][w][0][i][lane];
            B = affine(aw, B, s_map[buf][w][1][i][lane]);
            A *= aw;
          }
          to[i * 32 + lane] = A;
          to[(VEC + i) * 32 + lane] = B;
        }
      }
      cluster.sync();
    }
    float start[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float h = carry[i];
      if (kCluster) {
        float mine = h;
        for (int r = 0; r < cs; ++r) {
          if (r == rank) mine = h;
          h = affine(s_cta[buf][r][0][i][lane], h, s_cta[buf][r][1][i][lane]);
        }
        carry[i] = h;
        h = mine;
      }
      if (p.states && warp == 0 && live && tile < tiles)
        p.states[(b * tiles + tile) * p.D + c0 + i] = h;
      start[i] = h;
#pragma unroll 4
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) start[i] = h;
        h = affine(s_map[buf][w][0][i][lane], h, s_map[buf][w][1][i][lane]);
      }
      if (!kCluster) carry[i] = h;
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        start[i] = affine(a[s][i], start[i], u[s][i]);
        o[i] = t0 + s < len ? start[i] : 0.f;
      }
      if (live && t0 + s < p.T) store<In, VEC>(out + (t0 + s) * p.D, o);
    }
  }
  if (p.hT && rank == 0 && warp == 0 && live) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p.hT[b * p.D + c0 + i] = carry[i];
  }
}

// ----------------------------------------------------------------- backward
// The same tiles in reverse time order.  The states before each step are run
// again from the state saved at the tile's start (the forward's states, kept
// in float32, so no rounded output enters the gradients); the gradients are
// the reversed recurrence, whose maps compose from the last step to the first.
template <typename In, bool kSig, int VEC, bool kCluster>
__global__ void __launch_bounds__(kWarps * 32, 2) scan_bwd_kernel(ScanBwdArgs p, int cs, int64_t strips) {
  using Gate = typename std::conditional<kSig, In, float>::type;
  __shared__ float s_map[2][kWarps][3][VEC][32];  // decay, forward and reverse offsets
  __shared__ float s_cta[kCluster ? 2 : 1][kCluster ? kMaxCluster : 1][2][VEC][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kCluster ? (int)(blockIdx.x % cs) : 0;
  const int64_t id = kCluster ? blockIdx.x / cs : blockIdx.x;
  const int64_t b = id / strips, c0 = (id % strips) * (32 * VEC) + lane * VEC;
  const bool live = c0 < p.D;
  const int64_t len = row_length(p.lengths, b, p.T);
  const int64_t tiles = (p.T + kTile - 1) / kTile;
  const In *x = static_cast<const In *>(p.x) + b * p.x_sb + c0;
  const Gate *g = static_cast<const Gate *>(p.gate) + b * p.g_sb + c0;
  const In *dout = static_cast<const In *>(p.dout) + b * p.T * p.D + c0;
  In *dx = static_cast<In *>(p.dx) + b * p.T * p.D + c0;
  Gate *dg = static_cast<Gate *>(p.dgate) + b * p.T * p.D + c0;

  typename Raw<In, VEC>::type xr[kSteps], dr[kSteps];
  typename Raw<Gate, VEC>::type gr[kSteps];
  float hs[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) hs[i] = 0.f;
  auto fetch = [&](int64_t tile) {  // tile may be below 0: nothing is read
    const int64_t t0 = tile * kTile + warp * kSteps;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (live && tile >= 0 && t0 + s < len) {
        xr[s] = load<In, VEC>(x + (t0 + s) * p.x_st);
        gr[s] = load<Gate, VEC>(g + (t0 + s) * p.g_st);
        dr[s] = load<In, VEC>(dout + (t0 + s) * p.D);
      }
    if (live && tile >= 0) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) hs[i] = p.states[(b * tiles + tile) * p.D + c0 + i];
    }
  };

  float carry[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) carry[i] = live && p.dhT ? p.dhT[b * p.D + c0 + i] : 0.f;

  const int64_t rounds = (tiles + cs - 1) / cs;
  // every CTA of the cluster runs before any writes into its shared memory
  if (kCluster) cg::this_cluster().barrier_arrive();
  fetch(tiles - 1 - rank);
  if (kCluster) cg::this_cluster().barrier_wait();
  for (int64_t it = 0; it < rounds; ++it) {
    const int64_t tile = tiles - 1 - (it * cs + rank), t0 = tile * kTile + warp * kSteps;
    const int buf = (int)(it & 1);
    float a[kSteps][VEC], u[kSteps][VEC], ux[kSteps][VEC], d[kSteps][VEC], h[VEC];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (live && tile >= 0 && t0 + s < len) {
        float xv[VEC], gv[VEC];
        widen(xr[s], xv);
        widen(gr[s], gv);
        widen(dr[s], d[s]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          gates<kSig>(gv[i], a[s][i], u[s][i]);
          ux[s][i] = u[s][i] * xv[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[s][i] = 1.f, u[s][i] = 0.f, ux[s][i] = 0.f, d[s][i] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = hs[i];
    if (it + 1 < rounds) fetch(tile - cs);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float A = 1.f, F = 0.f, R = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        F = affine(a[s][i], F, ux[s][i]);
        A *= a[s][i];
        const int q = kSteps - 1 - s;
        R = a[q][i] == 0.f ? 0.f : a[q][i] * (d[q][i] + R);
      }
      s_map[buf][warp][0][i][lane] = A;
      s_map[buf][warp][1][i][lane] = F;
      s_map[buf][warp][2][i][lane] = R;
    }
    __syncthreads();
    if (kCluster) {
      cg::cluster_group cluster = cg::this_cluster();
      if (warp < cs) {
        float *to = cluster.map_shared_rank(&s_cta[buf][rank][0][0][0], warp);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float A = 1.f, R = 0.f;
#pragma unroll
          for (int w = kWarps - 1; w >= 0; --w) {
            const float aw = s_map[buf][w][0][i][lane];
            R = affine(aw, R, s_map[buf][w][2][i][lane]);
            A *= aw;
          }
          to[i * 32 + lane] = A;
          to[(VEC + i) * 32 + lane] = R;
        }
      }
      cluster.sync();
    }
    float c[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float r = carry[i];
      if (kCluster) {
        float mine = r;
        for (int k = 0; k < cs; ++k) {
          if (k == rank) mine = r;
          r = affine(s_cta[buf][k][0][i][lane], r, s_cta[buf][k][1][i][lane]);
        }
        carry[i] = r;
        r = mine;
      }
      c[i] = r;
      float f = h[i];
#pragma unroll 4
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) h[i] = f;
        f = affine(s_map[buf][w][0][i][lane], f, s_map[buf][w][1][i][lane]);
      }
#pragma unroll 4
      for (int w = kWarps - 1; w >= 0; --w) {
        if (w == warp) c[i] = r;
        r = affine(s_map[buf][w][0][i][lane], r, s_map[buf][w][2][i][lane]);
      }
      if (!kCluster) carry[i] = r;
    }
    // the state before each step takes the place of its input term: sigmoid
    // keeps u h_{t-1} - u x, linear keeps h_{t-1}
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float before = h[i];
        h[i] = affine(a[s][i], before, ux[s][i]);
        ux[s][i] = kSig ? u[s][i] * before - ux[s][i] : before;
      }
    }
#pragma unroll
    for (int s = kSteps - 1; s >= 0; --s) {
      float vx[VEC], vg[VEC];
      const bool in = t0 + s < len;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float dh = d[s][i] + c[i];
        c[i] = a[s][i] == 0.f ? 0.f : a[s][i] * dh;
        vx[i] = in ? u[s][i] * dh : 0.f;
        vg[i] = in ? (kSig ? dh * a[s][i] : dh) * ux[s][i] : 0.f;
      }
      if (live && tile >= 0 && t0 + s < p.T) {
        store<In, VEC>(dx + (t0 + s) * p.D, vx);
        store<Gate, VEC>(dg + (t0 + s) * p.D, vg);
      }
    }
  }
  if (p.dh0 && rank == 0 && warp == 0 && live) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p.dh0[b * p.D + c0 + i] = carry[i];
  }
}

// --------------------------------------------------------------------- step
// One token: the state is read, updated in place and written, elementwise.
template <typename In, bool kSig, int VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs p, int64_t n) {
  using Gate = typename std::conditional<kSig, In, float>::type;
  const int64_t i0 = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (i0 >= n) return;
  const int64_t b = i0 / p.D, c = i0 - b * p.D;
  float xv[VEC], gv[VEC], hv[VEC];
  widen(load<In, VEC>(static_cast<const In *>(p.x) + b * p.x_sb + c), xv);
  widen(load<Gate, VEC>(static_cast<const Gate *>(p.gate) + b * p.g_sb + c), gv);
  widen(load<float, VEC>(p.h0 + i0), hv);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    float a, u;
    gates<kSig>(gv[i], a, u);
    hv[i] = affine(a, hv[i], u * xv[i]);
  }
  store<float, VEC>(p.hT + i0, hv);
  store<In, VEC>(static_cast<In *>(p.out) + i0, hv);
}

// ------------------------------------------------------------------ launches
int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;
  return n;
}

// two channels per lane need even offsets everywhere
bool pairs(const ScanArgs &a) {
  const int gsz = a.sigmoid && a.bf16 ? 2 : 4, esz = a.bf16 ? 2 : 4;
  const auto ok = [](const void *q, int sz) { return (reinterpret_cast<uintptr_t>(q) % (2 * sz)) == 0; };
  return a.D % 2 == 0 && a.x_sb % 2 == 0 && a.x_st % 2 == 0 && a.g_sb % 2 == 0 && a.g_st % 2 == 0 &&
         ok(a.x, esz) && ok(a.gate, gsz);
}

// CTAs of a cluster along the time axis: enough to give every SM two CTAs,
// as far as there are tiles
int cluster_size(int64_t rows, int64_t tiles) {
  const int64_t want = 2 * (int64_t)sm_count();
  int cs = 1;
  while (cs < kMaxCluster && rows * cs < want && cs < tiles) cs *= 2;
  return cs;
}

template <typename K, typename A>
cudaError_t launch(K kern, const A &p, int64_t rows, int64_t strips, int cs, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cs));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cs;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cs > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, cs, strips);
}

template <typename In, bool kSig, int VEC>
cudaError_t launch_fwd(const ScanArgs &a, cudaStream_t s) {
  const int64_t strips = (a.D + 32 * VEC - 1) / (32 * VEC), rows = a.B * strips;
  const int cs = cluster_size(rows, (a.T + kTile - 1) / kTile);
  return cs > 1 ? launch(scan_fwd_kernel<In, kSig, VEC, true>, a, rows, strips, cs, s)
                : launch(scan_fwd_kernel<In, kSig, VEC, false>, a, rows, strips, cs, s);
}
template <typename In, bool kSig, int VEC>
cudaError_t launch_bwd(const ScanBwdArgs &a, cudaStream_t s) {
  const int64_t strips = (a.D + 32 * VEC - 1) / (32 * VEC), rows = a.B * strips;
  const int cs = cluster_size(rows, (a.T + kTile - 1) / kTile);
  return cs > 1 ? launch(scan_bwd_kernel<In, kSig, VEC, true>, a, rows, strips, cs, s)
                : launch(scan_bwd_kernel<In, kSig, VEC, false>, a, rows, strips, cs, s);
}
template <typename In, bool kSig, int VEC>
cudaError_t launch_one(const ScanArgs &a, cudaStream_t s) {
  const int64_t n = a.B * a.D, blocks = (n / VEC + 255) / 256;
  scan_step_kernel<In, kSig, VEC><<<(unsigned)blocks, 256, 0, s>>>(a, n);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s) {
  const bool v2 = pairs(a);
  if (a.bf16) {
    if (a.sigmoid) return v2 ? launch_fwd<__nv_bfloat16, true, 2>(a, s) : launch_fwd<__nv_bfloat16, true, 1>(a, s);
    return v2 ? launch_fwd<__nv_bfloat16, false, 2>(a, s) : launch_fwd<__nv_bfloat16, false, 1>(a, s);
  }
  if (a.sigmoid) return v2 ? launch_fwd<float, true, 2>(a, s) : launch_fwd<float, true, 1>(a, s);
  return v2 ? launch_fwd<float, false, 2>(a, s) : launch_fwd<float, false, 1>(a, s);
}

cudaError_t launch_scan_bwd(const ScanBwdArgs &a, cudaStream_t s) {
  const bool v2 = pairs(a);
  if (a.bf16) {
    if (a.sigmoid) return v2 ? launch_bwd<__nv_bfloat16, true, 2>(a, s) : launch_bwd<__nv_bfloat16, true, 1>(a, s);
    return v2 ? launch_bwd<__nv_bfloat16, false, 2>(a, s) : launch_bwd<__nv_bfloat16, false, 1>(a, s);
  }
  if (a.sigmoid) return v2 ? launch_bwd<float, true, 2>(a, s) : launch_bwd<float, true, 1>(a, s);
  return v2 ? launch_bwd<float, false, 2>(a, s) : launch_bwd<float, false, 1>(a, s);
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

cudaError_t launch_scan_passthrough(const float *h0, float *hT, int64_t n, cudaStream_t s) {
  if (!hT || hT == h0) return cudaSuccess;
  return h0 ? cudaMemcpyAsync(hT, h0, (size_t)n * 4, cudaMemcpyDeviceToDevice, s)
            : cudaMemsetAsync(hT, 0, (size_t)n * 4, s);
}

}  // namespace delta
