// linear.cu -- the linear layer outside the large tensor-core products: the
// form for few rows of x (decoding), float32 on the CUDA cores, and the
// elementwise part of the gradients.
#include <cooperative_groups.h>

#include "chain.cuh"
#include "linear.cuh"

namespace delta {
namespace {

namespace cg = cooperative_groups;
using namespace linear;

int sm_count() {
  int dev = 0, n = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}
bool aligned_to(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }

// ------------------------------------------------------------ few rows of x
// Bound by reading w once.  A CTA has 16 rows of w, its warps (and the CTAs of
// a cluster, where N alone does not fill the GPU) deal out k in blocks of
// kBlocks 64-byte pieces per row.  The products run on warp-level matrix
// instructions with w as the 16-row operand and up to 8 NT rows of x as the
// other: at M <= 16 the 5th-generation units would wait for the same bytes,
// and here a piece goes from memory to the operand's registers with nothing
// between.  The instruction's order of k within a block is free as long as
// both operands share it, so a lane takes 16 neighbouring bytes of its rows.
// The next turn's pieces are asked for before this one's products (M1 N8192
// K4096 bfloat16: 12.2 us, 5.5 TB/s; without, at four pieces a turn, 13.3).
// Partial sums meet in shared memory and in rank 0 in a fixed order.  More
// rows of x than 8 NT take the grid's second axis, each its own pass over w.
constexpr int kSmallWarps = 8;
constexpr int kBlocks = 2;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of a row from byte k on; zeros past the row's `bytes`.  kVec: rows
// are whole 16-byte pieces.  Else they are put together from the two aligned
// pieces that hold them (each read only if it holds a byte of the row), by
// words and then by bytes.
template <bool kVec, bool kStream>
__device__ __forceinline__ uint4 piece(const uint8_t *row, int64_t k, int64_t bytes) {
  if (k >= bytes) return make_uint4(0, 0, 0, 0);
  if constexpr (kVec) {
    const uint4 *p = reinterpret_cast<const uint4 *>(row + k);
    return kStream ? __ldcs(p) : *p;
  } else {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + k);
    const uint32_t sh = (uint32_t)(at & 15);
    const uint4 *p = reinterpret_cast<const uint4 *>(at - sh);
    const uint4 lo = *p;
    uint4 hi = make_uint4(0, 0, 0, 0);
    if (sh && bytes - k > 16 - (int)sh) hi = p[1];
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (sh & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (sh & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = 8 * (sh & 3);
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(w[i], w[i + 1], bits);
    if (bytes - k < 16) {
      const int have = (int)(bytes - k);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = have >= 4 * i + 4 ? v[i] : have <= 4 * i ? 0u : v[i] & (0xFFFFFFFFu >> (8 * (4 * i + 4 - have)));
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// The gated form (kGlu) takes 8 rows of either half of w for the 16 (one row through 2 x
// 8192 x 4096: 19.8 us, 6.8 TB/s of w).
template <bool kF8, int NT, bool kVec, bool kGlu>
__global__ void __launch_bounds__(kSmallWarps * 32) small_kernel(LinearArgs a, int cs) {
  constexpr int kSize = kF8 ? 1 : 2, kTok = 8 * NT;
  __shared__ float part[kSmallWarps][16][kTok + 1];
  __shared__ float ranks[kMaxCluster][16 * kTok];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = cs > 1 ? (int)(blockIdx.x % cs) : 0;
  chain_wait();
  constexpr int kRows = kGlu ? 8 : 16;  // output columns of a CTA
  const int64_t n0 = (int64_t)(blockIdx.x / cs) * kRows, m0 = (int64_t)blockIdx.y * kTok;
  if (cs > 1) cg::this_cluster().barrier_arrive();
  const int64_t bytes = a.K * kSize;
  // rows past the end repeat the last one; their results are not stored
  const uint8_t *w0 = static_cast<const uint8_t *>(a.w) + (n0 + g < a.N ? n0 + g : a.N - 1) * a.ldw * kSize;
  const uint8_t *w1 = kGlu ? w0 + a.N * a.ldw * kSize
                           : static_cast<const uint8_t *>(a.w) + (n0 + g + 8 < a.N ? n0 + g + 8 : a.N - 1) * a.ldw * kSize;
  const uint8_t *x[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    x[i] = static_cast<const uint8_t *>(a.x) + (m0 + 8 * i + g < a.M ? m0 + 8 * i + g : a.M - 1) * a.ldx * kSize;
  float c[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;

  constexpr int64_t kSpan = kBlocks * 64;  // bytes of a row per turn
  const int64_t step = kSpan * kSmallWarps * cs;
  int64_t k0 = (rank * kSmallWarps + warp) * kSpan;
  uint4 next0[kBlocks], next1[kBlocks];
  const auto ask = [&](int64_t k) {
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) {
      next0[j] = piece<kVec, true>(w0, k + j * 64 + t * 16, bytes);
      next1[j] = piece<kVec, true>(w1, k + j * 64 + t * 16, bytes);
    }
  };
  ask(k0);
  for (; k0 < bytes; k0 += step) {
    uint4 u0[kBlocks], u1[kBlocks];
#pragma unroll
    for (int j = 0; j < kBlocks; ++j) u0[j] = next0[j], u1[j] = next1[j];
    ask(k0 + step);
#pragma unroll
    for (int j = 0; j < kBlocks; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 v = piece<kVec, false>(x[i], k0 + j * 64 + t * 16, bytes);
        if constexpr (kF8) {
          mma_e4m3(c[i], u0[j].x, u1[j].x, u0[j].y, u1[j].y, v.x, v.y);
          mma_e4m3(c[i], u0[j].z, u1[j].z, u0[j].w, u1[j].w, v.z, v.w);
        } else {
          mma_bf16(c[i], u0[j].x, u1[j].x, u0[j].y, u1[j].y, v.x, v.y);
          mma_bf16(c[i], u0[j].z, u1[j].z, u0[j].w, u1[j].w, v.z, v.w);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    part[warp][g][8 * i + 2 * t] = c[i][0];
    part[warp][g][8 * i + 2 * t + 1] = c[i][1];
    part[warp][g + 8][8 * i + 2 * t] = c[i][2];
    part[warp][g + 8][8 * i + 2 * t + 1] = c[i][3];
  }
  __syncthreads();
  if (cs > 1) cg::this_cluster().barrier_wait();  // every CTA of the cluster has begun
  const auto sum = [&](int r, int tok) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) v += part[w][r][tok];
    return v;
  };
  const auto store = [&](int r, int tok, float v, float u) {  // (u: the other half's, gated alone)
    if (m0 + tok >= a.M || n0 + r >= a.N) return;
    if constexpr (kGlu)
      finish_glu<__nv_bfloat16>(a, m0 + tok, n0 + r, v, u);
    else
      finish<__nv_bfloat16>(a, m0 + tok, n0 + r, v);
  };
  if (cs == 1) {
    for (int i = threadIdx.x; i < kRows * kTok; i += kSmallWarps * 32) {
      const int r = i % kRows, tok = i / kRows;
      store(r, tok, sum(r, tok), kGlu ? sum(r + 8 & 15, tok) : 0.f);
    }
    return;
  }
  for (int i = threadIdx.x; i < 16 * kTok; i += kSmallWarps * 32)
    cg::this_cluster().map_shared_rank(&ranks[rank][0], 0)[i] = sum(i & 15, i >> 4);
  cg::this_cluster().sync();
  if (rank == 0)
    for (int i = threadIdx.x; i < kRows * kTok; i += kSmallWarps * 32) {
      const int r = i % kRows, tok = i / kRows;
      float v = 0.f, u = 0.f;
      for (int q = 0; q < cs; ++q) {
        v += ranks[q][tok * 16 + r];
        if constexpr (kGlu) u += ranks[q][tok * 16 + r + 8];
      }
      store(r, tok, v, u);
    }
}

template <bool kF8, int NT, bool kGlu = false>
cudaError_t run_small(const LinearArgs &a, cudaStream_t s) {
  const int64_t size = kF8 ? 1 : 2, e = 16 / size;
  const bool vec = a.K % e == 0 && a.ldx % e == 0 && a.ldw % e == 0 && aligned_to(a.x, 16) && aligned_to(a.w, 16);
  // CTAs along k until every SM has two, as far as k has a turn for each warp
  const int64_t groups = (a.N + (kGlu ? 7 : 15)) / (kGlu ? 8 : 16), passes = (a.M + 8 * NT - 1) / (8 * NT), turns = (a.K * size + kBlocks * 64 - 1) / (kBlocks * 64);
  int cs = 1;
  while (cs < kMaxCluster && groups * passes * cs < 2 * sm_count() && turns > (int64_t)kSmallWarps * cs) cs *= 2;
  return chain_launch(vec ? small_kernel<kF8, NT, true, kGlu> : small_kernel<kF8, NT, false, kGlu>,
                      dim3((unsigned)(groups * cs), (unsigned)passes), dim3(kSmallWarps * 32), 0, cs, true, s, a, cs);
}

// ------------------------------------------------------ float32, CUDA cores
// A correctness path: 64 x 64 tiles, 4 x 4 elements a thread, operands with
// any strides.
__global__ void __launch_bounds__(256) gemm_f32_kernel(LinearArgs e, const float *a, int64_t am, int64_t ak,
                                                       const float *b, int64_t bn, int64_t bk, int64_t K) {
  __shared__ float sa[16][65], sb[16][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t nt = (e.N + 63) / 64, m0 = (int64_t)blockIdx.x / nt * 64, n0 = (int64_t)blockIdx.x % nt * 64;
  float c[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      // neighbouring threads along the contiguous axis of each operand
      const int ka = ak == 1 ? i & 15 : i >> 6, ma = ak == 1 ? i >> 4 : i & 63;
      const int kb = bk == 1 ? i & 15 : i >> 6, nb = bk == 1 ? i >> 4 : i & 63;
      sa[ka][ma] = m0 + ma < e.M && k0 + ka < K ? a[(m0 + ma) * am + (k0 + ka) * ak] : 0.f;
      sb[kb][nb] = n0 + nb < e.N && k0 + kb < K ? b[(n0 + nb) * bn + (k0 + kb) * bk] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], c[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < e.M && n < e.N) finish<float>(e, m, n, c[i][j]);
    }
}

// ----------------------------------------------------------------- gradients
// Rows of `bytes` bytes, ld bytes apart, into rows of ldp bytes (a multiple of
// 16), whole 16-byte pieces; what lies past a row's end is not used.  A piece
// is put together from five aligned words; in the rows where one could lie
// outside the matrix, from the bytes that are in it.  A warp a row, four
// pieces a lane in flight.
__global__ void __launch_bounds__(256) pack_kernel(const unsigned char *src, unsigned char *dst, int64_t rows,
                                                   int64_t bytes, int64_t ld, int64_t ldp) {
  constexpr int kAhead = 4;
  chain_next();
  chain_wait();
  const uintptr_t lo = reinterpret_cast<uintptr_t>(src), hi = lo + (rows - 1) * ld + bytes;
  for (int64_t r = (int64_t)blockIdx.x * 8 + threadIdx.y; r < rows; r += (int64_t)gridDim.x * 8) {
    const uintptr_t row = lo + r * ld;
    const uint32_t shift = 8 * (uint32_t)(row & 3);
    const uintptr_t words = row & ~(uintptr_t)3;
    const bool inside = words >= lo && row + bytes + 20 <= hi;
    for (int64_t c0 = threadIdx.x * 16; c0 < bytes; c0 += 512 * kAhead) {
      uint32_t w[kAhead][5];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t c = c0 + 512 * k;
        if (c >= bytes) continue;
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const uintptr_t at = words + c + 4 * i;
          if (inside || (at >= lo && at + 4 <= hi)) {
            w[k][i] = *reinterpret_cast<const uint32_t *>(at);
          } else {
            w[k][i] = 0;
            for (int b = 0; b < 4; ++b)
              if (at + b >= lo && at + b < hi)
                w[k][i] |= (uint32_t)*reinterpret_cast<const unsigned char *>(at + b) << (8 * b);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (c0 + 512 * k < bytes)
          *reinterpret_cast<uint4 *>(dst + r * ldp + c0 + 512 * k) =
              make_uint4(__funnelshift_r(w[k][0], w[k][1], shift), __funnelshift_r(w[k][1], w[k][2], shift),
                         __funnelshift_r(w[k][2], w[k][3], shift), __funnelshift_r(w[k][3], w[k][4], shift));
    }
  }
}

// dpre = dout act'(pre) and its column sums: a CTA has 32 V columns and every
// parts-th group of 8 rows; one element (V = 1) or 16 bytes a lane.  The sums
// take the unrounded products; part sums meet in launch_column_sum.
// (The gated layer's is glu_dpre_kernel.)
template <typename T, int V>
__global__ void __launch_bounds__(256) dpre_kernel(DpreArgs p) {
  struct __align__(sizeof(T) * V) Vec { T v[V]; };
  __shared__ float sum[8][32 * V];
  const int64_t c = ((int64_t)blockIdx.x * 32 + threadIdx.x) * V;
  chain_next();
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.f;
  constexpr int kAhead = V == 1 ? 4 : 2;  // rows a thread asks for at a time
  const int64_t step = (int64_t)gridDim.y * 8;
  if (c < p.N)
    for (int64_t m0 = (int64_t)blockIdx.y * 8 + threadIdx.y; m0 < p.M; m0 += step * kAhead) {
      Vec d[kAhead], q[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t m = m0 + k * step;
        if (m >= p.M) continue;
        d[k] = *reinterpret_cast<const Vec *>(static_cast<const T *>(p.dout) + m * p.N + c);
        if (p.act != kActNone) q[k] = *reinterpret_cast<const Vec *>(static_cast<const T *>(p.pre) + m * p.N + c);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t m = m0 + k * step;
        if (m >= p.M) continue;
        Vec o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = to_f(d[k].v[i]);
          if (p.act != kActNone) v *= slope(p.act, to_f(q[k].v[i]));
          s[i] = __fadd_rn(s[i], v);  // not contracted: the same with dpre wanted and without
          from_f(v, o.v[i]);
        }
        if (p.dpre) *reinterpret_cast<Vec *>(static_cast<T *>(p.dpre) + m * p.ldp + c) = o;
      }
    }
  if (!p.dbias) return;
#pragma unroll
  for (int i = 0; i < V; ++i) sum[threadIdx.y][threadIdx.x * V + i] = s[i];
  __syncthreads();
  for (int i = threadIdx.y * 32 + threadIdx.x; i < 32 * V; i += 256) {
    const int64_t n = (int64_t)blockIdx.x * 32 * V + i;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sum[w][i];
    if (n < p.N) p.partial[(int64_t)blockIdx.y * p.N + n] = v;
  }
}

// The gated layer's: dpre [M][2 N] = (dout u act'(g), dout act(g)) from pre = (g, u),
// and the sums of its 2 N columns.  As above, a column of either half a lane.  One row at
// a time leaves room for four CTAs an SM, all of them resident at once (two rows, and two
// CTAs: 35 us for 26 at M4096 N4096, where reading and writing 168 MB takes 25).
template <typename T, int V>
__global__ void __launch_bounds__(256, 4) glu_dpre_kernel(DpreArgs p) {
  struct __align__(sizeof(T) * V) Vec { T v[V]; };
  __shared__ float sum[2][8][32 * V];
  const int64_t c = ((int64_t)blockIdx.x * 32 + threadIdx.x) * V;
  chain_next();
  float s[2][V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[0][i] = s[1][i] = 0.f;
  constexpr int kAhead = V == 1 ? 4 : 1;  // rows a thread asks for at a time
  const int64_t step = (int64_t)gridDim.y * 8;
  if (c < p.N)
    for (int64_t m0 = (int64_t)blockIdx.y * 8 + threadIdx.y; m0 < p.M; m0 += step * kAhead) {
      Vec d[kAhead], g[kAhead], u[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t m = m0 + k * step;
        if (m >= p.M) continue;
        d[k] = *reinterpret_cast<const Vec *>(static_cast<const T *>(p.dout) + m * p.N + c);
        g[k] = *reinterpret_cast<const Vec *>(static_cast<const T *>(p.pre) + m * 2 * p.N + c);
        u[k] = *reinterpret_cast<const Vec *>(static_cast<const T *>(p.pre) + m * 2 * p.N + p.N + c);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int64_t m = m0 + k * step;
        if (m >= p.M) continue;
        Vec o[2];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float dv = to_f(d[k].v[i]), gv = to_f(g[k].v[i]);
          float value, der;
          curve(p.act, gv, value, der);
          const float a = dv * to_f(u[k].v[i]) * der, b = dv * value;
          s[0][i] = __fadd_rn(s[0][i], a), s[1][i] = __fadd_rn(s[1][i], b);  // (as in dpre_kernel)
          from_f(a, o[0].v[i]), from_f(b, o[1].v[i]);
        }
        if (p.dpre) {
          *reinterpret_cast<Vec *>(static_cast<T *>(p.dpre) + m * p.ldp + c) = o[0];
          *reinterpret_cast<Vec *>(static_cast<T *>(p.dpre) + m * p.ldp + p.N + c) = o[1];
        }
      }
    }
  if (!p.dbias) return;
#pragma unroll
  for (int i = 0; i < V; ++i)
    sum[0][threadIdx.y][threadIdx.x * V + i] = s[0][i], sum[1][threadIdx.y][threadIdx.x * V + i] = s[1][i];
  __syncthreads();
  for (int i = threadIdx.y * 32 + threadIdx.x; i < 64 * V; i += 256) {
    const int h = i / (32 * V), j = i % (32 * V);
    const int64_t n = (int64_t)blockIdx.x * 32 * V + j;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sum[h][w][j];
    if (n < p.N) p.partial[((int64_t)blockIdx.y * 2 + h) * p.N + n] = v;
  }
}

// out = act(g) u from pre = (g, u), float32
__global__ void __launch_bounds__(256) glu_act_kernel(const float *pre, float *out, int64_t M, int64_t N, int act) {
  chain_wait();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * 256) {
    const float *at = pre + i / N * 2 * N + i % N;
    out[i] = activate(act, at[0]) * at[N];
  }
}

// Small gradients, all in one kernel: C[m][n] = sum_r A(r, m) B(r, n) with A
// formed on the way in as dpre = dout act'(pre), so that nothing is packed and
// dpre is not rounded.  For dx, m is the row and r the output channel, B is w;
// for dw, m is the output channel and r the row, B is x, and the column sums of
// dpre come out beside it.  The first CTAs have dx's tiles, the others dw's.  A
// CTA has 32 x 64 elements and every cs-th block of 32 r, 2 x 4 elements a thread
// on the CUDA cores in float32, the next block's elements on their way meanwhile;
// a cluster's sums meet through distributed shared memory in rank order.
constexpr int kBm = 32, kBn = 64, kBr = 32, kBwdCluster = 8;

struct SmallBwd {
  const __nv_bfloat16 *dout, *pre;  // [M][N]
  const __nv_bfloat16 *x, *w;       // [M][K], [N][K]
  __nv_bfloat16 *dx, *dw;           // nullptr: not wanted
  float *dbias;
  int64_t M, N, K, ldx, ldw;
  int64_t dx_tiles, dw_tiles;
  int act, cs;
};

// kGlu: the gated layer, whose N rows of w are two halves; dout is [M][N / 2]
template <bool kGlu>
__global__ void __launch_bounds__(256) small_bwd_kernel(SmallBwd p) {
  __shared__ float sa[kBr][kBm + 1];
  __shared__ __align__(16) float sb[kBr][kBn + 4];
  __shared__ __align__(16) float part[kBm][kBn + 4], bias[kBm];
  const int tid = threadIdx.x, cs = p.cs;
  const int rank = cs > 1 ? (int)(blockIdx.x % cs) : 0;
  if (cs > 1) cg::this_cluster().barrier_arrive();
  chain_wait();  // (chain_next(): 512 x 512 x 128 13 -> 17 us, the next CTAs crowd on free SMs)
  int64_t tile = blockIdx.x / cs;
  const bool of_w = tile >= p.dx_tiles;  // same for a cluster
  if (of_w) tile -= p.dx_tiles;
  const __nv_bfloat16 *const other = of_w ? p.x : p.w;
  __nv_bfloat16 *const out = of_w ? p.dw : p.dx;
  const int64_t ldo = of_w ? p.ldx : p.ldw;
  const int64_t rows = of_w ? p.N : p.M, red = of_w ? p.M : p.N;  // of C, and terms of its sums
  const int64_t across = out ? (p.K + kBn - 1) / kBn : 1;
  const int64_t m0 = tile / across * kBm, n0 = tile % across * kBn;
  const bool sums = of_w && p.dbias && n0 == 0;
  const int tm = tid / 16 * 2, tn = tid % 16 * 4;
  float c[2][4] = {}, s = 0.f;
  __nv_bfloat16 ra[kBr * kBm / 256], rp[kBr * kBm / 256], rb[kBr * kBn / 256], ru[kGlu ? kBr * kBm / 256 : 1];
  bool up[kGlu ? kBr * kBm / 256 : 1];
  const __nv_bfloat16 zero = __float2bfloat16_rn(0.f);
  const auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int k = 0; k < kBr * kBm / 256; ++k) {
      // neighbouring threads along a row of dout: its columns are r for dx, m for dw
      const int a = tid % 32, b = tid / 32 + 8 * k;
      const int64_t row = of_w ? r0 + b : m0 + b, col = of_w ? m0 + a : r0 + a;
      const bool in = row < p.M && col < p.N;
      if constexpr (kGlu) {
        const int64_t half = p.N / 2;
        up[k] = col >= half;
        const int64_t at = up[k] ? col - half : col;
        ra[k] = in ? p.dout[row * half + at] : zero;
        rp[k] = in ? p.pre[row * p.N + at] : zero;
        ru[k] = in && !up[k] ? p.pre[row * p.N + half + at] : zero;
      } else {
        ra[k] = in ? p.dout[row * p.N + col] : zero;
        rp[k] = in && p.act != kActNone ? p.pre[row * p.N + col] : zero;
      }
    }
    if (out) {
#pragma unroll
      for (int k = 0; k < kBr * kBn / 256; ++k) {
        const int a = tid % kBn, b = tid / kBn + 4 * k;
        rb[k] = r0 + b < red && n0 + a < p.K ? other[(r0 + b) * ldo + n0 + a] : zero;
      }
    }
  };
  int64_t r0 = (int64_t)rank * kBr;
  if (r0 < red) fetch(r0);
  for (; r0 < red; r0 += (int64_t)kBr * cs) {
#pragma unroll
    for (int k = 0; k < kBr * kBm / 256; ++k) {
      const int a = tid % 32, b = tid / 32 + 8 * k;
      const float g = __bfloat162float(ra[k]);
      // outside, dout stands as 0 and takes no factor
      float v;
      if constexpr (kGlu)
        v = up[k] ? g * activate(p.act, __bfloat162float(rp[k]))
                  : g * __bfloat162float(ru[k]) * slope(p.act, __bfloat162float(rp[k]));
      else
        v = p.act == kActNone ? g : g * slope(p.act, __bfloat162float(rp[k]));
      if (of_w)
        sa[b][a] = v;
      else
        sa[a][b] = v;
    }
    if (out) {
#pragma unroll
      for (int k = 0; k < kBr * kBn / 256; ++k) sb[tid / kBn + 4 * k][tid % kBn] = __bfloat162float(rb[k]);
    }
    __syncthreads();
    if (r0 + (int64_t)kBr * cs < red) fetch(r0 + (int64_t)kBr * cs);
    if (out) {
#pragma unroll 8
      for (int r = 0; r < kBr; ++r) {
        const float a0 = sa[r][tm], a1 = sa[r][tm + 1];
        const float4 b = *reinterpret_cast<const float4 *>(&sb[r][tn]);
        c[0][0] = fmaf(a0, b.x, c[0][0]), c[0][1] = fmaf(a0, b.y, c[0][1]);
        c[0][2] = fmaf(a0, b.z, c[0][2]), c[0][3] = fmaf(a0, b.w, c[0][3]);
        c[1][0] = fmaf(a1, b.x, c[1][0]), c[1][1] = fmaf(a1, b.y, c[1][1]);
        c[1][2] = fmaf(a1, b.z, c[1][2]), c[1][3] = fmaf(a1, b.w, c[1][3]);
      }
    }
    if (sums && tid < kBm) {
#pragma unroll 8
      for (int r = 0; r < kBr; ++r) s += sa[r][tid];
    }
    __syncthreads();
  }
  if (cs == 1) {
    if (sums && tid < kBm && m0 + tid < p.N) p.dbias[m0 + tid] = s;
    if (!out) return;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (m0 + tm + i < rows && n0 + tn + j < p.K)
          out[(m0 + tm + i) * p.K + n0 + tn + j] = __float2bfloat16_rn(c[i][j]);
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.barrier_wait();  // every CTA of the cluster has begun
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<float4 *>(&part[tm + i][tn]) = make_float4(c[i][0], c[i][1], c[i][2], c[i][3]);
  if (tid < kBm) bias[tid] = s;
  cluster.sync();
  // each CTA adds up and stores its share of the rows
  const int share = kBm / cs;
  for (int i = tid; i < share * kBn; i += 256) {
    const int m = rank * share + i / kBn, n = i % kBn;
    float v = 0.f;
    for (int q = 0; q < cs; ++q) v += *cluster.map_shared_rank(&part[m][n], q);
    if (out && m0 + m < rows && n0 + n < p.K) out[(m0 + m) * p.K + n0 + n] = __float2bfloat16_rn(v);
  }
  if (sums && tid < share && m0 + rank * share + tid < p.N) {
    float v = 0.f;
    for (int q = 0; q < cs; ++q) v += *cluster.map_shared_rank(&bias[rank * share + tid], q);
    p.dbias[m0 + rank * share + tid] = v;
  }
  cluster.sync();  // no CTA leaves while another may read from it
}

int64_t tiles_of(int64_t rows, int64_t cols) { return (rows + kBm - 1) / kBm * ((cols + kBn - 1) / kBn); }

int dpre_vec(const DpreArgs &p) {
  const int v = p.bf16 ? 8 : 4;
  return p.N % v == 0 && (!p.dpre || p.ldp % v == 0) && aligned_to(p.dout, 16) && aligned_to(p.pre, 16) &&
                 aligned_to(p.dpre, 16)
             ? v
             : 1;
}

}  // namespace

// From 30 measured sizes (M24..4000, N64..2048, K64..4096): 512 CTAs of 16 x 16
// outputs take a round, of 1.15 us and 1.06 us per KB of a row of w; twice as
// long where pieces are put together, three times of 8-bit elements.
double linear_small_us(int64_t M, int64_t N, int64_t K, bool f8, bool whole) {
  if (M > 65535 * 16) return 1e30;  // (a grid's height)
  const double ctas = (double)((M + 15) / 16) * (double)((N + 15) / 16);
  return (2.0 + ctas / 512.0 * (1.15 + 1.06 * (double)K * (f8 ? 1 : 2) / 1024.0)) * (whole ? 1.0 : f8 ? 3.0 : 2.0);
}

cudaError_t launch_linear_small(const LinearArgs &a, cudaStream_t s) {
  if (a.kind == kLinE4m3)
    return a.M <= 8 ? run_small<true, 1>(a, s) : run_small<true, 2>(a, s);
  return a.M <= 8 ? run_small<false, 1>(a, s) : run_small<false, 2>(a, s);
}

cudaError_t launch_glu_small(const LinearArgs &a, cudaStream_t s) {
  return a.M <= 8 ? run_small<false, 1, true>(a, s) : run_small<false, 2, true>(a, s);
}

cudaError_t launch_glu_act(const float *pre, float *out, int64_t M, int64_t N, int act, cudaStream_t s) {
  const int64_t want = (M * N + 255) / 256, cap = (int64_t)sm_count() * 8;
  return chain_launch(glu_act_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, 1, true, s, pre, out, M,
                      N, act);
}

cudaError_t launch_gemm_f32(const LinearArgs &epi, const float *a, int64_t am, int64_t ak, const float *b,
                            int64_t bn, int64_t bk, int64_t K, cudaStream_t s) {
  const int64_t grid = ((epi.M + 63) / 64) * ((epi.N + 63) / 64);
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  gemm_f32_kernel<<<(unsigned)grid, 256, 0, s>>>(epi, a, am, ak, b, bn, bk, K);
  return cudaGetLastError();
}

cudaError_t launch_pack(const void *src, void *dst, int64_t rows, int64_t cols, int64_t ld, int64_t ldp, int size,
                        bool dependent, cudaStream_t s) {
  const int64_t want = (rows + 7) / 8, cap = (int64_t)sm_count() * 8;
  return chain_launch(pack_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(32, 8), 0, 1, dependent, s,
                      static_cast<const unsigned char *>(src), static_cast<unsigned char *>(dst), rows, cols * size,
                      ld * size, ldp * size);
}

// (the gated layer's: as many as are resident; twice as many take 2 us more at M4096 N4096)
constexpr int64_t kGluCtas = 4;
int64_t dpre_parts(const DpreArgs &p) {
  // CTAs for every SM many times over, but no fewer than 4 rows a thread (M512
  // N2048: 24 us of gradients in all, for 28 with a quarter of the CTAs)
  const int64_t across = (p.N + 32 * dpre_vec(p) - 1) / (32 * dpre_vec(p));
  int64_t parts = ((p.glu ? kGluCtas : 32) * (int64_t)sm_count() + across - 1) / across;
  const int64_t most = (p.M + 31) / 32;
  if (parts > most) parts = most;
  return parts < 1 ? 1 : parts > 65535 ? 65535 : parts;
}

cudaError_t launch_dpre(const DpreArgs &p, cudaStream_t s) {
  const int v = dpre_vec(p);
  const int64_t parts = dpre_parts(p);
  const dim3 grid((unsigned)((p.N + 32 * v - 1) / (32 * v)), (unsigned)parts), block(32, 8);
  if (p.glu) {
    if (p.bf16)
      (v == 1 ? glu_dpre_kernel<__nv_bfloat16, 1> : glu_dpre_kernel<__nv_bfloat16, 8>)<<<grid, block, 0, s>>>(p);
    else
      (v == 1 ? glu_dpre_kernel<float, 1> : glu_dpre_kernel<float, 4>)<<<grid, block, 0, s>>>(p);
  } else if (p.bf16) {
    if (v == 1)
      dpre_kernel<__nv_bfloat16, 1><<<grid, block, 0, s>>>(p);
    else
      dpre_kernel<__nv_bfloat16, 8><<<grid, block, 0, s>>>(p);
  } else {
    if (v == 1)
      dpre_kernel<float, 1><<<grid, block, 0, s>>>(p);
    else
      dpre_kernel<float, 4><<<grid, block, 0, s>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dbias) return e;
  return launch_column_sum(p.partial, p.dbias, parts, (p.glu ? 2 : 1) * p.N, s);
}

namespace {

// CTAs along the sums while they do not fill the GPU and have blocks to share
int small_bwd_cluster(int64_t tiles, int64_t red) {
  int cs = 1;
  while (cs < kBwdCluster && tiles * cs < 3 * sm_count() && red > (int64_t)kBr * cs) cs *= 2;
  return cs;
}

}  // namespace

// The launch's time is 3.2 us, 1.85 us a block of 32 terms that follow one
// another in a CTA and 4 ns a block in all (14 measured sizes, M1..4096, N19..2048,
// K27..3712).  The tensor cores' way takes 10..13 us for small products from a
// graph, but is four to six launches, 16..20 us of a caller's time (M512 N512
// K128: 13 us a call for 16.5; M200 N300 K400: 16.6 for 15.9).
bool small_bwd_fits(int64_t M, int64_t N, int64_t K) {
  const int64_t m = (M + kBm - 1) / kBm, n = (N + kBm - 1) / kBm, k = (K + kBn - 1) / kBn;
  if (m > 4096 || n > 4096 || k > 4096) return false;
  const int64_t cs = small_bwd_cluster((m + n) * k, max(M, N)), chain = (max(m, n) + cs - 1) / cs;
  return 3.2 + 1.85 * (double)chain + 0.004 * (double)(2 * m * n * k) < kSmallBwdUs;
}

cudaError_t launch_small_bwd(const void *x, const void *w, const void *dout, const void *pre, void *dx, void *dw,
                             float *dbias, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw, int act,
                             bool glu, cudaStream_t s) {
  using T = __nv_bfloat16;
  SmallBwd p{};
  p.dout = static_cast<const T *>(dout), p.pre = static_cast<const T *>(pre);
  p.x = static_cast<const T *>(x), p.w = static_cast<const T *>(w);
  p.dx = static_cast<T *>(dx), p.dw = static_cast<T *>(dw), p.dbias = dbias;
  p.M = M, p.N = N, p.K = K, p.ldx = ldx, p.ldw = ldw, p.act = act;
  p.dx_tiles = dx ? tiles_of(M, K) : 0;
  p.dw_tiles = dw ? tiles_of(N, K) : dbias ? tiles_of(N, 1) : 0;
  const int64_t tiles = p.dx_tiles + p.dw_tiles;
  if (tiles == 0) return cudaSuccess;
  // of all gradients' tiles, whichever are wanted, so that each has the same value
  p.cs = small_bwd_cluster(tiles_of(M, K) + tiles_of(N, K), max(M, N));
  return chain_launch(glu ? small_bwd_kernel<true> : small_bwd_kernel<false>, dim3((unsigned)(tiles * p.cs)), dim3(256),
                      0, p.cs, true, s, p);
}

}  // namespace delta
