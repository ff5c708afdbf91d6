// linear_tc.cu -- the linear layer's matrix products on the 5th-generation
// tensor cores, D[M][N] = sum_k A(m, k) B(n, k), with the epilogue of
// linear.cuh, or that of the gated layer, D's columns in two halves (kGlu).
// The forward takes x and w with k contiguous; the gradients take them as they
// lie, with k as the row (w for dx, both operands for dw), which the
// shared-memory descriptors express as MN-major operands, so nothing is
// transposed in memory.
//
// One persistent CTA per SM, ten warps:
//   warp 0: TMA producer, a ring of kStages stages of 128 bytes of k;
//   warp 1: allocates TMEM and issues the products (one thread) into one of
//           two TMEM accumulators of 128 x BN;
//   warps 2-9: epilogue, two to a TMEM lane quarter (32 rows) that take turns
//           at its columns, while the next tile's products run into the other
//           accumulator.  A chunk of 32 x 32 is finished as TMEM gives it, a
//           row a lane, and goes out in 32-byte pieces: whole sectors, though a
//           lane's rows are apart.  (A turn through shared memory for coalesced
//           pieces, or for TMA, took its bandwidth from the operands and was
//           the slower way: 8192 x 4096 outputs at K = 512 in 31 and 34 us.)
// A large product takes CTAs in pairs (cta_group::2): a tile of 256 x 256 of
// which each CTA loads 128 rows of either operand, 32 KB a stage.  One CTA
// alone on 128 x 256 needs 48 KB for the same work, which at full rate is more
// than L2 gives 152 SMs (1.32 PFLOP/s).  Smaller ones take 128 x 128 or
// 128 x 64 tiles of one CTA.  Tiles are dealt out in bands of kBand tile rows,
// so that the CTAs at work at a time share operand rows in L2.  Every mbarrier
// wait is bounded: a timeout sets a device error word and the kernel winds
// down.
//
// The gated layer's product at M8192 N4096 K4096 is bound by the tensor cores'
// clock under power: 286 to 310 us, 1.8 to 1.92 PFLOP/s, and 340 after seconds
// of such load (1.6); the epilogue is hidden.
#include "chain.cuh"
#include "linear.cuh"
#include "sm100.cuh"
#include "tma_host.h"

namespace delta {
namespace {

using namespace sm100;

__device__ unsigned int g_linear_error = 0;

constexpr int kBM = 128;
constexpr int kEpi = 8;          // epilogue warps
constexpr int kThreads = 64 + 32 * kEpi;
constexpr int kBand = 8;
constexpr int kMaxSplit = 8;    // CTAs that share a tile's k: the portable cluster
constexpr int kPitch = 36;      // floats a row of an epilogue warp's stage (odd row widths)
constexpr int kEpiBytes = 32 * kPitch * 4;
constexpr int kRowBytes = 128;  // of k in a stage: 64 bfloat16 or 128 e4m3

// BN: columns of a tile; a pair's CTA loads half of B's rows
__host__ __device__ constexpr int b_rows(int BN, bool pair) { return pair ? BN / 2 : BN; }
__host__ __device__ constexpr int stage_bytes(int BN, bool pair) { return (kBM + b_rows(BN, pair)) * kRowBytes; }
__host__ __device__ constexpr int stages(int BN, bool pair) { return pair || BN == 128 ? 5 : 7; }
__host__ __device__ constexpr int smem_bytes(int BN, bool pair) {
  return 1024 + stages(BN, pair) * stage_bytes(BN, pair) + kEpi * kEpiBytes;
}

struct Shared {
  uint64_t full[8], empty[8], tfull[2], tempty[2], drain;
  uint32_t tmem;
  volatile int dead;
};

__device__ __noinline__ bool wait_slow(Shared *sh, uint64_t *bar, uint32_t parity, int role) {
  for (uint32_t i = 0; i < (1u << 22); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && sh->dead) return false;
  }
  sh->dead = 1;
  atomicCAS(&g_linear_error, 0u, (unsigned)(1 + role));
  return false;
}
__device__ __forceinline__ bool wait(Shared *sh, uint64_t *bar, uint32_t parity, int role) {
  return mbar_try_wait(bar, parity) || wait_slow(sh, bar, parity, role);
}

struct Tiles {
  int64_t m_tiles, n_tiles, total;
  int kblocks;
  int split, per;  // CTAs (or pairs) that share a tile's k, and blocks of k for each
};
__device__ __forceinline__ void tile_at(const Tiles &t, int64_t i, int64_t &m, int64_t &n) {
  // (fewer than 2^32 tiles: 32-bit divisions, an order of magnitude shorter)
  const uint32_t across = kBand * (uint32_t)t.n_tiles, band = (uint32_t)i / across, first = band * kBand;
  const uint32_t left = (uint32_t)t.m_tiles - first, high = left < kBand ? left : kBand;
  const uint32_t r = (uint32_t)i - band * across, down = r / high;
  m = first + (r - down * high);
  n = down;
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void widen8(const uint4 &q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 narrow8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// 8 columns of a row before the activation: scales and bias
__device__ __forceinline__ void raise8(const LinearArgs &e, int64_t n, float (&v)[8], float sx) {
  float q[8];
  if (e.x_scale) {
    load8(e.w_scale + n, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= sx * q[j];
  }
  if (e.bias) {
    if (e.bias_bf16)
      widen8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(e.bias) + n), q);
    else
      load8(static_cast<const float *>(e.bias) + n, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += q[j];
  }
}
__device__ __forceinline__ void activate8(const LinearArgs &e, float (&v)[8]) {
  if (e.act != kActNone) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = linear::activate(e.act, v[j]);
  }
}
__device__ __forceinline__ void add8(float (&v)[8], const uint4 &res) {
  float q[8];
  widen8(res, q);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += q[j];
}

// 16 neighbouring elements of a row: one 32-byte access, or two of 16 bytes
struct Half {
  uint4 a, b;
};
__device__ __forceinline__ Half load16(const __nv_bfloat16 *p, bool wide) {
  Half h;
  if (wide)
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(h.a.x), "=r"(h.a.y), "=r"(h.a.z), "=r"(h.a.w), "=r"(h.b.x), "=r"(h.b.y), "=r"(h.b.z), "=r"(h.b.w)
                 : "l"(p)
                 : "memory");
  else
    h.a = *reinterpret_cast<const uint4 *>(p), h.b = *reinterpret_cast<const uint4 *>(p + 8);
  return h;
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, const uint4 &a, const uint4 &b, bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  else
    *reinterpret_cast<uint4 *>(p) = a, *reinterpret_cast<uint4 *>(p + 8) = b;
}

// A row's 32 residuals of a chunk; the columns past N (a multiple of 8) are not
// read.
struct Residual {
  Half h[2];
};
__device__ __forceinline__ void ask_residual(const LinearArgs &e, int64_t m, int64_t n0, bool wide, Residual &r) {
  if (!e.residual || m >= e.M) return;
  const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(e.residual) + m * e.ldr + n0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (n0 + 16 * k + 16 <= e.N)
      r.h[k] = load16(p + 16 * k, wide);
    else if (n0 + 16 * k + 8 <= e.N)
      r.h[k].a = *reinterpret_cast<const uint4 *>(p + 16 * k);
  }
}

// One chunk of one row, start to end.  cols: the chunk's biases and column
// scales in shared memory, [2][32].
__device__ __forceinline__ void finish_row(const LinearArgs &e, int64_t m, int64_t n0, uint32_t (&r)[32], float sx,
                                           const float *cols, const Residual &res, bool wide) {
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e.out) + m * e.N + n0;
  __nv_bfloat16 *pre = static_cast<__nv_bfloat16 *>(e.pre) + m * e.N + n0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint4 po[2], pp[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      float v[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[16 * k + 8 * g + i]);
      if (e.x_scale) {
        load8(cols + 32 + 16 * k + 8 * g, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= sx * q[i];
      }
      if (e.bias) {
        load8(cols + 16 * k + 8 * g, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += q[i];
      }
      pp[g] = narrow8(v);
      activate8(e, v);
      if (e.residual) add8(v, g ? res.h[k].b : res.h[k].a);
      po[g] = narrow8(v);
    }
    if (n0 + 16 * k + 16 <= e.N) {
      if (e.pre) store16(pre + 16 * k, pp[0], pp[1], wide);
      store16(out + 16 * k, po[0], po[1], wide);
    } else if (n0 + 16 * k + 8 <= e.N) {
      if (e.pre) *reinterpret_cast<uint4 *>(pre + 16 * k) = pp[0];
      *reinterpret_cast<uint4 *>(out + 16 * k) = po[0];
    }
  }
}

// The same chunk where rows are not whole 16-byte pieces: a lane has one column
// of all 32 rows, single elements, eight rows asked for at a time.
__device__ __forceinline__ void finish_column(const LinearArgs &e, const float *stage, int lane, int64_t m0, int64_t n) {
  if (n >= e.N) return;
  constexpr int kRows = 8;
  const float bias = linear::bias_at(e, n), sw = e.x_scale ? e.w_scale[n] : 1.f;
  const int rows = e.M - m0 < 32 ? (int)(e.M - m0) : 32;
  const __nv_bfloat16 *res = static_cast<const __nv_bfloat16 *>(e.residual) + m0 * e.ldr + n;
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e.out) + m0 * e.N + n;
  __nv_bfloat16 *pre = static_cast<__nv_bfloat16 *>(e.pre) + m0 * e.N + n;
#pragma unroll 1
  for (int k = 0; k < rows; k += kRows) {
    float v[kRows];
    __nv_bfloat16 r[kRows];
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < kRows; ++i, res += e.ldr)
        if (k + i < rows) r[i] = *res;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i] = stage[(k + i) * kPitch + lane];
    if (e.x_scale) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        if (k + i < rows) v[i] *= e.x_scale[m0 + k + i] * sw;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i] += bias;
    if (e.pre) {
#pragma unroll
      for (int i = 0; i < kRows; ++i, pre += e.N)
        if (k + i < rows) *pre = __float2bfloat16_rn(v[i]);
    }
    if (e.act != kActNone) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) v[i] = linear::activate(e.act, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i, out += e.N)
      if (k + i < rows) *out = __float2bfloat16_rn(v[i] + (e.residual ? __bfloat162float(r[i]) : 0.f));
  }
}

// The gated form (kGlu): a tile's left half of columns are rows of w's gate half, its
// right half the same rows of the other half, so that one thread finds both in its row
// of TMEM: out = act(g + bg) (u + bu), pre [M][2 N] = g + bg beside u + bu.
// One chunk of one row; cols: the chunk's biases, the gate's [32] and the other's [32].
__device__ __forceinline__ void finish_row_glu(const LinearArgs &e, int64_t m, int64_t n0, const uint32_t (&g)[32],
                                               const uint32_t (&u)[32], const float *cols, bool wide) {
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e.out) + m * e.N + n0;
  __nv_bfloat16 *pre = static_cast<__nv_bfloat16 *>(e.pre) + m * 2 * e.N + n0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint4 po[2], pg[2], pu[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8], w[8], q[8];
      const int at = 16 * k + 8 * h;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(g[at + i]), w[i] = __uint_as_float(u[at + i]);
      if (e.bias) {
        load8(cols + at, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += q[i];
        load8(cols + 32 + at, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] += q[i];
      }
      pg[h] = narrow8(v), pu[h] = narrow8(w);
      activate8(e, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= w[i];
      po[h] = narrow8(v);
    }
    if (n0 + 16 * k + 16 <= e.N) {
      if (e.pre) {
        store16(pre + 16 * k, pg[0], pg[1], wide);
        store16(pre + e.N + 16 * k, pu[0], pu[1], wide);
      }
      store16(out + 16 * k, po[0], po[1], wide);
    } else if (n0 + 16 * k + 8 <= e.N) {
      if (e.pre) {
        *reinterpret_cast<uint4 *>(pre + 16 * k) = pg[0];
        *reinterpret_cast<uint4 *>(pre + e.N + 16 * k) = pu[0];
      }
      *reinterpret_cast<uint4 *>(out + 16 * k) = po[0];
    }
  }
}
// The same where rows are not whole 16-byte pieces: what each lane has of its row is
// turned through shared memory, and a lane stores one column of all 32 rows.
__device__ __forceinline__ void finish_columns_glu(const LinearArgs &e, float *stage, int lane, int64_t m0, int64_t n0,
                                                   uint32_t (&g)[32], uint32_t (&u)[32]) {
  const int64_t n = n0 + lane;
  const float bg = n < e.N ? linear::bias_at(e, n) : 0.f, bu = n < e.N ? linear::bias_at(e, e.N + n) : 0.f;
  const int rows = e.M - m0 < 32 ? (int)(e.M - m0) : 32;
  const auto turn = [&](const uint32_t(&r)[32]) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<uint4 *>(stage + lane * kPitch + 4 * k) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
    __syncwarp();
  };
  // after this g and u are this lane's column
  turn(g);
#pragma unroll
  for (int r = 0; r < 32; ++r) g[r] = __float_as_uint(stage[r * kPitch + lane] + bg);
  turn(u);
#pragma unroll
  for (int r = 0; r < 32; ++r) u[r] = __float_as_uint(stage[r * kPitch + lane] + bu);
  if (n >= e.N) return;
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e.out) + m0 * e.N + n;
  __nv_bfloat16 *pre = static_cast<__nv_bfloat16 *>(e.pre) + m0 * 2 * e.N + n;
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    if (r >= rows) break;
    const float a = __uint_as_float(g[r]), b = __uint_as_float(u[r]);
    if (e.pre) {
      pre[(int64_t)r * 2 * e.N] = __float2bfloat16_rn(a);
      pre[(int64_t)r * 2 * e.N + e.N] = __float2bfloat16_rn(b);
    }
    out[(int64_t)r * e.N] = __float2bfloat16_rn(linear::activate(e.act, a) * b);
  }
}

// A tile whose k was shared by `split` CTAs of the cluster, `apart` ranks from
// one another: each has its float32 sums in its own shared memory ([kBM] rows
// of BN + 4), and finishes 1 / split of the rows, adding in rank order.
template <int BN>
__device__ __forceinline__ void finish_split(const LinearArgs &e, const float *sums, int split, int apart, int rank,
                                             int64_t m0, int64_t n0, bool aligned) {
  const int rows = kBM / split, mine = rank / apart, first = rank % apart;
  for (int i = threadIdx.x; i < rows * (BN / 8); i += kThreads) {
    const int r = mine * rows + i / (BN / 8), c = i % (BN / 8) * 8;
    const int64_t row = m0 + r, n = n0 + c;
    if (row >= e.M || n >= e.N) continue;
    uint4 res = make_uint4(0, 0, 0, 0);
    if (aligned && e.residual)
      res = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(e.residual) + row * e.ldr + n);
    // all parts are asked for before any is added: a read takes about a microsecond
    float4 a[kMaxSplit], b[kMaxSplit];
#pragma unroll
    for (int q = 0; q < kMaxSplit; ++q)
      if (q < split) {
        const uint32_t at = map_cluster(sums + r * (BN + 4) + c, first + q * apart);
        a[q] = ld_cluster_f4(at);
        b[q] = ld_cluster_f4(at + 16);
      }
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kMaxSplit; ++q)
      if (q < split) {
        v[0] += a[q].x, v[1] += a[q].y, v[2] += a[q].z, v[3] += a[q].w;
        v[4] += b[q].x, v[5] += b[q].y, v[6] += b[q].z, v[7] += b[q].w;
      }
    if (aligned) {
      raise8(e, n, v, e.x_scale ? e.x_scale[row] : 1.f);
      if (e.pre) *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(e.pre) + row * e.N + n) = narrow8(v);
      activate8(e, v);
      if (e.residual) add8(v, res);
      *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(e.out) + row * e.N + n) = narrow8(v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j < e.N) linear::finish<__nv_bfloat16>(e, row, n + j, v[j]);
    }
  }
}

// The same for the gated form: 8 columns of either half a thread.
template <int BN>
__device__ __forceinline__ void finish_split_glu(const LinearArgs &e, const float *sums, int split, int apart, int rank,
                                                 int64_t m0, int64_t n0, bool aligned) {
  const int rows = kBM / split, mine = rank / apart, first = rank % apart;
  for (int i = threadIdx.x; i < rows * (BN / 16); i += kThreads) {
    const int r = mine * rows + i / (BN / 16), c = i % (BN / 16) * 8;
    const int64_t row = m0 + r, n = n0 + c;
    if (row >= e.M || n >= e.N) continue;
    float v[2][8] = {};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float4 a[kMaxSplit], b[kMaxSplit];
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (q < split) {
          const uint32_t at = map_cluster(sums + r * (BN + 4) + half * (BN / 2) + c, first + q * apart);
          a[q] = ld_cluster_f4(at);
          b[q] = ld_cluster_f4(at + 16);
        }
#pragma unroll
      for (int q = 0; q < kMaxSplit; ++q)
        if (q < split) {
          v[half][0] += a[q].x, v[half][1] += a[q].y, v[half][2] += a[q].z, v[half][3] += a[q].w;
          v[half][4] += b[q].x, v[half][5] += b[q].y, v[half][6] += b[q].z, v[half][7] += b[q].w;
        }
    }
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (n + j < e.N) v[0][j] += linear::bias_at(e, n + j), v[1][j] += linear::bias_at(e, e.N + n + j);
      o[j] = linear::activate(e.act, v[0][j]) * v[1][j];
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e.out) + row * e.N + n;
    __nv_bfloat16 *pre = static_cast<__nv_bfloat16 *>(e.pre) + row * 2 * e.N + n;
    if (aligned) {
      if (e.pre) {
        *reinterpret_cast<uint4 *>(pre) = narrow8(v[0]);
        *reinterpret_cast<uint4 *>(pre + e.N) = narrow8(v[1]);
      }
      *reinterpret_cast<uint4 *>(out) = narrow8(o);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (n + j >= e.N) continue;
        if (e.pre) pre[j] = __float2bfloat16_rn(v[0][j]), pre[e.N + j] = __float2bfloat16_rn(v[1][j]);
        out[j] = __float2bfloat16_rn(o[j]);
      }
    }
  }
}

template <int BN, bool kPair, bool kSplit, bool kAMn, bool kBMn, bool kF8, bool kGlu>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                Tiles tiles, LinearArgs epi, bool aligned, bool wide) {
  constexpr int kStages = stages(BN, kPair), kStage = stage_bytes(BN, kPair), kBRows = b_rows(BN, kPair);
  constexpr int kTM = kPair ? 2 * kBM : kBM;             // rows of a tile
  constexpr int kOut = kGlu ? BN / 2 : BN;               // columns of the output that a tile gives
  constexpr int kElems = kF8 ? 128 : 64;                 // of k in a stage
  constexpr uint32_t kCols = 2 * BN < 32 ? 32 : 2 * BN;  // TMEM columns: two accumulators
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  // swizzle atoms are 1024-byte aligned
  unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kWide = kPair ? 2 : 1;                   // CTAs of a tile, for one part of k
  const int crank = kPair || kSplit ? (int)cluster_rank() : 0;
  const int rank = crank % kWide, lead = crank - rank;   // rank 0 issues the products
  const int ctas = kSplit ? kWide * tiles.split : kWide;
  const int64_t worker = blockIdx.x / ctas, workers = gridDim.x / ctas;
  const int kb0 = kSplit ? crank / kWide * tiles.per : 0;
  const int kb1 = kSplit && kb0 + tiles.per < tiles.kblocks ? kb0 + tiles.per : tiles.kblocks;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.tfull[i], 1), mbar_init(&sh.tempty[i], kPair ? 2 * kEpi : kEpi);
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(&sh.tmem, kCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sh.tmem, kCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair || kSplit) cluster_sync();  // barriers and TMEM of all its CTAs are ready
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // (and no chain_next(): a next product's CTA could take tensor memory that a
  // CTA of this one has yet to ask for)
  chain_wait();

  // The producer's and the issuer's loops run warp-wide, with one elected lane
  // issuing: in code that only one lane reaches, the compiler cannot keep
  // descriptors and addresses in uniform registers.
  if (warp == 0) {
    if (elect_one()) {
      tma_prefetch_desc(&ma);
      tma_prefetch_desc(&mb);
    }
    int slot = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t i = worker; ok && i < tiles.total; i += workers) {
      int64_t tm, tn;
      tile_at(tiles, i, tm, tn);
      // (gated: w's halves are tiles' halves, so a pair's second CTA has the second)
      const int m0 = (int)(tm * kTM) + rank * kBM;
      const int n0 = (int)(tn * kOut) + rank * (kGlu ? (int)epi.N : kBRows);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = __all_sync(0xffffffffu, wait(&sh, &sh.empty[slot], phase ^ 1, 0)))) break;
        if (elect_one()) {
          unsigned char *st = base + slot * kStage, *stb = st + kBM * kRowBytes;
          // a pair's copies all count on the leader's barrier
          const uint32_t bar = kPair ? map_cluster(&sh.full[slot], lead) : 0;
          const auto copy = [&](unsigned char *to, const CUtensorMap *map, int c0, int c1) {
            if constexpr (kPair)
              tma_load_2d_pair(to, map, bar, c0, c1);
            else
              tma_load_2d(to, map, &sh.full[slot], c0, c1);
          };
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[slot], kPair ? 2 * kStage : kStage);
          if constexpr (kAMn) {
#pragma unroll
            for (int j = 0; j < kBM / 64; ++j) copy(st + j * 8192, &ma, m0 + 64 * j, kb * 64);
          } else {
            copy(st, &ma, kb * kElems, m0);
          }
          if constexpr (kBMn) {
#pragma unroll
            for (int j = 0; j < kBRows / 64; ++j) copy(stb + j * 8192, &mb, n0 + 64 * j, kb * 64);
          } else if constexpr (kGlu && !kPair) {
            copy(stb, &mb, kb * kElems, n0);
            copy(stb + kOut * kRowBytes, &mb, kb * kElems, (int)epi.N + n0);
          } else {
            copy(stb, &mb, kb * kElems, n0);
          }
        }
        __syncwarp();
        ++issued;
        if (++slot == kStages) slot = 0, phase ^= 1;
      }
    }
    if (!ok && rank != 0) {  // winding down: this warp's own copies land first
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);  // (the leader's barrier counts them)
    } else if (!ok) {
      for (int64_t i = issued < kStages ? 0 : issued - kStages; i < issued; ++i)
        for (uint32_t j = 0; j < (1u << 20) && !mbar_try_wait(&sh.full[i % kStages], (i / kStages) & 1); ++j) {
        }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t id = kF8 ? idesc_e4m3(kTM, BN) : idesc_bf16(kTM, BN, kAMn, kBMn);
      const auto commit = [&](uint64_t *bar) {
        if constexpr (kPair)
          mma_commit_pair(bar, (uint16_t)(3 << lead));
        else
          mma_commit(bar);
      };
      int slot = 0, acc = 0;
      uint32_t phase = 0, accphase = 0;
      bool ok = true;
      for (int64_t i = worker; ok && i < tiles.total; i += workers) {
        if (!(ok = __all_sync(0xffffffffu, wait(&sh, &sh.tempty[acc], accphase ^ 1, 1)))) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = __all_sync(0xffffffffu, wait(&sh, &sh.full[slot], phase, 1)))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t st = smem_u32(base + slot * kStage);
            // k-contiguous operands: a step of 16 (32) elements is 32 bytes of
            // the 128-byte row; MN-major ones: 16 rows of 128 bytes
            const uint64_t da = kAMn ? sdesc_sw128(st, 8192, 1024) : sdesc_sw128(st, 0, 1024);
            const uint64_t db = kBMn ? sdesc_sw128(st + kBM * kRowBytes, 8192, 1024)
                                     : sdesc_sw128(st + kBM * kRowBytes, 0, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t xa = da + (uint64_t)(k * (kAMn ? 2048 : 32) >> 4);
              const uint64_t xb = db + (uint64_t)(k * (kBMn ? 2048 : 32) >> 4);
              if constexpr (kPair)
                mma_ss_pair<kF8>(d, xa, xb, id, kb > kb0 || k > 0);
              else if constexpr (kF8)
                mma_ss_f8(d, xa, xb, id, kb > kb0 || k > 0);
              else
                mma_ss(d, xa, xb, id, kb > kb0 || k > 0);
            }
            commit(&sh.empty[slot]);
            if (kb + 1 == kb1) commit(&sh.tfull[acc]);
          }
          __syncwarp();
          if (++slot == kStages) slot = 0, phase ^= 1;
        }
        acc ^= 1;
        if (acc == 0) accphase ^= 1;
      }
      if (!ok) {  // products in flight end before TMEM is given back
        if (elect_one()) commit(&sh.drain);
        for (uint32_t j = 0; j < (1u << 20) && !mbar_try_wait(&sh.drain, 0); ++j) {
        }
      }
    }
  } else {
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const int half = (warp - 2) / 4;  // of the columns: every second chunk of 32
    float *stage = reinterpret_cast<float *>(base + kStages * kStage + (warp - 2) * kEpiBytes);
    int acc = 0;
    uint32_t accphase = 0;
    for (int64_t i = worker; i < tiles.total; i += workers) {
      int64_t tm, tn;
      tile_at(tiles, i, tm, tn);
      const int64_t m0 = tm * kTM + rank * kBM + quarter * 32, m = m0 + lane, n0 = tn * kOut;
      const int chunks = (int)(epi.N - n0 < kOut ? (epi.N - n0 + 31) / 32 : kOut / 32);
      // what a chunk needs from memory is asked for a chunk ahead; a lane has
      // the bias and scale of one column, which shared memory hands to all
      const bool rows = aligned && !kSplit;
      float sx = 1.f, bias = 0.f, sw = 0.f;
      Residual now, next;
      const auto ask = [&](int c) {
        if (!rows || c >= chunks) return;
        if constexpr (!kGlu) ask_residual(epi, m, n0 + c * 32, wide, next);
        const int64_t n = n0 + c * 32 + lane;
        if (n < epi.N) {
          bias = linear::bias_at(epi, n);
          if constexpr (kGlu)
            sw = linear::bias_at(epi, epi.N + n);  // (the other half's)
          else if (epi.x_scale)
            sw = epi.w_scale[n];
        }
      };
      if (rows && epi.x_scale && m < epi.M) sx = epi.x_scale[m];
      ask(half);
      if (!__all_sync(0xffffffffu, wait(&sh, &sh.tfull[acc], accphase, 2))) break;
      tc_fence_after();
      // this warp's part of the accumulator has been read: the products may
      // overwrite it.  Nothing but TMEM is handed over, and the fence orders that.
      const auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kPair)
            mbar_arrive_cluster_relaxed(map_cluster(&sh.tempty[acc], lead));
          else
            mbar_arrive(&sh.tempty[acc]);
        }
      };
      uint32_t r[32], r2[kGlu ? 32 : 1];
#pragma unroll 1
      for (int c = half; c < chunks; c += 2) {
        tmem_ld32(tmem_addr(tmem, quarter * 32, acc * BN + c * 32), r);
        if constexpr (kGlu) tmem_ld32(tmem_addr(tmem, quarter * 32, acc * BN + kOut + c * 32), r2);
        if (rows) {
          if (epi.bias) stage[lane] = bias;
          if (kGlu ? epi.bias != nullptr : epi.x_scale != nullptr) stage[32 + lane] = sw;
          __syncwarp();
          now = next;
          ask(c + 2);
        }
        tmem_wait_ld_regs(r);
        if constexpr (kGlu) tmem_wait_ld_regs(r2);
        if (c + 2 >= chunks) release();
        if constexpr (kSplit) {  // the one tile: its sums to shared memory, where the ring was
          float *row = reinterpret_cast<float *>(base) + (quarter * 32 + lane) * (BN + 4) + c * 32;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(row + 4 * k) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
          if constexpr (kGlu) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4 *>(row + kOut + 4 * k) =
                  make_uint4(r2[4 * k], r2[4 * k + 1], r2[4 * k + 2], r2[4 * k + 3]);
          }
        } else if constexpr (kGlu) {
          if (!aligned)
            finish_columns_glu(epi, stage, lane, m0, n0 + c * 32, r, r2);
          else if (m < epi.M)
            finish_row_glu(epi, m, n0 + c * 32, r, r2, stage, wide);
        } else if (aligned) {
          if (m < epi.M) finish_row(epi, m, n0 + c * 32, r, sx, stage, now, wide);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(stage + lane * kPitch + 4 * k) =
                make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
          __syncwarp();
          finish_column(epi, stage, lane, m0, n0 + c * 32 + lane);
        }
        __syncwarp();
      }
      if (half >= chunks) release();
      acc ^= 1;
      if (acc == 0) accphase ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (kSplit) {
    cluster_sync();
    int64_t tm, tn;
    tile_at(tiles, worker, tm, tn);
    (kGlu ? finish_split_glu<BN> : finish_split<BN>)(epi, reinterpret_cast<const float *>(base), tiles.split, kWide,
                                                     crank, tm * kTM + rank * kBM, tn * kOut, aligned);
  }
  if constexpr (kPair || kSplit) cluster_sync_relaxed();  // no CTA leaves while another may reach into it
  tc_fence_after();
  if (warp == 1) {
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, kCols);
    else
      tmem_dealloc(tmem, kCols);
  }
}

int sm_count() {
  int dev = 0, n = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

template <int BN, bool kPair, bool kSplit, bool kAMn, bool kBMn, bool kF8, bool kGlu>
cudaError_t run(const GemmArgs &g, int split, cudaStream_t s) {
  constexpr int kOut = kGlu ? BN / 2 : BN;
  const int size = kF8 ? 1 : 2;
  const LinearArgs &e = g.epi;
  CUtensorMap ma, mb;
  cudaError_t err;
  err = kAMn ? make_map_2d_sw128(&ma, g.a, (uint64_t)e.M, (uint64_t)g.K, (uint64_t)g.lda, size, 64)
             : make_map_2d_sw128(&ma, g.a, (uint64_t)g.K, (uint64_t)e.M, (uint64_t)g.lda, size, kBM);
  if (err != cudaSuccess) return err;
  err = kBMn ? make_map_2d_sw128(&mb, g.b, (uint64_t)e.N, (uint64_t)g.K, (uint64_t)g.ldb, size, 64)
             : make_map_2d_sw128(&mb, g.b, (uint64_t)g.K, (uint64_t)(kGlu ? 2 : 1) * e.N, (uint64_t)g.ldb, size,
                                 kGlu ? kOut : b_rows(BN, kPair));
  if (err != cudaSuccess) return err;
  Tiles t;
  constexpr int kTM = kPair ? 2 * kBM : kBM;
  t.m_tiles = (e.M + kTM - 1) / kTM;
  t.n_tiles = (e.N + kOut - 1) / kOut;
  t.total = t.m_tiles * t.n_tiles;
  if (t.total >= (int64_t(1) << 31) / kMaxSplit) return cudaErrorInvalidConfiguration;
  const int elems = kF8 ? 128 : 64;
  t.kblocks = (int)((g.K + elems - 1) / elems);
  t.per = (t.kblocks + split - 1) / split;
  t.split = split;
  const auto ok = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  const bool aligned = e.N % 8 == 0 && ok(e.out) && ok(e.pre) && ok(e.residual) && (!e.residual || e.ldr % 8 == 0) &&
                       ok(e.bias) && ok(e.w_scale);
  const auto ok32 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; };
  const bool wide = aligned && e.N % 16 == 0 && ok32(e.out) && ok32(e.pre) && ok32(e.residual) &&
                    (!e.residual || e.ldr % 16 == 0);
  auto kern = gemm_kernel<BN, kPair, kSplit, kAMn, kBMn, kF8, kGlu>;
  constexpr int smem = smem_bytes(BN, kPair);
  if ((err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return err;
  const int64_t ctas = (kPair ? 2 : 1) * split, fit = sm_count() / ctas;
  // persistent, but for a split product: one cluster a tile
  return chain_launch(kern, dim3((unsigned)((kSplit || t.total < fit ? t.total : fit) * ctas)), dim3(kThreads), smem,
                      (int)ctas, g.dependent, s, ma, mb, t, e, aligned, wide);
}

template <int BN, bool kPair, bool kAMn, bool kBMn, bool kF8, bool kGlu>
cudaError_t run(const GemmArgs &g, int split, cudaStream_t s) {
  return split > 1 ? run<BN, kPair, true, kAMn, kBMn, kF8, kGlu>(g, split, s)
                   : run<BN, kPair, false, kAMn, kBMn, kF8, kGlu>(g, 1, s);
}

// The tile and the split of k, by an estimate of the time.  A block of k takes
// 512 cycles for a pair's 256 x 256 (the tensor cores' own rate), and for the
// smaller tiles 300 to 375, what the copies take to issue and land; starting,
// filling the pipeline and writing out a tile cost about 4 us.  A split adds a
// turn through shared memory and (q - 1) / q of the tile's sums over the
// cluster's network, which carries about 20 GB/s a CTA.
struct Choice {
  int shape, split;  // shape: pair of 256, pair of 128, one CTA of 128, of 64 columns
  double us;
};
Choice choose(int64_t M, int64_t N, int64_t K, bool f8) {
  const int64_t sms = sm_count();
  const int64_t kblocks = (K + (f8 ? 127 : 63)) / (f8 ? 128 : 64);
  struct Shape { int bn, pair; double us; };
  constexpr Shape shapes[4] = {{256, 1, 0.26}, {128, 1, 0.15}, {128, 0, 0.19}, {64, 0, 0.16}};
  Choice c{0, 1, 1e30};
  for (int i = 0; i < 4; ++i) {
    const int bn = shapes[i].bn, wide = shapes[i].pair ? 2 : 1, bm = kBM * wide;
    const int64_t tiles = ((M + bm - 1) / bm) * ((N + bn - 1) / bn);
    for (int q = 1; q * wide <= kMaxSplit; q *= 2) {
      // (of clusters of 8 such CTAs only 15 are resident, of 4 only 36)
      const int64_t fit = q * wide == 8 ? 15 * 8 : q * wide == 4 ? 36 * 4 : sms;
      if (q > 1 && (tiles * q * wide > fit || kblocks < 4 * q)) break;
      if ((q - 1) * ((kblocks + q - 1) / q) >= kblocks) continue;  // every part has blocks
      const int64_t rounds = (tiles * q * wide + sms - 1) / sms;
      double us = (double)rounds * ((kblocks + q - 1) / q * shapes[i].us + bn * 0.005) + 3.0;
      if (q > 1) us += 1.3 + kBM * bn * 4 * (q - 1) / q / 20e3;
      if (us < 0.98 * c.us) c = Choice{i, q, us};
    }
  }
  return c;
}

template <bool kAMn, bool kBMn, bool kF8, bool kGlu = false>
cudaError_t pick(const GemmArgs &g, cudaStream_t s) {
  const Choice c = choose(g.epi.M, (kGlu ? 2 : 1) * g.epi.N, g.K, kF8);
  const int best = c.shape, split = c.split;
  switch (best) {
    case 0: return run<256, true, kAMn, kBMn, kF8, kGlu>(g, split, s);
    case 1: return run<128, true, kAMn, kBMn, kF8, kGlu>(g, split, s);
    case 2: return run<128, false, kAMn, kBMn, kF8, kGlu>(g, split, s);
    default: return run<64, false, kAMn, kBMn, kF8, kGlu>(g, split, s);
  }
}

// ------------------------------------------------------- both gradients at once
// dx and dw are two products whose tiles fill the last of their rounds badly (M4096
// K2048, 8192 rows of w: 1.7 and 3.4 rounds of 76 pairs), and one's tiles take longer than
// the other's, N and M long.  In one launch the pairs take the long tiles in turn, and
// then as many of the short ones as evens out what they have: those with one long tile
// fewer `extra` more, before the rest goes round.  A tile's sums are in the order that it
// has in a launch of its own.  After a second's rest, from graphs, the gated layer's
// gradients at M4096 N4096 K2048 take 170 us for 186, the linear layer's 98 for 104, at
// M2048 N8192 91 for 105; the gated ones as calls back to back, the clock down with power,
// 193 for 201.
struct Product {
  Tiles tiles;
  LinearArgs epi;
  bool aligned, wide, a_mn;
};
struct Deal {
  uint32_t workers, fewer, extra, total[2];  // the first `workers - fewer` have a long tile more
};
// the n-th task of a worker: which product, which tile
__device__ __forceinline__ bool task(const Deal &d, uint32_t w, uint32_t n, int &which, uint32_t &tile) {
  which = 0, tile = w + n * d.workers;
  if (tile < d.total[0]) return true;
  n -= w < d.total[0] ? (d.total[0] - w + d.workers - 1) / d.workers : 0u;
  which = 1;
  const uint32_t more = d.workers - d.fewer;
  if (w >= more) {
    if (n < d.extra) return (tile = n * d.fewer + (w - more)) < d.total[1];
    n -= d.extra;
  }
  return (tile = d.extra * d.fewer + n * d.workers + w) < d.total[1];
}

__global__ void __launch_bounds__(kThreads, 1)
    gradients_kernel(const __grid_constant__ CUtensorMap ma0, const __grid_constant__ CUtensorMap mb0,
                     const __grid_constant__ CUtensorMap ma1, const __grid_constant__ CUtensorMap mb1,
                     const __grid_constant__ Product p0, const __grid_constant__ Product p1, Deal deal) {
  constexpr int BN = 256, kStages = stages(BN, true), kStage = stage_bytes(BN, true);
  constexpr uint32_t kCols = 2 * BN;
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const uint32_t worker = blockIdx.x / 2;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.tfull[i], 1), mbar_init(&sh.tempty[i], 2 * kEpi);
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&sh.tmem, kCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  chain_wait();
  int which;
  uint32_t tile;

  // (roles and waits as in gemm_kernel)
  if (warp == 0) {
    int slot = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (uint32_t n = 0; ok && task(deal, worker, n, which, tile); ++n) {
      const Product &p = which ? p1 : p0;
      const CUtensorMap *ma = which ? &ma1 : &ma0, *mb = which ? &mb1 : &mb0;
      int64_t tm, tn;
      tile_at(p.tiles, tile, tm, tn);
      const int m0 = (int)(tm * 256) + rank * kBM, n0 = (int)(tn * BN) + rank * (BN / 2), kblocks = p.tiles.kblocks;
      const bool a_mn = p.a_mn;
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!(ok = __all_sync(0xffffffffu, wait(&sh, &sh.empty[slot], phase ^ 1, 0)))) break;
        if (elect_one()) {
          unsigned char *st = base + slot * kStage, *stb = st + kBM * kRowBytes;
          const uint32_t bar = map_cluster(&sh.full[slot], 0);
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[slot], 2 * kStage);
          if (a_mn) {
            tma_load_2d_pair(st, ma, bar, m0, kb * 64);
            tma_load_2d_pair(st + 8192, ma, bar, m0 + 64, kb * 64);
          } else {
            tma_load_2d_pair(st, ma, bar, kb * 64, m0);
          }
          tma_load_2d_pair(stb, mb, bar, n0, kb * 64);
          tma_load_2d_pair(stb + 8192, mb, bar, n0 + 64, kb * 64);
        }
        __syncwarp();
        ++issued;
        if (++slot == kStages) slot = 0, phase ^= 1;
      }
    }
    if (!ok && rank != 0) {
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    } else if (!ok) {
      for (int64_t i = issued < kStages ? 0 : issued - kStages; i < issued; ++i)
        for (uint32_t j = 0; j < (1u << 20) && !mbar_try_wait(&sh.full[i % kStages], (i / kStages) & 1); ++j) {
        }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      int slot = 0, acc = 0;
      uint32_t phase = 0, accphase = 0;
      bool ok = true;
      for (uint32_t n = 0; ok && task(deal, worker, n, which, tile); ++n) {
        const Product &p = which ? p1 : p0;
        const int kblocks = p.tiles.kblocks;
        const bool a_mn = p.a_mn;
        const uint32_t id = a_mn ? idesc_bf16(256, BN, true, true) : idesc_bf16(256, BN, false, true);
        const uint64_t step = (a_mn ? 2048 : 32) >> 4;
        if (!(ok = __all_sync(0xffffffffu, wait(&sh, &sh.tempty[acc], accphase ^ 1, 1)))) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!(ok = __all_sync(0xffffffffu, wait(&sh, &sh.full[slot], phase, 1)))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t st = smem_u32(base + slot * kStage);
            const uint64_t da = sdesc_sw128(st, a_mn ? 8192 : 0, 1024), db = sdesc_sw128(st + kBM * kRowBytes, 8192, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss_pair<false>(d, da + k * step, db + (uint64_t)(k * 2048 >> 4), id, kb > 0 || k > 0);
            mma_commit_pair(&sh.empty[slot], 3);
            if (kb + 1 == kblocks) mma_commit_pair(&sh.tfull[acc], 3);
          }
          __syncwarp();
          if (++slot == kStages) slot = 0, phase ^= 1;
        }
        acc ^= 1;
        if (acc == 0) accphase ^= 1;
      }
      if (!ok) {
        if (elect_one()) mma_commit_pair(&sh.drain, 3);
        for (uint32_t j = 0; j < (1u << 20) && !mbar_try_wait(&sh.drain, 0); ++j) {
        }
      }
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) / 4;
    float *stage = reinterpret_cast<float *>(base + kStages * kStage + (warp - 2) * kEpiBytes);
    int acc = 0;
    uint32_t accphase = 0;
    for (uint32_t n = 0; task(deal, worker, n, which, tile); ++n) {
      const Product &p = which ? p1 : p0;
      const LinearArgs &epi = p.epi;
      int64_t tm, tn;
      tile_at(p.tiles, tile, tm, tn);
      const int64_t m0 = tm * 256 + rank * kBM + quarter * 32, m = m0 + lane, n0 = tn * BN;
      const int chunks = (int)(epi.N - n0 < BN ? (epi.N - n0 + 31) / 32 : BN / 32);
      if (!__all_sync(0xffffffffu, wait(&sh, &sh.tfull[acc], accphase, 2))) break;
      tc_fence_after();
      const auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(map_cluster(&sh.tempty[acc], 0));
      };
      uint32_t r[32];
#pragma unroll 1
      for (int c = half; c < chunks; c += 2) {
        tmem_ld32(tmem_addr(tmem, quarter * 32, acc * BN + c * 32), r);
        tmem_wait_ld_regs(r);
        if (c + 2 >= chunks) release();
        if (p.aligned) {
          if (m < epi.M) finish_row(epi, m, n0 + c * 32, r, 1.f, stage, Residual{}, p.wide);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(stage + lane * kPitch + 4 * k) =
                make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
          __syncwarp();
          finish_column(epi, stage, lane, m0, n0 + c * 32 + lane);
        }
        __syncwarp();
      }
      if (half >= chunks) release();
      acc ^= 1;
      if (acc == 0) accphase ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();  // no CTA leaves while another may reach into it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kCols);
}

// Tiles of 256 x 256, their blocks of k and what one takes (as in choose())
struct Whole {
  int64_t tiles;
  double us;
};
Whole whole_of(int64_t M, int64_t N, int64_t K) {
  return {((M + 255) / 256) * ((N + 255) / 256), (double)((K + 63) / 64) * 0.26 + 256 * 0.005};
}
// The least time in which `workers` finish a's tiles, in turn, and then b's (each no
// longer), and how many more of b's those with a tile of a's fewer take.
double deal_out(const Whole &a, const Whole &b, int64_t workers, Deal &d) {
  const int64_t more = a.tiles % workers, fewer = workers - more, each = a.tiles / workers;
  d.workers = (uint32_t)workers, d.fewer = (uint32_t)fewer;
  d.total[0] = (uint32_t)a.tiles, d.total[1] = (uint32_t)b.tiles;
  int64_t extra = more ? (int64_t)(a.us / b.us) : 0;
  if (extra * fewer > b.tiles) extra = b.tiles / fewer;
  double best = 1e30;
  for (int64_t x = extra; x <= extra + (more ? 2 : 0); ++x) {
    const int64_t rest = b.tiles - x * fewer > 0 ? b.tiles - x * fewer : 0, rounds = rest / workers, left = rest % workers;
    // (what is left of the rounds goes to the first: those with a tile more, if there are any)
    const double first = (each + (more ? 1 : 0)) * a.us + (rounds + (left > 0)) * b.us;
    const double others = each * a.us + (x + rounds + (left > more)) * b.us;
    const double us = first > others ? first : others;
    if (us < best) best = us, d.extra = (uint32_t)x;
  }
  return best;
}

}  // namespace

bool gradients_fit(const GemmArgs &x, const GemmArgs &w) {
  const Choice a = choose(x.epi.M, x.epi.N, x.K, false), b = choose(w.epi.M, w.epi.N, w.K, false);
  // (parts of k, or other tiles, would be other sums than a product by itself has)
  if (a.shape != 0 || b.shape != 0 || a.split != 1 || b.split != 1) return false;
  Whole p = whole_of(x.epi.M, x.epi.N, x.K), q = whole_of(w.epi.M, w.epi.N, w.K);
  if (p.tiles + q.tiles >= (int64_t(1) << 30)) return false;
  Deal d;
  return deal_out(p.us >= q.us ? p : q, p.us >= q.us ? q : p, sm_count() / 2, d) + 3.0 < 0.97 * (a.us + b.us + 0.7);
}

cudaError_t launch_gradients_tc(const GemmArgs &x, const GemmArgs &w, cudaStream_t s) {
  const Whole px = whole_of(x.epi.M, x.epi.N, x.K), pw = whole_of(w.epi.M, w.epi.N, w.K);
  const bool first = px.us >= pw.us;  // dx has the longer tiles
  const GemmArgs *g[2] = {first ? &x : &w, first ? &w : &x};
  Deal d{};
  deal_out(first ? px : pw, first ? pw : px, sm_count() / 2, d);
  CUtensorMap ma[2], mb[2];
  Product p[2];
  for (int i = 0; i < 2; ++i) {
    const LinearArgs &e = g[i]->epi;
    cudaError_t err = g[i]->a_mn ? make_map_2d_sw128(&ma[i], g[i]->a, (uint64_t)e.M, (uint64_t)g[i]->K, (uint64_t)g[i]->lda, 2, 64)
                                 : make_map_2d_sw128(&ma[i], g[i]->a, (uint64_t)g[i]->K, (uint64_t)e.M, (uint64_t)g[i]->lda, 2, kBM);
    if (err == cudaSuccess) err = make_map_2d_sw128(&mb[i], g[i]->b, (uint64_t)e.N, (uint64_t)g[i]->K, (uint64_t)g[i]->ldb, 2, 64);
    if (err != cudaSuccess) return err;
    Tiles &t = p[i].tiles;
    t.m_tiles = (e.M + 255) / 256, t.n_tiles = (e.N + 255) / 256, t.total = t.m_tiles * t.n_tiles;
    t.kblocks = (int)((g[i]->K + 63) / 64), t.split = 1, t.per = t.kblocks;
    p[i].epi = e, p[i].a_mn = g[i]->a_mn;
    p[i].aligned = e.N % 8 == 0 && reinterpret_cast<uintptr_t>(e.out) % 16 == 0;
    p[i].wide = p[i].aligned && e.N % 16 == 0 && reinterpret_cast<uintptr_t>(e.out) % 32 == 0;
  }
  constexpr int smem = smem_bytes(256, true);
  const cudaError_t err = cudaFuncSetAttribute(gradients_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  return chain_launch(gradients_kernel, dim3(d.workers * 2), dim3(kThreads), smem, 2, x.dependent, s, ma[0], mb[0], ma[1],
                      mb[1], p[0], p[1], d);
}

double gemm_tc_us(int64_t M, int64_t N, int64_t K, bool f8) { return choose(M, N, K, f8).us + 0.7; }

cudaError_t launch_gemm_tc(const GemmArgs &g, cudaStream_t s) {
  if (g.epi.kind == kLinE4m3) return g.a_mn || g.b_mn ? cudaErrorNotSupported : pick<false, false, true>(g, s);
  if (!g.a_mn) return g.b_mn ? pick<false, true, false>(g, s) : pick<false, false, false>(g, s);
  return g.b_mn ? pick<true, true, false>(g, s) : cudaErrorNotSupported;
}

cudaError_t launch_glu_tc(const GemmArgs &g, cudaStream_t s) { return pick<false, false, false, true>(g, s); }

cudaError_t read_and_clear_linear_error(unsigned int *word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_linear_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(unsigned int));
}

}  // namespace delta
