// decay_tc.cu -- the pass of linear attention with a decay g for each head
// (decay.cu has the formulas) on the 5th-generation tensor cores: bfloat16, up to
// 128 key channels, value channels in groups of up to 128.
//
// A CTA takes a segment of one head in chunks of C = 128 tokens.  Five products a
// chunk, float32 in TMEM:
//
//   G  = Q K^T                      SS  M = tokens,  N = tokens,  K = dk
//   dS = K'^T V  (hi, then lo)      TS  M = dk,      N = dv,      K = tokens
//   O  = Q S                        SS  M = tokens,  N = dv,      K = dk
//   O += P V                        TS  M = tokens,  N = dv,      K = tokens
//
// K' is k_j g^(n-1-j) (in reverse g^(j+1)) in two bfloat16 parts, hi + lo, which
// hold it to 2^-16: the states are float32 and returned as such, and with hi alone
// they would be off by 1e-3.  P and the copy of S that O reads are single bfloat16:
// each is off by 2^-8 at most, at random, as the rounding of out itself.
//
// Both parts of O share one accumulator: with c_p the factor of S's part (g^(p+1),
// in reverse g^(n-1-p)), P is formed as G_pj g^|p-j| / c_p and the whole row is
// multiplied by c_p when it goes out.  c_p is taken no lower than 2^-100, so the
// quotient stays in range for any g; where that matters S's part is below 2^-100 of S.
//
// The state is float32 in registers, a row of dk a lane; what the chain from chunk
// to chunk costs is dS -> registers -> bfloat16 S in shared memory -> O.  All else
// (G, P, K', loads, stores) is work ahead of or behind it.
//
// Shared memory, 224 KB: two tiles each of Q, K and V (32 KB, 128-byte swizzle, as
// two blocks of 64 channels), S.  A finished O is staged where its Q was and leaves
// by TMA.  TMEM, all 512 columns: G (then P, packed over it), O, dS, K' hi and lo.
//
// Warps (640 threads):
//   0      TMA producer
//   1      issues the products
//   2      TMEM; stores finished tiles
//   4-7    P from G
//   8-11   K' from K, transposed on the way to TMEM; O to the staging tile
//   12-19  the state: 64 value columns each half
//
// Bound by HBM: 4 tensors of 32 KB a chunk.  Every mbarrier wait is bounded: a
// timeout sets a device error word and the kernel winds down.
#include <cuda_bf16.h>

#include "chain.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace delta {
namespace {

using namespace sm100;

__device__ unsigned int g_decay_error = 0;

constexpr int kC = kDecayChunk, kD = 128;
constexpr int kThreads = 640;
constexpr uint32_t kTile = 32768, kBlk = 16384;
constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffS = 6 * kTile;
constexpr int kSmem = 7 * kTile + 1024;
// TMEM columns
constexpr uint32_t kG = 0, kO = 128, kDs = 256, kHi = 384, kLo = 448;
constexpr float kFloor = -100.f;   // log2 of the least c_p
constexpr float kLogZero = -200.f; // log2 g of g = 0: any power of it vanishes, also over c_p

struct TcPass {
  CUtensorMap q, k, v, out;
  const float *init;
  float *final;
  __nv_bfloat16 *to;  // out
  float os, kvs;
  int dk, dv;
  bool reverse, init_t;
};
struct TcArgs {
  TcPass pass[3];
  int passes, groups, nseg;
  const float *decay;
  const int *lengths;
  int T, H, seg;
};

struct Shared {
  uint64_t qfull[2], qempty[2], kfull[2], kempty[2], vfull[2], vempty[2], staged[2];
  uint64_t gfull, pfull, ofull, oempty, dsfull, dsempty, kpfull, sfull, sempty, drain;
  uint32_t tmem;
  volatile int dead;
};

__device__ __noinline__ bool wait_slow(Shared *sh, uint64_t *bar, uint32_t parity, int role) {
  for (uint32_t i = 0; i < (1u << 22); ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && sh->dead) return false;
  }
  sh->dead = 1;
  atomicCAS(&g_decay_error, 0u, (unsigned)(1 + role));
  return false;
}
// by whole warps, so that they leave their loops together
__device__ __forceinline__ bool wait(Shared *sh, uint64_t *bar, uint32_t parity, int role) {
  const bool ok = mbar_try_wait(bar, parity) || wait_slow(sh, bar, parity, role);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tmem_st16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32"
      " [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// byte offset of 16-byte piece `piece` (0..7) of a row of a 64-channel block
__device__ __forceinline__ uint32_t piece_at(uint32_t row, uint32_t piece) {
  return row * 128u + ((piece ^ (row & 7u)) * 16u);
}

template <bool kStates>
__global__ void __launch_bounds__(kThreads, 1) decay_tc_kernel(const __grid_constant__ TcArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  int64_t item = blockIdx.x;
  const TcPass &p = a.pass[item % a.passes];
  item /= a.passes;
  const int sg = (int)(item % a.nseg);
  item /= a.nseg;
  const int c0 = (int)(item % a.groups) * kD;
  const int64_t bh = item / a.groups;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H);
  if (c0 >= p.dv) return;
  const int dk = p.dk, cols = min(kD, p.dv - c0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qfull[i], 1), mbar_init(&sh.qempty[i], 1);
      mbar_init(&sh.kfull[i], 1), mbar_init(&sh.kempty[i], kStates ? 4 : 5);
      mbar_init(&sh.vfull[i], 1), mbar_init(&sh.vempty[i], 1);
      mbar_init(&sh.staged[i], 4);
    }
    mbar_init(&sh.gfull, 1), mbar_init(&sh.pfull, 4), mbar_init(&sh.ofull, 1), mbar_init(&sh.oempty, 4);
    mbar_init(&sh.dsfull, 1), mbar_init(&sh.dsempty, 8), mbar_init(&sh.kpfull, 4);
    mbar_init(&sh.sfull, 8), mbar_init(&sh.sempty, 1), mbar_init(&sh.drain, 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  chain_wait();

  int len = a.lengths ? a.lengths[b] : a.T;
  len = len < 0 ? 0 : len > a.T ? a.T : len;
  const int t_lo = sg * a.seg, t_hi = min(t_lo + a.seg, a.T), t_end = min(t_hi, len);
  const int chunks = t_end > t_lo ? (t_end - t_lo + kC - 1) / kC : 0;
  const auto start_of = [&](int c) { return t_lo + (p.reverse ? chunks - 1 - c : c) * kC; };
  const float lg = fmaxf(log2f(a.decay[h]), kLogZero);
  const bool two = lg != 0.f || p.kvs != 1.f;  // else K' is K itself

  if (warp == 0) {
    bool ok = true;
    int issued = 0;
    if (elect_one()) {
      if (!kStates) tma_prefetch_desc(&p.q);
      tma_prefetch_desc(&p.k);
      tma_prefetch_desc(&p.v);
    }
    for (int c = 0; c < chunks; ++c, ++issued) {
      const int slot = c & 1, t0 = start_of(c);
      const uint32_t phase = (uint32_t)(c >> 1) & 1u ^ 1u;
      const auto load = [&](const CUtensorMap *map, uint32_t off, uint64_t *full, uint64_t *empty, int d0) {
        if (!(ok = wait(&sh, empty, phase, 0))) return;
        if (elect_one()) {
          mbar_arrive_expect_tx(full, kTile);
          tma_load_4d(base + off + slot * kTile, map, full, d0, h, t0, b);
          tma_load_4d(base + off + slot * kTile + kBlk, map, full, d0 + 64, h, t0, b);
        }
        __syncwarp();
      };
      load(&p.k, kOffK, &sh.kfull[slot], &sh.kempty[slot], 0);
      if (!kStates && ok) load(&p.q, kOffQ, &sh.qfull[slot], &sh.qempty[slot], 0);
      if (ok) load(&p.v, kOffV, &sh.vfull[slot], &sh.vempty[slot], c0);
      if (!ok) break;
    }
    // winding down: what is in flight lands first (a tile that was never asked
    // for lets its wait run out)
    if (!ok)
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  } else if (warp == 1) {
    const uint32_t nv = (uint32_t)(cols + 15) & ~15u;
    const int ksteps = (dk + 15) / 16;
    const uint32_t id_g = idesc_bf16(kC, kC, false, false), id_v = idesc_bf16(128, (int)nv, false, true);
    bool ok = true;
    // K-major: 16 channels are 32 bytes of a 128-byte row
    const auto step_k = [](int k) { return (uint64_t)((k >> 2) * kBlk + (k & 3) * 32) >> 4; };
    const auto product_g = [&](int c) {
      const int slot = c & 1;
      const uint32_t ph = (uint32_t)(c >> 1) & 1u;
      if (!(ok = wait(&sh, &sh.qfull[slot], ph, 1) && wait(&sh, &sh.kfull[slot], ph, 1))) return;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dq = sdesc_sw128(smem_u32(base + kOffQ + slot * kTile), 0, 1024);
        const uint64_t dkk = sdesc_sw128(smem_u32(base + kOffK + slot * kTile), 0, 1024);
        for (int k = 0; k < ksteps; ++k) mma_ss(tmem + kG, dq + step_k(k), dkk + step_k(k), id_g, k > 0);
        mma_commit(&sh.gfull);
        mma_commit(&sh.kempty[slot]);
      }
      __syncwarp();
    };
    if (!kStates && chunks > 0) product_g(0);
    for (int c = 0; ok && c < chunks; ++c) {
      const int slot = c & 1;
      const uint32_t ph = (uint32_t)(c >> 1) & 1u, one = (uint32_t)c & 1u;
      if (!(ok = wait(&sh, &sh.vfull[slot], ph, 1) && wait(&sh, &sh.kpfull, one, 1) &&
                 (c == 0 || wait(&sh, &sh.dsempty, one ^ 1u, 1))))
        break;
      tc_fence_after();
      // MN-major: 16 tokens are 16 rows of 128 bytes
      const uint64_t dvv = sdesc_sw128(smem_u32(base + kOffV + slot * kTile), kBlk, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_ts(tmem + kDs, tmem + kHi + 8 * k, dvv + (uint64_t)(k * 2048 >> 4), id_v, k > 0);
        if (two) {
#pragma unroll
          for (int k = 0; k < 8; ++k) mma_ts(tmem + kDs, tmem + kLo + 8 * k, dvv + (uint64_t)(k * 2048 >> 4), id_v, true);
        }
        mma_commit(&sh.dsfull);
        if (kStates) mma_commit(&sh.vempty[slot]);
      }
      __syncwarp();
      if constexpr (!kStates) {
        if (!(ok = wait(&sh, &sh.sfull, one, 1) && (c == 0 || wait(&sh, &sh.oempty, one ^ 1u, 1)))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dq = sdesc_sw128(smem_u32(base + kOffQ + slot * kTile), 0, 1024);
          const uint64_t ds = sdesc_sw128(smem_u32(base + kOffS), kBlk, 1024);
          for (int k = 0; k < ksteps; ++k) mma_ss(tmem + kO, dq + step_k(k), ds + (uint64_t)(k * 2048 >> 4), id_v, k > 0);
          mma_commit(&sh.sempty);
        }
        __syncwarp();
        if (!(ok = wait(&sh, &sh.pfull, one, 1))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) mma_ts(tmem + kO, tmem + kG + 8 * k, dvv + (uint64_t)(k * 2048 >> 4), id_v, true);
          mma_commit(&sh.ofull);
          mma_commit(&sh.vempty[slot]);
        }
        __syncwarp();
        if (c + 1 < chunks) product_g(c + 1);
      }
    }
    if (!ok) {  // products in flight end before TMEM is given back
      if (elect_one()) mma_commit(&sh.drain);
      for (uint32_t j = 0; j < (1u << 20) && !mbar_try_wait(&sh.drain, 0); ++j) {
      }
    }
  } else if (warp == 2) {
    if constexpr (!kStates) {
      for (int c = 0; c < chunks; ++c) {
        const int slot = c & 1;
        if (!wait(&sh, &sh.staged[slot], (uint32_t)(c >> 1) & 1u, 2)) break;
        if (elect_one()) {
          const unsigned char *from = base + kOffQ + slot * kTile;
          const int t0 = start_of(c);
          // 4-D tiled store of a block of 64 channels; past the tensor's end nothing is written
          for (int k = 0; 64 * k < cols; ++k)
            asm volatile(
                "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                    reinterpret_cast<uint64_t>(&p.out)),
                "r"(smem_u32(from + k * kBlk)), "r"(c0 + 64 * k), "r"(h), "r"(t0), "r"(b)
                : "memory");
          bulk_commit();
          bulk_wait_read0();
          mbar_arrive(&sh.qempty[slot]);
        }
        __syncwarp();
      }
      bulk_wait0();  // (of the lane that issued them; the others have none)
    }
  } else if (warp >= 4 && warp < 8) {
    if constexpr (!kStates) {
      const int quarter = warp & 3, row = quarter * 32 + lane;
      for (int c = 0; c < chunks; ++c) {
        const int n = min(kC, t_end - start_of(c));
        if (!wait(&sh, &sh.gfull, (uint32_t)c & 1u, 3)) break;
        tc_fence_after();
        // P = G 2^(lg |row - j| - log2 c_row); the difference of places is taken first,
        // so that a steep lg does not cancel
        const float cp = fmaxf(lg * (float)(p.reverse ? n - 1 - row : row + 1), kFloor);
        const float slope = p.reverse ? -lg : lg;
#pragma unroll 1
        for (int j0 = 0; j0 < kC; j0 += 32) {
          uint32_t out[16];
          // (whole warps: these columns are past every row of the warp, or before)
          const bool none = p.reverse ? j0 + 31 < quarter * 32 || j0 >= n : j0 > quarter * 32 + 31;
          if (none) {
#pragma unroll
            for (int i = 0; i < 16; ++i) out[i] = 0u;
          } else {
            uint32_t g[32];
            tmem_ld32(tmem_addr(tmem, quarter * 32, kG + j0), g);
            tmem_wait_ld_regs(g);
            const int lo = p.reverse ? row : 0, hi = p.reverse ? n - 1 : row;  // columns lo..hi count
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float v[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = j0 + 2 * i + e;
                const float w = ex2(fmaf(slope, (float)row - (float)j, -cp)) * p.kvs;
                v[e] = j >= lo && j <= hi ? __uint_as_float(g[2 * i + e]) * w : 0.f;
              }
              out[i] = pack_bf16(v[0], v[1]);
            }
          }
          // over columns of G that this warp has read
          tmem_st16(tmem_addr(tmem, quarter * 32, kG + j0 / 2), out);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pfull);
      }
    }
  } else if (warp >= 8 && warp < 12) {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    bool ok = true;
    const auto keys = [&](int c) {  // K' of chunk c
      const int slot = c & 1, n = min(kC, t_end - start_of(c));
      const uint32_t ph = (uint32_t)(c >> 1) & 1u;
      if (!(ok = wait(&sh, &sh.kfull[slot], ph, 4))) return;
      if (n < kC) {
        // tokens past the row's end: their values take no part, whatever they are
        if (!(ok = wait(&sh, &sh.vfull[slot], ph, 4))) return;
        for (int r = n + quarter; r < kC; r += 4)
          if (lane < 16)
            *reinterpret_cast<uint4 *>(base + kOffV + slot * kTile + (lane >> 3) * kBlk + r * 128 + (lane & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      // Tiles of 8 tokens x 8 channels, transposed by the load: a lane gets channel
      // lane / 4 of tokens 2 (lane % 4) and the next one.  That is what a 16-lane
      // store to TMEM takes, tokens 8 i.. in register pair i.
      const uint32_t tile = smem_u32(base + kOffK + slot * kTile);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {       // of the tokens
#pragma unroll 1
        for (int d16 = 0; d16 < 2; ++d16) {        // of the warp's 32 channels
          const uint32_t ch = (uint32_t)(quarter * 32 + d16 * 16 + ((lane >> 3) & 1) * 8);
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {            // 16 tokens
            const uint32_t tok = (uint32_t)(half * 64 + i * 16 + (lane >> 4) * 8 + (lane & 7));
            uint32_t x[4];
            ldsm_x4_trans(tile + (ch >> 6) * kBlk + piece_at(tok, (ch & 63) >> 3), x);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int j = half * 64 + i * 16 + g * 8 + 2 * (lane & 3);
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e)
                w[e] = ex2(lg * (float)(p.reverse ? j + e + 1 : n - 1 - j - e)) * p.kvs;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t u = x[2 * g + y];
                const float k0 = j < n ? __uint_as_float(u << 16) * w[0] : 0.f;
                const float k1 = j + 1 < n ? __uint_as_float(u & 0xFFFF0000u) * w[1] : 0.f;
                const uint32_t top = pack_bf16(k0, k1);
                hi[4 * i + 2 * g + y] = top;
                lo[4 * i + 2 * g + y] =
                    pack_bf16(k0 - __uint_as_float(top << 16), k1 - __uint_as_float(top & 0xFFFF0000u));
              }
            }
          }
          tmem_st16x128b_x8(tmem_addr(tmem, quarter * 32 + d16 * 16, kHi + half * 32), hi);
          if (two) tmem_st16x128b_x8(tmem_addr(tmem, quarter * 32 + d16 * 16, kLo + half * 32), lo);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.kpfull), mbar_arrive(&sh.kempty[slot]);
    };
    if (chunks > 0) keys(0);
    for (int c = 0; ok && c < chunks; ++c) {
      if (c + 1 < chunks) {
        if (!wait(&sh, &sh.dsfull, (uint32_t)c & 1u, 4)) break;  // K' has been read
        tc_fence_after();
        keys(c + 1);
        if (!ok) break;
      }
      if constexpr (!kStates) {
        const int slot = c & 1, n = min(kC, t_end - start_of(c));
        if (!wait(&sh, &sh.ofull, (uint32_t)c & 1u, 4)) break;
        tc_fence_after();
        const float cp = row < n ? p.os * ex2(fmaxf(lg * (float)(p.reverse ? n - 1 - row : row + 1), kFloor)) : 0.f;
        unsigned char *to = base + kOffQ + slot * kTile;
#pragma unroll 1
        for (int j0 = 0; j0 < cols; j0 += 32) {
          uint32_t o[32];
          tmem_ld32(tmem_addr(tmem, quarter * 32, kO + j0), o);
          tmem_wait_ld_regs(o);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = __uint_as_float(o[8 * i + 2 * e]) * cp, y = __uint_as_float(o[8 * i + 2 * e + 1]) * cp;
              w[e] = row < n ? pack_bf16(x, y) : 0u;
            }
            *reinterpret_cast<uint4 *>(to + (j0 >> 6) * kBlk + piece_at(row, ((j0 & 63) >> 3) + i)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.oempty), mbar_arrive(&sh.staged[slot]);
      }
    }
  } else if (warp >= 12) {
    const int quarter = warp & 3, d = quarter * 32 + lane, half = (warp - 12) / 4;
    const int v0 = c0 + half * 64, live = d < dk ? min(64, p.dv - v0) : 0;  // this lane's columns of the state
    const int64_t n_state = (int64_t)dk * p.dv;
    float S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    if (!kStates && p.init) {
      const float *from = p.init + (a.nseg > 1 ? bh * a.nseg + sg : bh) * n_state;
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (i < live) S[i] = p.init_t ? from[(int64_t)(v0 + i) * dk + d] : from[(int64_t)d * p.dv + v0 + i];
    }
    const auto publish = [&] {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4 *>(base + kOffS + half * kBlk + piece_at(d, i)) =
            make_uint4(pack_bf16(S[8 * i], S[8 * i + 1]), pack_bf16(S[8 * i + 2], S[8 * i + 3]),
                       pack_bf16(S[8 * i + 4], S[8 * i + 5]), pack_bf16(S[8 * i + 6], S[8 * i + 7]));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sfull);
    };
    if (!kStates) publish();
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      const int n = min(kC, t_end - start_of(c));
      const float keep = exp2f(lg * (float)n);
      if (!(ok = wait(&sh, &sh.dsfull, (uint32_t)c & 1u, 5))) break;
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t r[16];
        tmem_ld16(tmem_addr(tmem, quarter * 32, kDs + half * 64 + 16 * j), r);
        tmem_wait_ld_regs(r);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[16 * j + i] = fmaf(keep, S[16 * j + i], __uint_as_float(r[i]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.dsempty);
      if (!kStates && c + 1 < chunks) {
        if (!(ok = wait(&sh, &sh.sempty, (uint32_t)c & 1u, 5))) break;
        publish();
      }
    }
    if (ok && (kStates || (p.final && sg == (p.reverse ? 0 : a.nseg - 1)))) {
      float *to = p.final + (kStates ? bh * a.nseg + sg : bh) * n_state + (int64_t)d * p.dv + v0;
#pragma unroll
      for (int i = 0; i < 64; ++i)
        if (i < live) to[i] = S[i];
    }
  }
  if constexpr (!kStates) {  // tokens past the row's end, in chunks that no tile reached
    const int t0 = t_lo + chunks * kC, pieces = cols / 8;
    for (int64_t e = threadIdx.x; e < (int64_t)(t_hi - t0) * pieces; e += kThreads)
      *reinterpret_cast<uint4 *>(p.to + (((int64_t)b * a.T + t0 + e / pieces) * a.H + h) * p.dv + c0 + e % pieces * 8) =
          make_uint4(0, 0, 0, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// [B][T][H][d] with strides as a 4-D tensor {d, H, T, B} in tiles of 64 channels x
// 128 tokens, 128-byte swizzle; outside reads as zero and is not written
cudaError_t make_map(CUtensorMap *map, const void *p, int64_t d, int64_t H, int64_t T, int64_t B, const int64_t (&st)[3]) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
  // (the stride of an axis with one entry is never used)
  const auto bytes = [](int64_t n, int64_t s) { return (cuuint64_t)(n > 1 ? s * 2 : 16); };
  const cuuint64_t strides[3] = {bytes(H, st[2]), bytes(T, st[1]), bytes(B, st[0])};
  const cuuint32_t box[4] = {64, 1, kC, 1}, ones[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p), dims, strides, box, ones,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool kStates>
cudaError_t run(const DecayArgs &a, cudaStream_t s) {
  TcArgs t{};
  t.passes = a.passes; t.nseg = a.nseg; t.decay = a.decay; t.lengths = a.lengths;
  t.T = (int)a.T; t.H = (int)a.H; t.seg = (int)a.seg;
  t.groups = 1;
  for (int i = 0; i < a.passes; ++i) {
    const DecayPass &p = a.pass[i];
    TcPass &o = t.pass[i];
    const int64_t whole[3] = {a.T * a.H * p.dv, a.H * p.dv, p.dv};
    cudaError_t e = make_map(&o.k, p.k, p.dk, a.H, a.T, a.B, p.ks);
    if (e == cudaSuccess) e = make_map(&o.v, p.v, p.dv, a.H, a.T, a.B, p.vs);
    if (e == cudaSuccess && !kStates) e = make_map(&o.q, p.q, p.dk, a.H, a.T, a.B, p.qs);
    if (e == cudaSuccess && !kStates) e = make_map(&o.out, p.out, p.dv, a.H, a.T, a.B, whole);
    if (e != cudaSuccess) return e;
    o.init = p.init; o.final = p.final; o.to = static_cast<__nv_bfloat16 *>(p.out);
    o.os = p.os; o.kvs = p.kvs; o.dk = p.dk; o.dv = p.dv; o.reverse = p.reverse; o.init_t = p.init_t;
    const int g = (p.dv + kD - 1) / kD;
    if (g > t.groups) t.groups = g;
  }
  const int64_t grid = a.B * a.H * t.groups * a.nseg * a.passes;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  auto kern = decay_tc_kernel<kStates>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // (not as a dependent: it takes tensor memory before it waits)
  return chain_launch(kern, dim3((unsigned)grid), dim3(kThreads), kSmem, 1, false, s, t);
}

}  // namespace

// What the tensor maps can describe: addresses and strides in whole 16-byte
// pieces, no axis walked without a step, sizes in 32 bits.
bool decay_tc_fits(const DecayArgs &a) {
  if (!a.bf16 || a.T >= (int64_t(1) << 30)) return false;
  const int64_t n[3] = {a.B, a.T, a.H};
  const auto ok = [&](const void *p, const int64_t (&st)[3]) {
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && (st[i] % 8 || st[i] <= 0 || st[i] >= (int64_t(1) << 38))) return false;
    return true;
  };
  for (int i = 0; i < a.passes; ++i) {
    const DecayPass &p = a.pass[i];
    if (p.dk > kD || p.dk % 8 || p.dv % 8 || !ok(p.q, p.qs) || !ok(p.k, p.ks) || !ok(p.v, p.vs)) return false;
  }
  return true;
}

cudaError_t launch_decay_tc(const DecayArgs &a, bool states, cudaStream_t s) {
  return states ? run<true>(a, s) : run<false>(a, s);
}

cudaError_t read_and_clear_decay_error(unsigned int *word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_decay_error, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_decay_error, &zero, sizeof(unsigned int));
}

}  // namespace delta
