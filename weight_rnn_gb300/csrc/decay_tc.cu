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
// they would be off by 1e-3.  With both they are off by 2.4e-6 (plain float32 sums:
// 2.8e-7).  A third part finds no room in tensor memory: with K' in turns of 32 tokens
// the states were off by less than 1e-6, and B4 T8192 H32 took 197 us for 170, its
// gradients' three passes 272 for 236.  P and the copy of S that O reads are single bfloat16:
// each is off by 2^-8 at most, at random, as the rounding of out itself.
//
// Both parts of O share one accumulator: with c_p the factor of S's part (g^(p+1),
// in reverse g^(n-1-p)), P is formed as G_pj g^|p-j| / c_p and the whole row is
// multiplied by c_p when it goes out.  c_p is taken no lower than 2^-64, so that the
// quotient stays in range for any g while q k v stays below 2^63; where that matters S's
// part is 2^-64 of S in place of something less.
//
// The state is float32 in registers, a row of dk a lane; what the chain from chunk
// to chunk costs is dS -> registers -> bfloat16 S in shared memory -> O.  All else
// (G, P, K', loads, stores) is work ahead of or behind it.
//
// Shared memory, 224 KB: two tiles each of Q, K and V (32 KB, 128-byte swizzle, as
// two blocks of 64 channels), S.  TMEM, all 512 columns: G (then P, packed over it), O,
// dS, K' hi and lo.  O leaves from registers, a token a lane in 32-byte pieces: staged
// for TMA where its Q was, it kept that tile for 2500 cycles more, and the ring's wait
// for Q set the pace (6800 cycles a chunk).
//
// Warps (640 threads):
//   0      TMA producer
//   1      issues G, Q S and P V
//   2      TMEM
//   3      issues K'^T V
//   4-11   P from G, and K' from K, transposed on the way to TMEM: half of the columns,
//          of the tokens, each warpgroup
//   12-19  the state, and O: 64 value columns each warpgroup
//
// Bound by HBM where every SM has its share of a long call, 4 tensors of 32 KB a chunk
// (2.9 us at 152 CTAs): B4 T8192 H32 d128 170 us, 6.3 TB/s.  (Figures are of graphs after
// a second's rest; in calls back to back, the clock down with power, this one takes 180 to
// 187 us and the gradients below 253 to 263.)  The warps' own work takes 2.3 us a chunk,
// 4400 cycles, of which shared memory is busy for 3000: tiles in, 96 KB, what the products
// read, 224 (SS ones both operands, 64 cycles for 16 channels, where the tensor cores would
// take 32), K' and S, 64.  Bound by that are heads of 64 channels (B4 T8192 H32 125 us; what
// a narrow head has not is left out: 146 with it) and in part the gradients, three such
// passes at a time, which read 9.5 tensors from memory for the 7 of the call: B4 T4096 H32
// 236 us.  Where the time axis is cut, k and v are read twice: B1 T65536 H8 140 us.  Next is
// instruction fetch, with caches shared by five groups of warps (from 111 KB of code to 70
// KB: 204 -> 171 us).  (A warpgroup of its own for O's way out, 768 threads with registers
// moved by setmaxnreg: 205 us, 278 for the gradients.)  Every mbarrier wait is bounded: a
// timeout sets a device error word and the kernel winds down.
#include <cuda_bf16.h>

#include "chain.cuh"
#include "decay.cuh"
#include "decay_share.h"
#include "kernels.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace delta {
namespace {

using namespace sm100;
using decay::ex2;

__device__ unsigned int g_decay_error = 0;

constexpr int kC = kDecayChunk, kD = 128;
constexpr int kThreads = 640;
constexpr uint32_t kTile = 32768, kBlk = 16384;
constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffS = 6 * kTile;
constexpr int kSmem = 7 * kTile + 1024;
// TMEM columns
constexpr uint32_t kG = 0, kO = 128, kDs = 256, kHi = 384;  // (lo: 64 after hi)
constexpr float kFloor = -64.f;    // log2 of the least c_p
constexpr float kLogZero = -200.f; // log2 g of g = 0: any power of it vanishes, also over c_p

struct TcPass {
  CUtensorMap q, k, v;
  const float *init;
  float *final;
  __nv_bfloat16 *to;  // out
  float os, kvs;
  int dk, dv;
  int8_t rows[3], heads[3];    // of q, k, v: 1, or 0 where all share one batch row, one head
  bool reverse, init_t, wide;  // wide: out's rows are whole 32-byte pieces
};
struct TcArgs {
  TcPass pass[3];
  int passes, groups, nseg, chunks;  // chunks: of a whole segment
  uint32_t items;
  const float *decay;
  const int *lengths;
  int T, H, seg;
  bool shared;      // CTAs share items, and hand over states:
  uint32_t *flags;  // [CTA][8], zeroes
  float4 *handed;   // [CTA][8][16][32]
};

// A CTA's work: one of the passes, and of its items one, or a run of several that CTAs
// share (decay_share.h).  CTAs of different passes that are neighbours work on one head at
// one time, so that what both read comes from memory once (the two in reverse share two of
// three tensors).
using decay::kParts;
struct Part {
  int pass, c0, b, h;
  int t_lo, t_hi, t_end, chunks;  // of the item: tokens, those that count, their chunks
  int from, to;                   // the chunks of this part, in the order of the pass
  float lg;
  bool head, tail, two, last;     // begins, ends the item; K' needs two parts; ends the row
  int64_t state;                  // place among the states
};

template <bool kStates>
__device__ bool part_at(const TcArgs &a, int k, Part &r) {
  uint32_t item = blockIdx.x / (uint32_t)a.passes;
  r.pass = (int)(blockIdx.x % (uint32_t)a.passes);
  r.from = 0, r.to = a.chunks;
  if (a.shared) {
    decay::Run run;
    if (!decay::shared_part(a.items / (uint32_t)a.passes, (uint32_t)a.chunks, item, gridDim.x / (uint32_t)a.passes, k, run))
      return false;
    item = run.item, r.from = run.from, r.to = run.to;
  } else if (k > 0) {
    return false;
  }
  r.head = r.from == 0, r.tail = r.to == a.chunks;
  const TcPass &p = a.pass[r.pass];
  const int sg = (int)(item % (uint32_t)a.nseg);
  item /= (uint32_t)a.nseg;
  r.c0 = (int)(item % (uint32_t)a.groups) * kD;
  const uint32_t bh = item / (uint32_t)a.groups;
  r.b = (int)(bh / (uint32_t)a.H), r.h = (int)(bh % (uint32_t)a.H);
  int len = a.lengths ? a.lengths[r.b] : a.T;
  len = len < 0 ? 0 : len > a.T ? a.T : len;
  r.t_lo = sg * a.seg, r.t_hi = min(r.t_lo + a.seg, a.T), r.t_end = min(r.t_hi, len);
  r.chunks = r.t_end > r.t_lo ? (r.t_end - r.t_lo + kC - 1) / kC : 0;
  if (r.c0 >= p.dv) r.chunks = 0, r.t_hi = r.t_lo;  // a pass with fewer groups
  if (kStates && sg == (p.reverse ? 0 : a.nseg - 1)) r.chunks = 0;  // no segment begins with its state
  r.to = min(r.to, r.chunks);
  r.lg = log2f(a.decay[r.h]);
  if (r.lg < kLogZero) r.lg = kLogZero;  // (not fmaxf, which would drop the NaN of a decay that has no logarithm)
  r.two = r.lg != 0.f || p.kvs != 1.f;  // else K' is K itself
  r.last = kStates || sg == (p.reverse ? 0 : a.nseg - 1);
  r.state = kStates || a.nseg > 1 ? (int64_t)bh * a.nseg + sg : bh;
  return true;
}

struct Shared {
  uint64_t qfull[2], qempty[2], kfull[3], kempty[3], vfull[3], vempty[3];
  uint64_t gfull, pfull, ofull, oempty, dsfull[2], dsempty[2], kpfull[2], sfull, sempty, drain[2];
  uint32_t tmem;
  int parts;
  volatile int dead;
  Part part[kParts];
};

// The first wait of a CTA that gives up is the one reported.  (Barriers' other waits run
// out by themselves, all at about one time; those for another CTA's flag look at `dead`.)
__device__ __forceinline__ void give_up(Shared *sh, int role) {
  if (!sh->dead) atomicCAS(&g_decay_error, 0u, (unsigned)(1 + role));
  sh->dead = 1;
}
// By whole warps, so that they leave their loops together: a lane's try may time out where
// another's sees the phase, so the warp goes on only when all of its lanes have seen it.
// Few instructions, since they stand at every hand-over: the warps' loops have to share
// small instruction caches.
__device__ __forceinline__ bool wait(Shared *sh, uint64_t *bar, uint32_t parity, int role) {
#pragma unroll 1
  for (uint32_t n = 0; n < (1u << 21); ++n)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  give_up(sh, role);
  return false;
}

// The same for a flag that another CTA sets, after what it has for this warp.
__device__ __forceinline__ bool wait_flag(Shared *sh, const uint32_t *flag) {
  uint32_t there = 0;
#pragma unroll 1
  for (uint32_t i = 0; i < (1u << 22) && !sh->dead; ++i) {
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(there) : "l"(flag) : "memory");
    if (there) break;
    __nanosleep(200);
  }
  if (__all_sync(0xffffffffu, there != 0)) return true;
  give_up(sh, 6);
  return false;
}
// products in flight end before TMEM is given back
__device__ __noinline__ void drain(uint64_t *bar) {
  if (elect_one()) mma_commit(bar);
  for (uint32_t j = 0; j < (1u << 20) && !mbar_try_wait(bar, 0); ++j) {
  }
}
// K-major: 16 channels are 32 bytes of a 128-byte row
__device__ __forceinline__ uint64_t step_k(int k) { return (uint64_t)((k >> 2) * kBlk + (k & 3) * 32) >> 4; }

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void tmem_st16x128b_x2(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// float32 pairs: one instruction for two elements
__device__ __forceinline__ uint64_t pk(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pk(uint32_t a, uint32_t b) { return pk(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(pk(-1.f, -1.f)), "l"(a));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t narrow2(uint64_t v) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  return pack_bf16(a, b);
}
__device__ __forceinline__ uint64_t widen2(uint32_t u) { return pk(u << 16, u & 0xFFFF0000u); }

// A lane's row of the state, up to 64 columns (a multiple of 8), between registers and
// memory: 32 bytes at a time, or 16.  (Lanes' rows are apart, so an access takes as long
// as it has lines, whatever its width: by single columns 64 of them took 8 us.)
__device__ __forceinline__ void load_row(uint64_t (&S)[32], const float *from, int live) {
  const bool wide = (reinterpret_cast<uintptr_t>(from) & 31u) == 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (8 * i < live) {
      if (wide) {
        asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
                     : "=l"(S[4 * i]), "=l"(S[4 * i + 1]), "=l"(S[4 * i + 2]), "=l"(S[4 * i + 3])
                     : "l"(from + 8 * i)
                     : "memory");
      } else {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(from + 8 * i);
        const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(from + 8 * i + 4);
        S[4 * i] = x.x, S[4 * i + 1] = x.y, S[4 * i + 2] = y.x, S[4 * i + 3] = y.y;
      }
    }
}
__device__ __forceinline__ void store_row(const uint64_t (&S)[32], float *to, int live) {
  const bool wide = (reinterpret_cast<uintptr_t>(to) & 31u) == 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (8 * i < live) {
      if (wide) {
        asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(to + 8 * i), "l"(S[4 * i]), "l"(S[4 * i + 1]),
                     "l"(S[4 * i + 2]), "l"(S[4 * i + 3])
                     : "memory");
      } else {
        *reinterpret_cast<ulonglong2 *>(to + 8 * i) = make_ulonglong2(S[4 * i], S[4 * i + 1]);
        *reinterpret_cast<ulonglong2 *>(to + 8 * i + 4) = make_ulonglong2(S[4 * i + 2], S[4 * i + 3]);
      }
    }
}

// byte offset of 16-byte piece `piece` (0..7) of a row of a 64-channel block
__device__ __forceinline__ uint32_t piece_at(uint32_t row, uint32_t piece) {
  return row * 128u + ((piece ^ (row & 7u)) * 16u);
}

// where a ring stands at a chunk of the CTA's share
template <int kRing>
struct Turn {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kRing) slot = 0, phase ^= 1u;
  }
};

// tokens past a row's end, in chunks that no tile reached: every 17th row a warp
__device__ __noinline__ void zero_rest(const TcArgs &a, const Part &t, int share, int lane) {
  const TcPass &p = a.pass[t.pass];
  const int pieces = min(kD, p.dv - t.c0) / 8, first = t.t_lo + t.chunks * kC + share, t_hi = t.t_hi;
  if (!t.head || lane >= pieces) return;
  const int64_t row = (int64_t)a.H * p.dv;
  __nv_bfloat16 *to = p.to + ((int64_t)t.b * a.T + first) * row + (int64_t)t.h * p.dv + t.c0 + lane * 8;
  for (int i = first; i < t_hi; i += 17, to += 17 * row) *reinterpret_cast<uint4 *>(to) = make_uint4(0, 0, 0, 0);
}

template <bool kIs>
struct Bool {
  static constexpr bool value = kIs;
};

template <bool kStates>
__global__ void __launch_bounds__(kThreads, 1) decay_tc_kernel(const __grid_constant__ TcArgs a) {
  // The states alone have no Q, S, G and O: their tiles and tensor memory make the
  // rings of K and V one deeper, and K' and dS two.  They are sums, each chunk's own part
  // times a power of g, and the chunks are taken in the opposite order: what is read last
  // is what the pass with all products, which follows, reads first, from L2.
  constexpr int kRing = kStates ? 3 : 2, kBufs = kStates ? 2 : 1;
  extern __shared__ unsigned char raw[];
  __shared__ Shared sh;
  unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qfull[i], 1), mbar_init(&sh.qempty[i], 1);
      mbar_init(&sh.dsfull[i], 1), mbar_init(&sh.dsempty[i], 8), mbar_init(&sh.kpfull[i], 8);
      mbar_init(&sh.drain[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.kfull[i], 1), mbar_init(&sh.kempty[i], kStates ? 8 : 9);
      mbar_init(&sh.vfull[i], 1), mbar_init(&sh.vempty[i], kStates ? 1 : 2);
    }
    mbar_init(&sh.gfull, 1), mbar_init(&sh.pfull, 8), mbar_init(&sh.ofull, 1), mbar_init(&sh.oempty, 8);
    mbar_init(&sh.sfull, 8), mbar_init(&sh.sempty, 1);
    sh.dead = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (warp == 4) {
    bool there = false;
    if (lane < kParts) there = part_at<kStates>(a, lane, sh.part[lane]);
    const unsigned all = __ballot_sync(0xffffffffu, there);
    if (lane == 0) sh.parts = __popc(all);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int parts = sh.parts;
  const auto tile_q = [&](int slot) { return base + kOffQ + slot * kTile; };
  const auto tile_k = [&](int slot) { return base + (kStates ? 2 * slot * kTile : kOffK + slot * kTile); };
  const auto tile_v = [&](int slot) { return base + (kStates ? (2 * slot + 1) * kTile : kOffV + slot * kTile); };
  const auto cols_kp = [&](int buf) { return buf ? kG : kHi; };  // K' hi, lo 64 columns on
  const auto cols_ds = [&](int buf) { return buf ? kO : kDs; };
  bool ok = true;

  if (warp == 0) {
    Turn<kRing> g;
    for (int n = 0; ok && n < parts; ++n) {
      const Part &t = sh.part[n];
      const TcPass &p = a.pass[t.pass];
      const bool down = p.reverse != kStates;
      const int b = t.b, h = t.h, c0 = t.c0, to = t.to, step = down ? -kC : kC;
      int t0 = t.t_lo + (down ? t.chunks - 1 - t.from : t.from) * kC;
      for (int c = t.from; ok && c < to; ++c, g.next(), t0 += step) {
        // (a tile of each, in the order in which they are wanted)
#pragma unroll 1
        for (int i = 0; i < 3; ++i) {
          if (kStates && i == 1) continue;
          const CUtensorMap *map = i == 0 ? &p.k : i == 1 ? &p.q : &p.v;
          uint64_t *full = i == 0 ? &sh.kfull[g.slot] : i == 1 ? &sh.qfull[g.slot] : &sh.vfull[g.slot];
          uint64_t *empty = i == 0 ? &sh.kempty[g.slot] : i == 1 ? &sh.qempty[g.slot] : &sh.vempty[g.slot];
          unsigned char *tile = i == 0 ? tile_k(g.slot) : i == 1 ? tile_q(g.slot) : tile_v(g.slot);
          if (!(ok = wait(&sh, empty, g.phase ^ 1u, 0))) break;
          if (elect_one()) {
            const int x = i == 0 ? 1 : i == 1 ? 0 : 2, d0 = i == 2 ? c0 : 0;
            const int hx = h * p.heads[x], bx = b * p.rows[x];
            const bool both = (i == 2 ? p.dv - c0 : p.dk) > 64;  // (else nothing reads the second block)
            mbar_arrive_expect_tx(full, both ? kTile : kBlk);
            tma_load_4d(tile, map, full, d0, hx, t0, bx);
            if (both) tma_load_4d(tile + kBlk, map, full, d0 + 64, hx, t0, bx);
          }
          __syncwarp();
        }
      }
    }
    // winding down: what is in flight lands first (a tile that was never asked
    // for lets its wait run out)
    if (!ok) {
#pragma unroll 1
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
  } else if (warp == 1) {
    if constexpr (!kStates) {
      Turn<kRing> g;
      Turn<1> o;
      bool begun = false;
      for (int n = 0; ok && n < parts; ++n) {
        const Part &t = sh.part[n];
        const TcPass &p = a.pass[t.pass];
        const uint32_t nv = (uint32_t)(min(kD, p.dv - t.c0) + 15) & ~15u;
        const int ksteps = (p.dk + 15) / 16, to = t.to;
        constexpr uint32_t id_g = idesc_bf16(kC, kC, false, false);
        const uint32_t id_v = idesc_bf16(128, (int)nv, false, true);
        for (int c = t.from; c < to; ++c, g.next(), o.next()) {
          // G (over P, which this warp's products before have read)
          if (!(ok = wait(&sh, &sh.qfull[g.slot], g.phase, 1) && wait(&sh, &sh.kfull[g.slot], g.phase, 1))) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dq = sdesc_sw128(smem_u32(tile_q(g.slot)), 0, 1024);
            const uint64_t dkk = sdesc_sw128(smem_u32(tile_k(g.slot)), 0, 1024);
#pragma unroll 1
            for (int k = 0; k < ksteps; ++k) mma_ss(tmem + kG, dq + step_k(k), dkk + step_k(k), id_g, k > 0);
            mma_commit(&sh.gfull);
            mma_commit(&sh.kempty[g.slot]);
          }
          __syncwarp();
          // Q S, then P V
          if (!(ok = wait(&sh, &sh.sfull, o.phase, 2) && (!begun || wait(&sh, &sh.oempty, o.phase ^ 1u, 2)))) break;
          begun = true;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dq = sdesc_sw128(smem_u32(tile_q(g.slot)), 0, 1024);
            const uint64_t ds = sdesc_sw128(smem_u32(base + kOffS), kBlk, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (k < ksteps) mma_ss(tmem + kO, dq + step_k(k), ds + (uint64_t)(k * 2048 >> 4), id_v, k > 0);
            mma_commit(&sh.sempty);
            mma_commit(&sh.qempty[g.slot]);
          }
          __syncwarp();
          if (!(ok = wait(&sh, &sh.pfull, o.phase, 1) && wait(&sh, &sh.vfull[g.slot], g.phase, 1))) break;
          tc_fence_after();
          if (elect_one()) {
            // MN-major: 16 tokens are 16 rows of 128 bytes
            const uint64_t dvv = sdesc_sw128(smem_u32(tile_v(g.slot)), kBlk, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ts(tmem + kO, tmem + kG + 32 * (k >> 1) + 8 * (k & 1), dvv + (uint64_t)(k * 2048 >> 4), id_v, true);
            mma_commit(&sh.ofull);
            mma_commit(&sh.vempty[g.slot]);
          }
          __syncwarp();
        }
      }
      if (!ok) drain(&sh.drain[0]);
    }
  } else if (warp == 3) {
    Turn<kRing> g;
    Turn<kBufs> u;
    int gone = 0;  // chunks before, up to kBufs
    for (int n = 0; ok && n < parts; ++n) {
      const Part &t = sh.part[n];
      const TcPass &p = a.pass[t.pass];
      const uint32_t nv = (uint32_t)(min(kD, p.dv - t.c0) + 15) & ~15u;
      const int steps = t.two ? 16 : 8, to = t.to;
      const uint32_t id_v = idesc_bf16(128, (int)nv, false, true);
      for (int c = t.from; c < to; ++c, g.next(), u.next()) {
        if (!(ok = wait(&sh, &sh.kpfull[u.slot], u.phase, 2) && wait(&sh, &sh.vfull[g.slot], g.phase, 2) &&
                   (gone < kBufs || wait(&sh, &sh.dsempty[u.slot], u.phase ^ 1u, 2))))
          break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dvv = sdesc_sw128(smem_u32(tile_v(g.slot)), kBlk, 1024);
          const uint32_t kp = tmem + cols_kp(u.slot), ds = tmem + cols_ds(u.slot);
#pragma unroll 1
          for (int k = 0; k < steps; ++k)  // hi's 8 steps of 16 tokens, lo's 8
            mma_ts(ds, kp + 8 * k, dvv + (uint64_t)((k & 7) * 2048 >> 4), id_v, k > 0);
          mma_commit(&sh.dsfull[u.slot]);
          mma_commit(&sh.vempty[g.slot]);
        }
        __syncwarp();
        if (gone < kBufs) ++gone;
      }
    }
    if (!ok) drain(&sh.drain[1]);
  } else if (warp == 2) {
    if constexpr (!kStates)
      for (int n = 0; n < parts; ++n) zero_rest(a, sh.part[n], 0, lane);
  } else if (warp < 12) {
    const int quarter = warp & 3, half = (warp - 4) / 4;
    const int row = quarter * 32 + lane;
    Turn<kRing> g;
    Turn<kBufs> u;
    Turn<1> o;
    int gone = 0;
    const auto share = [&](const Part &t, auto direction) {
      constexpr bool kReverse = decltype(direction)::value;
      const float lg = t.lg, kvs = a.pass[t.pass].kvs;
      const bool two = t.two, mine = quarter * 32 < a.pass[t.pass].dk;  // else no such channels
      const float s16 = ex2(16.f * lg);
      const uint64_t step16 = pk(s16, s16);
      uint64_t c2[4];  // (see scores)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c2[i] = kReverse ? pk(ex2(-lg * (float)(7 - 2 * i)), ex2(-lg * (float)(6 - 2 * i)))
                         : pk(ex2(-lg * (float)(2 * i)), ex2(-lg * (float)(2 * i + 1)));
      const int to = t.to;
      constexpr bool kDown = kReverse != kStates;
      int left = t.t_end - t.t_lo - (kDown ? t.chunks - 1 - t.from : t.from) * kC;  // tokens from the chunk's first on
      for (int c = t.from; c < to; ++c, left += kDown ? kC : -kC) {
        const int n = min(kC, left);
        // ---- K': this warp's 32 channels, half of the tokens
        if (!wait(&sh, &sh.kfull[g.slot], g.phase, 4)) return false;
        if (n < kC) {
          // tokens past the row's end: their values take no part, whatever they are
          if (!wait(&sh, &sh.vfull[g.slot], g.phase, 4)) return false;
          for (int r = n + warp - 4; r < kC; r += 8)
            if (lane < 16)
              *reinterpret_cast<uint4 *>(tile_v(g.slot) + (lane >> 3) * kBlk + r * 128 + (lane & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        // Tiles of 8 tokens x 8 channels, transposed by the load: a lane gets channel
        // lane / 4 of tokens 2 (lane % 4) and the next one.  That is what a 16-lane
        // store to TMEM takes, tokens 8 i.. in register pair i.  16 tokens x 16 channels
        // at a time, from the heaviest tokens on: the next ones' weights are these times
        // g^16, which can only vanish.
        const uint32_t tile = smem_u32(tile_k(g.slot));
        const int j0 = half * 64 + 2 * (lane & 3);  // of the lane's first pair, and 8 on its second
        uint64_t w[2];
        if (!mine && gone == kBufs && !wait(&sh, &sh.dsfull[u.slot], u.phase ^ 1u, 4)) return false;
        if (!mine && gone < kBufs) ++gone;
#pragma unroll 1
        for (int i4 = mine ? 0 : 4; i4 < 4; ++i4) {
          const int i = kReverse ? i4 : 3 - i4;
          const uint32_t tok = (uint32_t)(half * 64 + i * 16 + (lane >> 4) * 8 + (lane & 7));
          if (i4 == 0 || n < kC) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int j = j0 + i * 16 + 8 * y;
              const int e = kReverse ? j + 1 : max(n - 1 - j, 0), f = kReverse ? j + 2 : max(n - 2 - j, 0);
              w[y] = pk(ex2(lg * (float)e) * kvs, ex2(lg * (float)f) * kvs);
            }
          }
#pragma unroll
          for (int d16 = 0; d16 < 2; ++d16) {  // of the warp's 32 channels
            const uint32_t ch = (uint32_t)(quarter * 32 + d16 * 16 + ((lane >> 3) & 1) * 8);
            uint32_t x[4], hi[4], lo[4];
            ldsm_x4_trans(tile + (ch >> 6) * kBlk + piece_at(tok, (ch & 63) >> 3), x);
            if (n < kC) {
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int j = j0 + i * 16 + 8 * (y >> 1);
                x[y] &= (j < n ? 0xFFFFu : 0u) | (j + 1 < n ? 0xFFFF0000u : 0u);
              }
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint64_t v = mul2(widen2(x[y]), w[y >> 1]);
              hi[y] = narrow2(v);
              lo[y] = narrow2(sub2(v, widen2(hi[y])));
            }
            if (i4 == 0 && d16 == 0) {  // what lay here has been read
              if (gone == kBufs) {
                if (!wait(&sh, &sh.dsfull[u.slot], u.phase ^ 1u, 4)) return false;
                tc_fence_after();
              } else {
                ++gone;
              }
            }
            const uint32_t at = tmem_addr(tmem, quarter * 32 + d16 * 16, cols_kp(u.slot) + half * 32 + i * 8);
            tmem_st16x128b_x2(at, hi);
            if (two) tmem_st16x128b_x2(at + 64, lo);
          }
          w[0] = mul2(w[0], step16), w[1] = mul2(w[1], step16);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kpfull[u.slot]), mbar_arrive(&sh.kempty[g.slot]);
        // ---- P: this lane's row, every second block of 32 columns
        if constexpr (!kStates) {
          if (!wait(&sh, &sh.gfull, o.phase, 3)) return false;
          tc_fence_after();
          // P = G 2^(lg |row - j| - log2 c_row).  The power is taken for one column of
          // eight, the one furthest from the row's own, and times eight constants
          // 2^(-lg i): below 2^-126 it is nothing beside the row's own 2^-log2 c_row.
          const float cp = fmaxf(lg * (float)(kReverse ? n - 1 - row : row + 1), kFloor);
#pragma unroll 1
          for (int i16 = 0; i16 < 4; ++i16) {  // 16 columns of the blocks half and half + 2
            const int blk = half * 32 + (i16 >> 1) * 64, j1 = blk + (i16 & 1) * 16;
            uint32_t out[8];
            // (whole warps: these columns are past every row of the warp, or before)
            const bool none = kReverse ? j1 + 15 < quarter * 32 || j1 >= n : j1 > quarter * 32 + 31;
            if (none) {
#pragma unroll
              for (int i = 0; i < 8; ++i) out[i] = 0u;
            } else {
              uint32_t s[16];
              tmem_ld16(tmem_addr(tmem, quarter * 32, kG + j1), s);
              tmem_wait_ld_regs(s);
              if (lg < -16.f) {  // 2^(-7 lg) would leave float32's range
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float apart = kReverse ? (float)(j1 + i - row) : (float)(row - j1 - i);
                  s[i] = __float_as_uint(__uint_as_float(s[i]) * (ex2(fmaf(lg, apart, -cp)) * kvs));
                }
              } else {
#pragma unroll
                for (int b8 = 0; b8 < 2; ++b8) {
                  const int j = j1 + 8 * b8 + (kReverse ? 7 : 0);
                  const float first = ex2(fmaf(lg, (float)(kReverse ? j - row : row - j), -cp)) * kvs;
                  const uint64_t f2 = pk(first, first);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const uint64_t v = mul2(pk(s[8 * b8 + 2 * i], s[8 * b8 + 2 * i + 1]), mul2(f2, c2[i]));
                    asm("mov.b64 {%0, %1}, %2;" : "=r"(s[8 * b8 + 2 * i]), "=r"(s[8 * b8 + 2 * i + 1]) : "l"(v));
                  }
                }
              }
              // (most pieces have no columns that do not count)
              if (kReverse ? j1 < quarter * 32 + 31 || j1 + 15 >= n : j1 + 15 > quarter * 32) {
                // bit i: column j1 + i counts, up to the row's own, or from it to the last
                const uint32_t upto = kReverse ? (n - j1 >= 16 ? 0xFFFFu : (1u << (n - j1)) - 1u)
                                               : (row - j1 >= 15 ? 0xFFFFu : row < j1 ? 0u : (2u << (row - j1)) - 1u);
                const uint32_t below = !kReverse || row <= j1 ? 0u : row - j1 >= 16 ? 0xFFFFu : (1u << (row - j1)) - 1u;
                const uint32_t keep = upto & ~below;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (!(keep >> i & 1u)) s[i] = 0u;
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) out[i] = pack_bf16(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
            }
            // over columns of the block that this warp has read
            tmem_st8(tmem_addr(tmem, quarter * 32, kG + blk + (i16 & 1) * 8), out);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.pfull);
        }
        g.next(), u.next(), o.next();
      }
      return true;
    };
    for (int n = 0; ok && n < parts; ++n) {
      const Part &t = sh.part[n];
      ok = a.pass[t.pass].reverse ? share(t, Bool<true>{}) : share(t, Bool<false>{});
      if constexpr (!kStates) zero_rest(a, t, warp - 3, lane);
    }
  } else {
    const int quarter = warp & 3, half = (warp - 12) / 4, d = quarter * 32 + lane;
    Turn<kBufs> u;
    Turn<1> o;
    bool begun = false, mine = true;  // mine: some of the warp's rows and columns are there
    uint64_t S[32];  // pairs of columns
    chain_wait();  // for the joined states: all else was there before that kernel began
    const auto publish = [&] {  // the bfloat16 copy that Q S reads, once the one before has been read
      if (begun && !wait(&sh, &sh.sempty, o.phase ^ 1u, 5)) return false;
      if (mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4 *>(base + kOffS + half * kBlk + piece_at(d, i)) =
              make_uint4(narrow2(S[4 * i]), narrow2(S[4 * i + 1]), narrow2(S[4 * i + 2]), narrow2(S[4 * i + 3]));
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.sfull);
      return true;
    };
    for (int m = 0; ok && m < parts; ++m) {
      const Part &t = sh.part[m];
      const TcPass &p = a.pass[t.pass];
      const int v0 = t.c0 + half * 64, live = d < p.dk ? min(64, p.dv - v0) : 0;  // this lane's columns
      mine = quarter * 32 < p.dk && v0 < p.dv;
      if (t.head) {
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = 0;
        if (!kStates && p.init) {
          const float *from = p.init + t.state * p.dk * p.dv;
          if (p.init_t) {
            from += (int64_t)v0 * p.dk + d;
#pragma unroll
            for (int i = 0; i < 32; ++i, from += 2 * p.dk)  // (an even number of columns)
              if (2 * i < live) S[i] = pk(from[0], from[p.dk]);
          } else {
            load_row(S, from + (int64_t)d * p.dv + v0, live);
          }
        }
      } else {  // from the CTA before
        if (!(ok = wait_flag(&sh, a.flags + (blockIdx.x - a.passes) * 8 + (warp - 12)))) break;
        const float4 *from = a.handed + ((int64_t)(blockIdx.x - a.passes) * 8 + (warp - 12)) * 512 + lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 v = __ldcg(from + i * 32);
          S[2 * i] = pk(v.x, v.y), S[2 * i + 1] = pk(v.z, v.w);
        }
      }
      const int to = t.to;
      if (!kStates && t.from < to && !(ok = publish())) break;
      const float lg = t.lg;
      decay::Keep keep = {0.f, 0.f};  // of a chunk of `kept` tokens
      float owed = 0.f;
      int kept = -1;
      const bool down = p.reverse != kStates;
      const int first = down ? t.chunks - 1 - t.from : t.from, step = down ? -kC : kC;
      int left = t.t_end - t.t_lo - first * kC, rest = t.t_hi - t.t_lo - first * kC - (quarter * 32 + lane);
      __nv_bfloat16 *out = kStates ? nullptr
                                   : p.to + (((int64_t)t.b * a.T + t.t_lo + (int64_t)first * kC + quarter * 32 + lane) * a.H + t.h) * p.dv + v0;
      const int64_t hop = (int64_t)step * a.H * p.dv;
      for (int c = t.from; c < to; ++c, left -= step, rest -= step, out += hop) {
        const int n = min(kC, left);
        float f;
        if constexpr (kStates) {  // the tokens between the chunk and the pass's end
          f = exp2f(lg * (float)(p.reverse ? t.t_end - t.t_lo - left : left - n));
        } else {
          if (n != kept) keep = decay::keep_of(lg, n), kept = n;  // (whole chunks, and the last)
          f = decay::keep_now(keep, owed);
        }
        const uint64_t f2 = pk(f, f);
        if (!(ok = wait(&sh, &sh.dsfull[u.slot], u.phase, 5))) break;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!mine) break;
          uint32_t r[16];
          tmem_ld16(tmem_addr(tmem, quarter * 32, cols_ds(u.slot) + half * 64 + 16 * j), r);
          tmem_wait_ld_regs(r);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t x = pk(r[2 * i], r[2 * i + 1]);
            S[8 * j + i] = kStates ? fma2(f2, x, S[8 * j + i]) : fma2(f2, S[8 * j + i], x);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.dsempty[u.slot]);
        u.next();
        if constexpr (!kStates) {
          const uint32_t phase = o.phase;
          o.next();
          begun = true;
          if (c + 1 < to && !(ok = publish())) break;
          // O, this half of its columns: a token a lane
          if (!(ok = wait(&sh, &sh.ofull, phase, 5))) break;
          tc_fence_after();
          const int row = quarter * 32 + lane;
          const float cp = p.os * ex2(fmaxf(lg * (float)(p.reverse ? n - 1 - row : row + 1), kFloor));
          const uint64_t cp2 = pk(cp, cp);
          const int have = rest > 0 ? p.dv - v0 : 0;
          const bool wide = p.wide;
          if (v0 >= p.dv && lane == 0) mbar_arrive(&sh.oempty);
#pragma unroll 1
          for (int j = v0 < p.dv ? 0 : 4; j < 4; ++j) {
            uint32_t x[16], w[8];
            tmem_ld16(tmem_addr(tmem, quarter * 32, kO + half * 64 + 16 * j), x);
            tmem_wait_ld_regs(x);
            if (j == 3) {  // O may be written again
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.oempty);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = narrow2(mul2(pk(x[2 * i], x[2 * i + 1]), cp2));
            if (n < kC) {  // (whatever their products are)
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = row < n ? w[i] : 0u;
            }
            if (wide && 16 * j + 16 <= have) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + 16 * j), "r"(w[0]),
                           "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                           : "memory");
            } else {
              if (16 * j + 8 <= have) *reinterpret_cast<uint4 *>(out + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
              if (16 * j + 16 <= have) *reinterpret_cast<uint4 *>(out + 16 * j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      if (!ok) break;
      if (!t.tail) {  // for the CTA after
        float4 *to4 = a.handed + ((int64_t)blockIdx.x * 8 + (warp - 12)) * 512 + lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float4 v;
          asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(S[2 * i]));
          asm("mov.b64 {%0, %1}, %2;" : "=f"(v.z), "=f"(v.w) : "l"(S[2 * i + 1]));
          __stcg(to4 + i * 32, v);
        }
        __threadfence();
        __syncwarp();
        if (lane == 0)
          asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(a.flags + blockIdx.x * 8 + (warp - 12)), "r"(1u) : "memory");
      } else if (p.final && t.last) {
        // (with segments, the states' own pass has a place for each, the row one)
        const int64_t at = kStates ? t.state : (int64_t)t.b * a.H + t.h;
        store_row(S, p.final + at * p.dk * p.dv + (int64_t)d * p.dv + v0, live);
      }
      if constexpr (!kStates) zero_rest(a, t, warp - 3, lane);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

int sm_count() {
  int dev = 0, n = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// [B][T][H][d] with strides as a 4-D tensor {d, H, T, B} in tiles of 64 channels x
// 128 tokens, 128-byte swizzle; outside reads as zero and is not written
cudaError_t make_map(CUtensorMap *map, const void *p, int64_t d, int64_t H, int64_t T, int64_t B, const int64_t (&st)[3]) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  if (st[2] == 0) H = 1;  // (shared)
  if (st[0] == 0) B = 1;
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

int64_t tc_items(const DecayArgs &a) {
  int dv = 1;
  for (int i = 0; i < a.passes; ++i) dv = max(dv, a.pass[i].dv);
  return a.B * a.H * ((dv + kD - 1) / kD) * a.nseg * a.passes;
}
// (rows of differing lengths are better dealt out one by one)
bool tc_shared(const DecayArgs &a) { return !a.lengths && decay::share_items(tc_items(a), a.passes, sm_count()); }
int64_t flag_bytes(int sms) { return ((int64_t)sms * 32 + 255) / 256 * 256; }

// (Not launched as a dependent, but where this call's own joining of states goes before:
// it takes tensor memory before it waits, which a caller's kernel may have yet to take.)
template <bool kStates>
cudaError_t run(const DecayArgs &a, cudaStream_t s) {
  TcArgs t{};
  t.passes = a.passes; t.nseg = a.nseg; t.decay = a.decay; t.lengths = a.lengths;
  t.T = (int)a.T; t.H = (int)a.H; t.seg = (int)a.seg;
  t.groups = 1;
  for (int i = 0; i < a.passes; ++i) {
    const DecayPass &p = a.pass[i];
    TcPass &o = t.pass[i];
    cudaError_t e = make_map(&o.k, p.k, p.dk, a.H, a.T, a.B, p.ks);
    if (e == cudaSuccess) e = make_map(&o.v, p.v, p.dv, a.H, a.T, a.B, p.vs);
    if (e == cudaSuccess && !kStates) e = make_map(&o.q, p.q, p.dk, a.H, a.T, a.B, p.qs);
    if (e != cudaSuccess) return e;
    o.init = p.init; o.final = p.final; o.to = static_cast<__nv_bfloat16 *>(p.out);
    o.os = p.os; o.kvs = p.kvs; o.dk = p.dk; o.dv = p.dv; o.reverse = p.reverse; o.init_t = p.init_t;
    const int64_t *strides[3] = {p.qs, p.ks, p.vs};
    for (int x = 0; x < 3; ++x) o.rows[x] = strides[x][0] != 0, o.heads[x] = strides[x][2] != 0;
    o.wide = p.dv % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
    const int g = (p.dv + kD - 1) / kD;
    if (g > t.groups) t.groups = g;
  }
  const int64_t items = tc_items(a);
  if (items >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  t.items = (uint32_t)items;
  t.chunks = (int)(a.seg / kC);
  auto kern = decay_tc_kernel<kStates>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  // CTAs that hand states to one another are resident together
  const int sms = sm_count();
  t.shared = tc_shared(a);
  if (t.shared) {
    t.flags = static_cast<uint32_t *>(a.handed);
    t.handed = reinterpret_cast<float4 *>(static_cast<unsigned char *>(a.handed) + flag_bytes(sms));
    if ((e = cudaMemsetAsync(t.flags, 0, (size_t)sms * 32, s)) != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(t.shared ? decay::shared_ctas(a.passes, sms) * a.passes : items));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  if (t.shared) {
    at.id = cudaLaunchAttributeCooperative;
    at.val.cooperative = 1;
  } else {
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = &at;
  cfg.numAttrs = t.shared || a.joined ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, t);
}

}  // namespace

// What the tensor maps can describe: addresses and strides in whole 16-byte
// pieces, sizes in 32 bits; heads or batch rows that share their values as one.
bool decay_tc_fits(const DecayArgs &a) {
  if (!a.bf16 || a.T >= (int64_t(1) << 30)) return false;
  const int64_t n[3] = {a.B, a.T, a.H};
  const auto ok = [&](const void *p, const int64_t (&st)[3]) {
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && (st[i] % 8 || (i == 1 && st[i] == 0) || st[i] >= (int64_t(1) << 38))) return false;
    return true;
  };
  for (int i = 0; i < a.passes; ++i) {
    const DecayPass &p = a.pass[i];
    if (p.dk > kD || p.dk % 8 || p.dv % 8 || !ok(p.q, p.qs) || !ok(p.k, p.ks) || !ok(p.v, p.vs)) return false;
  }
  return true;
}

// what CTAs hand over
int64_t decay_tc_scratch(const DecayArgs &a) {
  const int sms = sm_count();
  return tc_shared(a) ? flag_bytes(sms) + (int64_t)sms * 65536 : 0;
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
