// gdn_linear_tc.cu -- the scan of linear attention (gdn_linear.cuh) on the
// Blackwell tensor cores: tcgen05 with TMEM accumulators, TMA tiles; bf16 operands
// and output, head dims 128 or 64, fp32 state.
//
// Chunks of 128 tokens, so that every product is a full 128 x 128 x 128 tile:
//     P  = A B^T                     A, B, C: the chunk's rows of a, b, c
//     Oi = A X^T                     X (Dc x Da) the state before the chunk
//     Oa = (P . lam^{|t-s|}) C       causal
//     dX = (w C)^T B                 w_t = s_upd lam^{rest}
//     out_t = s_inter lam^{p+1} Oi_t + s_intra Oa_t,   X <- lam^len X + dX.
// A head dim of 64 runs on the same tiles: TMA fills the columns past it with zeros and
// does not store them.  (The products are then up to four times what is needed, and the
// halved bytes buy little: 8192 tokens at 16/48 heads take 120 us against 130.)
// Precision.  A, B, C are exact bf16.  The state is fp32 in registers; w C enters dX
// as bf16 terms cut from its fp32 value, 8 bits each: three (all 24 bits) where the
// state is returned or handed to another segment, two where it only serves outputs;
// each chunk's dX is summed apart and added once, rounded to nearest.  P . lam^{..}
// and X are rounded to bf16 once as operands of the output, whose own rounding to
// bf16 is as large.
//
// Bound and measured (8192 tokens, 16/48 heads of 128).  The outputs kernel takes 76 us
// at 243 MB of HBM traffic, 3.0 TB/s, with the tensor pipe active 39 % of the time: the
// products read 224 KB of operands a chunk from shared memory (A, B, X, C, and B again
// for the second term of w C), and loads, w C, X and the output tiles move as much again:
// about 450 KB or 3,500 cycles of the 5,800 that a chunk takes, beside 3,000 for its share
// of HBM.  So none of the three is full (shared memory 44 %), and the rest is waiting:
// there is one P in tensor memory, and the next chunk's is issued after the product with
// this one's, which waits for the warps that form P and scale A X^T.  The states kernel
// takes 40 us.  The whole prefill takes 130 us by itself and 140 in a loop of many, where
// the board is at its power limit (980 W) and the clock falls to 1.67 GHz; a packed batch
// of 65,000 tokens 664 and 770 (1.53 GHz).  A batch of 256 prompts of 100 tokens takes 897
// us: one CTA per (prompt, head), 10.8 us each, whose start and end do not overlap with
// another's.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_chunk_ops.cuh"
#include "gdn_common.cuh"
#include "gdn_linear.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace lin {

using namespace sm100;
using chunk::CTL_ABORT;
using chunk::CTL_LIMIT;

namespace {

constexpr int CH = 128;
constexpr int NTHREADS = 640;   // states: warp 0 TMA, 1 MMA, 2 wait limit, 4-19 elementwise
constexpr int NTHREADS_O = 1024;  // outputs: warp 0 loads, 1 and 3 MMA, 2 stores, 4-7 w C, 8-15 X, 16-23 P, 24-31 out
constexpr uint32_t TILE = 32768;  // 128 rows x 128 bf16: [d 0-63 | d 64-127], 128-byte rows, swizzled

// ---- instruction descriptors ----
constexpr uint32_t IDESC_KK = idesc_bf16(128, 128, 0, 0);  // A B^T, A X^T: both K-major
constexpr uint32_t IDESC_KM = idesc_bf16(128, 128, 0, 1);  // (wC)^T B, P C: B operand MN-major

struct Weights {        // fp32 tables in shared memory
  float pw[CH + 4];     // lam^i
  float pm[CH + 4];     // lam^i - 1, or 2 (Power)
  Carry carry[8];       // of the X warps
  float pwi[CH];        // s_intra lam^i
  float wfull[CH], wtail[CH];  // w_t of a full chunk and of the segment's last one
};

__device__ __forceinline__ void fill_weights(const Scan &p, Weights *w, float gh, int tail, int tid) {
  if (tid <= CH) {
    const Power x = decay_power(gh, tid);
    w->pw[tid] = x.value;
    w->pm[tid] = x.m;
  }
  if (tid < CH) {
    const int rf = p.back ? tid : CH - 1 - tid, rt = p.back ? tid : tail - 1 - tid;
    w->wfull[tid] = p.s_upd * expf(gh * (float)rf);
    w->wtail[tid] = tid < tail ? p.s_upd * expf(gh * (float)rt) : 0.f;
  }
  if (tid < 8) w->carry[tid].rest = 0.f;
  if (tid < CH) w->pwi[tid] = p.s_intra * expf(gh * (float)tid);
}

// Rows [len, 128) of a tile <- 0, by `n` threads: what TMA read there belongs to the
// next sequence, and 0 * NaN would carry it over.
__device__ __forceinline__ void zero_tail(unsigned char *tile, int len, int thread, int n) {
  for (int x = thread; x < (CH - len) * 16; x += n) {
    const int r = len + (x >> 4), ch = x & 15;
    *reinterpret_cast<uint4 *>(tile + (ch >> 3) * 16384 + r * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// The kernels here run five roles at once on each SM sub-core, so their code is kept
// short (few loops unrolled, a small wait): with everything unrolled the roles did not
// fit the instruction caches together and ran at about five cycles an instruction.
//
// All lanes of a warp wait for a phase, for at most the limit in ctl[CTL_LIMIT] (in
// 1024 clock cycles) and only while no role has given up.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int *ctl, int32_t *status) {
  bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
  if (!ok) {
    const long long t0 = clock64();
    bool over;
    do {
      ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
      over = __any_sync(0xffffffffu, ctl[CTL_ABORT] != 0 || ((clock64() - t0) >> 10) > ctl[CTL_LIMIT]);
    } while (!ok && !over);
    if (!ok) {
      ctl[CTL_ABORT] = 1;
      if ((threadIdx.x & 31) == 0) report_status(status, GDN_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
  tc_fence_after();
  return true;
}
// The same for one thread, which then acts alone (the TMA producer).
__device__ __forceinline__ bool wait_phase_alone(uint32_t bar, uint32_t parity, volatile int *ctl) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (ctl[CTL_ABORT] != 0 || ((clock64() - t0) >> 10) > ctl[CTL_LIMIT]) return false;
  return true;
}
// The limit of a workspace header in units of 1024 cycles: microseconds at 2 GHz (the
// clock is at most that), 2 s by default.
__device__ __forceinline__ int wait_limit(const int32_t *status) {
  const uint32_t us = header_wait_limit_us(status);
  return us ? (int)(2u * min(us, 0x3fffffffu)) : 4000000;
}

// 8 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// One 16-bit term of two fp32 values: their upper halves in one word, and what they
// leave.  Three such terms hold all 24 bits of a value.
__device__ __forceinline__ uint32_t cut_term(float &x0, float &x1) {
  const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
  x0 -= __uint_as_float(u0 & 0xffff0000u);
  x1 -= __uint_as_float(u1 & 0xffff0000u);
  return __byte_perm(u0, u1, 0x7632);
}

// Four 8 x 8 blocks of 16-bit values, transposed: word of lane l in block m = rows
// 2 (l mod 4), + 1 of column l / 4.
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16 lanes x 8 columns: lane l holds row l / 4 (+ 8: odd words), column l mod 4 (+ 4:
// words 2, 3).
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// (w C)^T as the A operand of dX: 32 rows of X (columns 32 lq .. of C) by the tokens
// [t0, t0 + 16 TT), a pair of tokens in a word, 8 columns for 16 tokens (lane 32 lq of
// TMEM).  TERMS: 3, the high, middle and low terms at t1, t2, t3; 2, the first two;
// 1, the low term alone at t1.  C is read by transposing 8 x 8 blocks, whose lane
// layout is that of the 16-lane TMEM stores.
template <int TERMS, int TT>
__device__ __forceinline__ void scale_split(uint32_t tile, const float *wt, int lq, int lane, int t0, uint32_t t1,
                                            uint32_t t2, uint32_t t3) {
  // block m of a load: tokens 8 (m / 2) .., columns 8 (m mod 2) ..
  const int tr = t0 + 8 * (lane >> 4) + (lane & 7);
  const uint32_t base = tile + (lq >> 1) * 16384 + tr * 128;
  const uint32_t ch = 4 * (lq & 1) + ((lane >> 3) & 1);
  const float *wl = wt + t0 + 2 * (lane & 3);
#pragma unroll 1
  for (int i = 0; i < TT; ++i) {
    const float2 w0 = *reinterpret_cast<const float2 *>(wl + 16 * i);
    const float2 w1 = *reinterpret_cast<const float2 *>(wl + 16 * i + 8);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      uint32_t r[4], h[4], m[4], l[4];
      ldmatrix_x4_t(base + i * 2048 + (((ch + 2 * d) ^ (tr & 7)) << 4), r);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 wk = k < 2 ? w0 : w1;
        float x0 = wk.x * __uint_as_float(r[k] << 16), x1 = wk.y * __uint_as_float(r[k] & 0xffff0000u);
        h[k] = cut_term(x0, x1);
        m[k] = cut_term(x0, x1);
        if (TERMS != 2) l[k] = cut_term(x0, x1);
      }
      const uint32_t at = ((uint32_t)(16 * d) << 16) + 8 * i;
      if (TERMS > 1) {
        tmem_st_16x8(t1 + at, h);
        tmem_st_16x8(t2 + at, m);
      }
      if (TERMS == 3) tmem_st_16x8(t3 + at, l);
      if (TERMS == 1) tmem_st_16x8(t1 + at, l);
    }
  }
}

// Registers of a thread, set by each warpgroup: a CTA is launched with 1024 x 64, and
// 128 x 32 + 128 x 48 + 256 x 104 + 256 x 64 + 256 x 48 is the same sum.
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A row of a state is 512 bytes and a thread holds a piece of one, so states pass
// through shared memory, where a piece has a slot of its own with 16 bytes to spare
// (no bank conflicts), and are copied piece by piece.  (Rows of 32 scattered pieces
// loaded and stored directly took 4 us of a CTA each.)
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}

// ---------------------------------------------------------------- outputs
// Shared memory of the output kernel: 2 stages of A, B, C tiles, X as an operand.
constexpr uint32_t STAGE = 3 * TILE;
constexpr uint32_t OFF_X = 2 * STAGE;
constexpr uint32_t OFF_W = OFF_X + TILE;
constexpr uint32_t OFF_BAR = OFF_W + ((sizeof(Weights) + 15) / 16) * 16;
constexpr uint32_t OFF_CTL = OFF_BAR + 256;  // TMEM base, control words
constexpr uint32_t OFF_UNIT = OFF_CTL + 32;  // the unit, for the end of the X warps
constexpr uint32_t SMEM_OUT = OFF_UNIT + 32;
static_assert(SMEM_OUT <= 232448, "shared memory of a CTA");

// TMEM columns: P (fp32), whose two halves are overwritten by their bf16 form (32
// columns each); O; two terms of w C; dX.  (MMAs of one issuer run in order, so P may
// be written where the product before read.)
constexpr uint32_t R_P = 0, T_PB = 0, R_O = 128, T_VH = 256, T_VM = 320, R_DX = 384;
__host__ __device__ constexpr uint32_t pcol(int kk) { return 64 * (kk >> 2) + 8 * (kk & 3); }  // of T_PB

enum { B_FULL = 0, B_EMPTY = 2, B_P = 4, B_PB = 6, B_V = 7, B_VFREE = 9, B_DX = 11, B_DXFREE = 12, B_OI = 13,
       B_OA = 14, B_OFREE = 15, B_X = 16, B_FIX = 17, B_DRAIN = 18, B_EMPTYA = 19, B_OUT = 21, B_X0 = 23, B_VL = 25, B_VUSED = 27, B_DXO = 29, NBAR = 31 };
static_assert(NBAR * 8 <= 256, "barrier area");

// One CTA per (segment, head).  Only X <- lam^len X + dX is carried from chunk to
// chunk; dX, P and the rest of a chunk do not wait for the one before, except for the
// buffers.  So each kind of work has its own warps, which run as far ahead as the
// buffers let them:
//   warps 4-7    w C as two bf16 terms, in two halves of 64 tokens with a buffer each
//   warps 8-15   X: adds dX, writes X as an operand; where a third term of w C is
//                wanted, writes it into a half's buffer when the first two have been used
//   warps 16-23  P to its causal bf16 form
//   warps 24-31  scale A X^T in place (the product with P then adds to it), and put the
//                outputs where the chunk's A tile was (fp32: A and B tiles)
//   warp 2 stores them from there by TMA (a direct store of 32 rows by a warp is 32
//   scattered pieces, about 85 cycles of the load-store unit); warp 1 issues P, A X^T
//   and the product with P; warp 3 issues dX.
template <typename TO, bool BACK>
__global__ void __launch_bounds__(NTHREADS_O, 1)
scan_out_tc_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_o, const Scan p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tm_a);
    prefetch_tensormap(&tm_b);
    prefetch_tensormap(&tm_c);
    prefetch_tensormap(&tm_o);
  }
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  Unit u;
  if (!get_unit(p, blockIdx.x, u)) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_addr(smem);
  const int nch = (u.t1 - u.t0 + CH - 1) / CH;
  const int tail = u.t1 - u.t0 - (nch - 1) * CH;  // tokens of the last chunk
  volatile int *ctl = reinterpret_cast<volatile int *>(smem + OFF_CTL + 4);
  Weights *wts = reinterpret_cast<Weights *>(smem + OFF_W);
  auto bar = [&](int i) { return sb + OFF_BAR + 8u * i; };
  if (sb & 1023u) {  // swizzled operand tiles need 1024-byte alignment
    if (tid == 0) report_status(p.status, GDN_ERR_UNSUPPORTED);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NBAR; ++i) {
      // one arrival per warp of the group that signals; a stage is freed by both issuers
      const bool eight = i == B_DXFREE || i == B_OFREE || i == B_X || i == B_OUT || i == B_X0 || i == B_X0 + 1;
      const bool four = i == B_V || i == B_V + 1 || i == B_VL || i == B_VL + 1 || i == B_FIX;
      const int empty = sizeof(TO) == 4 ? 3 : 2;  // fp32: its B tile's place is stored from, too
      mbar_init(bar(i), i == B_PB ? 16 : eight ? 8 : four ? 4 : i == B_EMPTY || i == B_EMPTY + 1 ? empty :
                        i == B_DRAIN ? 2 : 1);
    }
    ctl[CTL_ABORT] = 0;
    ctl[CTL_LIMIT] = 4000000;  // until warp 2 has read the header
    fence_barrier_init();
    *reinterpret_cast<Unit *>(smem + OFF_UNIT) = u;
  }
  const float gh = head_decay(p, u.h);
  fill_weights(p, wts, gh, tail, tid);
  if (warp == 1) {
    tmem_alloc(sb + OFF_CTL, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + OFF_CTL);
  const bool exact = u.first && u.last && p.xf;  // the state is returned: three terms
  const int parts = exact ? 4 : 2;               // of dX
  auto chunk_of = [&](int ci) { return BACK ? nch - 1 - ci : ci; };
  auto arrive = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  auto warp_wait = [&](int b, uint32_t parity) { return wait_phase(bar(b), parity, ctl, p.status); };

  if (warp < 4) fewer_registers<32>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const int ha = u.h / (p.Hv / p.Ha), hb = u.h / (p.Hv / p.Hb), hc = u.h / (p.Hv / p.Hc);
      int issued = 0;
      auto prefetch = [&](int ci) {  // into L2, two chunks before the stage is free
        if (ci >= nch) return;
        const int t = u.t0 + chunk_of(ci) * CH;
        for (int half = 0; half < 2; ++half) {
          tma_prefetch_3d(&tm_a, 64 * half, ha, t);
          tma_prefetch_3d(&tm_b, 64 * half, hb, t);
          tma_prefetch_3d(&tm_c, 64 * half, hc, t);
        }
      };
      prefetch(2);
      prefetch(3);
      for (int ci = 0; ci < nch; ++ci) {
        const int s = ci & 1, t = u.t0 + chunk_of(ci) * CH;
        if (ci >= 2) prefetch(ci + 2);
        if (!wait_phase_alone(bar(B_EMPTY + s), ((ci >> 1) & 1) ^ 1, ctl)) break;
        // (the second stage holds the starting state at first)
        if (ci == 1 && !wait_phase_alone(bar(B_X0 + 1), 0, ctl)) break;
        const uint32_t st = sb + s * STAGE, fb = bar(B_FULL + s);
        mbar_arrive_expect_tx(fb, STAGE);
        for (int half = 0; half < 2; ++half) {
          tma_load_3d(st + TILE + half * 16384, &tm_b, fb, 64 * half, hb, t);
          tma_load_3d(st + 2 * TILE + half * 16384, &tm_c, fb, 64 * half, hc, t);
        }
        // the outputs have left the place of A
        const bool a_free = wait_phase_alone(bar(B_EMPTYA + s), ((ci >> 1) & 1) ^ 1, ctl);
        for (int half = 0; half < 2; ++half) tma_load_3d(st + half * 16384, &tm_a, fb, 64 * half, ha, t);
        issued = ci + 1;
        if (!a_free) break;
      }
      if (issued < nch || ctl[CTL_ABORT]) {
        ctl[CTL_ABORT] = 1;
        report_status(p.status, GDN_ERR_DEVICE_TIMEOUT);
      }
      // every load this thread issued lands before the CTA can exit
      for (int ci = max(issued - 2, 0); ci < issued; ++ci)
        mbar_wait_landed(bar(B_FULL + (ci & 1)), (ci >> 1) & 1, 50000000ull);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer of the outputs
    const uint64_t dA0 = sdesc_sw128(sb, 16, 1024), dB0 = sdesc_sw128(sb + TILE, 16, 1024);
    const uint64_t dCm0 = sdesc_sw128(sb + 2 * TILE, 16384, 1024), dX = sdesc_sw128(sb + OFF_X, 16, 1024);
    for (int ci = 0; ci < nch; ++ci) {
      const int s = ci & 1;
      const uint32_t ph = ci & 1;
      const uint64_t so = (uint64_t)(s * (STAGE >> 4));
      if (!warp_wait(B_FULL + s, (ci >> 1) & 1)) break;
      if (chunk_of(ci) == nch - 1 && tail < CH && !warp_wait(B_FIX, 0)) break;
      if (elect_one()) {
#pragma unroll 1
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t k16 = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
          mma_bf16(tmem + R_P, dA0 + so + k16, dB0 + so + k16, IDESC_KK, ks > 0);
        }
        mma_commit(bar(B_P));
      }
      __syncwarp();
      if (!warp_wait(B_X, ph) || (ci > 0 && !warp_wait(B_OFREE, (ci - 1) & 1))) break;
      if (elect_one()) {
#pragma unroll 1
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t k16 = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
          mma_bf16(tmem + R_O, dA0 + so + k16, dX + k16, IDESC_KK, ks > 0);
        }
        mma_commit(bar(B_OI));
      }
      __syncwarp();
      if (!warp_wait(B_PB, ph)) break;
      if (elect_one()) {
#pragma unroll 1
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(tmem + R_O, tmem + T_PB + pcol(kk), dCm0 + so + ((kk * 2048) >> 4), IDESC_KM, 1);
        mma_commit(bar(B_OA));
        mma_commit(bar(B_EMPTY + s));
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(bar(B_DRAIN));
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ MMA issuer of dX
    const uint64_t dBm0 = sdesc_sw128(sb + TILE, 16384, 1024);
    for (int ci = 0; ci < nch; ++ci) {
      const int s = ci & 1;
      const uint32_t ph = ci & 1;
      const uint64_t so = (uint64_t)(s * (STAGE >> 4));
      if (!warp_wait(B_FULL + s, (ci >> 1) & 1)) break;
      if (ci > 0 && !warp_wait(B_DXFREE, (ci - 1) & 1)) break;
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < parts; ++j) {  // halves of the tokens; again for the third term
        const int hf = j & 1;
        // (the terms are written after a short tile was zeroed)
        if (!(ok = warp_wait(j < 2 ? B_V + hf : B_VL + hf, ph))) break;
        if (elect_one()) {
#pragma unroll 1
          for (int kk = 4 * hf; kk < 4 * hf + 4; ++kk) {
            const uint64_t db = dBm0 + so + ((kk * 2048) >> 4);
            mma_bf16_ts(tmem + R_DX, tmem + T_VH + 8 * kk, db, IDESC_KM, j + kk > 0);
            if (j < 2) mma_bf16_ts(tmem + R_DX, tmem + T_VM + 8 * kk, db, IDESC_KM, 1);
          }
          mma_commit(bar((j + 2 < parts ? B_VUSED : B_VFREE) + hf));  // used by two terms; by all
          if (j == parts - 1) {
            mma_commit(bar(B_DX));
            mma_commit(bar(B_DXO + s));
            mma_commit(bar(B_EMPTY + s));
          }
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    // Drain: every MMA that the two issuers sent finishes before TMEM is freed.
    if (elect_one()) {
      mma_commit(bar(B_DRAIN));
      mbar_wait_landed(bar(B_DRAIN), 0, 50000000ull);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ stores
    if (lane == 0) ctl[CTL_LIMIT] = wait_limit(p.status);
    __syncwarp();
    constexpr int BOXES = 4 * (int)sizeof(TO);  // of 32 rows by 128 bytes
    for (int ci = 0; ci < nch; ++ci) {
      const int c = chunk_of(ci), s = ci & 1;
      const int len = c == nch - 1 ? tail : CH;
      if (!warp_wait(B_OUT, ci & 1)) break;
      if (lane == 0) {
#pragma unroll 1
        for (int i = 0; i < BOXES; ++i) {
          const int hf = (i >> 2) & 1, r = 32 * (i & 3), col = 64 * hf + 32 * (i >> 3);
          if (r + 32 <= len && 64 * hf < p.Dc)  // boxes that end inside the sequence
            tma_store_3d(&tm_o, sb + s * STAGE + (i >> 2) * 16384 + r * 128, col, u.h, u.t0 + c * CH + r);
        }
        bulk_commit_group();
        bulk_wait_read_all();
        mbar_arrive(bar(B_EMPTYA + s));
        if (sizeof(TO) == 4) mbar_arrive(bar(B_EMPTY + s));
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_all();
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ w C
    fewer_registers<48>();
    const int gt = tid - 128, lq = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16);
    for (int ci = 0; ci < nch; ++ci) {
      const int s = ci & 1;
      const bool last = chunk_of(ci) == nch - 1;
      if (!warp_wait(B_FULL + s, (ci >> 1) & 1)) break;
      if (last && tail < CH) {
        unsigned char *st = smem + s * STAGE;
        zero_tail(st + TILE, tail, gt, 128);
        zero_tail(st + 2 * TILE, tail, gt, 128);
        fence_proxy_async_smem();
        arrive(B_FIX);
        if (!warp_wait(B_FIX, 0)) break;  // rows that other warps have zeroed are read
      }
      const float *wt = last ? wts->wtail : wts->wfull;
      const uint32_t ct = sb + s * STAGE + 2 * TILE;
      bool ok = true;
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        if (ci > 0 && !(ok = warp_wait(B_VFREE + hf, (ci - 1) & 1))) break;
        scale_split<2, 4>(ct, wt, lq, lane, 64 * hf, tl + T_VH + 32 * hf, tl + T_VM + 32 * hf, 0);
        tmem_wait_st();
        tc_fence_before();
        arrive(B_V + hf);
      }
      if (!ok) break;
    }
  } else if (warp >= 8 && warp < 16) {
    // ------------------------------------------------------------ X
    more_registers<104>();
    const int hf = (warp - 8) >> 2;                 // half of the columns of X
    const int lq = warp & 3, row = 32 * lq + lane;  // TMEM lane: row of X and dX
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16);
    float X[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) X[i] = 0.f;
    // (a warp's lanes agree on all of these)
    const bool mine = row < p.Dc && 64 * hf < p.Da, own = u.first && u.last;  // own: starts from x0
    const bool some = mine && (!own || p.x0), by_copy = some && !(own && p.x0_tr), bf = own && p.x_bf16 && by_copy;
    const uint32_t slot = (128 * hf + row) * 272;
    if (by_copy) {
      const size_t e0 = (((size_t)(own ? u.n : u.seg) * p.Hv + u.h) * p.Dc + row) * p.Da + 64 * hf;
      const unsigned char *src = static_cast<const unsigned char *>(own ? p.x0 : p.seg_state) + e0 * (bf ? 2 : 4);
      const uint32_t bytes = bf ? 128 : 256;
      if (lane == 0) mbar_arrive_expect_tx(bar(B_X0), 32 * bytes);
      __syncwarp();
      bulk_load(sb + STAGE + slot, src, bytes, bar(B_X0));
    } else {
      if (some) {
#pragma unroll 4
        for (int i = 0; i < 64; ++i)
          *reinterpret_cast<float *>(smem + STAGE + slot + 4 * i) = initial_state(p, u, row, 64 * hf + i);
        fence_proxy_async_smem();  // these ordinary stores come before the tiles that TMA writes there
      }
      arrive(B_X0);
    }
    bool ok = warp_wait(B_X0, 0);
    if (!ok) mbar_wait_landed(bar(B_X0), 0, 50000000ull);  // the copies land before the CTA can exit
    if (ok && some) {
      const unsigned char *at = smem + STAGE + slot;
      if (bf) {
#pragma unroll
        for (int i = 0; i < 64; i += 4) load4(reinterpret_cast<const __nv_bfloat16 *>(at) + i, X + i);
      } else {
#pragma unroll
        for (int i = 0; i < 64; i += 4) load4(reinterpret_cast<const float *>(at) + i, X + i);
      }
    }
    arrive(B_X0 + 1);
    auto put_x = [&]() {
      unsigned char *xo = smem + OFF_X + hf * 16384;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float *x = X + 8 * c;
        *reinterpret_cast<uint4 *>(xo + sw128_off(row, c)) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      }
      fence_proxy_async_smem();
      arrive(B_X);
    };
    if (nch > 0) put_x();
    for (int ci = 0; ok && ci < nch; ++ci) {
      const uint32_t ph = ci & 1;
      const int len = chunk_of(ci) == nch - 1 ? tail : CH, skip = BACK && u.first && ci == 0 ? 1 : 0;
      if (exact) {
        const int s = ci & 1;
        const bool last = chunk_of(ci) == nch - 1;
        if (!(ok = warp_wait(B_FULL + s, (ci >> 1) & 1) && (!last || tail == CH || warp_wait(B_FIX, 0)) &&
                   warp_wait(B_VUSED + hf, ph)))
          break;
        scale_split<1, 4>(sb + s * STAGE + 2 * TILE, last ? wts->wtail : wts->wfull, lq, lane, 64 * hf,
                          tl + T_VH + 32 * hf, 0, 0);
        tmem_wait_st();
        tc_fence_before();
        arrive(B_VL + hf);
      }
      if (!(ok = warp_wait(B_DX, ph))) break;
      Carry carry = wts->carry[warp - 8];
      const float lx = carry.next(Power{wts->pw[len - skip], wts->pm[len - skip]});
      __syncwarp();
      if (lane == 0) wts->carry[warp - 8] = carry;  // (not kept in a register beside X)
#pragma unroll
      for (int i = 0; i < 64; i += 8) {
        float d[8];
        tmem_ld8(tl + R_DX + 64 * hf + i, d);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k) X[i + k] = fmaf(lx, X[i + k], d[k]);
      }
      tc_fence_before();
      arrive(B_DXFREE);
      if (ci + 1 < nch) {
        if (!(ok = warp_wait(B_OI, ph))) break;  // A X^T has read the operand
        put_x();
      }
    }
    if (exact && ok && nch > 1) {  // the stage before the last one, once all have left it
      const int s = nch & 1;
      ok = warp_wait(B_EMPTY + s, ((nch - 2) >> 1) & 1) && warp_wait(B_EMPTYA + s, ((nch - 2) >> 1) & 1);
    }
    if (exact && ok) {
      // what only the end needs is read again, not kept through the loop beside X
      uint32_t t2;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t2));
      const volatile Unit *u2 = reinterpret_cast<const volatile Unit *>(smem + OFF_UNIT);
      const int half = (t2 - 256) >> 7, r = t2 & 127;
      if (r < p.Dc && 64 * half < p.Da) {
        const float f = BACK && nch > 0 ? wts->pw[1] : 1.f;
        const size_t e0 = (((size_t)u2->n * p.Hv + u2->h) * p.Dc + r) * p.Da + 64 * half;
        const uint32_t at = (nch & 1) * STAGE + (128 * half + r) * 272;
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const float y[4] = {f * X[i], f * X[i + 1], f * X[i + 2], f * X[i + 3]};
          store_state4(smem + at, i, p.x_bf16, y);
        }
        fence_proxy_async_smem();
        bulk_store(static_cast<unsigned char *>(p.xf) + e0 * (p.x_bf16 ? 2 : 4), sb + at, p.x_bf16 ? 128 : 256);
        bulk_commit_group();
        bulk_wait_all();
      }
    }
  } else if (warp >= 16 && warp < 24) {
    // ------------------------------------------------------------ P -> its causal, decayed part in bf16
    fewer_registers<64>();
    const int hf = (warp - 16) >> 2;                // half of the columns of P
    const int lq = warp & 3, row = 32 * lq + lane;  // TMEM lane: token
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16);
    const float lam = wts->pw[1];
    for (int ci = 0; ci < nch; ++ci) {
      if (!warp_wait(B_P, ci & 1)) break;
      uint32_t pb[16];
#pragma unroll 1
      for (int j = 0; j < 2; ++j) {
        const int q = 2 * hf + j;  // 32-wide column block
        if (BACK ? q >= lq : q <= lq) {
          float v[32];
          tmem_ld32(tl + R_P + 32 * q, v);
          tmem_wait_ld();
          // times s_intra lam^{|t-s|}, from the nearest column of the block to the farthest
          if (q != lq) {
            float w = wts->pwi[BACK ? 32 * q - row : row - 32 * q - 31];
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              const int i = BACK ? n : 31 - n;
              v[i] *= w;
              w *= lam;
            }
          } else {
            float w = 0.f;
#pragma unroll
            for (int n = 0; n < 32; ++n) {
              const int i = BACK ? n : 31 - n;
              if (i == lane) w = p.s_intra;
              v[i] = (BACK ? i >= lane : i <= lane) ? v[i] * w : 0.f;
              w *= lam;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) pb[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) pb[i] = 0u;
        }
        // (over columns of P that this warp has read)
        tmem_st16(tl + T_PB + 64 * hf + 16 * j, pb);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(B_PB);
    }
  } else if (warp >= 24) {
    // ------------------------------------------------------------ A X^T scaled in place; outputs
    fewer_registers<48>();
    const int hf = (warp - 24) >> 2;                // half of the columns of O
    const int lq = warp & 3, row = 32 * lq + lane;  // TMEM lane: token
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16) + R_O + 64 * hf;
    for (int ci = 0; ci < nch; ++ci) {
      const int c = chunk_of(ci), s = ci & 1;
      const uint32_t ph = ci & 1;
      const int len = c == nch - 1 ? tail : CH, skip = BACK && u.first && ci == 0 ? 1 : 0;
      if (!warp_wait(B_OI, ph)) break;
      const float wi = row < len ? p.s_inter * wts->pw[(BACK ? len - 1 - row : row) + 1 - skip] : 0.f;
#pragma unroll 1
      for (int i = 0; i < 64; i += 32) {
        float v[32];
        tmem_ld32(tl + i, v);
        tmem_wait_ld();
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(wi * v[k]);
        tmem_st32(tl + i, w);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(B_PB);
      if (!warp_wait(B_OA, ph)) break;
      if (sizeof(TO) == 4 && !warp_wait(B_DXO + s, (ci >> 1) & 1)) break;  // dX has used the B tile
      // rows of this warp: boxes of 32 rows by 128 bytes, 32 (fp32) or 64 columns, at their
      // places in the tiles
      unsigned char *box = smem + s * STAGE + hf * 16384 + lq * 4096;
      const bool whole = 32 * lq + 32 <= len;
#pragma unroll
      for (int j = 0; j < 64; j += 32) {
        float v[32];
        tmem_ld32(tl + j, v);
        tmem_wait_ld();
        if (j == 32) {
          tc_fence_before();
          arrive(B_OFREE);
        }
        constexpr int W = 32 * sizeof(TO) / 4;  // words
        uint32_t w[W];
#pragma unroll
        for (int k = 0; k < W; ++k)
          w[k] = sizeof(TO) == 2 ? pack_bf16x2(v[(2 * k) % 32], v[(2 * k + 1) % 32]) : __float_as_uint(v[k]);
        unsigned char *at = sizeof(TO) == 4 ? box + (j / 32) * TILE : box;
        const int ch0 = sizeof(TO) == 4 ? 0 : j / 8;
        if (whole) {
#pragma unroll
          for (int k = 0; k < W; k += 4)
            *reinterpret_cast<uint4 *>(at + sw128_off(lane, ch0 + k / 4)) =
                make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
        } else if (row < len && 64 * hf < p.Dc) {  // the rows after belong to the next sequence
          TO *o = static_cast<TO *>(p.out) + ((size_t)(u.t0 + c * CH + row) * p.Hv + u.h) * p.Dc + 64 * hf + j;
#pragma unroll
          for (int k = 0; k < W; k += 4)
            *reinterpret_cast<uint4 *>(o + k * 4 / (int)sizeof(TO)) = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
        }
      }
      fence_proxy_async_smem();
      arrive(B_OUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- states
// What a segment adds to the state: 3 stages of B, C tiles; w C double-buffered in
// TMEM, so that the next chunk's terms are formed while this one's product runs.
constexpr uint32_t STAGE_S = 2 * TILE;
constexpr int NST_S = 3;
constexpr uint32_t OFF_W_S = NST_S * STAGE_S;
constexpr uint32_t OFF_BAR_S = OFF_W_S + ((sizeof(Weights) + 15) / 16) * 16;
constexpr uint32_t OFF_CTL_S = OFF_BAR_S + 128;
constexpr uint32_t SMEM_STATE = OFF_CTL_S + 32;
static_assert(SMEM_STATE <= 232448, "shared memory of a CTA");
enum { S_FULL = 0, S_EMPTY = 3, S_V = 6, S_DX = 8, S_FREE = 9, S_FIX = 10, S_DRAIN = 11, S_NBAR = 12 };
constexpr uint32_t S_TV = 0, S_RDX = 384;  // 2 x 192 columns of terms, 128 of dX

__global__ void __launch_bounds__(NTHREADS, 1)
scan_state_tc_kernel(const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                     const Scan p) {
  extern __shared__ __align__(1024) unsigned char smem[];
  if (threadIdx.x == 0) {
    prefetch_tensormap(&tm_b);
    prefetch_tensormap(&tm_c);
  }
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  Unit u;
  if (!get_unit(p, blockIdx.x, u)) return;
  if (u.last && (u.first || !p.xf)) return;  // nothing starts from its end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sb = smem_addr(smem);
  const int nch = (u.t1 - u.t0 + CH - 1) / CH;
  const int tail = u.t1 - u.t0 - (nch - 1) * CH;
  volatile int *ctl = reinterpret_cast<volatile int *>(smem + OFF_CTL_S + 4);
  Weights *wts = reinterpret_cast<Weights *>(smem + OFF_W_S);
  auto bar = [&](int i) { return sb + OFF_BAR_S + 8u * i; };
  if (sb & 1023u) {  // swizzled operand tiles need 1024-byte alignment
    if (tid == 0) report_status(p.status, GDN_ERR_UNSUPPORTED);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < S_NBAR; ++i)
      mbar_init(bar(i), i == S_V || i == S_V + 1 || i == S_FREE || i == S_FIX ? 16 : 1);
    ctl[CTL_ABORT] = 0;
    ctl[CTL_LIMIT] = 4000000;  // until warp 2 has read the header
    fence_barrier_init();
  }
  const float gh = head_decay(p, u.h);
  fill_weights(p, wts, gh, tail, tid);
  if (warp == 1) {
    tmem_alloc(sb + OFF_CTL_S, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + OFF_CTL_S);
  auto chunk_of = [&](int ci) { return p.back ? nch - 1 - ci : ci; };
  auto warp_wait = [&](int b, uint32_t parity) { return wait_phase(bar(b), parity, ctl, p.status); };

  if (warp == 0) {
    if (lane == 0) {
      const int hb = u.h / (p.Hv / p.Hb), hc = u.h / (p.Hv / p.Hc);
      int issued = 0;
      for (int ci = 0; ci < nch; ++ci) {
        const int s = ci % NST_S, t = u.t0 + chunk_of(ci) * CH;
        if (!wait_phase_alone(bar(S_EMPTY + s), ((ci / NST_S) & 1) ^ 1, ctl)) break;
        const uint32_t st = sb + s * STAGE_S, fb = bar(S_FULL + s);
        mbar_arrive_expect_tx(fb, STAGE_S);
        for (int half = 0; half < 2; ++half) {
          tma_load_3d(st + half * 16384, &tm_b, fb, 64 * half, hb, t);
          tma_load_3d(st + TILE + half * 16384, &tm_c, fb, 64 * half, hc, t);
        }
        issued = ci + 1;
      }
      if (issued < nch) {
        ctl[CTL_ABORT] = 1;
        report_status(p.status, GDN_ERR_DEVICE_TIMEOUT);
      }
      for (int ci = max(issued - NST_S, 0); ci < issued; ++ci)
        mbar_wait_landed(bar(S_FULL + ci % NST_S), (ci / NST_S) & 1, 50000000ull);
    }
  } else if (warp == 1) {
    const uint64_t dBm0 = sdesc_sw128(sb, 16384, 1024);
    for (int ci = 0; ci < nch; ++ci) {
      const int s = ci % NST_S;
      const uint64_t so = (uint64_t)(s * (STAGE_S >> 4));
      // (the terms are written after the tile landed and, if short, was zeroed)
      if (!warp_wait(S_FULL + s, (ci / NST_S) & 1)) break;
      if (!warp_wait(S_V + (ci & 1), (ci >> 1) & 1)) break;
      if (ci > 0 && !warp_wait(S_FREE, (ci - 1) & 1)) break;  // the last dX has been read
      if (elect_one()) {
        const uint32_t tv = tmem + S_TV + 192 * (ci & 1);
#pragma unroll
        for (int ks = 0; ks < 24; ++ks) {  // low terms first
          const int kk = ks & 7;
          mma_bf16_ts(tmem + S_RDX, tv + 64 * (2 - (ks >> 3)) + 8 * kk, dBm0 + so + ((kk * 2048) >> 4), IDESC_KM,
                      ks > 0);
        }
        mma_commit(bar(S_DX));
        mma_commit(bar(S_EMPTY + s));
      }
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(bar(S_DRAIN));
      mbar_wait_landed(bar(S_DRAIN), 0, 50000000ull);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) ctl[CTL_LIMIT] = wait_limit(p.status);
  } else if (warp >= 4) {
    const int etid = tid - 128, q = etid >> 7, lq = warp & 3, row = 32 * lq + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16);
    auto arrive = [&](int b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    float X[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) X[i] = 0.f;
    auto terms = [&](int ci) {
      const int s = ci % NST_S;
      unsigned char *st = smem + s * STAGE_S;
      const bool last = chunk_of(ci) == nch - 1;
      if (!warp_wait(S_FULL + s, (ci / NST_S) & 1)) return false;
      if (last && tail < CH) {
        zero_tail(st, tail, etid, 512);
        zero_tail(st + TILE, tail, etid, 512);
        fence_proxy_async_smem();
        arrive(S_FIX);
        if (!warp_wait(S_FIX, 0)) return false;
      }
      const uint32_t tv = tl + S_TV + 192 * (ci & 1);
      scale_split<3, 2>(sb + s * STAGE_S + TILE, last ? wts->wtail : wts->wfull, lq, lane, 32 * q, tv + 16 * q,
                        tv + 64 + 16 * q, tv + 128 + 16 * q);
      tmem_wait_st();
      tc_fence_before();
      arrive(S_V + (ci & 1));
      return true;
    };
    Carry carry{0.f};
    bool ok = nch == 0 || terms(0);
    for (int ci = 0; ci < nch && ok; ++ci) {
      if (ci + 1 < nch && !(ok = terms(ci + 1))) break;
      if (!(ok = warp_wait(S_DX, ci & 1))) break;
      float d[32];
      tmem_ld32(tl + S_RDX + 32 * q, d);
      tmem_wait_ld();
      tc_fence_before();
      arrive(S_FREE);
      const int len = chunk_of(ci) == nch - 1 ? tail : CH;
      const float lx = carry.next(Power{wts->pw[len], wts->pm[len]});
#pragma unroll
      for (int i = 0; i < 32; ++i) X[i] = fmaf(lx, X[i], d[i]);
    }
    if (ok && row < p.Dc && 32 * q < p.Da) {  // (every tile has been used)
      const uint32_t at = (128 * q + row) * 144;
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<float4 *>(smem + at + 4 * i) = make_float4(X[i], X[i + 1], X[i + 2], X[i + 3]);
      fence_proxy_async_smem();
      bulk_store(p.seg_state + (((size_t)u.seg * p.Hv + u.h) * p.Dc + row) * p.Da + 32 * q, sb + at, 128);
      bulk_commit_group();
      bulk_wait_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Tensor map of a packed [T, H, D] bf16 (or fp32) tensor viewed as (d, head, token), box
// 128 bytes of d x 1 head x `rows` tokens, 128-byte swizzle.  Tokens past T and columns
// past D read as zeros and are not written.
bool make_map(CUtensorMap *m, const void *base, int H, int T, int D, bool fp32 = false, int rows = CH) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t eb = fp32 ? 4 : 2;
  const cuuint64_t strides[2] = {D * eb, (cuuint64_t)H * D * eb};
  const cuuint32_t box[3] = {fp32 ? 32u : 64u, 1, (cuuint32_t)rows}, elem[3] = {1, 1, 1};
  return encode(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, elem,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool scan_tc_supported(const Scan &p, int dtype) {
  return dtype == GDN_DTYPE_BF16 && p.T > 0 && p.T <= INT32_MAX - CH;
}

cudaError_t launch_scan_tc(const Scan &p, int units, int out_dtype, cudaStream_t stream) {
  static std::atomic<bool> f0[64], f1[64], f2[64], f3[64], f4[64];
  CUtensorMap ma, mb, mc, mo;
  if (!make_map(&mb, p.b, p.Hb, p.T, p.Da) || !make_map(&mc, p.c, p.Hc, p.T, p.Dc)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (p.states_only) {
    if ((e = set_smem_once(scan_state_tc_kernel, SMEM_STATE, f0)) != cudaSuccess) return e;
    return launch_pdl(scan_state_tc_kernel, dim3((unsigned)units), dim3(NTHREADS), SMEM_STATE, stream, mb, mc, p);
  }
  if (!make_map(&ma, p.a, p.Ha, p.T, p.Da) || !make_map(&mo, p.out, p.Hv, p.T, p.Dc, out_dtype == GDN_DTYPE_FP32, 32))
    return cudaErrorInvalidValue;
  auto go = [&](auto kern, std::atomic<bool>(&flags)[64]) {
    const cudaError_t r = set_smem_once(kern, SMEM_OUT, flags);
    if (r != cudaSuccess) return r;
    return launch_pdl(kern, dim3((unsigned)units), dim3(NTHREADS_O), SMEM_OUT, stream, ma, mb, mc, mo, p);
  };
  if (out_dtype == GDN_DTYPE_BF16)
    return p.back ? go(scan_out_tc_kernel<__nv_bfloat16, true>, f1) : go(scan_out_tc_kernel<__nv_bfloat16, false>, f2);
  return p.back ? go(scan_out_tc_kernel<float, true>, f3) : go(scan_out_tc_kernel<float, false>, f4);
}

}  // namespace lin
}  // namespace gdn
