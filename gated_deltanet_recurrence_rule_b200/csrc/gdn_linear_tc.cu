// gdn_linear_tc.cu -- the scan of linear attention (gdn_linear.cuh) on the
// Blackwell tensor cores: tcgen05 with TMEM accumulators, TMA tiles; bf16 operands
// and output, head dims 128, fp32 state.
//
// Chunks of 128 tokens, so that every product is a full 128 x 128 x 128 tile:
//     P  = A B^T                     A, B, C: the chunk's rows of a, b, c
//     Oi = A X^T                     X (Dc x Da) the state before the chunk
//     Oa = (P . lam^{|t-s|}) C       causal
//     dX = (w C)^T B                 w_t = s_upd lam^{rest}
//     out_t = s_inter lam^{p+1} Oi_t + s_intra Oa_t,   X <- lam^len X + dX.
// Precision.  A, B, C are exact bf16.  The state is fp32 in registers; w C enters dX
// as three bf16 terms (24 bits: exact to fp32), each chunk's dX is summed apart and
// added once, rounded to nearest.  P . lam^{..} and X are rounded to bf16 once as
// operands of the output, whose own rounding to bf16 is as large.
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

constexpr int CH = 128, HD = 128;
constexpr int NTHREADS = 640;  // warp 0 TMA, warp 1 MMA, warp 2 wait limit, warps 4-19 epilogue
constexpr uint32_t TILE = 32768;  // 128 rows x 128 bf16: [d 0-63 | d 64-127], 128-byte rows, swizzled

// ---- instruction descriptors ----
constexpr uint32_t IDESC_KK = idesc_bf16(128, 128, 0, 0);  // A B^T, A X^T: both K-major
constexpr uint32_t IDESC_KM = idesc_bf16(128, 128, 0, 1);  // (wC)^T B, P C: B operand MN-major

struct Weights {        // fp32 tables in shared memory
  float pw[CH + 4];     // lam^i
  float wfull[CH], wtail[CH];  // w_t of a full chunk and of the segment's last one
  float cf[32];         // column factors of a 32-wide block of P
};

__device__ __forceinline__ void fill_weights(const Scan &p, Weights *w, float gh, int tail, int tid) {
  if (tid <= CH) w->pw[tid] = expf(gh * (float)tid);
  if (tid < CH) {
    const int rf = p.back ? tid : CH - 1 - tid, rt = p.back ? tid : tail - 1 - tid;
    w->wfull[tid] = p.s_upd * expf(gh * (float)rf);
    w->wtail[tid] = tid < tail ? p.s_upd * expf(gh * (float)rt) : 0.f;
  }
  if (tid < 32) w->cf[tid] = expf(gh * (float)(p.back ? tid : 31 - tid));
}

// Rows [len, 128) of a tile <- 0, by the 512 epilogue threads: what TMA read there
// belongs to the next sequence, and 0 * NaN would carry it over.
__device__ __forceinline__ void zero_tail(unsigned char *tile, int len, int etid) {
  for (int x = etid; x < (CH - len) * 16; x += 512) {
    const int r = len + (x >> 4), ch = x & 15;
    *reinterpret_cast<uint4 *>(tile + (ch >> 3) * 16384 + r * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// (w C)^T as the A operand of dX: lane = row of X (column `row` of C), token pairs
// [32 q, 32 q + 32) in three bf16 terms of 16 words each.
__device__ __forceinline__ void scale_split(const unsigned char *tile, const float *wt, int row, int q,
                                            uint32_t t_hi, uint32_t t_mid, uint32_t t_lo) {
  const unsigned char *base = tile + (row >> 6) * 16384 + 32 * q * 128 + (row & 7) * 2;
  const uint32_t ch = (row & 63) >> 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t hi[8], mid[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 w4 = *reinterpret_cast<const float4 *>(wt + 32 * q + 16 * half + 2 * i);
      const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = 16 * half + 2 * (i + k);
        const uint32_t c0 = *reinterpret_cast<const unsigned short *>(base + t * 128 + ((ch ^ (t & 7)) << 4));
        const uint32_t c1 =
            *reinterpret_cast<const unsigned short *>(base + (t + 1) * 128 + ((ch ^ ((t + 1) & 7)) << 4));
        float x0 = w[2 * k] * __uint_as_float(c0 << 16), x1 = w[2 * k + 1] * __uint_as_float(c1 << 16);
        hi[i + k] = pack_bf16x2(x0, x1);
        x0 -= __uint_as_float(hi[i + k] << 16);
        x1 -= __uint_as_float(hi[i + k] & 0xffff0000u);
        mid[i + k] = pack_bf16x2(x0, x1);
        x0 -= __uint_as_float(mid[i + k] << 16);
        x1 -= __uint_as_float(mid[i + k] & 0xffff0000u);
        lo[i + k] = pack_bf16x2(x0, x1);
      }
    }
    tmem_st8(t_hi + 16 * q + 8 * half, hi);
    tmem_st8(t_mid + 16 * q + 8 * half, mid);
    tmem_st8(t_lo + 16 * q + 8 * half, lo);
  }
}

__device__ __forceinline__ void st_global_32b(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// ---------------------------------------------------------------- outputs
// Shared memory of the output kernel: 2 stages of A, B, C tiles, X as an operand.
constexpr uint32_t STAGE = 3 * TILE;
constexpr uint32_t OFF_X = 2 * STAGE;
constexpr uint32_t OFF_W = OFF_X + TILE;
constexpr uint32_t OFF_BAR = OFF_W + ((sizeof(Weights) + 15) / 16) * 16;
constexpr uint32_t OFF_CTL = OFF_BAR + 128;  // TMEM base, control words
constexpr uint32_t SMEM_OUT = OFF_CTL + 32;
static_assert(SMEM_OUT <= 232448, "shared memory of a CTA");

// TMEM columns.  P (fp32) is overwritten by its own bf16 form, and the columns that
// frees take the low terms of w C; the others share the columns of Oa, which dX, issued
// before, has finished reading when Oa is written.
constexpr uint32_t R_P = 0, T_PB = 0, T_VL = 64, R_OI = 128, R_OA = 256, T_VH = 256, T_VM = 320, R_DX = 384;

enum { B_FULL = 0, B_EMPTY = 2, B_P = 4, B_PREAD = 5, B_PB = 9, B_V = 10, B_DX = 11, B_OA = 12, B_X = 13, B_FIX = 14,
       B_DRAIN = 15, NBAR = 16 };
static_assert(NBAR * 8 <= 128, "barrier area");

// One CTA per (segment, head).  The 16 epilogue warps go through a chunk's four
// elementwise phases together (P, w C, X, out), 32 elements a thread each, while the
// tensor pipe works on the products already fed.
template <typename TO>
__global__ void __launch_bounds__(NTHREADS, 1)
scan_out_tc_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ CUtensorMap tm_c, const Scan p) {
  extern __shared__ __align__(1024) unsigned char smem[];
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
      const bool all = i == B_PB || i == B_V || i == B_X || i == B_FIX;  // every epilogue warp
      mbar_init(bar(i), all ? 16 : (i >= B_PREAD && i < B_PREAD + 4) ? 4 : 1);
    }
    ctl[CTL_ABORT] = 0;
    ctl[CTL_LIMIT] = 0;
    fence_barrier_init();
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
  // the chunk of a step, and whether it is the segment's short last one
  auto chunk_of = [&](int ci) { return p.back ? nch - 1 - ci : ci; };
  auto warp_wait = [&](int b, uint32_t parity) {
    int ok = 1;
    if (lane == 0 && !(ok = mbar_wait(bar(b), parity, ctl))) {
      ctl[CTL_ABORT] = 1;
      report_status(p.status, GDN_ERR_DEVICE_TIMEOUT);
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    if (ok) tc_fence_after();
    return ok != 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const int ha = u.h / (p.Hv / p.Ha), hb = u.h / (p.Hv / p.Hb), hc = u.h / (p.Hv / p.Hc);
      int issued = 0;
      for (int ci = 0; ci < nch; ++ci) {
        const int s = ci & 1, t = u.t0 + chunk_of(ci) * CH;
        if (!mbar_wait(bar(B_EMPTY + s), ((ci >> 1) & 1) ^ 1, ctl)) break;
        const uint32_t st = sb + s * STAGE, fb = bar(B_FULL + s);
        mbar_arrive_expect_tx(fb, STAGE);
        for (int half = 0; half < 2; ++half) {
          tma_load_3d(st + half * 16384, &tm_a, fb, 64 * half, ha, t);
          tma_load_3d(st + TILE + half * 16384, &tm_b, fb, 64 * half, hb, t);
          tma_load_3d(st + 2 * TILE + half * 16384, &tm_c, fb, 64 * half, hc, t);
        }
        issued = ci + 1;
      }
      if (issued < nch) {
        ctl[CTL_ABORT] = 1;
        report_status(p.status, GDN_ERR_DEVICE_TIMEOUT);
      }
      // every load this thread issued lands before the CTA can exit
      for (int ci = max(issued - 2, 0); ci < issued; ++ci)
        mbar_wait_landed(bar(B_FULL + (ci & 1)), (ci >> 1) & 1, 50000000ull);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint64_t dA0 = sdesc_sw128(sb, 16, 1024), dB0 = sdesc_sw128(sb + TILE, 16, 1024);
    const uint64_t dBm0 = sdesc_sw128(sb + TILE, 16384, 1024), dCm0 = sdesc_sw128(sb + 2 * TILE, 16384, 1024);
    const uint64_t dX = sdesc_sw128(sb + OFF_X, 16, 1024);
    for (int ci = 0; ci < nch; ++ci) {
      const int s = ci & 1;
      const uint32_t ph = ci & 1;
      const uint64_t so = (uint64_t)(s * (STAGE >> 4));
      if (!warp_wait(B_FULL + s, (ci >> 1) & 1)) break;
      if (chunk_of(ci) == nch - 1 && tail < CH && !warp_wait(B_FIX, 0)) break;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t k16 = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
          mma_bf16(tmem + R_P, dA0 + so + k16, dB0 + so + k16, IDESC_KK, ks > 0);
        }
        mma_commit(bar(B_P));
      }
      __syncwarp();
      if (!warp_wait(B_X, ph)) break;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t k16 = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
          mma_bf16(tmem + R_OI, dA0 + so + k16, dX + k16, IDESC_KK, ks > 0);
        }
      }
      __syncwarp();
      if (!warp_wait(B_V, ph)) break;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 24; ++ks) {  // low terms first
          const int kk = ks & 7;
          const uint32_t ta = ks < 8 ? T_VL : ks < 16 ? T_VM : T_VH;
          mma_bf16_ts(tmem + R_DX, tmem + ta + 8 * kk, dBm0 + so + ((kk * 2048) >> 4), IDESC_KM, ks > 0);
        }
        mma_commit(bar(B_DX));
      }
      __syncwarp();
      if (!warp_wait(B_PB, ph)) break;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_bf16_ts(tmem + R_OA, tmem + T_PB + 8 * ks, dCm0 + so + ((ks * 2048) >> 4), IDESC_KM, ks > 0);
        mma_commit(bar(B_OA));
        mma_commit(bar(B_EMPTY + s));
      }
      __syncwarp();
    }
    // Drain: every MMA this warp issued finishes before TMEM is freed.
    if (elect_one()) {
      mma_commit(bar(B_DRAIN));
      mbar_wait_landed(bar(B_DRAIN), 0, 50000000ull);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) ctl[CTL_LIMIT] = (int)header_wait_limit_us(p.status);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int etid = tid - 128, q = etid >> 7;  // column quarter
    const int lq = warp & 3, row = 32 * lq + lane;  // TMEM lane: token of P, Oi, Oa; row of X and dX
    const uint32_t tl = tmem + ((uint32_t)(32 * lq) << 16);
    float X[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) X[i] = start_state(p, u, row, 32 * q + i);
    auto put_x = [&]() {
      unsigned char *xo = smem + OFF_X + (q >> 1) * 16384;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float *x = X + 8 * c;
        *reinterpret_cast<uint4 *>(xo + sw128_off(row, 4 * (q & 1) + c)) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      }
      fence_proxy_async_smem();
    };
    auto arrive = [&](int b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    if (nch > 0) {
      put_x();
      arrive(B_X);
    }
    bool ok = true;
    for (int ci = 0; ci < nch; ++ci) {
      const int s = ci & 1, c = chunk_of(ci);
      const uint32_t ph = ci & 1;
      const bool last = c == nch - 1;
      const int len = last ? tail : CH, skip = p.back && u.first && ci == 0 ? 1 : 0;
      unsigned char *st = smem + s * STAGE;
      if (!(ok = warp_wait(B_FULL + s, (ci >> 1) & 1))) break;
      if (len < CH) {
        zero_tail(st + TILE, len, etid);
        zero_tail(st + 2 * TILE, len, etid);
        fence_proxy_async_smem();
        arrive(B_FIX);
        // the w C phase reads rows that other warps have zeroed
        if (!(ok = warp_wait(B_FIX, 0))) break;
      }
      // ---- P -> its causal, decayed part in bf16
      if (!(ok = warp_wait(B_P, ph))) break;
      uint32_t pb[16];
      const bool off = p.back ? q > lq : q < lq;
      if (off || q == lq) {
        float v[32];
        tmem_ld32(tl + R_P + 32 * q, v);
        tmem_wait_ld();
        if (off) {
          const float f = wts->pw[p.back ? 32 * q - row : row - 32 * q - 31];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 c4 = *reinterpret_cast<const float4 *>(wts->cf + i);
            pb[i / 2] = pack_bf16x2(v[i] * (f * c4.x), v[i + 1] * (f * c4.y));
            pb[i / 2 + 1] = pack_bf16x2(v[i + 2] * (f * c4.z), v[i + 3] * (f * c4.w));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int d = p.back ? i - lane : lane - i;
            v[i] = d >= 0 ? v[i] * wts->pw[d] : 0.f;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) pb[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) pb[i] = 0u;
      }
      // the columns of P are reused once the four warps of this lane quarter have read them
      tc_fence_before();
      arrive(B_PREAD + lq);
      if (!(ok = warp_wait(B_PREAD + lq, ph))) break;
      tmem_st16(tl + T_PB + 16 * q, pb);
      // ---- w C -> three bf16 terms
      scale_split(st + 2 * TILE, last ? wts->wtail : wts->wfull, row, q, tl + T_VH, tl + T_VM, tl + T_VL);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(B_V));
        mbar_arrive(bar(B_PB));
      }
      // ---- X
      if (!(ok = warp_wait(B_DX, ph))) break;
      {
        float d[32];
        tmem_ld32(tl + R_DX + 32 * q, d);
        tmem_wait_ld();
        const float lx = wts->pw[len - skip];
#pragma unroll
        for (int i = 0; i < 32; ++i) X[i] = fmaf(lx, X[i], d[i]);
      }
      if (ci + 1 < nch) put_x();
      // ---- out
      if (!(ok = warp_wait(B_OA, ph))) break;
      {
        float oi[32], oa[32];
        tmem_ld32(tl + R_OI + 32 * q, oi);
        tmem_ld32(tl + R_OA + 32 * q, oa);
        tmem_wait_ld();
        tc_fence_before();
        arrive(B_X);
        if (row < len) {
          const float wi = p.s_inter * wts->pw[(p.back ? len - 1 - row : row) + 1 - skip];
          TO *o = static_cast<TO *>(p.out) + ((size_t)(u.t0 + c * CH + row) * p.Hv + u.h) * HD + 32 * q;
          if (sizeof(TO) == 2) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack_bf16x2(fmaf(wi, oi[2 * i], p.s_intra * oa[2 * i]),
                                 fmaf(wi, oi[2 * i + 1], p.s_intra * oa[2 * i + 1]));
            st_global_32b(o, w);
            st_global_32b(o + 16, w + 8);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(fmaf(wi, oi[i + k], p.s_intra * oa[i + k]));
              st_global_32b(o + i, w);
            }
          }
        }
      }
    }
    if (ok && u.last && p.xf) {
      const float f = p.back && nch > 0 ? expf(gh) : 1.f;
      const size_t e0 = (((size_t)u.n * p.Hv + u.h) * HD + row) * HD + 32 * q;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float y[4] = {f * X[i], f * X[i + 1], f * X[i + 2], f * X[i + 3]};
        store_state4(p.xf, e0 + i, p.x_bf16, y);
      }
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
  Unit u;
  if (!get_unit(p, blockIdx.x, u)) return;
  if (u.last) return;  // no segment starts from its end
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
    ctl[CTL_LIMIT] = 0;
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
  auto warp_wait = [&](int b, uint32_t parity) {
    int ok = 1;
    if (lane == 0 && !(ok = mbar_wait(bar(b), parity, ctl))) {
      ctl[CTL_ABORT] = 1;
      report_status(p.status, GDN_ERR_DEVICE_TIMEOUT);
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    __syncwarp();
    if (ok) tc_fence_after();
    return ok != 0;
  };

  if (warp == 0) {
    if (lane == 0) {
      const int hb = u.h / (p.Hv / p.Hb), hc = u.h / (p.Hv / p.Hc);
      int issued = 0;
      for (int ci = 0; ci < nch; ++ci) {
        const int s = ci % NST_S, t = u.t0 + chunk_of(ci) * CH;
        if (!mbar_wait(bar(S_EMPTY + s), ((ci / NST_S) & 1) ^ 1, ctl)) break;
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
    if (lane == 0) ctl[CTL_LIMIT] = (int)header_wait_limit_us(p.status);
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
        zero_tail(st, tail, etid);
        zero_tail(st + TILE, tail, etid);
        fence_proxy_async_smem();
        arrive(S_FIX);
        if (!warp_wait(S_FIX, 0)) return false;
      }
      const uint32_t tv = tl + S_TV + 192 * (ci & 1);
      scale_split(st + TILE, last ? wts->wtail : wts->wfull, row, q, tv, tv + 64, tv + 128);
      tmem_wait_st();
      tc_fence_before();
      arrive(S_V + (ci & 1));
      return true;
    };
    bool ok = nch == 0 || terms(0);
    for (int ci = 0; ci < nch && ok; ++ci) {
      if (ci + 1 < nch && !(ok = terms(ci + 1))) break;
      if (!(ok = warp_wait(S_DX, ci & 1))) break;
      float d[32];
      tmem_ld32(tl + S_RDX + 32 * q, d);
      tmem_wait_ld();
      tc_fence_before();
      arrive(S_FREE);
      const float lx = wts->pw[chunk_of(ci) == nch - 1 ? tail : CH];
#pragma unroll
      for (int i = 0; i < 32; ++i) X[i] = fmaf(lx, X[i], d[i]);
    }
    if (ok) {
      float *x = p.seg_state + (((size_t)u.seg * p.Hv + u.h) * HD + row) * HD + 32 * q;
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<float4 *>(x + i) = make_float4(X[i], X[i + 1], X[i + 2], X[i + 3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Tensor map of a packed [T, H, 128] bf16 tensor viewed as (d, head, token), box
// 64 d x 1 head x 128 tokens, 128-byte swizzle.  Tokens past T read as zeros.
bool make_map(CUtensorMap *m, const void *base, int H, int T) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &res) != cudaSuccess ||
        res != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {HD, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {HD * 2, (cuuint64_t)H * HD * 2};
  const cuuint32_t box[3] = {64, 1, CH}, elem[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, elem,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool scan_tc_supported(const Scan &p, int dtype) {
  return p.Da == HD && p.Dc == HD && dtype == GDN_DTYPE_BF16 && p.T > 0 &&
         (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;  // 32-byte stores
}

cudaError_t launch_scan_tc(const Scan &p, int units, int out_dtype, cudaStream_t stream) {
  static std::atomic<bool> f0[64], f1[64], f2[64];
  CUtensorMap ma, mb, mc;
  if (!make_map(&mb, p.b, p.Hb, p.T) || !make_map(&mc, p.c, p.Hc, p.T)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (!p.out) {
    if ((e = set_smem_once(scan_state_tc_kernel, SMEM_STATE, f0)) != cudaSuccess) return e;
    scan_state_tc_kernel<<<(unsigned)units, NTHREADS, SMEM_STATE, stream>>>(mb, mc, p);
    return cudaGetLastError();
  }
  if (!make_map(&ma, p.a, p.Ha, p.T)) return cudaErrorInvalidValue;
  auto go = [&](auto kern, std::atomic<bool>(&flags)[64]) {
    const cudaError_t r = set_smem_once(kern, SMEM_OUT, flags);
    if (r != cudaSuccess) return r;
    kern<<<(unsigned)units, NTHREADS, SMEM_OUT, stream>>>(ma, mb, mc, p);
    return cudaGetLastError();
  };
  if (out_dtype == GDN_DTYPE_BF16) return go(scan_out_tc_kernel<__nv_bfloat16>, f1);
  return go(scan_out_tc_kernel<float>, f2);
}

}  // namespace lin
}  // namespace gdn
