// gdn_linear_scan.cu -- linear attention with a decay for each head: the plan and
// prefix kernels, the scan for every element type and head dim on warp-level tf32
// MMAs, and the host drivers of prefill and backward.  gdn_linear.cuh has the
// mathematics; gdn_linear_tc.cu the tcgen05 form of the scan.
#include <algorithm>

#include "gdn_chunk_ops.cuh"
#include "gdn_common.cuh"
#include "gdn_linear.cuh"

namespace gdn {
namespace lin {

using chunk::mma_tf32_16x8x8;

// ---------------------------------------------------------------- plan
// The segments of the packed sequences (an empty one has one, of no tokens), by one
// CTA: `units` all of them, `cuts` the sequences of several (x the sequence, y the slot
// of the first segment's state, z how many, w the tokens) and `cut_units` their
// segments, which alone take part in (1) and (2).  Units of unequal length are started
// longest first, so that the last ones to finish are short; beyond kMaxSorted segments
// there are enough waves of units for the order not to matter.  Entries past the last
// of a table, and all of them where cu_seqlens is inconsistent, are marked.
struct Plan {
  int4 *units, *cut_units, *cuts;
  int max_seg, max_cut_seg, max_cut;  // entries of the tables
};
constexpr int kMaxSorted = 512;
__global__ void __launch_bounds__(1024)
plan_segments_kernel(const int32_t *__restrict__ cu, int N, int T, int L, const Plan p, int32_t *status) {
  __shared__ int wsum[32], wcut[32], run_s, run_c, cuts_s;
  __shared__ int4 table[kMaxSorted];
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int bad = 0;
  for (int i = tid; i <= N; i += 1024) {
    const int c = cu[i];
    bad |= c < 0 || c > T || (i == 0 && c != 0) || (i == N && c != T) || (i < N && cu[i + 1] < c);
  }
  if (tid == 0) run_s = run_c = cuts_s = 0;
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) report_status(status, GDN_ERR_BAD_SEQLENS);
  auto scan = [&](int x) {  // inclusive, of a warp
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    return x;
  };
  for (int base = 0; base < (bad ? 0 : N); base += 1024) {
    const int n = base + tid;
    const int c0 = n < N ? cu[n] : 0, c1 = n < N ? cu[n + 1] : 0;
    const int cnt = n < N ? max(1, (int)(((long long)c1 - c0 + L - 1) / L)) : 0;
    const int cut = cnt > 1 ? cnt : 0;
    const int inc = scan(cnt), inc_cut = scan(cut);
    if (lane == 31) {
      wsum[wid] = inc;
      wcut[wid] = inc_cut;
    }
    __syncthreads();
    if (wid == 0) {
      wsum[lane] = scan(wsum[lane]);
      wcut[lane] = scan(wcut[lane]);
    }
    __syncthreads();
    const int start = run_s + (wid ? wsum[wid - 1] : 0) + inc - cnt;
    const int slot = run_c + (wid ? wcut[wid - 1] : 0) + inc_cut - cut;
    auto put = [&](int n, int c0, int c1, int i, int cnt, int sg, int slot) {
      const int4 s = make_int4(slot | (i == 0 ? kFirst : 0) | (i == cnt - 1 ? kLast : 0), n, c0 + i * L,
                               i == cnt - 1 ? c1 : c0 + (i + 1) * L);
      p.units[sg] = s;
      if (sg < kMaxSorted) table[sg] = s;
      if (cnt > 1) p.cut_units[slot] = s;
    };
    if (cnt == 1) put(n, c0, c1, 0, 1, start, 0);
    if (cut) p.cuts[atomicAdd(&cuts_s, 1)] = make_int4(n, slot, cnt, c1 - c0);
    for (unsigned m = __ballot_sync(0xffffffffu, cut); m; m &= m - 1) {  // the segments of one, by its warp
      const int src = __ffs(m) - 1;
      const int b0 = __shfl_sync(0xffffffffu, c0, src), b1 = __shfl_sync(0xffffffffu, c1, src);
      const int segs = __shfl_sync(0xffffffffu, cut, src), sg = __shfl_sync(0xffffffffu, start, src);
      const int sl = __shfl_sync(0xffffffffu, slot, src);
      for (int i = lane; i < segs; i += 32) put(n - lane + src, b0, b1, i, segs, sg + i, sl + i);
    }
    __syncthreads();
    if (tid == 0) {
      run_s += wsum[31];
      run_c += wcut[31];
    }
    __syncthreads();
  }
  const int total = run_s;
  for (int i = total + tid; i < p.max_seg; i += 1024) p.units[i].x = -1;
  for (int i = run_c + tid; i < p.max_cut_seg; i += 1024) p.cut_units[i].x = -1;
  for (int i = cuts_s + tid; i < p.max_cut; i += 1024) p.cuts[i].x = -1;
  if (total <= kMaxSorted && tid < total) {
    const int len = table[tid].w - table[tid].z;
    int rank = 0;
    for (int i = 0; i < total; ++i) {
      const int other = table[i].w - table[i].z;
      rank += other > len || (other == len && i < tid);
    }
    p.units[rank] = table[tid];
  }
}

// ---------------------------------------------------------------- prefix
// Per (sequence of several segments, head): the states that the segments add become
// the states that they start from, in place (`nat`) and/or transposed (`tr`), and what
// follows the last is the final state.  One CTA per 32 x 32 tile of one state: 4
// elements a thread, four segments' loads in flight.  Bound: HBM, or L2 where the states
// are still there: 7.5 us for 144 states of 64 KB read and written (2.5 TB/s with the
// launch), in place of a walk through the segments by one CTA a head.
struct Prefix {
  const float *g;
  const int4 *cuts;  // of the plan
  int Hv, L, Da, Dc, back;
  float *nat, *tr;
  int keep_nat;      // the starting states are wanted in nat
  const void *x0;    // [N, Hv, Dc, Da]
  void *xf;          // final states; NULL to skip
  int x_bf16;
};

__global__ void __launch_bounds__(256) prefix_kernel(const Prefix p) {
  __shared__ float tile[32][33];
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  const int tiles = (p.Da / 32) * (p.Dc / 32);
  const int unit = blockIdx.x / tiles, tl = blockIdx.x - unit * tiles;
  const int ci = unit / p.Hv, h = unit - ci * p.Hv;
  const int4 seq = p.cuts[ci];
  const int n = seq.x, s0 = seq.y, cnt = seq.z, len = seq.w;
  const float gh = floor_decay(p.g[h]);
  if (n < 0) return;
  const int i0 = 32 * (tl / (p.Da / 32)), j0 = 32 * (tl % (p.Da / 32));
  const int r = threadIdx.x >> 3, c = 4 * (threadIdx.x & 7);
  const size_t in_state = (size_t)(i0 + r) * p.Da + j0 + c;
  const size_t state = (size_t)p.Da * p.Dc;
  const size_t e0 = ((size_t)n * p.Hv + h) * state + in_state;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.x0) load_state4(p.x0, e0, p.x_bf16, x);
  const Power whole = decay_power(gh, p.L);
  Carry carry{0.f};
  // what the last segment adds is there only where the final state is wanted
  const int adds = p.xf ? cnt : cnt - 1;
  for (int b = 0; b < cnt; b += 4) {
    float add[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int sg = p.back ? cnt - 1 - (b + i) : b + i;
      if (b + i < adds) load4(p.nat + ((size_t)(s0 + sg) * p.Hv + h) * state + in_state, add[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (b + i >= cnt) break;
      const int sg = p.back ? cnt - 1 - (b + i) : b + i;
      const size_t at = ((size_t)(s0 + sg) * p.Hv + h) * state;
      if (p.keep_nat) *reinterpret_cast<float4 *>(p.nat + at + in_state) = make_float4(x[0], x[1], x[2], x[3]);
      if (p.tr) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) tile[c + k][r] = x[k];
        __syncthreads();
        *reinterpret_cast<float4 *>(p.tr + at + (size_t)(j0 + r) * p.Dc + i0 + c) =
            make_float4(tile[r][c], tile[r][c + 1], tile[r][c + 2], tile[r][c + 3]);
      }
      if (b + i >= adds) break;
      const int tokens = min(p.L, len - sg * p.L) - (p.back && b + i == 0 ? 1 : 0);
      const float f = carry.next(tokens == p.L ? whole : decay_power(gh, tokens));
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = fmaf(f, x[k], add[i][k]);
    }
  }
  if (p.xf) {
    const float f = p.back ? expf(gh) : 1.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] *= f;
    store_state4(p.xf, e0, p.x_bf16, x);
  }
}

// ---------------------------------------------------------------- the scan
// d += A (16 x 8) B (8 x 8) in tf32 with the operands split in two terms (three
// products, about fp32) where they are not exact in tf32 (EXA, EXB: bf16 inputs).  The
// first term is the value rounded to 11 bits, by integers (with cvt.rna.tf32
// in its place, 8 warps and no tiles fetched ahead, fp32 prefill of 8192 tokens at 16/48
// heads took 2.35 ms against 1.36); the second what that
// leaves, of which the tensor core takes 11 of 12 bits, with a sum of its own (dl), because a
// tensor core cuts what an addition shifts out: one cut a step on d instead of three.  A NaN stays in the second.
template <bool EX>
__device__ __forceinline__ uint32_t first_term(float x) {
  return EX ? __float_as_uint(x) : (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
}
template <bool EXA, bool EXB>
__device__ __forceinline__ void mma_split(float *d, float *dl, const float *a, const float *b) {
  uint32_t ah[4], bh[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) ah[i] = first_term<EXA>(a[i]);
#pragma unroll
  for (int i = 0; i < 2; ++i) bh[i] = first_term<EXB>(b[i]);
  if (!EXB) {
    const uint32_t bl[2] = {__float_as_uint(b[0] - __uint_as_float(bh[0])), __float_as_uint(b[1] - __uint_as_float(bh[1]))};
    mma_tf32_16x8x8(dl, ah, bl);
  }
  if (!EXA) {
    const uint32_t al[4] = {__float_as_uint(a[0] - __uint_as_float(ah[0])), __float_as_uint(a[1] - __uint_as_float(ah[1])),
                            __float_as_uint(a[2] - __uint_as_float(ah[2])), __float_as_uint(a[3] - __uint_as_float(ah[3]))};
    mma_tf32_16x8x8(dl, al, bh);
  }
  mma_tf32_16x8x8(d, ah, bh);
}

constexpr int C = 64;    // chunk length
constexpr int DCT = 64;  // columns of out (rows of X) of one CTA

template <int DA>
struct Smem {
  float a[C][DA + 4], b[C][DA + 4], c[C][DCT + 8], P[C][C + 4], X[DCT][DA + 4], pw[C + 1];
  Power whole;  // of a full chunk
  Carry carry;
  float lx;     // what the chunk's state is carried over by
};

// 4 elements on their way from global memory.
template <typename T> struct Quad;
template <> struct Quad<float> {
  float4 x;
  __device__ __forceinline__ void load(const float *p) { x = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void zero() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float4 get() const { return x; }
};
template <> struct Quad<__nv_bfloat16> {
  uint2 x;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { x = *reinterpret_cast<const uint2 *>(p); }
  __device__ __forceinline__ void zero() { x = make_uint2(0u, 0u); }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xffff0000u));
  }
};
// A thread's part of a chunk's 64 rows x W columns, from row `base` on; rows past `len`
// read as zeros.
template <typename T, int W, int NTH>
struct TilePart {
  static constexpr int N = C * W / 4 / NTH;
  Quad<T> q[N];
  __device__ __forceinline__ void load(const T *base, size_t step, int len, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = tid + i * NTH, r = x / (W / 4), d = 4 * (x - r * (W / 4));
      if (r < len) q[i].load(base + (size_t)r * step + d);
      else q[i].zero();
    }
  }
  __device__ __forceinline__ void store(float *dst, int ld, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int x = tid + i * NTH, r = x / (W / 4), d = 4 * (x - r * (W / 4));
      *reinterpret_cast<float4 *>(dst + r * ld + d) = q[i].get();
    }
  }
};

// One CTA per (segment, head, 64 columns of out), 16 warps.  Per chunk of 64
// tokens: P = (A B^T) . lam^{|t-s|}; out = s_intra P C + s_inter lam^{p+1} A X^T;
// X <- lam^len X + (w C)^T B.  X stays in fp32 accumulator registers, with a copy
// in shared memory as an operand; the next chunk's tiles are on their way in registers
// meanwhile.  Bound: the tf32 products (three for each fp32 one) and their operands'
// shared-memory reads.  This form serves fp32 inputs and fp32 outputs: 8192 tokens at
// 16/48 heads of 128 take 1.41 ms from fp32 inputs and 0.99 ms from bf16 ones.
constexpr int NTHREADS = 512;
template <typename T, typename TO, int DA, bool OUT>
__global__ void __launch_bounds__(NTHREADS) scan_kernel(const Scan p) {
  constexpr bool EX = sizeof(T) == 2;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<DA> &s = *reinterpret_cast<Smem<DA> *>(smem_raw);
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  const int splits = p.Dc / DCT;
  const int unit = blockIdx.x / splits, dc0 = DCT * (blockIdx.x - unit * splits);
  Unit w;
  if (!get_unit(p, unit, w)) return;
  if (!OUT && w.last && (w.first || !p.xf)) return;  // nothing starts from its end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const float gh = head_decay(p, w.h);
  const int mt = warp >> 2, nq = warp & 3;  // this warp's 16 rows and quarter of the columns
  constexpr int NX = DA / 32;               // 8-column tiles of X per warp
  const int nch = (w.t1 - w.t0 + C - 1) / C;
  auto chunk_of = [&](int ci) { return p.back ? nch - 1 - ci : ci; };

  TilePart<T, DA, NTHREADS> ta, tb;
  TilePart<T, DCT, NTHREADS> tc;
  auto fetch = [&](int ci) {
    const int t0 = w.t0 + chunk_of(ci) * C, len = min(C, w.t1 - t0);
    auto at = [&](const void *base, int H, int D) {
      return static_cast<const T *>(base) + ((size_t)t0 * H + w.h / (p.Hv / H)) * D;
    };
    if (OUT) ta.load(at(p.a, p.Ha, DA), (size_t)p.Ha * DA, len, tid);
    tb.load(at(p.b, p.Hb, DA), (size_t)p.Hb * DA, len, tid);
    tc.load(at(p.c, p.Hc, p.Dc) + dc0, (size_t)p.Hc * p.Dc, len, tid);
  };
  if (nch > 0) fetch(0);
  if (tid <= C) s.pw[tid] = expf(gh * (float)tid);
  if (tid == 0) {
    s.whole = decay_power(gh, C);
    s.carry.rest = 0.f;
  }

  float X[NX][4];
#pragma unroll
  for (int n = 0; n < NX; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      X[n][e] = OUT ? start_state(p, w, dc0 + 16 * mt + gid + 8 * (e >> 1), 8 * (nq * NX + n) + 2 * tig + (e & 1)) : 0.f;
  auto put_x = [&]() {
#pragma unroll
    for (int n = 0; n < NX; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s.X[16 * mt + gid + 8 * (e >> 1)][8 * (nq * NX + n) + 2 * tig + (e & 1)] = X[n][e];
  };
  if (OUT) put_x();

  for (int ci = 0; ci < nch; ++ci) {
    const int t0 = w.t0 + chunk_of(ci) * C, len = min(C, w.t1 - t0);
    const int skip = p.back && w.first && ci == 0 ? 1 : 0;
    __syncthreads();  // the last chunk's tiles have been used
    if (OUT) ta.store(&s.a[0][0], DA + 4, tid);
    tb.store(&s.b[0][0], DA + 4, tid);
    tc.store(&s.c[0][0], DCT + 8, tid);
    if (tid == 0) s.lx = s.carry.next(len - skip == C ? s.whole : decay_power(gh, len - skip));
    __syncthreads();
    if (ci + 1 < nch) fetch(ci + 1);
    if (OUT) {
      // P, rows t of tile mt, columns s of quarter nq; A X^T beside it
      float acc[2][4] = {}, oi[2][4] = {}, oa[2][4] = {};
      float accl[2][4] = {}, oil[2][4] = {}, oal[2][4] = {};
#pragma unroll 4
      for (int k = 0; k < DA; k += 8) {
        const float af[4] = {s.a[16 * mt + gid][k + tig], s.a[16 * mt + gid + 8][k + tig],
                             s.a[16 * mt + gid][k + tig + 4], s.a[16 * mt + gid + 8][k + tig + 4]};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int col = 8 * (2 * nq + n) + gid;
          const float bf[2] = {s.b[col][k + tig], s.b[col][k + tig + 4]};
          mma_split<EX, EX>(acc[n], accl[n], af, bf);
          const float xf[2] = {s.X[col][k + tig], s.X[col][k + tig + 4]};
          mma_split<EX, false>(oi[n], oil[n], af, xf);
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 16 * mt + gid + 8 * (e >> 1), sc = 8 * (2 * nq + n) + 2 * tig + (e & 1);
          const int d = p.back ? sc - t : t - sc;
          s.P[t][sc] = d >= 0 ? (acc[n][e] + accl[n][e]) * s.pw[d] : 0.f;
        }
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < C; k += 8) {
        const float af[4] = {s.P[16 * mt + gid][k + tig], s.P[16 * mt + gid + 8][k + tig],
                             s.P[16 * mt + gid][k + tig + 4], s.P[16 * mt + gid + 8][k + tig + 4]};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int dc = 8 * (2 * nq + n) + gid;
          const float bf[2] = {s.c[k + tig][dc], s.c[k + tig + 4][dc]};
          mma_split<false, EX>(oa[n], oal[n], af, bf);
        }
      }
      TO *out = static_cast<TO *>(p.out);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int t = 16 * mt + gid + 8 * r;
        if (t >= len) continue;
        const float wi = p.s_inter * s.pw[(p.back ? len - 1 - t : t) + 1 - skip];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          TO *o = out + ((size_t)(t0 + t) * p.Hv + w.h) * p.Dc + dc0 + 8 * (2 * nq + n) + 2 * tig;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            o[e] = from_f32<TO>(fmaf(wi, oi[n][2 * r + e] + oil[n][2 * r + e],
                                     p.s_intra * (oa[n][2 * r + e] + oal[n][2 * r + e])));
        }
      }
    }
    // X <- lam^len X + sum_t (s_upd lam^{rest} c_t) b_t^T
    // (the chunk's sum on its own: tensor cores cut what an addition shifts out, which
    // over many additions to a large X would be a drift)
    float dx[NX][4] = {}, dxl[NX][4] = {};
#pragma unroll 4
    for (int k = 0; k < C; k += 8) {
      float wt[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = k + tig + 4 * i, rest = p.back ? t : len - 1 - t;
        wt[i] = t < len ? p.s_upd * s.pw[rest] : 0.f;
      }
      const float af[4] = {wt[0] * s.c[k + tig][16 * mt + gid], wt[0] * s.c[k + tig][16 * mt + gid + 8],
                           wt[1] * s.c[k + tig + 4][16 * mt + gid], wt[1] * s.c[k + tig + 4][16 * mt + gid + 8]};
#pragma unroll
      for (int n = 0; n < NX; ++n) {
        const int da = 8 * (nq * NX + n) + gid;
        const float bf[2] = {s.b[k + tig][da], s.b[k + tig + 4][da]};
        mma_split<false, EX>(dx[n], dxl[n], af, bf);
      }
    }
    const float lx = s.lx;
#pragma unroll
    for (int n = 0; n < NX; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) X[n][e] = fmaf(lx, X[n][e], dx[n][e] + dxl[n][e]);
    if (OUT) put_x();  // (its readers have passed the barrier after P)
  }
  const bool fin = OUT && w.first && w.last && p.xf;
  if (OUT && !fin) return;
  const float f = fin && p.back && nch > 0 ? expf(gh) : 1.f;
  const size_t base = fin ? ((size_t)w.n * p.Hv + w.h) * p.Dc * p.Da
                          : ((size_t)w.seg * p.Hv + w.h) * p.Dc * p.Da;
#pragma unroll
  for (int n = 0; n < NX; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const size_t at = base + (size_t)(dc0 + 16 * mt + gid + 8 * (e >> 1)) * p.Da +
                        8 * (nq * NX + n) + 2 * tig + (e & 1);
      if (fin && p.x_bf16) static_cast<__nv_bfloat16 *>(p.xf)[at] = __float2bfloat16_rn(f * X[n][e]);
      else (fin ? static_cast<float *>(p.xf) : p.seg_state)[at] = f * X[n][e];
    }
}

template <typename T, typename TO, int DA>
static cudaError_t launch_scan_t(const Scan &p, int units, cudaStream_t stream) {
  static std::atomic<bool> f0[64], f1[64];
  constexpr int bytes = (int)sizeof(Smem<DA>);
  static_assert(bytes <= 232448, "shared memory of a CTA");
  const unsigned grid = (unsigned)units * (unsigned)(p.Dc / DCT);
  cudaError_t e;
  if (!p.states_only) {
    if ((e = set_smem_once(scan_kernel<T, TO, DA, true>, bytes, f1)) != cudaSuccess) return e;
    return launch_pdl(scan_kernel<T, TO, DA, true>, dim3(grid), dim3(NTHREADS), bytes, stream, p);
  }
  if ((e = set_smem_once(scan_kernel<T, T, DA, false>, bytes, f0)) != cudaSuccess) return e;
  return launch_pdl(scan_kernel<T, T, DA, false>, dim3(grid), dim3(NTHREADS), bytes, stream, p);
}

cudaError_t launch_scan(const Scan &p, int units, int dtype, int out_dtype, cudaStream_t stream) {
  return dispatch_types(dtype, out_dtype, [&](auto t, auto to) {
    using T = decltype(t);
    using TO = decltype(to);
    if (p.Da == 128) return launch_scan_t<T, TO, 128>(p, units, stream);
    return launch_scan_t<T, TO, 64>(p, units, stream);
  });
}

// ---------------------------------------------------------------- group sums
// out[t, j] = sum over the G value heads of query/key head j of part[t, jG + r]
// (fp32 partials, summed in order, rounded once: atomics on a bf16 or fp32 gradient
// would depend on the order).  4 columns a thread.  Bound: HBM, 39 us for 201 MB read
// and 34 MB written (8192 tokens, 16/48 heads), 6.0 TB/s.
template <typename TO>
__global__ void __launch_bounds__(256)
group_sum_kernel(const float *__restrict__ part, TO *__restrict__ out, size_t quads, int D, int G) {
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  const size_t x = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (x >= quads) return;
  const size_t row = x / (D / 4), d = 4 * (x - row * (D / 4));
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r = 0; r < G; ++r) {
    const float4 y = __ldcs(reinterpret_cast<const float4 *>(part + (row * G + r) * D + d));
    s[0] += y.x; s[1] += y.y; s[2] += y.z; s[3] += y.w;
  }
  store_state4(out, row * D + d, sizeof(TO) == 2, s);
}

// ---------------------------------------------------------------- host drivers
namespace {

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Segment length in tokens.  Cutting lets the multiprocessors that a call's heads leave
// idle work on a sequence, but its chunks then cost more (the segments' states) and
// there are launches, starts and state moves on top; so the total's chunks are counted
// in microseconds both ways, with costs taken from timings.  At 48 heads of 128, us for
// one segment and for 3: tcgen05 form, 1024 tokens 41 and 44, 2048 68 and 58, 8192 223
// and 130; its backward, 1024 tokens 135 and 118.  The other form (fp32), 256 tokens 59
// and 94, 1024 201 and 224, 8192 1550 and 1422.  Segments for more waves than these cost
// more again (8192 tokens in 6: 154), and so do segments of one 64-token chunk (4096
// tokens, 4 heads, fp32: 89 us in 16 segments, 99 in 32).  Other head counts and head dim 64 go by the
// same costs, which were not timed for them.
struct Cutting {
  int ch, max_waves;           // tokens of a chunk; waves of segments that are tried
  int64_t min_per, ctas, sms;  // chunks of the shortest segment; CTAs of one over all heads
  double chunk, cut, fixed;    // a chunk uncut and cut, and what cutting costs (us)
  Cutting(int Hv, int Dv, bool tc, bool backward)
      : ch(tc ? 128 : 64), max_waves(tc ? 1 : 2), min_per(tc ? 1 : 2), ctas(tc ? Hv : Hv * (Dv / DCT)),
        sms(sm_count()) {
    chunk = (backward ? 3 : 1) * (tc ? 3.2 : 11.8);
    cut = chunk + (backward ? 2 : 1) * (tc ? 1.2 : 4.3);
    fixed = tc ? (backward ? 28 : 22) : 25;
  }
  int64_t chunks(int64_t T) const { return std::max<int64_t>(1, (T + ch - 1) / ch); }
  int segment_len(int64_t T) const {
    const int64_t n = chunks(T);
    int64_t best = n;
    double least = chunk * (double)n;
    for (int waves = 1; waves <= max_waves; ++waves) {
      const int64_t s = waves * sms / ctas;
      if (s < 2) continue;
      const int64_t per = std::max(min_per, (n + s - 1) / s);
      const double us = fixed + cut * (double)(per * waves);
      if (us < least) {
        least = us;
        best = per;
      }
    }
    return (int)std::min<int64_t>(best * ch, INT32_MAX);
  }
  // At least T' / (its segment length) of every T' <= T that is cut.
  int64_t most(int64_t T) const {
    const int64_t n = chunks(T), s = max_waves * sms / ctas;
    return s < 2 || chunk * (double)n <= fixed + cut * (double)min_per ? 0 : std::min(s, n / min_per);
  }
};

struct Layout {
  int L;
  int64_t max_seg, max_cut, max_cut_seg;  // segments; sequences of several, and their segments
  size_t units, nat, tr, part, total;
};

// Where things lie in a workspace; `reserve`: as for the call of at most N sequences and
// T tokens that needs most, so that a workspace of its size serves all of them.
Layout layout(int64_t N, int64_t T, int Hqk, int Hv, int Dk, int Dv, bool tc, bool backward, bool reserve = false) {
  Layout l;
  const Cutting c(Hv, Dv, tc, backward);
  l.L = c.segment_len(T);
  const int64_t per_seq = reserve ? c.most(T) : T <= l.L ? 0 : T / l.L;
  const bool one = per_seq == 0;
  l.max_seg = per_seq + N;
  l.max_cut = std::min(N, per_seq);
  l.max_cut_seg = per_seq + l.max_cut;
  size_t at = kWorkspaceHeaderBytes;
  l.units = at;
  if (!one) at = round_up(at + sizeof(int4) * (size_t)(l.max_seg + l.max_cut_seg + l.max_cut), 1024);
  const size_t states = round_up((size_t)l.max_cut_seg * Hv * Dk * Dv * sizeof(float), 1024);
  l.nat = at;
  at += states;
  l.tr = at;
  if (backward) at += states;
  l.part = at;
  if (backward && Hv > Hqk) at = round_up(at + (size_t)T * Hv * Dk * sizeof(float), 1024);
  l.total = at;
  return l;
}

}  // namespace
}  // namespace lin

size_t linear_workspace_bytes(int64_t N, int64_t T, int Hqk, int Hv, int Dk, int Dv, bool backward) {
  // of both forms: the output's type, which decides between them, is not known here
  return std::max(lin::layout(N, T, Hqk, Hv, Dk, Dv, true, backward, true).total,
                  lin::layout(N, T, Hqk, Hv, Dk, Dv, false, backward, true).total);
}

namespace lin {

// Whether a call whose results end up in bf16 (or not) runs the tcgen05 form: 8192 tokens
// at 16/48 heads of 128 take 130 us there and 990 us in the other, which keeps about 24
// bits where tcgen05's bf16 operands keep 8.
static bool use_tc(const Scan &p, int dtype, int result_dtype) {
  return result_dtype == GDN_DTYPE_BF16 && scan_tc_supported(p, dtype);
}

static cudaError_t run_scan(const Scan &p, bool tc, int units, int dtype, int out_dtype, cudaStream_t stream) {
  return tc ? launch_scan_tc(p, units, out_dtype, stream) : launch_scan(p, units, dtype, out_dtype, stream);
}

// Plan the segments of p's sequences.
static cudaError_t run_plan(const Scan &p, const Layout &l, unsigned char *ws, Plan &plan, cudaStream_t stream) {
  plan.units = reinterpret_cast<int4 *>(ws + l.units);
  plan.cut_units = plan.units + l.max_seg;
  plan.cuts = plan.cut_units + l.max_cut_seg;
  plan.max_seg = (int)l.max_seg; plan.max_cut_seg = (int)l.max_cut_seg; plan.max_cut = (int)l.max_cut;
  return launch_pdl(plan_segments_kernel, dim3(1), dim3(1024), 0, stream, p.cu, p.N, p.T, l.L, plan, p.status);
}

// What the segments add to the states, into p.seg_state.
static cudaError_t run_states(Scan p, bool tc, const Plan &plan, int dtype, cudaStream_t stream) {
  p.units = plan.cut_units;
  p.states_only = 1;
  return run_scan(p, tc, plan.max_cut_seg * p.Hv, dtype, dtype, stream);
}

static cudaError_t run_prefix(const Prefix &p, const Plan &plan, cudaStream_t stream) {
  const unsigned grid = (unsigned)plan.max_cut * (unsigned)p.Hv * (unsigned)((p.Da / 32) * (p.Dc / 32));
  return launch_pdl(prefix_kernel, dim3(grid), dim3(256), 0, stream, p);
}

}  // namespace lin

cudaError_t launch_linear_prefill(const void *q, const void *k, const void *v, const float *g,
                                  const int32_t *cu, int N, int64_t T, int Hqk, int Hv, int Dk, int Dv,
                                  int dtype, int o_dtype, int state_dtype, float scale, const void *s0,
                                  void *sf, void *o, void *ws, cudaStream_t stream) {
  using namespace lin;
  unsigned char *w = static_cast<unsigned char *>(ws);
  Scan p = {};
  p.a = q; p.b = k; p.c = v; p.Ha = p.Hb = Hqk; p.Hc = Hv; p.g = g; p.cu = cu; p.N = N; p.T = (int)T;
  p.Hv = Hv; p.Da = Dk; p.Dc = Dv; p.s_intra = p.s_inter = scale; p.s_upd = 1.f;
  const bool tc = use_tc(p, dtype, o_dtype);
  const lin::Layout l = layout(N, T, Hqk, Hv, Dk, Dv, tc, false);
  p.L = l.L;
  p.status = static_cast<int32_t *>(ws);
  p.x0 = s0; p.xf = sf; p.x_bf16 = state_dtype == GDN_DTYPE_BF16;
  if (T <= l.L) {
    p.out = o;
    return run_scan(p, tc, N * Hv, dtype, o_dtype, stream);
  }
  Plan plan;
  cudaError_t e = run_plan(p, l, w, plan, stream);
  if (e != cudaSuccess) return e;
  p.seg_state = reinterpret_cast<float *>(w + l.nat);
  if ((e = run_states(p, tc, plan, dtype, stream)) != cudaSuccess) return e;
  Prefix x = {};
  x.g = g; x.cuts = plan.cuts; x.Hv = Hv; x.L = l.L; x.Da = Dk; x.Dc = Dv;
  x.nat = p.seg_state; x.keep_nat = 1; x.x0 = s0; x.xf = sf; x.x_bf16 = p.x_bf16;
  if ((e = run_prefix(x, plan, stream)) != cudaSuccess) return e;
  p.out = o;
  p.units = plan.units;
  return run_scan(p, tc, plan.max_seg * Hv, dtype, o_dtype, stream);
}

cudaError_t launch_linear_backward(const void *q, const void *k, const void *v, const float *g,
                                   const int32_t *cu, int N, int64_t T, int Hqk, int Hv, int Dk, int Dv,
                                   int dtype, float scale, const float *s0, const void *d_o,
                                   const float *dsf, void *dq, void *dk, void *dv, float *ds0, void *ws,
                                   cudaStream_t stream) {
  using namespace lin;
  unsigned char *w = static_cast<unsigned char *>(ws);
  Scan base = {};
  base.g = g; base.cu = cu; base.N = N; base.T = (int)T; base.Hv = Hv;
  const bool tc = use_tc(base, dtype, dtype);
  const lin::Layout l = layout(N, T, Hqk, Hv, Dk, Dv, tc, true);
  base.L = l.L;
  const bool one = T <= l.L, grouped = Hv > Hqk;
  base.status = static_cast<int32_t *>(ws);
  float *nat = reinterpret_cast<float *>(w + l.nat), *tr = reinterpret_cast<float *>(w + l.tr);
  float *part = reinterpret_cast<float *>(w + l.part);
  const int units = (int)l.max_seg * Hv;
  cudaError_t e = cudaSuccess;
  Plan plan = {};
  if (!one) {
    if ((e = run_plan(base, l, w, plan, stream)) != cudaSuccess) return e;
    base.units = plan.units;
  }
  Prefix x = {};
  x.g = g; x.cuts = plan.cuts; x.Hv = Hv; x.L = l.L; x.Da = Dk; x.Dc = Dv;
  x.nat = nat; x.tr = tr;

  // dq (and dk) of a query/key head: fp32 partials of its value heads, then their sum
  auto into = [&](Scan p, void *out) -> cudaError_t {
    p.out = grouped ? part : out;
    cudaError_t r = run_scan(p, tc, units, dtype, grouped ? GDN_DTYPE_FP32 : dtype, stream);
    if (r != cudaSuccess || !grouped || T == 0) return r;  // (no rows: a grid of no blocks is refused)
    const size_t quads = (size_t)T * Hqk * Dk / 4;
    const unsigned blocks = (unsigned)((quads + 255) / 256);
    const float *from = part;
    if (dtype == GDN_DTYPE_BF16)
      return launch_pdl(group_sum_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0, stream, from,
                        static_cast<__nv_bfloat16 *>(out), quads, Dk, Hv / Hqk);
    return launch_pdl(group_sum_kernel<float>, dim3(blocks), dim3(256), 0, stream, from, static_cast<float *>(out),
                      quads, Dk, Hv / Hqk);
  };

  Scan p = base;  // S, for dq
  p.a = q; p.Ha = Hqk; p.b = k; p.Hb = Hqk; p.c = v; p.Hc = Hv; p.Da = Dk; p.Dc = Dv; p.s_upd = 1.f;
  if (!one) {
    p.seg_state = nat;
    if ((e = run_states(p, tc, plan, dtype, stream)) != cudaSuccess) return e;
    x.x0 = s0; x.back = 0; x.keep_nat = 0;
    if ((e = run_prefix(x, plan, stream)) != cudaSuccess) return e;
  }
  p = base;
  p.a = d_o; p.Ha = Hv; p.b = v; p.Hb = Hv; p.c = k; p.Hc = Hqk; p.Da = Dv; p.Dc = Dk;
  p.s_intra = p.s_inter = scale; p.s_upd = 1.f; p.seg_state = tr; p.x0 = s0; p.x0_tr = 1;
  if ((e = into(p, dq)) != cudaSuccess) return e;

  p = base;  // D, for dv and dk
  p.back = 1;
  p.a = k; p.Ha = Hqk; p.b = q; p.Hb = Hqk; p.c = d_o; p.Hc = Hv; p.Da = Dk; p.Dc = Dv;
  p.s_intra = p.s_upd = scale; p.s_inter = 1.f; p.seg_state = nat; p.x0 = dsf; p.xf = ds0;
  if (!one) {
    if ((e = run_states(p, tc, plan, dtype, stream)) != cudaSuccess) return e;
    x.x0 = dsf; x.back = 1; x.keep_nat = 1; x.xf = ds0;
    if ((e = run_prefix(x, plan, stream)) != cudaSuccess) return e;
  }
  p.out = dv;
  if ((e = run_scan(p, tc, units, dtype, dtype, stream)) != cudaSuccess) return e;
  p.a = v; p.Ha = Hv; p.b = d_o; p.Hb = Hv; p.c = q; p.Hc = Hqk; p.Da = Dv; p.Dc = Dk;
  p.seg_state = tr; p.x0_tr = 1; p.xf = nullptr;
  return into(p, dk);
}

}  // namespace gdn
