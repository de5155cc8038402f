// gdn_tree.cu -- verification of a tree of drafted tokens against cached
// recurrent states, and the commit of the accepted path.
//
// A tree has M nodes; node i continues its parent p (the cached state S0 of the
// sequence where p = -1).  With a_i = e^{g_i} and b_i the write strength,
//     delta rule:  S_i = a_i S_p (I - b_i k_i k_i^T) + b_i v_i k_i^T
//     linear rule: S_i = lam S_p + v_i k_i^T            (lam = e^g of the head)
//     o_i = scale S_i q_i.
// Unrolled along the path from S0 to i, with E_ij the product of a over the path
// after j up to and including i (1 for j = i) and E_i0 the one from S0:
//     S_i = E_i0 S0 + sum_{j on the path} E_ij u_j k_j^T
//     u_i = b_i (v_i - E_i0 S0 k_i - sum_{j on the path, j != i} E_ij (k_j . k_i) u_j)
//     o_i = scale (E_i0 S0 q_i + sum_{j on the path} E_ij (k_j . q_i) u_j)
// (u_i = v_i for the linear rule).  So every node's output follows from the one
// state S0, which is read once and left as it is.
#include "gdn_common.cuh"
#include "gdn_rows.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace tree {

constexpr int kMaxNodes = 64;

// d (16 x 8, fp32) += a (16 x 16, row) * b (16 x 8, col), bf16 operands.
__device__ __forceinline__ void mma_16x8x16(float *d, const uint32_t *a, const uint32_t *b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Four consecutive values as NP bf16 planes whose sum is the value to 8 NP bits:
// plane 0 the value rounded, each further plane the rounded rest.
template <int NP>
__device__ __forceinline__ void split4(const float x[4], uint32_t (*w)[2]) {
  float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    w[p][0] = pack2(r[0], r[1]);
    w[p][1] = pack2(r[2], r[3]);
    if (p + 1 < NP) {
      r[0] -= lo_of(w[p][0]); r[1] -= hi_of(w[p][0]);
      r[2] -= lo_of(w[p][1]); r[3] -= hi_of(w[p][1]);
    }
  }
}

// d += A B with A in PA and B in PB terms, products whose weight is below the last term
// kept left out.  A tensor core cuts what an addition shifts out of 24 bits, always
// towards zero: with three terms in B (fp32 inputs), a K step is summed apart, small
// products first, and added once, rounded to nearest.  (With all of them added to d
// as they come, 48 cuts in a row at the size of d, fp32 trees were off by 9.6e-7 in rms where
// they are by 1e-7 now; 64 trees of 32 nodes took 228 us against 237, of 16 nodes 93 against
// 102.  Three terms against one, 24 cuts, are off by 4e-7 and stay as they are.)
template <int PA, int PB>
__device__ __forceinline__ void mma_terms(float *d, const uint32_t (*a)[4], const uint32_t (*b)[2]) {
  constexpr int P = PA > PB ? PA : PB;
  if (PB < 3) {
#pragma unroll
    for (int tb = 0; tb < PB; ++tb)
#pragma unroll
      for (int ta = 0; ta < PA && ta + tb < P; ++ta) mma_16x8x16(d, a[ta], b[tb]);
    return;
  }
  float s[4] = {};
#pragma unroll
  for (int w = P - 1; w >= 0; --w)
#pragma unroll
    for (int tb = 0; tb < PB; ++tb)
      if (w - tb >= 0 && w - tb < PA) mma_16x8x16(s, a[w - tb], b[tb]);
#pragma unroll
  for (int e = 0; e < 4; ++e) d[e] += s[e];
}

struct Params {
  const void *q, *k, *v;
  const float *g, *beta;  // beta NULL: linear rule, g one per value head
  const int32_t *parent;
  const void *state;
  const int32_t *src_slot;
  int num_slots;
  void *o;
  int o_bf16, M, Hqk, Hv, raw;
  float scale;
  int32_t *status;
};

// Shared memory of decode_tree_kernel, in bytes from its start.
template <typename T, int XP, int DK, int DV, int MP>
struct Layout {
  static constexpr int LDX = DK + 16;  // bf16; 4-lane groups of a fragment read distinct banks
  static constexpr int LDU = DV + 4;   // fp32; the fragments' column writes hit distinct banks
  static constexpr int X = 0;                                  // [XP][2 MP][LDX]: rows of k, then of q
  static constexpr int XB = XP * 2 * MP * LDX * 2;
  static constexpr int U = 0;                                  // [MP][LDU] over X, once X has been used
  static constexpr int O = MP * LDU * 4;                       // [MP][LDU]
  static constexpr int V = XB > 2 * O ? XB : 2 * O;            // [MP][DV] T
  // by node i and place s along its path (0: the parent), j the ancestor there
  static constexpr int AC = V + MP * DV * (int)sizeof(T);      // [MP][MP] {E_ij (k_j . k_i), E_ij (k_j . q_i)}
  static constexpr int IDX = AC + MP * MP * 8;                 // [MP][MP] bytes: j
  static constexpr int S = IDX + MP * MP;                      // per-node scalars
  static constexpr int BYTES = S + MP * 4 * 11 + 16;
  // CTAs of a multiprocessor: 4 or 2 by registers, fewer where shared memory (228 KB, 1 KB
  // of it for each CTA) does not hold them; the registers then need not be kept for more
  static constexpr int FIT = 233472 / (BYTES + 1024), MOST = MP <= 32 ? 4 : 2, CTAS = FIT < MOST ? FIT : MOST;
};

__device__ __forceinline__ void cp_async_16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// One CTA per (sequence, value head).  S0 [k; q]^T (Dv x 2 M) and [k; q] k^T
// (2 M x M) run on warp-level bf16 MMAs (fp32 accumulation); S0 goes straight
// from HBM into A fragments, a lane's float4 holding the four K positions that
// lane owns (the order of K within a 16-wide step is free as long as both
// operands use the same).  Values that bf16 does not hold are split into SP (S0)
// or XP (fp32 k, q) bf16 terms; products of terms whose weight is below the last
// term kept are dropped.  Then u is solved for depth by depth, a warp for a node
// (nodes of one depth do not depend on one another), along the node's path only, so
// that nothing of a branch (a NaN, say) reaches another; a path's indices and factors
// lie in its order, four to a load.  Every global load of the CTA is issued before the
// first is waited for.
// Bound: HBM, one read of each state; the products are 4 M flops an element.  Measured at
// 64 trees of 32 nodes, 16/48 heads of 128, bf16 over fp32 states: 86 us for 269 MB, 3.1
// TB/s: products, the solve's shared-memory reads and its barriers share the time (tensor
// pipe 29 %, shared memory 57 % busy, a third of the issue slots used).  8 nodes 54 us,
// 16 nodes 60; a chain of 32, one node a depth, 180.
template <typename T, typename ST, int SP, int XP, int DK, int DV, int MP>
__global__ void __launch_bounds__(DV == 128 && MP == 64 ? 256 : 128, Layout<T, XP, DK, DV, MP>::CTAS)
decode_tree_kernel(const Params p) {
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  constexpr int NT = DV == 128 && MP == 64 ? 256 : 128, NW = NT / 32;
  constexpr int MT = DV / (16 * NW);   // 16-row tiles of S0 per warp
  constexpr int NX = 2 * MP / 8;       // 8-node column tiles of [k; q]^T
  constexpr int KS = DK / 16;
  constexpr int PF = MP <= 32 ? 2 : 4; // k steps of S0 in flight (all of it is on its way to L2)
  using L = Layout<T, XP, DK, DV, MP>;
  extern __shared__ __align__(16) unsigned char smem[];
  __nv_bfloat16 *X = reinterpret_cast<__nv_bfloat16 *>(smem + L::X);
  float *U = reinterpret_cast<float *>(smem + L::U), *O = reinterpret_cast<float *>(smem + L::O);
  T *V = reinterpret_cast<T *>(smem + L::V);
  float2 *AC = reinterpret_cast<float2 *>(smem + L::AC);
  unsigned char *idx = smem + L::IDX;
  unsigned long long *anc = reinterpret_cast<unsigned long long *>(smem + L::S);  // strict ancestors
  float *alpha = reinterpret_cast<float *>(smem + L::S + MP * 8), *bet = alpha + MP, *E0 = bet + MP;
  float *rn = E0 + MP;         // [2 MP] 1/|k_i|, 1/|q_i| (1 for prepared inputs)
  float *cself = rn + 2 * MP;  // k_i . q_i
  int32_t *par = reinterpret_cast<int32_t *>(cself + MP);
  int32_t *order = par + MP;                   // the nodes by depth
  int32_t *level = order + MP;                 // [MP + 1] first place of each depth; then the end
  int32_t *nodes = level + MP + 1;             // how many there are

  const int b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv;
  const int j = h / (p.Hv / p.Hqk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tig = lane & 3;
  const int M = p.M;
  const bool delta = p.beta != nullptr;
  const int src = p.src_slot ? p.src_slot[b] : b;
  if (src < 0) return;  // padding entry
  if (src >= p.num_slots) {
    if (tid == 0) report_status(p.status, GDN_ERR_INVALID_ARG);
    return;
  }
  const ST *S = static_cast<const ST *>(p.state) + ((size_t)src * p.Hv + h) * DV * DK;

  if (tid == 0) sm100::bulk_prefetch_l2(S, DV * DK * (int)sizeof(ST));
  // S0 fragments: rows 16 (warp MT + mt) + gid, + 8; columns 16 ks + 4 tig .. + 3
  float sf[PF][MT][2][4];
  auto load_ks = [&](int slot, int ks) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        load4(S + (size_t)(16 * (warp * MT + mt) + gid + 8 * r) * DK + 16 * ks + 4 * tig, sf[slot][mt][r]);
  };
#pragma unroll
  for (int ks = 0; ks < PF; ++ks) load_ks(ks, ks);

  // stage k, q (as bf16 terms), v and the gates (rows past the last node as zeros)
  const T *kb = static_cast<const T *>(p.k) + ((size_t)b * M * p.Hqk + j) * DK;
  const T *qb = static_cast<const T *>(p.q) + ((size_t)b * M * p.Hqk + j) * DK;
  const T *vb = static_cast<const T *>(p.v) + ((size_t)b * M * p.Hv + h) * DV;
  constexpr int EV = 16 / (int)sizeof(T);  // elements of a 16-byte copy
#pragma unroll
  for (int x = tid; x < MP * (DV / EV); x += NT) {
    const int i = x / (DV / EV), d = EV * (x - i * (DV / EV));
    if (i < M) cp_async_16(V + i * DV + d, vb + (size_t)i * p.Hv * DV + d);
  }
  if (XP == 1) {  // bf16: the rows as they are
#pragma unroll
    for (int x = tid; x < 2 * MP * (DK / 8); x += NT) {
      const int r = x / (DK / 8), d = 8 * (x - r * (DK / 8)), i = r < MP ? r : r - MP;
      __nv_bfloat16 *dst = X + (size_t)r * L::LDX + d;
      if (i < M) cp_async_16(dst, (r < MP ? kb : qb) + (size_t)i * p.Hqk * DK + d);
      else *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  int bad = 0;
  for (int i = tid; i < MP; i += NT) {
    const size_t gi = ((size_t)b * M + i) * p.Hv + h;
    const int32_t pi = i < M ? p.parent[(size_t)b * M + i] : -2;
    const float gv = i < M ? p.g[delta ? gi : (size_t)h] : 0.f, bv = i < M && delta ? p.beta[gi] : 1.f;
    par[i] = pi;
    bad |= pi >= i;
    alpha[i] = delta ? (p.raw ? alpha_raw(gv) : expf(gv)) : expf(floor_decay(gv));
    bet[i] = p.raw ? beta_raw(bv) : bv;
  }
  if (XP > 1) {  // fp32: as XP bf16 terms, four loads of a thread in flight
    constexpr int N = 2 * MP * (DK / 4) / NT;
#pragma unroll 1
    for (int o = 0; o < N; o += 4) {
      float y[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int x = tid + (o + n) * NT, r = x / (DK / 4), d = 4 * (x - r * (DK / 4)), i = r < MP ? r : r - MP;
        y[n][0] = y[n][1] = y[n][2] = y[n][3] = 0.f;
        if (i < M) load4((r < MP ? kb : qb) + (size_t)i * p.Hqk * DK + d, y[n]);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int x = tid + (o + n) * NT, r = x / (DK / 4), d = 4 * (x - r * (DK / 4));
        uint32_t w[XP][2];
        split4<XP>(y[n], w);
#pragma unroll
        for (int t = 0; t < XP; ++t)
          *reinterpret_cast<uint2 *>(X + (size_t)(t * 2 * MP + r) * L::LDX + d) = make_uint2(w[t][0], w[t][1]);
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < M; i += NT) bad |= par[i] >= 0 && par[i] < i && par[par[i]] < -1;
  if (__syncthreads_or(bad)) {  // a parent that is no earlier node of the tree
    if (tid == 0) report_status(p.status, GDN_ERR_INVALID_ARG);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  // paths: E_ij, E_i0 and the set of strict ancestors of each node.  (Powers of one decay
  // are taken as such: 64 factors with the same rounding were off by 1.3e-6.)
  const float gh = delta ? 0.f : floor_decay(p.g[h]);
  for (int i = tid; i < MP; i += NT) {
    unsigned long long m = 0;
    float e = alpha[i];
    int s = 0, a = par[i];
    for (; a >= 0; a = par[a], ++s) {
      m |= 1ull << a;
      AC[i * MP + s] = make_float2(e, e);  // E_ij, times the products below
      idx[i * MP + s] = (unsigned char)a;
      e = delta ? e * alpha[a] : expf(gh * (float)(s + 2));
    }
    // to a multiple of four: the parent again, with factors of zero
    for (; s & 3; ++s) {
      idx[i * MP + s] = idx[i * MP];
      AC[i * MP + s] = make_float2(0.f, 0.f);
    }
    anc[i] = m;
    E0[i] = e;
    rn[i] = rn[MP + i] = 1.f;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (warp == NW - 1) {  // places by depth
    constexpr int PL = (MP + 31) / 32;
    int depth[PL], base = 0, todo = 0;
#pragma unroll
    for (int n = 0; n < PL; ++n) {
      const int i = lane + 32 * n;
      depth[n] = i < M && par[i] >= -1 ? __popcll(anc[i]) : -1;
      todo += __popc(__ballot_sync(0xffffffffu, depth[n] >= 0));
    }
    for (int l = 0; base < todo; ++l) {
      if (lane == 0) level[l] = base;
#pragma unroll
      for (int n = 0; n < PL; ++n) {
        const unsigned m = __ballot_sync(0xffffffffu, depth[n] == l);
        if (depth[n] == l) order[base + __popc(m & ((1u << lane) - 1))] = lane + 32 * n;
        base += __popc(m);
      }
      if (lane == 0) level[l + 1] = base;
    }
    if (lane == 0 && todo == 0) level[0] = 0;
    if (lane == 0) *nodes = todo;
  }
  if (p.raw) {
    for (int r = warp; r < 2 * MP; r += NW) {
      float ss = 0.f;
      for (int d = lane; d < DK; d += 32) {
        float y = 0.f;
#pragma unroll
        for (int t = XP - 1; t >= 0; --t) y += to_f32(X[(size_t)(t * 2 * MP + r) * L::LDX + d]);
        ss = fmaf(y, y, ss);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (lane == 0) rn[r] = inv_norm(ss);
    }
    __syncthreads();
  }

  // fragment words of X: rows r (A: r = tile row; B: r = node), K positions 16 ks + 4 tig
  auto xw = [&](int t, int r, int ks) {
    return *reinterpret_cast<const uint2 *>(X + (size_t)(t * 2 * MP + r) * L::LDX + 16 * ks + 4 * tig);
  };
  // [k; q] k^T -> AC (ancestors only)
  for (int mt = warp; mt < 2 * MP / 16; mt += NW) {
    float acc[MP / 8][4] = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a[XP][4];
#pragma unroll
      for (int t = 0; t < XP; ++t) {
        const uint2 u0 = xw(t, 16 * mt + gid, ks), u1 = xw(t, 16 * mt + gid + 8, ks);
        a[t][0] = u0.x; a[t][1] = u1.x; a[t][2] = u0.y; a[t][3] = u1.y;
      }
#pragma unroll
      for (int n = 0; n < MP / 8; ++n) {
        uint32_t bb[XP][2];
#pragma unroll
        for (int t = 0; t < XP; ++t) {
          const uint2 w = xw(t, 8 * n + gid, ks);
          bb[t][0] = w.x; bb[t][1] = w.y;
        }
        mma_terms<XP, XP>(acc[n], a, bb);
      }
    }
#pragma unroll
    for (int n = 0; n < MP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * mt + gid + 8 * (e >> 1), c = 8 * n + 2 * tig + (e & 1);
        const int i = r < MP ? r : r - MP;
        const float y = acc[n][e] * (rn[r] * rn[c]);
        if (anc[i] >> c & 1) {
          const int s = i * MP + __popcll(anc[i] >> c) - 1;  // its place on the path
          (r < MP ? AC[s].x : AC[s].y) *= y;
        } else if (i == c && r >= MP) {
          cself[i] = y;
        }
      }
  }
  // S0 [k; q]^T
  float acc[MT][NX][4] = {};
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    uint32_t a[MT][SP][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t w0[SP][2], w1[SP][2];
      split4<SP>(sf[ks % PF][mt][0], w0);
      split4<SP>(sf[ks % PF][mt][1], w1);
#pragma unroll
      for (int t = 0; t < SP; ++t) {
        a[mt][t][0] = w0[t][0]; a[mt][t][1] = w1[t][0]; a[mt][t][2] = w0[t][1]; a[mt][t][3] = w1[t][1];
      }
    }
    if (ks + PF < KS) load_ks(ks % PF, ks + PF);
#pragma unroll
    for (int n = 0; n < NX; ++n) {
      if (n < MP / 8 && !delta) continue;  // the linear rule needs no S0 k
      uint32_t bb[XP][2];
#pragma unroll
      for (int t = 0; t < XP; ++t) {
        const uint2 w = xw(t, 8 * n + gid, ks);
        bb[t][0] = w.x; bb[t][1] = w.y;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) mma_terms<SP, XP>(acc[mt][n], a[mt], bb);
    }
  }
  __syncthreads();  // X has been used: U and O take its place
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int n = 0; n < NX; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 16 * (warp * MT + mt) + gid + 8 * (e >> 1), r = 8 * n + 2 * tig + (e & 1);
        const int i = r < MP ? r : r - MP;
        (r < MP ? U : O)[i * L::LDU + d] = E0[i] * rn[r] * acc[mt][n][e];
      }
  __syncthreads();

  const int total = *nodes, d = 4 * lane;
  for (int l = 0, begin = 0; begin < total; ++l) {
    const int end = level[l + 1];
    for (int at = begin + warp; at < end; at += NW) {
      const int i = order[at];
      if (d < DV) {
        float r[4], y[4], u[4];
        load4(V + i * DV + d, r);
        load4(O + i * L::LDU + d, y);
        load4(U + i * L::LDU + d, u);
        if (delta)
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] -= u[e];
        for (int s = 0; s < l; s += 4) {  // l: the length of the path before i
          const uchar4 a = *reinterpret_cast<const uchar4 *>(idx + i * MP + s);
          const float4 f0 = *reinterpret_cast<const float4 *>(AC + i * MP + s);
          const float4 f1 = *reinterpret_cast<const float4 *>(AC + i * MP + s + 2);
          float ua[4][4];
          load4(U + a.x * L::LDU + d, ua[0]);
          load4(U + a.y * L::LDU + d, ua[1]);
          load4(U + a.z * L::LDU + d, ua[2]);
          load4(U + a.w * L::LDU + d, ua[3]);
          const float fa[4] = {f0.x, f0.z, f1.x, f1.z}, fc[4] = {f0.y, f0.w, f1.y, f1.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (delta) r[e] = fmaf(-fa[k], ua[k][e], r[e]);
              y[e] = fmaf(fc[k], ua[k][e], y[e]);
            }
        }
        const float bt = delta ? bet[i] : 1.f, cs = cself[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] = bt * r[e];
          y[e] = p.scale * fmaf(cs, u[e], y[e]);
        }
        *reinterpret_cast<float4 *>(U + i * L::LDU + d) = make_float4(u[0], u[1], u[2], u[3]);
        store_state4(p.o, (((size_t)b * M + i) * p.Hv + h) * DV + d, p.o_bf16, y);
      }
    }
    begin = end;
    __syncthreads();  // the next depth reads these u
  }
}

template <typename T, typename ST, int SP, int XP, int DK, int DV, int MP>
cudaError_t launch_mp(const Params &p, int B, cudaStream_t stream) {
  static std::atomic<bool> flags[64];
  auto kern = decode_tree_kernel<T, ST, SP, XP, DK, DV, MP>;
  constexpr int bytes = Layout<T, XP, DK, DV, MP>::BYTES;
  static_assert(bytes <= 232448, "shared memory of a CTA");
  const cudaError_t e = set_smem_once(kern, bytes, flags);
  if (e != cudaSuccess) return e;
  const unsigned threads = DV == 128 && MP == 64 ? 256 : 128;
  return launch_pdl(kern, dim3((unsigned)B * (unsigned)p.Hv), dim3(threads), bytes, stream, p);
}

// ---------------------------------------------------------------------------
// Commit: state_out[dst] <- the state after node accept[b] of each tree (the
// cached state itself where accept is -1).  The path is applied token by token
// in registers between one read and one write of each state; only the path's k
// and v are read.  Rows are laid out as in the decode kernels.  Bound: HBM: 64 trees of
// 32 random nodes 69.6 us, 403 MB of fp32 states at 5.8 TB/s; paths
// of 32 tokens 143 us, where the fp32 pipe binds.
struct CommitParams {
  const void *k, *v;
  const float *g, *beta;
  const int32_t *parent, *accept;
  const void *state_in;
  void *state_out;
  const int32_t *src_slot, *dst_slot;
  int num_slots, M, Hqk, Hv, raw;
  int32_t *status;
};

template <typename T, typename ST, int DK, int DV>
__global__ void __launch_bounds__(128, 4)
tree_commit_kernel(const CommitParams p) {
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  using L = rows::Lane<ST, DK>;
  constexpr int NV4 = L::NV4, ROWS = DV / 4, GROUPS = ROWS / 4, BATCH = GROUPS < 4 ? GROUPS : 4;
  extern __shared__ __align__(16) float stage[];  // k [M][DK] in lane order, v [M][DV], along the path
  __shared__ int path[kMaxNodes], par[kMaxNodes];
  __shared__ int len_s;
  __shared__ float al[kMaxNodes], bt[kMaxNodes];
  const int b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv;
  const int j = h / (p.Hv / p.Hqk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c8 = lane & 7, rr = lane >> 3;
  const int M = p.M;
  const int src = p.src_slot ? p.src_slot[b] : b;
  if (src < 0) return;  // padding entry
  const int dst = p.dst_slot ? p.dst_slot[b] : src;
  if (src >= p.num_slots || dst < 0 || dst >= p.num_slots) {
    if (tid == 0) report_status(p.status, GDN_ERR_INVALID_ARG);
    return;
  }
  const size_t row0 = (size_t)h * DV + warp * ROWS;
  const ST *Sin = static_cast<const ST *>(p.state_in) + ((size_t)src * p.Hv * DV + row0) * DK;
  ST *Sout = static_cast<ST *>(p.state_out) + ((size_t)dst * p.Hv * DV + row0) * DK;
  typename L::Raw raw[BATCH];
#pragma unroll
  for (int x = 0; x < BATCH; ++x) L::load(raw[x], Sin + (size_t)(x * 4 + rr) * DK, c8);

  const int accept = p.accept[b];
  for (int i = tid; i < M; i += 128) par[i] = p.parent[(size_t)b * M + i];
  __syncthreads();
  if (tid == 0) {  // the path, last node first; parents strictly decrease, so the walk ends
    int n = 0, a = accept;
    bool ok = a >= -1 && a < M;
    while (ok && a >= 0) {
      path[n++] = a;
      const int pa = par[a];
      ok = pa >= -1 && pa < a;
      a = pa;
    }
    len_s = ok ? n : -1;
  }
  __syncthreads();
  const int n = len_s;
  if (n < 0) {
    if (tid == 0) report_status(p.status, GDN_ERR_INVALID_ARG);
    return;
  }
  const bool delta = p.beta != nullptr;
  // The linear rule's powers are taken as such (64 factors with the same rounding were off
  // by 1.9e-6): S = lam^n S0 + sum_t (lam^{n-1-t} v_t) k_t^T.
  const float gh = delta ? 0.f : floor_decay(p.g[h]);
  float *ks = stage, *vs = stage + n * DK;
#pragma unroll 2
  for (int x = tid; x < n * (DK / 8); x += 128) {
    const int t = x / (DK / 8), d = 8 * (x - t * (DK / 8));
    float y[8];
    rows::load8(static_cast<const T *>(p.k) + (((size_t)b * M + path[n - 1 - t]) * p.Hqk + j) * DK + d, y);
#pragma unroll
    for (int e = 0; e < 8; e += 4)
      *reinterpret_cast<float4 *>(ks + t * DK + L::pos(d + e)) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
  }
#pragma unroll 2
  for (int x = tid; x < n * (DV / 8); x += 128) {
    const int t = x / (DV / 8), d = 8 * (x - t * (DV / 8));
    float y[8];
    rows::load8(static_cast<const T *>(p.v) + (((size_t)b * M + path[n - 1 - t]) * p.Hv + h) * DV + d, y);
    if (!delta) {
      const float w = expf(gh * (float)(n - 1 - t));
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= w;
    }
#pragma unroll
    for (int e = 0; e < 8; e += 4)
      *reinterpret_cast<float4 *>(vs + t * DV + d + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
  }
  for (int t = tid; t < n; t += 128) {
    if (delta) {
      const size_t gi = ((size_t)b * M + path[n - 1 - t]) * p.Hv + h;
      al[t] = p.raw ? alpha_raw(p.g[gi]) : expf(p.g[gi]);
      bt[t] = p.raw ? beta_raw(p.beta[gi]) : p.beta[gi];
    } else {
      al[t] = t == 0 ? expf(gh * (float)n) : 1.f;
    }
  }
  __syncthreads();
  if (p.raw) {  // unit L2 norm of each k
    for (int t = warp; t < n; t += 4) {
      float ss = 0.f;
      for (int d = lane; d < DK; d += 32) ss = fmaf(ks[t * DK + d], ks[t * DK + d], ss);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float r = inv_norm(ss);
      for (int d = lane; d < DK; d += 32) ks[t * DK + d] *= r;
    }
    __syncthreads();
  }

#pragma unroll
  for (int gb = 0; gb < GROUPS; gb += BATCH) {
    if (gb > 0) {
#pragma unroll
      for (int x = 0; x < BATCH; ++x) L::load(raw[x], Sin + (size_t)((gb + x) * 4 + rr) * DK, c8);
    }
    float2 s[BATCH][NV4 * 2];
#pragma unroll
    for (int x = 0; x < BATCH; ++x) L::widen(raw[x], reinterpret_cast<float *>(s[x]));
    for (int t = 0; t < n; ++t) {
      float2 kf[NV4 * 2];
#pragma unroll
      for (int m = 0; m < NV4; ++m)
        *reinterpret_cast<float4 *>(kf + 2 * m) = *reinterpret_cast<const float4 *>(ks + t * DK + 32 * m + 4 * c8);
      const float alpha = al[t];
      const float2 alpha2 = make_float2(alpha, alpha);
      float c[BATCH];
#pragma unroll
      for (int x = 0; x < BATCH; ++x) c[x] = vs[t * DV + warp * ROWS + (gb + x) * 4 + rr];
      if (delta) {
        float2 u2[BATCH];
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
          u2[x] = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < NV4 * 2; ++e) u2[x] = __ffma2_rn(s[x][e], kf[e], u2[x]);
        }
        static_assert(BATCH == 4, "four row groups at a time");
        const float sums[4] = {u2[0].x + u2[0].y, u2[1].x + u2[1].y, u2[2].x + u2[2].y, u2[3].x + u2[3].y};
        const float mine = rows::reduce4(sums, c8);  // of row group c8 mod 4
#pragma unroll
        for (int x = 0; x < BATCH; ++x)
          c[x] = bt[t] * (c[x] - alpha * __shfl_sync(0xffffffffu, mine, (lane & ~7) | x));
      }
#pragma unroll
      for (int x = 0; x < BATCH; ++x) {
        const float2 c2 = make_float2(c[x], c[x]);
#pragma unroll
        for (int e = 0; e < NV4 * 2; ++e) s[x][e] = __ffma2_rn(alpha2, s[x][e], __fmul2_rn(c2, kf[e]));
      }
    }
#pragma unroll
    for (int x = 0; x < BATCH; ++x)
      L::store(Sout + (size_t)((gb + x) * 4 + rr) * DK, reinterpret_cast<const float *>(s[x]), c8);
  }
}

}  // namespace tree

int tree_max_nodes() { return tree::kMaxNodes; }

cudaError_t launch_decode_tree(const void *q, const void *k, const void *v, const float *g,
                               const float *beta, const int32_t *parent, const void *state,
                               const int32_t *src_slot, int num_slots, void *o, int B, int M, int Hqk,
                               int Hv, int Dk, int Dv, int dtype, int o_dtype, int state_dtype,
                               int input_form, float scale, int32_t *status, cudaStream_t stream) {
  tree::Params p;
  p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.parent = parent; p.state = state;
  p.src_slot = src_slot; p.num_slots = num_slots; p.o = o; p.o_bf16 = o_dtype == GDN_DTYPE_BF16;
  p.M = M; p.Hqk = Hqk; p.Hv = Hv; p.raw = input_form == GDN_INPUT_RAW; p.scale = scale; p.status = status;
  // Terms: an fp32 value has 24 significant bits, three bf16 terms; where the
  // output is rounded to bf16, two (16 bits) leave its rounding the largest error.
  return rows::dispatch_state_dims(state_dtype, Dk, Dv, [&](auto st, auto dk, auto dv) {
    using ST = decltype(st);
    constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
    constexpr bool fp32_state = sizeof(ST) == 4;
    auto nodes = [&](auto t, auto sp, auto xp) {
      using T = decltype(t);
      constexpr int SP = decltype(sp)::value, XP = decltype(xp)::value;
      // Node counts are padded to 16, 32 or 64.  In the next larger instances, 8 nodes (64
      // trees, 16/48 heads) take 76 and 203 us against 57 from a flushed L2, 17 nodes 217
      // against 84.
      if (M <= 16) return tree::launch_mp<T, ST, SP, XP, DK, DV, 16>(p, B, stream);
      if (M <= 32) return tree::launch_mp<T, ST, SP, XP, DK, DV, 32>(p, B, stream);
      return tree::launch_mp<T, ST, SP, XP, DK, DV, 64>(p, B, stream);
    };
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    using S2 = std::conditional_t<fp32_state, I2, I1>;
    using S3 = std::conditional_t<fp32_state, I3, I1>;
    if (dtype == GDN_DTYPE_BF16) {
      if (fp32_state && !p.o_bf16) return nodes(__nv_bfloat16{}, S3{}, I1{});
      return nodes(__nv_bfloat16{}, S2{}, I1{});
    }
    return nodes(float{}, S3{}, I3{});
  });
}

cudaError_t launch_tree_commit(const void *k, const void *v, const float *g, const float *beta,
                               const int32_t *parent, const int32_t *accept, const void *state_in,
                               void *state_out, const int32_t *src_slot, const int32_t *dst_slot,
                               int num_slots, int B, int M, int Hqk, int Hv, int Dk, int Dv, int dtype,
                               int state_dtype, int input_form, int32_t *status, cudaStream_t stream) {
  tree::CommitParams p;
  p.k = k; p.v = v; p.g = g; p.beta = beta; p.parent = parent; p.accept = accept; p.state_in = state_in;
  p.state_out = state_out; p.src_slot = src_slot; p.dst_slot = dst_slot; p.num_slots = num_slots;
  p.M = M; p.Hqk = Hqk; p.Hv = Hv; p.raw = input_form == GDN_INPUT_RAW; p.status = status;
  return rows::dispatch_state_dims(state_dtype, Dk, Dv, [&](auto st, auto dk, auto dv) {
    using ST = decltype(st);
    constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
    auto go = [&](auto t) {
      using T = decltype(t);
      static std::atomic<bool> flags[64];
      auto kern = tree::tree_commit_kernel<T, ST, DK, DV>;
      const cudaError_t e = set_smem_once(kern, tree::kMaxNodes * (DK + DV) * 4, flags);
      if (e != cudaSuccess) return e;
      return launch_pdl(kern, dim3((unsigned)B * (unsigned)Hv), dim3(128), (size_t)M * (DK + DV) * 4, stream, p);
    };
    return dtype == GDN_DTYPE_BF16 ? go(__nv_bfloat16{}) : go(float{});
  });
}

}  // namespace gdn
