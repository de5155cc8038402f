// gdn_linear_decode.cu -- 1 to 16 new tokens of linear attention with a decay
// for each head, states in a slot pool.
//
// Per (sequence b, value head h), S the Dv x Dk state, lam = e^{g_h}:
//     S_t = lam S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t.
// Nothing that is written depends on what was read before (unlike the delta
// rule, where v_t is corrected by S k_t), so the call's tokens are taken
// together from the state S0 that was read:
//     o_t  = scale (lam^{t+1} S0 q_t + sum_{s<=t} lam^{t-s} (k_s . q_t) v_s)
//     S_Tn = lam^Tn S0 + sum_s (lam^{Tn-1-s} v_s) k_s^T.
// The token x token factors lam^{t-s} (k_s . q_t) are formed once per CTA.
//
// Bound: HBM (each state read once and written once; 4 Tn flops an element).
// One 128-thread CTA per (b, h), 8 lanes per row, lane c8 of a row holding
// float4 pieces so that a warp's load covers four whole 128-byte segments;
// four row groups (16 rows of a warp) are in flight before the first is used.
#include "gdn_common.cuh"
#include "gdn_rows.cuh"

namespace gdn {
namespace {
constexpr int kMaxLinearTokens = 16;
}

template <typename T, typename TO, typename ST, int DK, int DV, bool ONE>
__global__ void __launch_bounds__(128, 4)
linear_decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                     const float *__restrict__ g, const ST *state_in, ST *state_out,
                     const int32_t *__restrict__ src_slot, const int32_t *__restrict__ dst_slot,
                     int num_slots, TO *__restrict__ o, int Tn_, int Hqk, int Hv, float scale,
                     int32_t *status) {
  pdl_wait();  // nothing is read before the previous kernel on the stream is done
  pdl_allow_next();
  using L = rows::Lane<ST, DK>;
  constexpr int NV4 = L::NV4;
  constexpr int ROWS = DV / 4;        // rows of a warp
  constexpr int GROUPS = ROWS / 4;    // 4 rows per warp instruction
  constexpr int BATCH = GROUPS < 4 ? GROUPS : 4;
  constexpr int MT = ONE ? 1 : kMaxLinearTokens;
  const int Tn = ONE ? 1 : Tn_;
  __shared__ __align__(16) float ks[MT][DK], qs[MT][DK];  // in lane order
  __shared__ float vs[MT][DV];
  __shared__ float os[MT][DV];    // the tokens' own part of o
  __shared__ float qk[MT][MT];    // lam^{t-s} (k_s . q_t)
  __shared__ float lp[MT + 1];    // lam^i

  const int b = blockIdx.x / Hv, h = blockIdx.x - b * Hv;
  const int j = h / (Hv / Hqk);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c8 = lane & 7, rr = lane >> 3;
  const int src = src_slot ? src_slot[b] : b;
  if (src < 0) return;  // padding entry: nothing read or written
  const int dst = dst_slot ? dst_slot[b] : src;
  if (src >= num_slots || dst < 0 || dst >= num_slots) {
    if (tid == 0) report_status(status, GDN_ERR_INVALID_ARG);
    return;
  }
  const size_t row0 = (size_t)h * DV + warp * ROWS;  // first row of this warp in a slot
  const ST *Sin = state_in + ((size_t)src * Hv * DV + row0) * DK;
  ST *Sout = state_out + ((size_t)dst * Hv * DV + row0) * DK;

  typename L::Raw raw[BATCH];
#pragma unroll
  for (int x = 0; x < BATCH; ++x) L::load(raw[x], Sin + (size_t)(x * 4 + rr) * DK, c8);

  const float gh = fmaxf(g[h], rows::kDecayFloor);
  for (int x = tid; x < Tn * DK; x += 128) {
    const int t = x / DK, d = x - t * DK;
    const size_t off = (((size_t)b * Tn + t) * Hqk + j) * DK + d;
    ks[t][L::pos(d)] = to_f32(k[off]);
    qs[t][L::pos(d)] = to_f32(q[off]);
  }
  for (int x = tid; x < Tn * DV; x += 128) {
    const int t = x / DV, d = x - t * DV;
    vs[t][d] = to_f32(v[(((size_t)b * Tn + t) * Hv + h) * DV + d]);
  }
  if (tid <= Tn) lp[tid] = expf(gh * (float)tid);
  __syncthreads();
  // token x token factors, one pair per warp in turn
  for (int x = warp; x < Tn * Tn; x += 4) {
    const int t = x / Tn, s = x - t * Tn;
    if (s > t) continue;
    float a = 0.f;
#pragma unroll
    for (int d = lane; d < DK; d += 32) a = fmaf(ks[s][d], qs[t][d], a);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    if (lane == 0) qk[t][s] = a * lp[t - s];
  }
  __syncthreads();
  for (int x = tid; x < Tn * DV; x += 128) {
    const int t = x / DV, d = x - t * DV;
    float a = 0.f;
    for (int s = 0; s <= t; ++s) a = fmaf(qk[t][s], vs[s][d], a);
    os[t][d] = a;
  }
  __syncthreads();
  for (int x = tid; x < Tn * DV; x += 128) {  // from here vs holds lam^{Tn-1-t} v_t
    const int t = x / DV, d = x - t * DV;
    vs[t][d] *= lp[Tn - 1 - t];
  }
  __syncthreads();

#pragma unroll
  for (int gb = 0; gb < GROUPS; gb += BATCH) {
    if (gb > 0) {
#pragma unroll
      for (int x = 0; x < BATCH; ++x) L::load(raw[x], Sin + (size_t)((gb + x) * 4 + rr) * DK, c8);
    }
    float s[BATCH][NV4 * 4];
#pragma unroll
    for (int x = 0; x < BATCH; ++x) L::widen(raw[x], s[x]);
    for (int t = 0; t < Tn; ++t) {
      float p[BATCH];
#pragma unroll
      for (int x = 0; x < BATCH; ++x) p[x] = 0.f;
#pragma unroll
      for (int m = 0; m < NV4; ++m) {
        const float4 a = *reinterpret_cast<const float4 *>(&qs[t][32 * m + 4 * c8]);
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
          p[x] = fmaf(s[x][4 * m + 0], a.x, p[x]);
          p[x] = fmaf(s[x][4 * m + 1], a.y, p[x]);
          p[x] = fmaf(s[x][4 * m + 2], a.z, p[x]);
          p[x] = fmaf(s[x][4 * m + 3], a.w, p[x]);
        }
      }
#pragma unroll
      for (int off = 1; off < 8; off <<= 1)
#pragma unroll
        for (int x = 0; x < BATCH; ++x) p[x] += __shfl_xor_sync(0xffffffffu, p[x], off);
      if (c8 < BATCH) {  // lane c8 of a row group writes the row of group gb + c8
        float px = p[0];
#pragma unroll
        for (int x = 1; x < BATCH; ++x) px = c8 == x ? p[x] : px;
        const int row = warp * ROWS + (gb + c8) * 4 + rr;
        o[(((size_t)b * Tn + t) * Hv + h) * DV + row] =
            from_f32<TO>(scale * fmaf(lp[t + 1], px, os[t][row]));
      }
    }
    const float lT = lp[Tn];
#pragma unroll
    for (int x = 0; x < BATCH; ++x)
#pragma unroll
      for (int e = 0; e < NV4 * 4; ++e) s[x][e] *= lT;
    for (int t = 0; t < Tn; ++t) {
      float c[BATCH];
#pragma unroll
      for (int x = 0; x < BATCH; ++x) c[x] = vs[t][warp * ROWS + (gb + x) * 4 + rr];
#pragma unroll
      for (int m = 0; m < NV4; ++m) {
        const float4 a = *reinterpret_cast<const float4 *>(&ks[t][32 * m + 4 * c8]);
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
          s[x][4 * m + 0] = fmaf(c[x], a.x, s[x][4 * m + 0]);
          s[x][4 * m + 1] = fmaf(c[x], a.y, s[x][4 * m + 1]);
          s[x][4 * m + 2] = fmaf(c[x], a.z, s[x][4 * m + 2]);
          s[x][4 * m + 3] = fmaf(c[x], a.w, s[x][4 * m + 3]);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < BATCH; ++x) L::store(Sout + (size_t)((gb + x) * 4 + rr) * DK, s[x], c8);
  }
}

int linear_decode_tokens_max() { return kMaxLinearTokens; }

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *g,
                                 const void *state_in, void *state_out, const int32_t *src_slot,
                                 const int32_t *dst_slot, int num_slots, void *o, int B, int Tn,
                                 int Hqk, int Hv, int Dk, int Dv, int dtype, int o_dtype,
                                 int state_dtype, float scale, int32_t *status, cudaStream_t stream) {
  return dispatch_types(dtype, o_dtype, [&](auto t, auto to) {
    using T = decltype(t);
    using TO = decltype(to);
    return rows::dispatch_state_dims(state_dtype, Dk, Dv, [&](auto st, auto dk, auto dv) {
      using ST = decltype(st);
      constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
      auto go = [&](auto kern) {
        return launch_pdl(kern, dim3((unsigned)B * (unsigned)Hv), dim3(128), 0, stream,
                          static_cast<const T *>(q), static_cast<const T *>(k),
                          static_cast<const T *>(v), g, static_cast<const ST *>(state_in),
                          static_cast<ST *>(state_out), src_slot, dst_slot, num_slots,
                          static_cast<TO *>(o), Tn, Hqk, Hv, scale, status);
      };
      if (Tn == 1) return go(linear_decode_kernel<T, TO, ST, DK, DV, true>);
      return go(linear_decode_kernel<T, TO, ST, DK, DV, false>);
    });
  });
}

}  // namespace gdn
