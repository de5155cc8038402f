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
// Measured, 16/48 heads of 128, fp32 states in place: 64 sequences x 1 token 63.9 us
// (403 MB, 6.3 TB/s, 97 % of the copy bandwidth), x 4 81 us, x 16 166 us, where the
// fp32 pipe binds; bf16 states 38 us for one token.
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
  __shared__ __align__(16) float ks[MT][DK + 4], qs[MT][DK + 4];  // in lane order
  __shared__ __align__(16) float vs[MT][DV];
  __shared__ float os[MT][DV];                  // the tokens' own part of o
  __shared__ __align__(16) float qk[MT][16];    // [s][t]: lam^{t-s} (k_s . q_t)
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

  const float gh = floor_decay(g[h]);
#pragma unroll 2
  for (int x = tid; x < Tn * (DK / 8); x += 128) {
    const int t = x / (DK / 8), d = 8 * (x - t * (DK / 8));
    const size_t off = (((size_t)b * Tn + t) * Hqk + j) * DK + d;
    float y[8], z[8];
    rows::load8(k + off, y);
    rows::load8(q + off, z);
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      *reinterpret_cast<float4 *>(&ks[t][L::pos(d + e)]) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
      *reinterpret_cast<float4 *>(&qs[t][L::pos(d + e)]) = make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]);
    }
  }
#pragma unroll 2
  for (int x = tid; x < Tn * (DV / 8); x += 128) {
    const int t = x / (DV / 8), d = 8 * (x - t * (DV / 8));
    float y[8];
    rows::load8(v + (((size_t)b * Tn + t) * Hv + h) * DV + d, y);
    *reinterpret_cast<float4 *>(&vs[t][d]) = make_float4(y[0], y[1], y[2], y[3]);
    *reinterpret_cast<float4 *>(&vs[t][d + 4]) = make_float4(y[4], y[5], y[6], y[7]);
  }
  if (tid <= Tn) lp[tid] = expf(gh * (float)tid);
  __syncthreads();
  // token x token factors, a thread for a pair (16 lanes read one q and 16 k)
  for (int x = tid; x < Tn * 16; x += 128) {
    const int t = x >> 4, s = x & 15;
    if (s > t) continue;
    float a = 0.f;
#pragma unroll 8
    for (int d = 0; d < DK; d += 4) {
      const float4 y = *reinterpret_cast<const float4 *>(&ks[s][d]), z = *reinterpret_cast<const float4 *>(&qs[t][d]);
      a = fmaf(y.x, z.x, fmaf(y.y, z.y, fmaf(y.z, z.z, fmaf(y.w, z.w, a))));
    }
    qk[s][t] = a * lp[t - s];
  }
  __syncthreads();
  // each column's own part of every token's output, then vs <- lam^{Tn-1-t} v_t
  if (tid < DV) {
    float a[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) a[t] = 0.f;
    for (int s = 0; s < Tn; ++s) {
      const float y = vs[s][tid];
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if (t >= s) a[t] = fmaf(qk[s][t], y, a[t]);  // (rows past Tn are not used)
      vs[s][tid] = y * lp[Tn - 1 - s];
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
      if (t < Tn) os[t][tid] = a[t];
  }
  __syncthreads();

#pragma unroll
  for (int gb = 0; gb < GROUPS; gb += BATCH) {
    if (gb > 0) {
#pragma unroll
      for (int x = 0; x < BATCH; ++x) L::load(raw[x], Sin + (size_t)((gb + x) * 4 + rr) * DK, c8);
    }
    float2 s[BATCH][NV4 * 2];
#pragma unroll
    for (int x = 0; x < BATCH; ++x) L::widen(raw[x], reinterpret_cast<float *>(s[x]));
    for (int t = 0; t < Tn; ++t) {
      float2 p[BATCH];
#pragma unroll
      for (int x = 0; x < BATCH; ++x) p[x] = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < NV4; ++m) {
        const float4 a = *reinterpret_cast<const float4 *>(&qs[t][32 * m + 4 * c8]);
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
          p[x] = __ffma2_rn(s[x][2 * m], make_float2(a.x, a.y), p[x]);
          p[x] = __ffma2_rn(s[x][2 * m + 1], make_float2(a.z, a.w), p[x]);
        }
      }
      static_assert(BATCH == 4, "four row groups at a time");
      const float sums[4] = {p[0].x + p[0].y, p[1].x + p[1].y, p[2].x + p[2].y, p[3].x + p[3].y};
      const float px = rows::reduce4(sums, c8);
      if (c8 < BATCH) {  // lane c8 of a row group writes the row of group gb + c8
        const int row = warp * ROWS + (gb + c8) * 4 + rr;
        o[(((size_t)b * Tn + t) * Hv + h) * DV + row] =
            from_f32<TO>(scale * fmaf(lp[t + 1], px, os[t][row]));
      }
    }
    const float2 lT = make_float2(lp[Tn], lp[Tn]);
#pragma unroll
    for (int x = 0; x < BATCH; ++x)
#pragma unroll
      for (int e = 0; e < NV4 * 2; ++e) s[x][e] = __fmul2_rn(s[x][e], lT);
    for (int t = 0; t < Tn; ++t) {
      float2 c[BATCH];
#pragma unroll
      for (int x = 0; x < BATCH; ++x) {
        const float cx = vs[t][warp * ROWS + (gb + x) * 4 + rr];
        c[x] = make_float2(cx, cx);
      }
#pragma unroll
      for (int m = 0; m < NV4; ++m) {
        const float4 a = *reinterpret_cast<const float4 *>(&ks[t][32 * m + 4 * c8]);
#pragma unroll
        for (int x = 0; x < BATCH; ++x) {
          s[x][2 * m] = __ffma2_rn(c[x], make_float2(a.x, a.y), s[x][2 * m]);
          s[x][2 * m + 1] = __ffma2_rn(c[x], make_float2(a.z, a.w), s[x][2 * m + 1]);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < BATCH; ++x)
      L::store(Sout + (size_t)((gb + x) * 4 + rr) * DK, reinterpret_cast<const float *>(s[x]), c8);
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
      // One token has no token x token part and no loop over tokens: from a flushed L2, 64
      // sequences take 71.7 us against 73.7 for the general kernel, with bf16 states 41.0
      // against 45.1, one sequence 10.2 against 12.3.
      if (Tn == 1) return go(linear_decode_kernel<T, TO, ST, DK, DV, true>);
      return go(linear_decode_kernel<T, TO, ST, DK, DV, false>);
    });
  });
}

}  // namespace gdn
