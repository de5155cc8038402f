// gdn_linear.cuh -- the scan that linear attention with a head decay and its
// gradients are made of, and the layouts its kernels share.
//
// One scan over a sequence, lam = e^g of the head, X a (Dc x Da) state:
//     X_t = lam X_{t-1} + s_upd c_t b_t^T
//     out_t = s_inter lam^{..} X0 a_t + s_intra sum_s lam^{|t-s|} (b_s . a_t) c_s
// over s <= t, or (back) from the last token to the first, over s >= t.
//     o  : a = q,  b = k,  c = v          X = S
//     dq : a = do, b = v,  c = k          X = S^T
//     dv : a = k,  b = q,  c = do, back   X = D,   D_t = lam D_{t+1} + scale do_t q_t^T
//     dk : a = v,  b = do, c = q,  back   X = D^T
// (out_t uses the state with token t in it, so X0 enters token i of a sequence with
// lam^{i+1}; dL/dS_final is a gradient of the state after the last token, so going
// back it enters with one factor less: `first`.)
//
// Sequences are cut into segments of L tokens.  (1) The state each segment adds
// for the ones after it, all segments at once; (2) a prefix over the segments of each
// sequence turns those into the state each segment starts from; (3) the outputs, all
// segments at once, each walking its chunks from its start state.  The final state of
// a sequence of several segments comes from (2), that of one from (3).  (1) and (2)
// only concern sequences longer than L; where no sequence can be, (3) alone is launched.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "gdn_common.cuh"

namespace gdn {
namespace lin {

struct Scan {
  const void *a, *b, *c;  // [T, Ha | Hb | Hc, Da | Da | Dc], element type T
  int Ha, Hb, Hc;         // their heads: Hv or Hqk
  void *out;              // [T, Hv, Dc], and NULL where T = 0
  const float *g;         // [Hv]
  const int32_t *cu;
  int N, T, Hv, Da, Dc;
  int back;
  int states_only;        // what each segment adds, into seg_state; no outputs
  float s_intra, s_inter, s_upd;
  const int4 *units;         // [segments] the segments, longest first (below); NULL where each
                             // sequence is one segment
  int L;
  float *seg_state;          // [cut segments, Hv, Dc, Da] added (states only) or starting state;
                             // a sequence of one segment starts from x0 (and x0 may be xf: of
                             // several, the last may end before the first has started)
  const void *x0;            // [N, Hv, Dc, Da], or (x0_tr) [N, Hv, Da, Dc]; NULL: zeros
  void *xf;                  // [N, Hv, Dc, Da], NULL to skip; back: times lam
  int x0_tr, x_bf16;
  int32_t *status;
};

// What one CTA works on: tokens [t0, t1) of sequence n, head h.
struct Unit {
  int n, h, t0, t1, seg;
  int first, last;  // the segment its sequence's scan starts, ends with
};

// A segment of the plan: x the slot of its state (of a sequence of several), with kFirst
// and kLast where it is the first or last of its sequence (-1: no segment), y the
// sequence, z and w its tokens.
constexpr int kFirst = 1 << 30, kLast = 1 << 29;

// False where unit `u` does not exist or cu_seqlens is inconsistent.
__device__ __forceinline__ bool get_unit(const Scan &p, int u, Unit &w) {
  w.seg = u / p.Hv;
  w.h = u - w.seg * p.Hv;
  if (p.units) {
    const int4 s = p.units[w.seg];
    if (s.x < 0) return false;
    w.seg = s.x & (kLast - 1);
    w.n = s.y;
    w.t0 = s.z;
    w.t1 = s.w;
    const int first = (s.x & kFirst) != 0, last = (s.x & kLast) != 0;
    w.first = p.back ? last : first;
    w.last = p.back ? first : last;
    return true;
  }
  w.n = w.seg;
  const int c0 = p.cu[w.n], c1 = p.cu[w.n + 1];
  if (c0 < 0 || c1 < c0 || c1 > p.T || (w.n == 0 && c0 != 0) || (w.n == p.N - 1 && c1 != p.T)) {
    if (threadIdx.x == 0) report_status(p.status, GDN_ERR_BAD_SEQLENS);
    return false;
  }
  w.t0 = c0;
  w.t1 = c1;
  w.first = w.last = 1;
  return true;
}

__device__ __forceinline__ float head_decay(const Scan &p, int h) { return floor_decay(p.g[h]); }

// lam^n for a state that is carried over many stretches of n tokens.  Rounded to fp32 it
// would be off the same way each time, by as many half steps in the end as there are
// stretches in the head's memory (3.4e-6 after 16,000 tokens of a slow head).  So a power
// near one is held as 1 + m, and what a factor's rounding leaves goes into the next one:
// every product of factors is then right to a step or two.
struct Power {
  float value, m;  // value = lam^n, and m = lam^n - 1 where that is above -1/2; else 2
};
__device__ __forceinline__ Power decay_power(float g, int n) {
  const float x = g * (float)n;
  return Power{expf(x), x > -0.6931f ? expm1f(x) : 2.f};
}
struct Carry {
  float rest;  // 0 at first
  __device__ __forceinline__ float next(const Power &p) {
    if (p.m == 2.f) return p.value;
    const float t = rest + p.m, f = 1.f + t;
    rest = t - (f - 1.f);
    return f;
  }
};

// Element (i, j) of a sequence's initial state.
__device__ __forceinline__ float initial_state(const Scan &p, const Unit &w, int i, int j) {
  if (!p.x0) return 0.f;
  const size_t base = ((size_t)w.n * p.Hv + w.h) * p.Dc * p.Da;
  const size_t e = base + (p.x0_tr ? (size_t)j * p.Dc + i : (size_t)i * p.Da + j);
  return p.x_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.x0)[e])
                  : static_cast<const float *>(p.x0)[e];
}

// Element (i, j) of the state a unit starts from.
__device__ __forceinline__ float start_state(const Scan &p, const Unit &w, int i, int j) {
  if (!w.first || !w.last) return p.seg_state[(((size_t)w.seg * p.Hv + w.h) * p.Dc + i) * p.Da + j];
  return initial_state(p, w, i, j);
}

// ---- host ----
// The CUDA-core-and-mma.sync form, every type and head dim (gdn_linear_scan.cu).
cudaError_t launch_scan(const Scan &p, int units, int dtype, int out_dtype, cudaStream_t stream);
// The tcgen05 form (gdn_linear_tc.cu): bf16 operands.  States that are returned or
// handed to another segment are summed from products of all 24 bits; its outputs carry
// the roundings of bf16 operands, whatever type they are stored in.
bool scan_tc_supported(const Scan &p, int dtype);
cudaError_t launch_scan_tc(const Scan &p, int units, int out_dtype, cudaStream_t stream);

}  // namespace lin
}  // namespace gdn
