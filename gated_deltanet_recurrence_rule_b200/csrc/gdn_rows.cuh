// gdn_rows.cuh -- state rows spread over 8 lanes, for the kernels that stream
// recurrent states (fp32, or bf16 at rest) from HBM and back.
//
// Lane c8 (0..7) of a row holds DK / 8 elements as NV4 float4 pieces.  fp32
// rows: piece i at columns 32 i + 4 c8; bf16 rows: 16-byte loads at columns
// 64 m + 8 c8, pieces 2m and 2m + 1.  Either way a warp's load instruction
// covers four whole 128-byte segments.  pos(d) is where column d is staged in
// shared memory so that lane c8 reads its i-th piece at 32 i + 4 c8, free of
// bank conflicts, whatever the state's type.
#pragma once

#include <type_traits>

#include "gdn_common.cuh"

namespace gdn {
namespace rows {

// Four rows' sums over the 8 lanes of a row group, each lane c8 left with the sum of
// row c8 mod 4 (two rows change places at each of two steps: 4 shuffles, not 12).
__device__ __forceinline__ float reduce4(const float p[4], int c8) {
  const bool b0 = c8 & 1, b1 = c8 & 2;
  const float a = (b0 ? p[1] : p[0]) + __shfl_xor_sync(0xffffffffu, b0 ? p[0] : p[1], 1);
  const float b = (b0 ? p[3] : p[2]) + __shfl_xor_sync(0xffffffffu, b0 ? p[2] : p[3], 1);
  const float c = (b1 ? b : a) + __shfl_xor_sync(0xffffffffu, b1 ? a : b, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 4);
}

template <typename ST, int DK>
struct Lane;

template <int DK>
struct Lane<float, DK> {
  static constexpr int NV4 = DK / 32;
  struct Raw { float4 x[NV4]; };
  static __device__ __forceinline__ int pos(int d) { return d; }
  static __device__ __forceinline__ void load(Raw &r, const float *row, int c8) {
#pragma unroll
    for (int i = 0; i < NV4; ++i) r.x[i] = ld_stream(reinterpret_cast<const float4 *>(row + 32 * i + 4 * c8));
  }
  static __device__ __forceinline__ void widen(const Raw &r, float *s) {
#pragma unroll
    for (int i = 0; i < NV4; ++i) {
      s[4 * i] = r.x[i].x; s[4 * i + 1] = r.x[i].y; s[4 * i + 2] = r.x[i].z; s[4 * i + 3] = r.x[i].w;
    }
  }
  static __device__ __forceinline__ void store(float *row, const float *s, int c8) {
#pragma unroll
    for (int i = 0; i < NV4; ++i)
      st_stream(reinterpret_cast<float4 *>(row + 32 * i + 4 * c8),
                make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]));
  }
};

template <int DK>
struct Lane<__nv_bfloat16, DK> {
  static constexpr int NV4 = DK / 32;
  struct Raw { uint4 x[NV4 / 2]; };
  static __device__ __forceinline__ int pos(int d) {
    return 32 * (2 * (d >> 6) + ((d >> 2) & 1)) + 4 * ((d >> 3) & 7) + (d & 3);
  }
  static __device__ __forceinline__ void load(Raw &r, const __nv_bfloat16 *row, int c8) {
#pragma unroll
    for (int m = 0; m < NV4 / 2; ++m) r.x[m] = __ldcs(reinterpret_cast<const uint4 *>(row + 64 * m + 8 * c8));
  }
  static __device__ __forceinline__ void widen(const Raw &r, float *s) {
#pragma unroll
    for (int m = 0; m < NV4 / 2; ++m) {
      const uint32_t w[4] = {r.x[m].x, r.x[m].y, r.x[m].z, r.x[m].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[8 * m + 2 * e] = __uint_as_float(w[e] << 16);
        s[8 * m + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *row, const float *s, int c8) {
#pragma unroll
    for (int m = 0; m < NV4 / 2; ++m) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(s[8 * m + 2 * e], s[8 * m + 2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t *>(&y);
      }
      __stcs(reinterpret_cast<uint4 *>(row + 64 * m + 8 * c8), make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
};

// 8 consecutive elements as fp32 (16-byte aligned; fp32: 32 bytes).
__device__ __forceinline__ void load8(const float *p, float out[8]) {
  load4(p, out);
  load4(p + 4, out + 4);
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float out[8]) {
  const uint4 x = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    out[2 * e] = __uint_as_float(w[e] << 16);
    out[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// Call f(ST{}, DK, DV) with the state's element type and the head dims as
// integral constants (64 or 128 each).
template <class F>
__host__ auto dispatch_state_dims(int state_dtype, int Dk, int Dv, F &&f) {
  auto dims = [&](auto st) {
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (Dk == 128) return Dv == 128 ? f(st, I128{}, I128{}) : f(st, I128{}, I64{});
    return Dv == 128 ? f(st, I64{}, I128{}) : f(st, I64{}, I64{});
  };
  if (state_dtype == GDN_DTYPE_BF16) return dims(__nv_bfloat16{});
  return dims(float{});
}

}  // namespace rows
}  // namespace gdn
