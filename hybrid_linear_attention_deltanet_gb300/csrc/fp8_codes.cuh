// e4m3 codes with a scale a block: what the norm, the quantisation and the
// attention cache share.  m = max(|x|, 2^-100) over the block, scale = m / 448,
// code = e4m3(448 x / m).
#pragma once

#include <cuda_fp8.h>

#include "gdn_internal.cuh"

namespace gdn {

constexpr float kTiny = 0x1p-100f;     // the smallest block maximum: its scale stays normal
constexpr float kE4m3Max = 448.f;

// a NaN wins, so that a block with one shows it
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float amax8(const float (&y)[8]) {
  float m = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(y[i]));
  return m;
}
// 8 e4m3 codes of v (round to nearest even, ties in v as they stand; a NaN
// keeps a NaN code).
__device__ __forceinline__ uint2 codes8(const float (&v)[8]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t c =
        __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    w[i >> 1] |= (uint32_t)c << (16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}
// 448 / m to a few units in the last place (scaled, so that no m from 2^-100 up
// has a subnormal reciprocal), and m / 448 rounded to nearest: the product with
// the rounded reciprocal, corrected by its exact remainder (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34, 1990).
__device__ __forceinline__ float codes_per(float m) { return 1.75f * rcp_sfu(m * 0x1p-8f); }
__device__ __forceinline__ float scale_of(float m) {
  constexpr float r = 1.f / kE4m3Max;
  const float q = __fmul_rn(m, r);
  return isinf(q) ? q : __fmaf_rn(__fmaf_rn(-kE4m3Max, q, m), r, q);
}
// The codes of 448 x / m, x bf16 numbers of a block whose largest magnitude is m.
__device__ __forceinline__ uint2 quantise8_bf16(const float (&x)[8], float m) {
  float v[8];
  // 0.875 x is exact, so one step with the quotient's exact remainder (scale_of's)
  // gives the rounded quotient, and the quotient itself where it has few
  // bits, as the middle between two codes does (no other is so near one that
  // fp32 rounds to it: it is apart by 2^-13 at least)
  const float d = m * 0x1p-9f, r = rcp_sfu(d);   // 448 / m = 0.875 / d
  const F2 rr = f2(r, r), dd = f2(-d, -d), k = f2(0.875f, 0.875f);   // two at a time
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const F2 a = f2_mul(f2(x[i], x[i + 1]), k), q = f2_mul(a, rr);
    f2_split(f2_fma(f2_fma(q, dd, a), rr, q), v[i], v[i + 1]);
  }
  return codes8(v);
}

}  // namespace gdn
