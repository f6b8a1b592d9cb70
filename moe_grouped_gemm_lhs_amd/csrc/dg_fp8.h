// dg_fp8.h -- the fp8 rounding shared by every kernel that writes codes (dg_quant.hip,
// dg_norm.hip, dg_gated.hip): quotients by a block's scale and their conversion.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_internal.h"

namespace dg {
namespace {

template <int FMT>
__device__ __forceinline__ float fp8_max() {
  return FMT == kFmtE5M2 ? 57344.0f : 448.0f;
}

// Smallest scale whose quotients take the reciprocal path below.  From 2^-64 up, 1/scale
// is finite and, for every quotient that can round to a non-zero fp8 code (|x/scale| >=
// 2^-18), x >= 2^-82 and y*scale is a multiple of 2^-128, so the residual below is an
// exact fp32 value; smaller quotients give the zero code whatever their last bits.
constexpr float kMinReciprocalScale = 0x1p-64f;

// x / scale rounded to nearest fp32, from a correctly rounded reciprocal r = 1/scale:
// y = x*r is within an ulp of the quotient and the residual x - y*scale is exact (one
// fma), so y + r*residual rounded once is the correctly rounded quotient (Markstein's
// theorem; no overflow: |x| <= amax = scale * FMAX).  The sign comes from x (scale > 0),
// which also keeps the sign of a zero.  Blocks with a scale under kMinReciprocalScale
// (amax below FMAX * 2^-64: tiny and subnormal inputs, where 1/scale overflows or the
// residual underflows) take the IEEE division instead; there a scale that underflowed to
// zero gives +-inf (saturated below) and 0/0 a zero with the sign of x.
// TINY: some lane of the wave holds such a block (decided once per wave by the caller,
// so that the usual case carries no division at all).
template <bool TINY>
__device__ __forceinline__ float div_by_scale(float x, float scale, float r) {
  if (!TINY || scale >= kMinReciprocalScale) {
    const float y = x * r;
    const float e = __builtin_fmaf(-y, scale, x);
    return __builtin_copysignf(__builtin_fmaf(e, r, y), x);
  }
  const float q = x / scale;                      // correctly rounded fp32 division
  return q != q ? __builtin_copysignf(0.0f, x) : q;
}

// Four codes: the quotients saturated to +-FMAX, then converted by the hardware's
// round-to-nearest-even fp8 conversion (OCP E4M3 / E5M2 on gfx950).
template <int FMT, bool TINY>
__device__ __forceinline__ uint32_t pack4(const float* x, float scale, float r) {
  const float m = fp8_max<FMT>();
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = fminf(fmaxf(div_by_scale<TINY>(x[i], scale, r), -m), m);
  int v;
  if (FMT == kFmtE5M2) {
    v = __builtin_amdgcn_cvt_pk_bf8_f32(q[0], q[1], 0, false);
    v = __builtin_amdgcn_cvt_pk_bf8_f32(q[2], q[3], v, true);
  } else {
    v = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], v, true);
  }
  return (uint32_t)v;
}

}  // namespace
}  // namespace dg
