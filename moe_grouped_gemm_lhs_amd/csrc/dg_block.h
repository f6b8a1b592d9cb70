// dg_block.h -- 1x128 blocks of a row as the elementwise kernels of dg_norm.hip and
// dg_gated.hip hold them: 16 lanes (one DPP row) with 8 consecutive values each.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_fp8.h"

namespace dg {
namespace {

// Sum over a wave's 64 lanes, in every lane: in each row of 16 by DPP, then across the rows.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ unsigned dpp(unsigned v) {
  return (unsigned)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// lanes ^1, ^2 (quad_perm), then mirrors of 8 and of 16
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// Largest magnitude of a block, in its 16 lanes.  Magnitudes are compared as unsigned
// integers, where every NaN is above infinity: a NaN in a block is its maximum.
__device__ __forceinline__ unsigned magnitude(float v) {
  return __builtin_bit_cast(unsigned, v) & 0x7FFFFFFFu;
}
__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }
__device__ __forceinline__ float block_amax(const float (&x)[8]) {
  unsigned m = magnitude(x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) m = umax(m, magnitude(x[e]));
  m = umax(m, dpp<kXor1>(m));
  m = umax(m, dpp<kXor2>(m));
  m = umax(m, dpp<kHalfMirror>(m));
  m = umax(m, dpp<kMirror>(m));
  return __builtin_bit_cast(float, m);
}

// Scale of a block, and its eight codes of this lane.
__device__ __forceinline__ float block_scale(float amax, int fmt) {
  return amax == 0.0f ? 1.0f : amax / (fmt == kFmtE5M2 ? fp8_max<kFmtE5M2>() : fp8_max<kFmtE4M3>());
}
// Four codes by the scale's reciprocal (correctly rounded): the quotients are off by 1.5 units of
// their last place at most, so the largest, FMAX, needs no clamp, and only a quotient that near
// the border between two codes may go to the other one, which is as near to it.  A third of the
// exact division's instructions (pack4), and two fewer a value than with the residual added but no
// clamps.  Measured against pack4 and that: gated backward pass 16384 x 2048 38.5 us against 43.7 and
// 40.7; norm without a residual 16384 x 4096 49.4 against 53.2 and 51.8; with one, 4096 x 7168, 41.1
// against 41.4 and 41.2; gated block 16384 x (2048, 7168) with the checkpoint 855 against 858 and 862,
// of few rows no difference.  Scales whose reciprocal may leave fp32's range take the exact division
// (pack4).
template <int FMT>
__device__ __forceinline__ unsigned quick4(const float* x, float r) {
  int v;
  if (FMT == kFmtE5M2) {
    v = __builtin_amdgcn_cvt_pk_bf8_f32(x[0] * r, x[1] * r, 0, false);
    v = __builtin_amdgcn_cvt_pk_bf8_f32(x[2] * r, x[3] * r, v, true);
  } else {
    v = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * r, x[1] * r, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * r, x[3] * r, v, true);
  }
  return (unsigned)v;
}
// N codes (a multiple of four) of a lane in N / 4 words.
template <int FMT, int N>
__device__ __forceinline__ void codes_as(const float (&x)[N], float scale, unsigned (&c)[N / 4]) {
  const float r = 1.0f / scale;
  if (__builtin_amdgcn_ballot_w64(scale < kMinReciprocalScale) == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) c[i] = quick4<FMT>(x + 4 * i, r);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) c[i] = pack4<FMT, true>(x + 4 * i, scale, r);
  }
}
template <int N>
__device__ __forceinline__ void codes(const float (&x)[N], float scale, int fmt, unsigned (&c)[N / 4]) {
  if (fmt == kFmtE5M2)
    codes_as<kFmtE5M2, N>(x, scale, c);
  else
    codes_as<kFmtE4M3, N>(x, scale, c);
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale, int fmt) {
  unsigned c[2];
  codes<8>(x, scale, fmt, c);
  return make_uint2(c[0], c[1]);
}

// Eight consecutive bf16 or fp32 values as they lie in memory, and as fp32.
template <bool BF16>
struct Eight {
  uint4 v[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* s = (const uint4*)((const uint8_t*)p + i * (BF16 ? 2 : 4));
    v[0] = s[0];
    if (!BF16) v[BF16 ? 0 : 1] = s[1];
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    uint4* s = (uint4*)((uint8_t*)p + i * (BF16 ? 2 : 4));
    s[0] = v[0];
    if (!BF16) s[1] = v[BF16 ? 0 : 1];
  }
  __device__ __forceinline__ void zero() {
    v[0] = make_uint4(0, 0, 0, 0);
    v[BF16 ? 0 : 1] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if (BF16) {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16);
        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
    } else {
      const uint4 a = v[0], b = v[BF16 ? 0 : 1];
      x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
      x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
      x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
      x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
    }
  }
  // rounded to nearest even (bf16)
  __device__ __forceinline__ void set(const float (&x)[8]) {
    if (BF16) {
      typedef __bf16 pair __attribute__((ext_vector_type(2)));
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const pair p = {(__bf16)x[2 * k], (__bf16)x[2 * k + 1]};
        w[k] = __builtin_bit_cast(uint32_t, p);
      }
      v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                        __float_as_uint(x[3]));
      v[BF16 ? 0 : 1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]),
                                   __float_as_uint(x[6]), __float_as_uint(x[7]));
    }
  }
};

}  // namespace
}  // namespace dg
