// dg_wgrad.hip -- a weight's gradient from two matrices of fp8 codes with 1x128 scales, for
// gfx950:  dW_g[n,k] = sum over the rows t of group g of (sP[t,n/128] P[t,n]) (sQ[t,k/128] Q[t,k]).
//
// The sum runs over rows, so each row's scales are inside it and no fp8 product can carry
// them: the codes become bf16 on their way into LDS (P with both scales, rounded once; Q's
// codes are bf16 numbers) and v_mfma_f32_32x32x16_bf16 multiplies them, accumulating in fp32.
// Both operands lie row by row in memory and in LDS (the order of the sum, 8 rows deep per
// lane, is down the columns): ds_read_b64_tr_b16 turns 4 rows x 16 columns at a time.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_ffn.h"
#include "dg_fp8.h"

namespace dg {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

constexpr int kDeep = 64;          // rows of a step
constexpr int kTile = 128;         // columns of P and of Q a tile
constexpr int kRowBytes = kTile * 2;
constexpr int kStageBytes = 2 * kDeep * kRowBytes;

// Two codes of a word as fp32.
template <int FMT, bool HI>
__device__ __forceinline__ v2f two(unsigned w) {
  return FMT == kFmtE5M2 ? __builtin_amdgcn_cvt_pk_f32_bf8((int)w, HI) : __builtin_amdgcn_cvt_pk_f32_fp8((int)w, HI);
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  const v2b v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(unsigned, v);
}

// Eight codes times a scale, as bf16 (exact for scale 1: a code has at most 4 bits).
template <int FMT>
__device__ __forceinline__ uint4 to_bf16(uint2 c, float s) {
  const v2f a = two<FMT, false>(c.x), b = two<FMT, true>(c.x), d = two<FMT, false>(c.y), e = two<FMT, true>(c.y);
  return make_uint4(pack_bf16(a[0] * s, a[1] * s), pack_bf16(b[0] * s, b[1] * s),
                    pack_bf16(d[0] * s, d[1] * s), pack_bf16(e[0] * s, e[1] * s));
}

// The 128-row blocks of a group in [b, end), in order: those whose first row names it.
struct Blocks {
  const int32_t* idx;              // nullptr: all of them
  int g, lane;
  int64_t T;
  int b, end;                      // the 64 blocks in `mask` are b .. b + 63
  uint64_t mask;
  __device__ __forceinline__ void look() {
    const int at = b + lane;
    const bool in = at < end;
    const int64_t row = (int64_t)at * kAlignM;
    mask = __builtin_amdgcn_ballot_w64(in && (!idx || idx[row] == g));
  }
  __device__ __forceinline__ int next() {       // -1: none left
    while (mask == 0) {
      b += 64;
      if (b >= end) return -1;
      look();
    }
    const int i = (int)__builtin_ctzll(mask);
    mask &= mask - 1;
    return b + i;
  }
};

template <int FP, int FQ>
__global__ void __launch_bounds__(256) wgrad_kernel(WgradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2][kStageBytes];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int tiles_n = a.N / kTile, tiles_k = a.K / kTile;
  int64_t id = blockIdx.x;
  const int tk = (int)(id % tiles_k);
  id /= tiles_k;
  const int tn = (int)(id % tiles_n);
  id /= tiles_n;
  const int g = (int)(id % a.G), split = (int)(id / a.G);
  const int n0 = tn * kTile, k0 = tk * kTile;
  const int nblocks = (int)((a.T + kAlignM - 1) / kAlignM);

  Blocks blocks;
  blocks.idx = a.group_idx;
  blocks.g = g;
  blocks.lane = lane;
  blocks.T = a.T;
  blocks.b = (int)((int64_t)nblocks * split / a.splits);
  blocks.end = (int)((int64_t)nblocks * (split + 1) / a.splits);
  blocks.look();

  // staging: 16 threads a row, 8 codes each, 16 rows a pass
  const int sr = t >> 4, sc = (t & 15) * 8;
  uint2 cp[4], cq[4];
  float s[4];
  auto load = [&](int64_t row0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = row0 + 16 * i + sr;
      const bool live = row < a.T && (!a.group_idx || a.group_idx[row] == g);
      cp[i] = cq[i] = make_uint2(0, 0);
      s[i] = 0.0f;
      if (live) {
        cp[i] = *(const uint2*)(a.P + row * a.N + n0 + sc);
        cq[i] = *(const uint2*)(a.Q + row * a.K + k0 + sc);
        s[i] = a.sP[row * tiles_n + tn] * a.sQ[row * tiles_k + tk];
      }
    }
  };
  // 64-byte pieces of a row are swapped by the row's last two bits: the four rows that a
  // transposing read takes lie in different banks
  auto stage = [&](uint8_t* st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * i + sr;
      const int at = r * kRowBytes + (((sc >> 5) ^ (r & 3)) << 6) + (sc & 31) * 2;
      *(uint4*)(st + at) = to_bf16<FP>(cp[i], s[i]);
      *(uint4*)(st + kDeep * kRowBytes + at) = to_bf16<FQ>(cq[i], 1.0f);
    }
  };
  // one operand fragment: columns 32 c .. + 31, rows r0 + 8 (lane / 32) .. + 7
  const int fr = (lane >> 5) * 8 + ((lane & 15) >> 2);
  const int fc = ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
  auto fragment = [&](const uint8_t* st, int c, int r0) {
    const int at = (r0 + fr) * kRowBytes + ((c ^ (fr & 3)) << 6) + fc;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(st + at));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(st + at + 4 * kRowBytes));
    const short v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    v8b r;
    __builtin_memcpy(&r, v, 16);
    return r;
  };

  const int wn = wave & 1, wk = wave >> 1;      // 64 columns of P and of Q a wave
  v16f acc[2][2];                                // [n][k]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  int block = blocks.next(), half = 0, cur = 0;
  if (block >= 0) {
    load((int64_t)block * kAlignM);
    stage(smem[0]);
  }
  while (block >= 0) {
    int next = block, next_half = half ^ 1;
    if (half) next = blocks.next();
    if (next >= 0) load((int64_t)next * kAlignM + next_half * kDeep);
    __syncthreads();                             // this step is staged, the last one read
    const uint8_t* P = smem[cur];
    const uint8_t* Q = P + kDeep * kRowBytes;
#pragma unroll
    for (int r = 0; r < kDeep; r += 16) {
      v8b fp[2], fq[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fp[i] = fragment(P, 2 * wn + i, r);
        fq[i] = fragment(Q, 2 * wk + i, r);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fq[j], fp[i], acc[i][j], 0, 0, 0);
    }
    cur ^= 1;
    if (next >= 0) stage(smem[cur]);
    block = next;
    half = next_half;
  }

  // lane l has column n = l % 32 and, four at a time, k = 8 e + 4 (l / 32) .. + 3
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t n = n0 + 64 * wn + 32 * i + (lane & 31);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = k0 + 64 * wk + 32 * j + 8 * e + 4 * (lane >> 5);
        v4f v = {acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
        const int64_t at = ((int64_t)g * a.N + n) * a.K + k;
        if (a.splits > 1) {
          *(v4f*)(a.partial + (int64_t)split * a.G * a.N * a.K + at) = v;
        } else if (a.bf16) {
          uint16_t* w = (uint16_t*)a.dW + at;
          if (a.accumulate) {
            const uint2 o = *(const uint2*)w;
            v += (v4f){__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xFFFF0000u),
                       __uint_as_float(o.y << 16), __uint_as_float(o.y & 0xFFFF0000u)};
          }
          *(uint2*)w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
          v4f* w = (v4f*)((float*)a.dW + at);
          *w = a.accumulate ? *w + v : v;
        }
      }
  }
}

// The parts of a gradient added up, in order.
__global__ void __launch_bounds__(256) wgrad_sum_kernel(WgradArgs a, int64_t n4) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  v4f v = ((const v4f*)a.partial)[i];
  for (int s = 1; s < a.splits; ++s) v += ((const v4f*)a.partial)[(int64_t)s * n4 + i];
  if (a.bf16) {
    uint2* w = (uint2*)a.dW + i;
    if (a.accumulate) {
      const uint2 o = *w;
      v += (v4f){__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xFFFF0000u), __uint_as_float(o.y << 16),
                 __uint_as_float(o.y & 0xFFFF0000u)};
    }
    *w = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
    v4f* w = (v4f*)a.dW + i;
    *w = a.accumulate ? *w + v : v;
  }
}

template <int FP, int FQ>
void launch(const WgradArgs& a, hipStream_t stream) {
  const int64_t grid = (int64_t)(a.N / kTile) * (a.K / kTile) * a.G * a.splits;
  hipLaunchKernelGGL((wgrad_kernel<FP, FQ>), dim3((unsigned)grid), dim3(256), 0, stream, a);
}

}  // namespace

// Parts of the sum over rows: one.
int wgrad_splits(int64_t, int64_t, int64_t, int64_t) { return 1; }

void launch_wgrad(const WgradArgs& a, hipStream_t stream) {
  if (a.p_fmt == kFmtE4M3)
    a.q_fmt == kFmtE4M3 ? launch<0, 0>(a, stream) : launch<0, 1>(a, stream);
  else
    a.q_fmt == kFmtE4M3 ? launch<1, 0>(a, stream) : launch<1, 1>(a, stream);
  if (a.splits > 1) {
    const int64_t n4 = (int64_t)a.G * a.N * a.K / 4;
    hipLaunchKernelGGL(wgrad_sum_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, stream, a, n4);
  }
}

}  // namespace dg
