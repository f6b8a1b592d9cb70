// dg_lora.hip -- low-rank adapters of many requests beside a shared projection, gfx950:
//
//   out[t] = base[t] + scale_i (x[t] A_i^T) B_i^T      with i = ids[t]
//
// Two kernels.  The first ("down") forms h[t] = scale_i x[t] A_i^T in fp32, the second
// ("up") adds h[t] B_i^T to the base row and rounds once to bf16.  Both work on tiles of 16
// consecutive rows with v_mfma_f32_16x16x32_bf16 and, for each adapter that the tile's rows
// name, compute all 16 rows and keep those that are the adapter's: the products are few,
// the bytes of x, A, B and the outputs are what costs, and no row ever meets another
// adapter's values (a row's result depends on its own adapter alone, whatever the others
// hold).
//
// h is kept in fp32 between the two (the workspace); the second product takes it as the sum
// of two bf16 numbers, the value rounded and the rest rounded, so that 16 bits of it take
// part and the only rounding that shows is the output's.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_ops.h"

namespace dg {
namespace {

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using f32x4 = __attribute__((ext_vector_type(4))) float;

constexpr int kTile = 16;                 // rows of a tile
constexpr int kDownWaves = 8;
constexpr int kFrags = kLoraDownFrags;    // 32-deep pieces of K that a wave holds
constexpr int kUpWaves = 4;
constexpr int kUpCols = 64;               // output columns of a wave

__device__ __forceinline__ f32x4 mfma(const uint4& a, const uint4& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t round_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
__device__ __forceinline__ float from_bf16(uint32_t b) { return __uint_as_float(b << 16); }

// The adapters of a tile: lane l holds the id of row l % 16 (-1: none).  next() gives the
// adapters one by one, in the order of their first rows, with the rows that are theirs.
struct TileAdapters {
  int id;                  // of row lane % 16
  uint32_t left;           // rows whose adapter has not been given out
  __device__ __forceinline__ TileAdapters(const LoraArgs& a, int64_t t0, int lane) {
    const int64_t t = t0 + (lane & 15);
    int i = t < a.T ? a.ids[t] : -1;
    id = i >= 0 && i < a.L ? i : -1;
    left = (uint32_t)__builtin_amdgcn_ballot_w64(id >= 0) & 0xFFFFu;
  }
  __device__ __forceinline__ bool next(int* adapter, uint32_t* rows) {
    if (!left) return false;
    *adapter = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    *rows = (uint32_t)__builtin_amdgcn_ballot_w64(id == *adapter) & 0xFFFFu;
    left &= ~*rows;
    return true;
  }
};

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter) {
  if (!a.ranks) return a.R;
  const int r = a.ranks[adapter];
  return r < 0 ? 0 : r < a.R ? r : a.R;
}

// h of a tile's rows over one share of K: workgroup (tile, share s, q) takes every
// down_q-th adapter of the tile, its waves an eighth each of the share, and the waves'
// sums are added up in wave order.  A row of h without an adapter is not written.
__global__ void __launch_bounds__(64 * kDownWaves)
lora_down_kernel(LoraArgs a) {
  extern __shared__ float red[];          // [wave][rank tile][row][rank]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x, s = blockIdx.y, q = blockIdx.z;
  const int64_t t0 = (int64_t)tile * kTile;
  const int rt_all = (a.R + 15) / 16;
  TileAdapters ad(a, t0, lane);

  // this wave's pieces of K
  const int pieces = a.K / 32, shares = a.S * kDownWaves, share = s * kDownWaves + wave;
  const int f0 = (int)((int64_t)pieces * share / shares);
  const int nf = (int)((int64_t)pieces * (share + 1) / shares) - f0;
  const int64_t row = t0 + l16 < a.T ? t0 + l16 : a.T - 1;
  uint4 xf[kFrags];
  const uint16_t* xp = a.x + row * a.ldx + (int64_t)f0 * 32 + g * 8;
  bool loaded = false;

  int adapter;
  uint32_t rows;
  for (int n = 0; ad.next(&adapter, &rows); ++n) {
    if (n % a.Q != q) continue;
    if (!loaded) {
      loaded = true;
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        if (f < nf) xf[f] = *(const uint4*)(xp + f * 32);
    }
    const int r = rank_of(a, adapter), rts = (r + 15) / 16;
    const float scale = a.scales ? a.scales[adapter] : 1.0f;
    for (int rt = 0; rt < rts; ++rt) {
      const int rr = rt * 16 + l16 < a.R ? rt * 16 + l16 : a.R - 1;
      const uint16_t* ap = a.A + ((int64_t)adapter * a.R + rr) * a.K + (int64_t)f0 * 32 + g * 8;
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        if (f < nf) acc = mfma(xf[f], *(const uint4*)(ap + f * 32), acc);
      // row 4g + j, rank l16
#pragma unroll
      for (int j = 0; j < 4; ++j)
        red[((wave * rt_all + rt) * kTile + 4 * g + j) * 16 + l16] = acc[j];
    }
    __syncthreads();
    for (int i = tid; i < rt_all * 256; i += 64 * kDownWaves) {
      const int rt = i >> 8, m = (i >> 4) & 15, c = rt * 16 + (i & 15);
      if (c >= a.R || !((rows >> m) & 1)) continue;
      float sum = 0.0f;
      if (c < r)
        for (int w = 0; w < kDownWaves; ++w)
          sum += red[((w * rt_all + rt) * kTile + m) * 16 + (i & 15)];
      a.h[((int64_t)s * a.T + t0 + m) * a.R + c] = sum * scale;
    }
    __syncthreads();
  }
}

// out = base + h B^T for a tile's rows and kUpWaves * kUpCols columns.  Weights are the
// MFMA's row operand and rows of the tile its columns, so a lane's four results are
// consecutive output columns; two products over interleaved weights give it eight, one
// 16-byte load of base and one store.
template <bool VEC>
__global__ void __launch_bounds__(64 * kUpWaves)
lora_up_kernel(LoraArgs a) {
  extern __shared__ uint16_t hs[];        // [row][2 R rounded up to 32]: rounded, then rest
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * kTile;
  const int64_t n0 = ((int64_t)blockIdx.y * kUpWaves + wave) * kUpCols;
  TileAdapters ad(a, t0, lane);
  const int chunks = a.R / 8;             // 8-rank pieces of an adapter
  const int steps = (2 * chunks + 3) / 4; // MFMA steps over [rounded | rest]
  const int hw = steps * 32 + 8;          // LDS row, 16 bytes past a multiple of 64
  const uint32_t mine = ad.left;
  for (int i = tid; i < kTile * a.R; i += 64 * kUpWaves) {
    const int m = i / a.R, c = i - m * a.R;
    float sum = 0.0f;
    if ((mine >> m) & 1)
      for (int s = 0; s < a.S; ++s) sum += a.h[((int64_t)s * a.T + t0 + m) * a.R + c];
    const uint32_t hi = round_bf16(sum);
    const float rest = sum - from_bf16(hi);
    hs[m * hw + c] = (uint16_t)hi;
    hs[m * hw + a.R + c] = (uint16_t)(fabsf(rest) < INFINITY ? round_bf16(rest) : 0u);
  }
  for (int i = tid; i < kTile * (steps * 32 - 2 * a.R); i += 64 * kUpWaves) {
    const int w = steps * 32 - 2 * a.R;
    hs[(i / w) * hw + 2 * a.R + i % w] = 0;
  }
  __syncthreads();

  const int64_t t = t0 + l16;
  f32x4 out[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) out[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int adapter;
  uint32_t rows;
  while (ad.next(&adapter, &rows)) {
    const int r = rank_of(a, adapter);
    f32x4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int st = 0; st < steps; ++st) {
      const int piece = 4 * st + g;
      const uint4 hf = *(const uint4*)(hs + l16 * hw + piece * 8);
      const int rank0 = (piece < chunks ? piece : piece < 2 * chunks ? piece - chunks : chunks) * 8;
      const int have = r - rank0;         // ranks of this piece that the adapter has
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // weight row of MFMA row m of product c: its four results per lane group lie at
        // column 32 (c / 2) + 8 g + 4 (c % 2) + j
        const int64_t n = n0 + 32 * (c / 2) + 8 * (l16 / 4) + 4 * (c & 1) + (l16 & 3);
        const int64_t nn = n < a.N ? n : a.N - 1;
        uint4 b = make_uint4(0, 0, 0, 0);
        if (have > 0) b = *(const uint4*)(a.B + ((int64_t)adapter * a.N + nn) * a.R + rank0);
        if (have > 0 && have < 8) {
          uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = 2 * i >= have ? 0u : 2 * i + 1 >= have ? w[i] & 0xFFFFu : w[i];
          b = make_uint4(w[0], w[1], w[2], w[3]);
        }
        acc[c] = mfma(b, hf, acc[c]);
      }
    }
    if ((rows >> l16) & 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) out[c] = acc[c];
    }
  }
  if (t >= a.T) return;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int64_t n = n0 + 32 * p + 8 * g;
    if (n >= a.N) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = out[2 * p + i / 4][i & 3];
    if (VEC && n + 8 <= a.N) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (a.base) {
        const uint4 u = *(const uint4*)(a.base + t * a.ld_base + n);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = v[2 * i] + from_bf16(w[i] & 0xFFFFu);
        const float hi = v[2 * i + 1] + __uint_as_float(w[i] & 0xFFFF0000u);
        w[i] = round_bf16(lo) | (round_bf16(hi) << 16);
      }
      *(uint4*)(a.out + t * a.ld_out + n) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < a.N) {
          const float b = a.base ? from_bf16(a.base[t * a.ld_base + n + i]) : 0.0f;
          a.out[t * a.ld_out + n + i] = (uint16_t)round_bf16(v[i] + b);
        }
    }
  }
}

}  // namespace

void lora_split(int64_t T, int64_t K, int64_t R, int* S, int* Q) {
  (void)R;
  const int64_t tiles = (T + kTile - 1) / kTile, deep = (int64_t)kDownWaves * kFrags * 32;
  int64_t s = (K + deep - 1) / deep;                       // what the registers need
  int64_t q = 1;
  while (q < kTile && tiles * s * q < 512 && q < T) q *= 2;
  while (tiles * s * q < 512 && K / s > 1024) ++s;
  *S = (int)s;
  *Q = (int)q;
}

void launch_lora(const LoraArgs& a, hipStream_t stream) {
  const unsigned tiles = (unsigned)((a.T + kTile - 1) / kTile);
  const int rt = (a.R + 15) / 16, steps = (2 * (a.R / 8) + 3) / 4;
  hipLaunchKernelGGL(lora_down_kernel, dim3(tiles, a.S, a.Q), dim3(64 * kDownWaves),
                     (size_t)kDownWaves * rt * 256 * 4, stream, a);
  const unsigned cols = (unsigned)((a.N + kUpWaves * kUpCols - 1) / (kUpWaves * kUpCols));
  const size_t lds = (size_t)kTile * (steps * 32 + 8) * 2;
  const bool vec = (((uintptr_t)a.out | (uintptr_t)a.base) & 15) == 0 && a.ld_out % 8 == 0 &&
                   (!a.base || a.ld_base % 8 == 0);
  if (vec)
    hipLaunchKernelGGL((lora_up_kernel<true>), dim3(tiles, cols), dim3(64 * kUpWaves), lds, stream, a);
  else
    hipLaunchKernelGGL((lora_up_kernel<false>), dim3(tiles, cols), dim3(64 * kUpWaves), lds, stream, a);
}

}  // namespace dg
