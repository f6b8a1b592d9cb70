// dg_norm.hip -- root-mean-square norm with the residual's addition in front and fp8 codes
// with 1x128 scales behind, and its backward pass, for gfx950.
//
//   forward    h = x + r (rounded to x's type), rstd = 1 / sqrt(mean h^2 + eps),
//              y = h rstd w; codes and scales of y as the quantisation's, bf16 y on request
//   backward   g = w dy, dx = rstd (g - h rstd^2 mean(g h)) + grad_h, dw = sum_t dy h rstd
//
// Memory-bound: every value is loaded once, in 16-byte accesses, and stays in registers
// between the row's sum and its use.  NW waves share a row and each lane holds C pieces of
// 8 values, 64 NW 8 apart, so 16 lanes hold one 128-block.  Rows longer than 16384 values
// (backward) or 32768 (forward, fp32) do not fit the 128 registers that 16 waves leave a lane: the
// backward pass keeps 200 (C = 4) or 830 (C = 8) bytes a lane in scratch, the forward one 92.
//
// Forward, 4096 x 7168 bf16 with a residual and bf16 out too: 51 us for 265 MB, 5.2 TB/s (a copy of
// 256 MB: 5.4); one row 3.4 us, of which an empty launch takes 1.6; 512 x 65536 62 us, 3.8 TB/s (fp32
// 128, 3.4).  Backward, 8192 x 7168 bf16 with both incoming gradients: 92 us for 470 MB, 5.1 TB/s,
// and 4.8 for the weight's sums; 1024 x 32768 129 us, 2.1 TB/s, and 512 x 65536 275, 1.0, out of scratch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_block.h"
#include "dg_ffn.h"

namespace dg {
namespace {

// Eight weights from column c on: bf16, fp32 or ones; none past the row's end.
__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&w)[8]) {
  if (c >= a.K) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 0.0f;
  } else if (!a.w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
  } else if (a.w_bf16) {
    Eight<true> v;
    v.load(a.w, c);
    v.get(w);
  } else {
    Eight<false> v;
    v.load(a.w, c);
    v.get(w);
  }
}

// Workgroups of max(NW, 4) waves: four rows for NW = 1, else one.
template <bool BF16, int NW, int C>
__global__ void __launch_bounds__(NW < 4 ? 256 : NW * 64)
norm_kernel(NormArgs a) {
  constexpr int ROWS = NW < 4 ? 4 / NW : 1;
  static_assert(NW == 1 || NW >= 4, "one wave or whole workgroups a row");
  __shared__ float part[NW < 4 ? 1 : NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? wave : 0);
  if (row >= a.T) return;                      // a wave alone (NW = 1: no barrier below)
  const int t = NW == 1 ? lane : (int)threadIdx.x;
  constexpr bool KEEP = C <= 2;                // the weights on their way with the row (4096 x 7168 bf16
  float kept[KEEP ? C : 1][8];                 // 41.3 us against 42.4); longer rows have no registers
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < C; ++i) load_weight(a, (i * NW * 64 + t) * 8, kept[i % (KEEP ? C : 1)]);
  }
  Eight<BF16> v[C];
  float sum = 0.0f;
  {
    Eight<BF16> r[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = (i * NW * 64 + t) * 8;
      v[i].zero();
      r[i].zero();
      if (c < a.K) {
        v[i].load(a.x, row * a.ldx + c);
        if (a.r) r[i].load(a.r, row * a.ldr + c);
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float x[8];
      v[i].get(x);
      if (a.r) {
        float y[8];
        r[i].get(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += y[e];
        v[i].set(x);
        v[i].get(x);
        const int c = (i * NW * 64 + t) * 8;
        if (c < a.K) v[i].store(a.h, row * a.ldh + c);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(x[e], x[e], sum);
    }
  }
  sum = wave_sum(sum);
  if constexpr (NW > 1) {
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    sum = part[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) sum += part[i];
  }
  const float rstd = 1.0f / sqrtf(sum / (float)a.K + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
  const int nkb = a.K / kBlockK;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = (i * NW * 64 + t) * 8;
    if (c >= a.K) continue;                    // whole groups of 16 lanes: K is 128 n
    float x[8], w[8];
    v[i].get(x);
    if constexpr (KEEP) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = kept[i][e];
    } else {
      load_weight(a, c, w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * w[e];
    if (a.y) {
      Eight<true> y;
      y.set(x);
      y.store(a.y, row * a.ldy + c);
    }
    if (a.q) {
      const float scale = block_scale(block_amax(x), a.fmt);
      *(uint2*)(a.q + row * a.K + c) = codes8(x, scale, a.fmt);
      if ((lane & 15) == 0) a.s[row * nkb + c / kBlockK] = scale;
    }
  }
}

// Backward: a workgroup takes rows blockIdx, blockIdx + gridDim, ... and keeps its columns'
// weights (C <= 2) and sums of dy h rstd in registers (C <= 2; longer rows' partly in scratch).  The
// weights loaded again for each row, four pieces a
// lane and 1024 workgroups, whose rows of sums the second kernel reads, took 120 + 21 us of 8192 x
// 7168, where this takes 92 + 4.8.
template <bool BF16, int NW, int C>
__global__ void __launch_bounds__(NW * 64)
norm_backward_kernel(NormArgs a) {
  __shared__ float part[2][NW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = threadIdx.x;
  constexpr bool KEEP = C <= 2;                // longer rows have no registers for the weights
  float dw[C][8], kept[KEEP ? C : 1][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = (i * NW * 64 + t) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    if (KEEP) load_weight(a, c, kept[i % (KEEP ? C : 1)]);
  }
  auto weight = [&](int i, float (&w)[8]) {
    if constexpr (KEEP) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = kept[i][e];
    } else {
      load_weight(a, (i * NW * 64 + t) * 8, w);
    }
  };
  int flip = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, flip ^= 1) {
    const float rstd = a.rstd[row];
    Eight<BF16> vy[C], vh[C], vg[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = (i * NW * 64 + t) * 8;
      vy[i].zero();
      vh[i].zero();
      vg[i].zero();
      if (c < a.K) {
        vy[i].load(a.x, row * a.ldx + c);
        vh[i].load(a.r, row * a.ldr + c);
        if (KEEP && a.grad_h) vg[i].load(a.grad_h, row * a.ld_gh + c);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float y[8], h[8], w[8];
      vy[i].get(y);
      vh[i].get(h);
      weight(i, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = y[e] * h[e];
        dw[i][e] = __builtin_fmaf(p, rstd, dw[i][e]);
        sum = __builtin_fmaf(p, w[e], sum);
      }
    }
    sum = wave_sum(sum);
    if (lane == 0) part[flip][wave] = sum;
    __syncthreads();
    sum = part[flip][0];
#pragma unroll
    for (int i = 1; i < NW; ++i) sum += part[flip][i];
    const float m = sum / (float)a.K * rstd * rstd;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c = (i * NW * 64 + t) * 8;
      if (c >= a.K) continue;
      float y[8], h[8], g[8], w[8];
      if (!KEEP && a.grad_h) vg[i].load(a.grad_h, row * a.ld_gh + c);
      vy[i].get(y);
      vh[i].get(h);
      vg[i].get(g);
      weight(i, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(rstd, y[e] * w[e] - h[e] * m, g[e]);
      Eight<BF16> o;
      o.set(y);
      o.store(a.h, row * a.ldh + c);
    }
  }
  if (!a.grad_w) return;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int c = (i * NW * 64 + t) * 8;
    if (c >= a.K) continue;
    Eight<false> o;
    o.set(dw[i]);
    o.store(a.partial, (int64_t)blockIdx.x * a.K + c);
  }
}

// The workgroups' sums added up: 64 columns a workgroup, 16 waves over its rows, eight loads of
// each in flight.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* partial, float* grad_w, int K, int n) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;        // K is a multiple of 64
  float sum = 0.0f;
  for (int i = wave; i < n; i += 128) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + 16 * k < n ? partial[(int64_t)(i + 16 * k) * K + c] : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += v[k];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += part[i][lane];
    grad_w[c] = sum;
  }
}

// Backward of few rows, in one launch.  The weight's gradient needs no sum over a row, so that
// workgroups of their own can form it beside the rows': the first `strips` take a strip of columns
// each (eight lanes of 16 bytes, 128 rows at a time, KEEP of such loads of both matrices in flight),
// the others 16 / NW rows each, a piece of 8 values a lane.
template <bool BF16, int NW>
__global__ void __launch_bounds__(1024)
norm_backward_few_kernel(NormArgs a, int strips) {
  constexpr int CPL = BF16 ? 8 : 4, COLS = 8 * CPL, KEEP = 4;
  __shared__ float part[16 * COLS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x < strips) {
    const int c = blockIdx.x * COLS + (lane & 7) * CPL;
    float sum[CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) sum[e] = 0.0f;
    for (int64_t r0 = wave * 8 + (lane >> 3); r0 < a.T; r0 += 128 * KEEP) {
      uint4 y[KEEP], h[KEEP];
      float rstd[KEEP];
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        const int64_t row = r0 + 128 * k;
        y[k] = h[k] = make_uint4(0, 0, 0, 0);
        rstd[k] = 0.0f;
        if (row < a.T) {
          y[k] = *(const uint4*)((const uint8_t*)a.x + (row * a.ldx + c) * (BF16 ? 2 : 4));
          h[k] = *(const uint4*)((const uint8_t*)a.r + (row * a.ldr + c) * (BF16 ? 2 : 4));
          rstd[k] = a.rstd[row];
        }
      }
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        const uint32_t wy[4] = {y[k].x, y[k].y, y[k].z, y[k].w}, wh[4] = {h[k].x, h[k].y, h[k].z, h[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (BF16) {
            sum[(2 * e) % CPL] = __builtin_fmaf(__uint_as_float(wy[e] << 16) * __uint_as_float(wh[e] << 16), rstd[k],
                                                sum[(2 * e) % CPL]);
            sum[(2 * e + 1) % CPL] = __builtin_fmaf(
                __uint_as_float(wy[e] & 0xFFFF0000u) * __uint_as_float(wh[e] & 0xFFFF0000u), rstd[k],
                sum[(2 * e + 1) % CPL]);
          } else {
            sum[e] = __builtin_fmaf(__uint_as_float(wy[e]) * __uint_as_float(wh[e]), rstd[k], sum[e]);
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      sum[e] += __shfl_xor(sum[e], 8, 64);
      sum[e] += __shfl_xor(sum[e], 16, 64);
      sum[e] += __shfl_xor(sum[e], 32, 64);
      if (lane < 8) part[wave * COLS + lane * CPL + e] = sum[e];
    }
    __syncthreads();
    if (threadIdx.x < COLS) {
      float total = part[threadIdx.x];
#pragma unroll
      for (int w = 1; w < 16; ++w) total += part[w * COLS + threadIdx.x];
      a.grad_w[blockIdx.x * COLS + threadIdx.x] = total;
    }
    return;
  }
  const int sub = wave / NW;                   // of the workgroup's rows
  const int64_t row = (int64_t)(blockIdx.x - strips) * (16 / NW) + sub;
  const int c = ((int)threadIdx.x - sub * NW * 64) * 8;
  const bool on = row < a.T && c < a.K;
  Eight<BF16> vy, vh, vg;
  vy.zero();
  vh.zero();
  vg.zero();
  float rstd = 0.0f, w[8];
  if (on) {
    vy.load(a.x, row * a.ldx + c);
    vh.load(a.r, row * a.ldr + c);
    if (a.grad_h) vg.load(a.grad_h, row * a.ld_gh + c);
    rstd = a.rstd[row];
  }
  load_weight(a, c, w);
  float y[8], h[8], g[8], sum = 0.0f;
  vy.get(y);
  vh.get(h);
  vg.get(g);
#pragma unroll
  for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(y[e] * h[e], w[e], sum);
  sum = wave_sum(sum);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  sum = part[sub * NW];
#pragma unroll
  for (int i = 1; i < NW; ++i) sum += part[sub * NW + i];
  if (!on) return;
  const float m = sum / (float)a.K * rstd * rstd;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(rstd, y[e] * w[e] - h[e] * m, g[e]);
  Eight<BF16> o;
  o.set(y);
  o.store(a.h, row * a.ldh + c);
}

template <bool BF16, int NW, int C>
void launch_forward(const NormArgs& a, hipStream_t stream) {
  constexpr int rows = NW < 4 ? 4 / NW : 1;
  hipLaunchKernelGGL((norm_kernel<BF16, NW, C>), dim3((unsigned)((a.T + rows - 1) / rows)),
                     dim3(NW < 4 ? 256 : NW * 64), 0, stream, a);
}

template <bool BF16>
void forward_for(const NormArgs& a, hipStream_t stream) {
  // Eight waves a row from 2048 values on: 4096 x 7168 bf16 42.4 us against 47.4 by four, fp32 72.9
  // against 78.5, 4096 x 4096 24.7 against 26.7.  Of few rows 16 where each then has a piece: one row
  // of 7168 3.3 us against 3.5, 256 rows 4.7 against 5.0, 512 7.8 against 7.9, 768 10.0 against 9.6; of
  // 4096 values 768 rows 7.6 against 6.6.
  const int pieces = (a.K + 511) / 512;        // of 512 values, a wave's worth
  if (pieces <= 1) return launch_forward<BF16, 1, 1>(a, stream);
  if (pieces <= 4) return launch_forward<BF16, 4, 1>(a, stream);
  if (pieces <= 8) return launch_forward<BF16, 8, 1>(a, stream);
  if (a.T <= 512 && pieces <= 16) return launch_forward<BF16, 16, 1>(a, stream);
  if (pieces <= 16) return launch_forward<BF16, 8, 2>(a, stream);
  if (pieces <= 32) return launch_forward<BF16, 16, 2>(a, stream);
  if (pieces <= 64) return launch_forward<BF16, 16, 4>(a, stream);
  return launch_forward<BF16, 16, 8>(a, stream);
}

template <bool BF16, int NW, int C>
void launch_back(const NormArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL((norm_backward_kernel<BF16, NW, C>), dim3(grid), dim3(NW * 64), 0, stream, a);
}

template <bool BF16>
void backward_for(const NormArgs& a, int grid, hipStream_t stream) {
  // A piece a lane up to 8192 values: 8192 x 7168 fp32 175 us against 182 with two (bf16 97.8 against
  // 97.7), 2048 x 4096 fp32 30.4 against 32.3.
  const int pieces = (a.K + 511) / 512;
  if (pieces <= 4) return launch_back<BF16, 4, 1>(a, grid, stream);
  if (pieces <= 8) return launch_back<BF16, 8, 1>(a, grid, stream);
  if (pieces <= 16) return launch_back<BF16, 16, 1>(a, grid, stream);
  if (pieces <= 32) return launch_back<BF16, 16, 2>(a, grid, stream);
  if (pieces <= 64) return launch_back<BF16, 16, 4>(a, grid, stream);
  return launch_back<BF16, 16, 8>(a, grid, stream);
}

template <bool BF16, int NW>
void launch_few(const NormArgs& a, hipStream_t stream) {
  int strips = a.grad_w ? a.K / (BF16 ? 64 : 32) : 0;
  const unsigned rows = (unsigned)((a.T + 16 / NW - 1) / (16 / NW));
  if (strips && (a.h == a.x || a.h == a.r)) {  // in grad_y's or h's place: the strips have to read it first
    hipLaunchKernelGGL((norm_backward_few_kernel<BF16, NW>), dim3(strips), dim3(1024), 0, stream, a, strips);
    strips = 0;
  }
  hipLaunchKernelGGL((norm_backward_few_kernel<BF16, NW>), dim3(strips + rows), dim3(1024), 0, stream, a, strips);
}
template <bool BF16>
void few_for(const NormArgs& a, hipStream_t stream) {
  if (a.K <= 2048) return launch_few<BF16, 4>(a, stream);
  if (a.K <= 4096) return launch_few<BF16, 8>(a, stream);
  return launch_few<BF16, 16>(a, stream);
}

}  // namespace

// Two workgroups a CU; of few rows one a CU, and a row each at least: the second kernel reads a row
// of sums for each (517 x 2048 by these two kernels: 5.7 + 3.3 us, with a workgroup a row 6.4 + 11.4).
int norm_backward_grid(int64_t T) {
  const int64_t most = T / 4 > 256 ? T / 4 : 256;
  return (int)(T < most ? T : most < kNormMaxGrid ? most : kNormMaxGrid);
}

// In slices of rows: a launch has less than 2^32 threads.
void launch_norm(const NormArgs& args, hipStream_t stream) {
  NormArgs a = args;
  const int64_t e = a.bf16 ? 2 : 4;
  for (int64_t left = args.T; left > 0; left -= a.T) {
    a.T = left < kNormRows ? left : kNormRows;
    a.bf16 ? forward_for<true>(a, stream) : forward_for<false>(a, stream);
    a.x = (const uint8_t*)a.x + a.T * a.ldx * e;
    if (a.r) {
      a.r = (const uint8_t*)a.r + a.T * a.ldr * e;
      a.h = (uint8_t*)a.h + a.T * a.ldh * e;
    }
    if (a.q) {
      a.q += a.T * a.K;
      a.s += a.T * (a.K / kBlockK);
    }
    if (a.y) a.y += a.T * a.ldy;
    if (a.rstd) a.rstd += a.T;
  }
}

void launch_norm_backward(const NormArgs& a, hipStream_t stream) {
  // One launch up to 1024 rows: 517 x 2048 fp32 6.6 us against 9.6, 256 x 7168 bf16 6.7 against 11.6,
  // 1024 x 7168 bf16 15.9 against 16.6, fp32 29.9 against 29.6; 2048 rows 31.6 against 31.7 and 61.7
  // against 52.6, as the strips read both matrices again.
  if (a.T > 0 && a.T <= kNormFewRows && a.K <= 8192)
    return a.bf16 ? few_for<true>(a, stream) : few_for<false>(a, stream);
  const int grid = norm_backward_grid(a.T);
  if (grid > 0) a.bf16 ? backward_for<true>(a, grid, stream) : backward_for<false>(a, grid, stream);
  if (a.grad_w)
    hipLaunchKernelGGL(norm_weight_kernel, dim3(a.K / 64), dim3(1024), 0, stream, a.partial, a.grad_w, a.K,
                       grid);
}

}  // namespace dg
