// dg_route.hip -- the gate of a mixture of experts for gfx950: scores, the k experts of
// each row, their weights, rows per expert and the balance loss in one pass over the
// logits, and the gradient of weights and loss by the logits in another.
//
// A row of E logits is held by L lanes of a wave, V of them in each lane's registers
// (L * V >= E), 64 / L rows a wave; element 4 (c L + l) + i of the row is register 4c + i
// of lane l, so that a chunk c is one 16-byte (fp32) or 8-byte (bf16) load a lane and
// consecutive lanes read consecutive addresses.
//
// Choice of experts.  The key fp32(z + bias) is widened to a double, whose low 29 mantissa
// bits are then zero, and the expert's index goes into the lowest ten of them, so that of
// two equal keys the lower index is the larger double.  All keys of a row differ, and one
// maximum finds both the largest key and, among equals, the lowest expert.
//
// Scores are recomputed in the backward pass rather than kept: reading T x E logits again
// costs what reading T x E scores would.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_ops.h"

namespace dg {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWaves = kRouteThreads / 64;

// exp(x) for x <= 0 within about an ulp: 2^(x log2 e) with the rounding of the product
// put back to first order.  Below -104 (where fp32 has nothing left) the result is 0; NaN
// stays NaN.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.69314718f;
  const float y = x < -104.0f ? -104.0f : x;
  const float t = y * kLog2e;
  const float r = __builtin_fmaf(y, kLog2eLow, __builtin_fmaf(y, kLog2e, -t));
  const float p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p * kLn2, r, p);
}

// sigmoid(z) and 1 - sigmoid(z), each without cancellation; exact 0 and 1 at -inf and inf.
__device__ __forceinline__ void sigmoid(float z, float* s, float* c) {
  const float e = exp_neg(-fabsf(z));
  const float r = 1.0f / (1.0f + e);
  const float er = e * r;
  *s = z >= 0.0f ? r : er;
  *c = z >= 0.0f ? er : r;
  if (z != z) *s = *c = z;
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, L));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off, L);
  return v;
}
template <int L>
__device__ __forceinline__ double group_max(double v) {
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) v = fmax(v, __shfl_xor(v, off, L));
  return v;
}

constexpr double kNoKey = -1.0e300;       // below every widened fp32 key

// The key of expert e as described above; -inf and NaN keys cannot be chosen.
__device__ __forceinline__ double pack_key(float key, int e) {
  if (!(key > -INFINITY)) return kNoKey;
  const double d = key == INFINITY ? 1.0e300 : (double)(key + 0.0f);   // -0 counts as 0
  const uint64_t u = (uint64_t)__double_as_longlong(d) & ~(uint64_t)1023;
  return __longlong_as_double((long long)(u | (uint64_t)(d < 0.0 ? e : 1023 - e)));
}
__device__ __forceinline__ int key_expert(double d) {
  const int low = (int)(__double_as_longlong(d) & 1023);
  return d <= kNoKey ? -1 : (d < 0.0 ? low : 1023 - low);
}

__device__ __forceinline__ float load_one(const void* p, int64_t i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}
__device__ __forceinline__ uint16_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0;
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

// A row's V logits of this lane; `fill` past the last expert.
template <int L, int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t row, int l, float fill,
                                         float (&z)[V]) {
  const int64_t at = row * a.ld;
#pragma unroll
  for (int c = 0; c < V / 4; ++c) {
    const int e = 4 * (c * L + l);
    if (a.vec) {
      if (e < a.E) {
        if (a.bf16) {
          const uint2 u = *(const uint2*)((const uint16_t*)a.logits + at + e);
          z[4 * c] = __uint_as_float(u.x << 16);
          z[4 * c + 1] = __uint_as_float(u.x & 0xFFFF0000u);
          z[4 * c + 2] = __uint_as_float(u.y << 16);
          z[4 * c + 3] = __uint_as_float(u.y & 0xFFFF0000u);
        } else {
          const float4 f = *(const float4*)((const float*)a.logits + at + e);
          z[4 * c] = f.x; z[4 * c + 1] = f.y; z[4 * c + 2] = f.z; z[4 * c + 3] = f.w;
        }
      } else {
        z[4 * c] = z[4 * c + 1] = z[4 * c + 2] = z[4 * c + 3] = fill;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[4 * c + i] = e + i < a.E ? load_one(a.logits, at + e + i, a.bf16) : fill;
    }
  }
}

// A row's softmax: its maximum and 1 / sum of exp(z - max), by which a score is
// exp(z - max) * inv.  A row of -inf only (nothing left of it) has max = 0 and inv = 0.
struct RowNorm {
  float max, inv;
};

template <int L, int V>
__device__ __forceinline__ RowNorm softmax_row(const float (&z)[V], float (&s)[V]) {
  float m = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, z[v]);
  m = group_max<L>(m);
  const bool none = m == -INFINITY;
  m = none ? 0.0f : m;
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = exp_neg(z[v] - m);
    sum += s[v];
  }
  sum = group_sum<L>(sum);
  return {m, none ? 0.0f : 1.0f / sum};
}

// ------------------------------------------------------------------------------ forward
// Grid-stride over row blocks.  With `counts` every workgroup leaves its sums over its
// rows (chosen rows and, with `loss`, probabilities of each expert, live rows) in the
// workspace, and the last workgroup to arrive adds them up in workgroup order: the result
// does not depend on which one that is.
template <int L, int V>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(RouteArgs a) {
  constexpr int RW = 64 / L, EP = L * V;
  __shared__ int hist[EP];
  __shared__ float psum[kRouteWaves][EP];
  __shared__ int live_rows;
  __shared__ int is_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % L, sub = lane / L;
  const bool sums = a.counts != nullptr;
  for (int e = tid; e < EP; e += kRouteThreads) hist[e] = 0;
  if (tid == 0) live_rows = 0;
  __syncthreads();

  float bias[V], acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 4 * ((v / 4) * L + l) + (v & 3);
    bias[v] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    acc[v] = 0.0f;
  }
  int nlive = 0;
  const int64_t step = (int64_t)gridDim.x * kRouteWaves * RW;
  for (int64_t row0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * RW; row0 < a.T; row0 += step) {
    const int64_t row = row0 + sub;
    const bool in = row < a.T;
    const bool live = in && (!a.row_valid || a.row_valid[row] != 0);
    float z[V], s[V];
    if (live) {
      load_row<L, V>(a, row, l, -INFINITY, z);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = -INFINITY;
    }
    RowNorm n{0.0f, 0.0f};
    if (a.sigmoid) {
      if (a.loss) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float c;
          sigmoid(z[v], &s[v], &c);
          sum += s[v];
        }
        sum = group_sum<L>(sum);
        n.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      }
    } else {
      n = softmax_row<L, V>(z, s);
    }
    if (a.loss) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = __builtin_fmaf(s[v], n.inv, acc[v]);
    }
    double key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = pack_key(z[v] + bias[v], 4 * ((v / 4) * L + l) + (v & 3));
    if (live && l == 0) ++nlive;

    // k rounds: the largest key left; lane j % L keeps the choices j, j + L, ...
    constexpr int KP = L >= kRouteMaxK ? 1 : kRouteMaxK / L;
    int ids[KP];
#pragma unroll
    for (int q = 0; q < KP; ++q) ids[q] = -1;
    for (int j = 0; j < a.k; ++j) {
      double m = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = fmax(m, key[v]);
      m = group_max<L>(m);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = key[v] == m ? kNoKey : key[v];
      const int e = key_expert(m);
#pragma unroll
      for (int q = 0; q < KP; ++q)
        if (j == q * L + l) ids[q] = e;
    }
    // scores of the chosen experts, recomputed by the lane that keeps each
    float w[KP], total = 0.0f;
#pragma unroll
    for (int q = 0; q < KP; ++q) {
      w[q] = 0.0f;
      if (ids[q] >= 0) {
        const float zc = load_one(a.logits, row * a.ld + ids[q], a.bf16);
        float c;
        if (a.sigmoid) sigmoid(zc, &w[q], &c);
        else w[q] = exp_neg(zc - n.max) * n.inv;
        if (sums) atomicAdd(&hist[ids[q]], 1);
      }
      total += w[q];
    }
    float f = a.scale;
    if (a.normalize) {
      total = group_sum<L>(total);
      f = total == 0.0f ? 0.0f : a.scale / total;
    }
#pragma unroll
    for (int q = 0; q < KP; ++q) {
      const int j = q * L + l;
      if (in && j < a.k) {
        a.ids[row * a.k + j] = ids[q];
        a.weights[row * a.k + j] = ids[q] >= 0 ? w[q] * f : 0.0f;
      }
    }
  }
  if (!sums) return;

  // this workgroup's sums
  atomicAdd(&live_rows, nlive);
  if (a.loss) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float p = acc[v];
#pragma unroll
      for (int off = 32; off >= L; off >>= 1) p += __shfl_xor(p, off, 64);
      if (sub == 0) psum[wave][4 * ((v / 4) * L + l) + (v & 3)] = p;
    }
  }
  __syncthreads();
  const int G = (int)gridDim.x, b = blockIdx.x;
  float* part_p = (float*)((uint8_t*)a.workspace + kRouteWsHeader);
  int* part_n = (int*)(part_p + (int64_t)G * a.E);
  int* part_live = part_n + (int64_t)G * a.E;
  for (int e = tid; e < a.E; e += kRouteThreads) {
    if (a.loss) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < kRouteWaves; ++w) p += psum[w][e];
      __hip_atomic_store(part_p + (int64_t)b * a.E + e, p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __hip_atomic_store(part_n + (int64_t)b * a.E + e, hist[e], __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
  }
  if (tid == 0)
    __hip_atomic_store(part_live + b, live_rows, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __threadfence();                      // this thread's stores before its workgroup's arrival
  __syncthreads();
  if (tid == 0)
    is_last = __hip_atomic_fetch_add((int*)a.workspace, 1, __ATOMIC_ACQ_REL,
                                     __HIP_MEMORY_SCOPE_AGENT) == G - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  if (tid == 0) {
    __hip_atomic_store((int*)a.workspace, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    live_rows = 0;
  }
  __syncthreads();
  for (int g = tid; g < G; g += kRouteThreads)
    atomicAdd(&live_rows, __hip_atomic_load(part_live + g, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  __syncthreads();
  const float rows = (float)live_rows;
  float part = 0.0f;
  for (int e = tid; e < a.E; e += kRouteThreads) {
    int n = 0;
    float p = 0.0f;
    for (int g = 0; g < G; ++g) {
      n += __hip_atomic_load(part_n + (int64_t)g * a.E + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (a.loss)
        p += __hip_atomic_load(part_p + (int64_t)g * a.E + e, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    a.counts[e] = n;
    if (a.loss) {
      const float c = live_rows ? a.balance * (float)a.E / (float)a.k * (float)n / rows / rows : 0.0f;
      a.coef[e] = c;
      part += live_rows ? c * p : 0.0f;
    }
  }
  if (a.loss) {
    part = group_sum<64>(part);
    if (lane == 0) psum[wave][0] = part;
    __syncthreads();
    if (tid == 0) {
      float sum = 0.0f;
      for (int w = 0; w < kRouteWaves; ++w) sum += psum[w][0];
      *a.loss = sum;
    }
  }
}

// ----------------------------------------------------------------------------- backward
// dz from the weights' gradients (scattered to the chosen experts through a row of LDS)
// and the loss's (coef, the same for every row).
template <int L, int V>
__global__ void __launch_bounds__(kRouteThreads)
route_backward_kernel(RouteArgs a) {
  constexpr int RW = 64 / L, EP = L * V;
  constexpr int KP = L >= kRouteMaxK ? 1 : kRouteMaxK / L;
  __shared__ float rows_d[kRouteWaves * RW][EP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % L, sub = lane / L;
  float* d = rows_d[wave * RW + sub];
#pragma unroll
  for (int v = 0; v < V; ++v) d[4 * ((v / 4) * L + l) + (v & 3)] = 0.0f;

  float u[V];
  const float g_loss = a.coef ? (a.grad_loss ? *a.grad_loss : 1.0f) : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 4 * ((v / 4) * L + l) + (v & 3);
    u[v] = a.coef && e < a.E ? g_loss * a.coef[e] : 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * kRouteWaves * RW;
  for (int64_t row0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * RW; row0 < a.T; row0 += step) {
    const int64_t row = row0 + sub;
    const bool in = row < a.T;
    const bool live = in && (!a.row_valid || a.row_valid[row] != 0);
    float z[V], s[V], c[V];
    if (live) {
      load_row<L, V>(a, row, l, -INFINITY, z);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = -INFINITY;
    }
    RowNorm n{0.0f, 0.0f};
    float us = 0.0f;                              // sum of u p over the row
    if (a.sigmoid) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sigmoid(z[v], &s[v], &c[v]);
        sum += s[v];
        us = __builtin_fmaf(u[v], s[v], us);
      }
      sum = group_sum<L>(sum);
      n.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      us = group_sum<L>(us) * n.inv;
    } else {
      n = softmax_row<L, V>(z, s);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] *= n.inv;
        us = __builtin_fmaf(u[v], s[v], us);
      }
      us = group_sum<L>(us);
    }
    // the chosen experts' score gradients
    int id[KP];
    float gw[KP], sc[KP], total = 0.0f, dot = 0.0f;
#pragma unroll
    for (int q = 0; q < KP; ++q) {
      const int j = q * L + l;
      id[q] = -1;
      gw[q] = sc[q] = 0.0f;
      if (live && a.grad_weights && j < a.k) {
        const int e = a.ids_in[row * a.k + j];
        if (e >= 0 && e < a.E) {
          id[q] = e;
          gw[q] = a.scale * a.grad_weights[row * a.k + j];
          const float zc = load_one(a.logits, row * a.ld + e, a.bf16);
          float cc;
          if (a.sigmoid) sigmoid(zc, &sc[q], &cc);
          else sc[q] = exp_neg(zc - n.max) * n.inv;
        }
      }
      total += sc[q];
      dot = __builtin_fmaf(gw[q], sc[q], dot);
    }
    if (a.normalize) {
      total = group_sum<L>(total);
      dot = group_sum<L>(dot);
      const float it = total == 0.0f ? 0.0f : 1.0f / total;
      const float mean = dot * it;
#pragma unroll
      for (int q = 0; q < KP; ++q) gw[q] = (gw[q] - mean) * it;
    }
    float ds = 0.0f;                              // sum of D s over the chosen
#pragma unroll
    for (int q = 0; q < KP; ++q)
      if (id[q] >= 0) {
        d[id[q]] = gw[q];
        ds = __builtin_fmaf(gw[q], sc[q], ds);
      }
    ds = group_sum<L>(ds);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    float dz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float dv = d[4 * ((v / 4) * L + l) + (v & 3)];
      dz[v] = a.sigmoid ? ((u[v] - us) * n.inv + dv) * s[v] * c[v] : s[v] * (u[v] + dv - (us + ds));
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int q = 0; q < KP; ++q)
      if (id[q] >= 0) d[id[q]] = 0.0f;
    if (!in) continue;
    const int64_t at = row * a.ld_grad;
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const int e = 4 * (q * L + l);
      if (!live)
        for (int i = 0; i < 4; ++i) dz[4 * q + i] = 0.0f;
      if (a.vec_grad) {
        if (e < a.E) {
          if (a.bf16)
            *(uint2*)((uint16_t*)a.grad_logits + at + e) =
                make_uint2(to_bf16(dz[4 * q]) | ((uint32_t)to_bf16(dz[4 * q + 1]) << 16),
                           to_bf16(dz[4 * q + 2]) | ((uint32_t)to_bf16(dz[4 * q + 3]) << 16));
          else
            *(float4*)((float*)a.grad_logits + at + e) =
                make_float4(dz[4 * q], dz[4 * q + 1], dz[4 * q + 2], dz[4 * q + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < a.E) {
            if (a.bf16) ((uint16_t*)a.grad_logits)[at + e + i] = to_bf16(dz[4 * q + i]);
            else ((float*)a.grad_logits)[at + e + i] = dz[4 * q + i];
          }
      }
    }
  }
}

template <int L, int V>
void launch(const RouteArgs& a, bool backward, int grid, hipStream_t stream) {
  if (backward)
    hipLaunchKernelGGL((route_backward_kernel<L, V>), dim3(grid), dim3(kRouteThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((route_kernel<L, V>), dim3(grid), dim3(kRouteThreads), 0, stream, a);
}

// Lanes a row: as few as hold it at 16 experts each.
int lanes_of(int64_t E) {
  return E <= 64 ? 4 : E <= 128 ? 8 : E <= 256 ? 16 : E <= 512 ? 32 : 64;
}

}  // namespace

int route_grid(int64_t T, int64_t E) {
  const int64_t rows = (int64_t)kRouteWaves * 64 / lanes_of(E);
  const int64_t blocks = (T + rows - 1) / rows;
  return (int)(blocks < 1 ? 1 : blocks < kRouteMaxGrid ? blocks : kRouteMaxGrid);
}

void launch_route(const RouteArgs& a, bool backward, int grid, hipStream_t stream) {
  switch (lanes_of(a.E)) {
    case 4: launch<4, 16>(a, backward, grid, stream); break;
    case 8: launch<8, 16>(a, backward, grid, stream); break;
    case 16: launch<16, 16>(a, backward, grid, stream); break;
    case 32: launch<32, 16>(a, backward, grid, stream); break;
    default: launch<64, 16>(a, backward, grid, stream); break;
  }
}

}  // namespace dg
