// dg_route.hip -- the gate of a mixture of experts for gfx950: scores, the k experts of
// each row, their weights, rows per expert and the balance loss in one pass over the
// logits, and the gradient of weights and loss by the logits in another.
//
// A row of E logits is held by L lanes of a wave, V of them in each lane's registers
// (L * V >= E), 64 / L rows a wave; element 4 (c L + l) + i of the row is register 4c + i
// of lane l, so that a chunk c is one 16-byte (fp32) or 8-byte (bf16) load a lane and
// consecutive lanes read consecutive addresses.
//
// Choice of experts.  A key fp32(z + bias) becomes a double whose high word is the key's
// bits and whose low word says the expert: both formats order by sign, then magnitude, so
// doubles made this way compare as the keys do (an fp32 infinity is an ordinary double),
// and between equal keys the low word decides, in favour of the lower expert.  No two of a
// row are equal, so one v_max_f64 / v_min_f64 pair orders two candidates completely: each
// lane sorts its candidates by blocks, keeps the best KM >= k, and the lanes' lists are
// merged in pairs (the maximum of one list with the other reversed holds the best KM of
// both, as a bitonic sequence).
//
// Scores are recomputed in the backward pass rather than kept: reading T x E logits again
// costs what reading T x E scores would.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_ops.h"

namespace dg {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// --------------------------------------------------------------------------- arithmetic
constexpr float kLog2e = 1.44269504f;

// exp(x) as 2^(x log2 e): two roundings of the exponent, which cost |x| 2^-24 of the result
// (the weights that matter have small |x|).  0 at -inf, NaN at NaN.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// sigmoid(z) = s and s (1 - s), without cancellation on either side; 0 at -inf, 1 at inf.
// Shifted, both times exp(-by): for z up to -18 only, where 1 + exp(z) is 1.
struct Shift {
  float by = 0.0f, one = 1.0f;           // one: what exp(z) counts for beside 1
};
__device__ __forceinline__ float sigmoid(float z, float* slope, Shift shift = {}) {
  const float e = exp_of(-fabsf(z) - shift.by);
  const float r = __builtin_amdgcn_rcpf(__builtin_fmaf(e, shift.one, 1.0f)), er = e * r;
  *slope = r * er;
  return z >= 0.0f ? r : er;
}
__device__ __forceinline__ float sigmoid(float z) {
  float slope;
  return sigmoid(z, &slope);
}

// Scores that leave fp32's range.  Normalized weights and the shares of a sigmoid's row in the
// loss are quotients of scores, and keep their precision where the scores do not: they are
// formed from scores relative to the largest of theirs (not below e^-600: sigmoid scores under
// that or so count as 0).  The sigmoid's in the loss always are.  Otherwise rows with a choice
// whose score is below kTinyScore, or in the backward pass with sigmoid scores that sum to less
// than kTinySum (every logit is below -18 then), are done once more.  Ordinary rows have
// neither, and a ballot leaves both out: done for every row, the first costs 1.5% of a decode
// step and 2.6% of a backward pass (32768 x 256), the second 8% of one under sigmoid.
constexpr float kTinyScore = 0x1p-80f, kTinySum = 0x1p-26f;

__device__ __forceinline__ bool any(bool lane) {
  return __builtin_expect(__builtin_amdgcn_ballot_w64(lane) != 0, 0);
}
// Whether it holds in one of the L lanes of this lane's row.
template <int L>
__device__ __forceinline__ bool in_row(bool lane) {
  const uint64_t lanes = __builtin_amdgcn_ballot_w64(lane);
  if constexpr (L == 64) return lanes != 0;
  else return ((lanes >> (__lane_id() & ~(L - 1))) & ((1ull << L) - 1)) != 0;
}
__device__ __forceinline__ float relative_to(float top) { return fmaxf(fminf(top, 0.0f), -600.0f); }
__device__ __forceinline__ Shift shift_for(float max) {
  return max < -18.0f ? Shift{relative_to(max), 0.0f} : Shift{};
}
// A choice's score relative to that of the row's choice with the largest logit, and in *rest
// 1 - s (softmax: 1).
__device__ __forceinline__ float relative_score(const RouteArgs& a, float z, float top, float* rest) {
  *rest = 1.0f;
  if (!a.sigmoid) return exp_of(z - top);
  const float e = exp_of(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
  *rest = z >= 0.0f ? e * r : r;
  return exp_of(fminf(z, 0.0f) - relative_to(top)) * r;
}

// What the wave's lanes have written to memory is there, and is followed by what they write next.
__device__ __forceinline__ void wave_memory_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// ------------------------------------------------------------------------ across lanes
// The value of another lane of the group, for combining groups of X lanes (whose lanes all
// hold the same) into groups of 2 X: lane ^ X, or any other lane of the other half.
template <int X>
__device__ __forceinline__ int across(int v) {
  if constexpr (X == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);    // quad 1 0 3 2
  else if constexpr (X == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);  // 2 3 0 1
  else if constexpr (X == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true); // 8 mirrored
  else if constexpr (X == 8) return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true); // 16 mirrored
  else return __shfl_xor(v, X, 64);
}
template <int X>
__device__ __forceinline__ float across(float v) {
  return __int_as_float(across<X>(__float_as_int(v)));
}
template <int X>
__device__ __forceinline__ double across(double v) {
  const long long u = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)across<X>((int)(uint32_t)u), hi = (uint32_t)across<X>((int)(u >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

template <int L, int X = 1>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (X < L) return group_max<L, 2 * X>(fmaxf(v, across<X>(v)));
  else return v;
}
template <int L, int X = 1>
__device__ __forceinline__ float group_sum(float v) {
  if constexpr (X < L) return group_sum<L, 2 * X>(v + across<X>(v));
  else return v;
}

// What the wave's lanes have written to LDS is there for the others, and stays as it is until
// all have read it (a wave's LDS accesses are carried out in order).
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// --------------------------------------------------------------------- choosing experts
__device__ __forceinline__ double pack_key(float key, int e) {
  const int bits = __float_as_int(fmaxf(key, -INFINITY));      // NaN: -inf
  const uint32_t low = (uint32_t)((bits >> 31) ^ (1023 - e));
  return __longlong_as_double((long long)(((uint64_t)(uint32_t)bits << 32) | low));
}
__device__ __forceinline__ double no_key() {                   // below every finite key
  return __longlong_as_double((long long)0xFF800000FFFFFFFFull);
}
__device__ __forceinline__ float key_value(double d) {
  return __int_as_float((int)(__double_as_longlong(d) >> 32));
}
__device__ __forceinline__ int key_expert(double d) {          // -1: a key of -inf
  const int bits = (int)(__double_as_longlong(d) >> 32);
  const int low = (int)__double_as_longlong(d);
  return bits == (int)0xFF800000 ? -1 : 1023 - (low ^ (bits >> 31));
}

__device__ __forceinline__ void order(double& a, double& b) {  // a >= b
  const double hi = fmax(a, b), lo = fmin(a, b);
  a = hi;
  b = lo;
}

// Comparators of Batcher's odd-even merge sort of N = 2^n numbers.
template <int N>
struct SortNet {
  int n = 0;
  int a[80] = {}, b[80] = {};
  constexpr SortNet() {
    for (int p = 1; p < N; p *= 2)
      for (int k = p; k >= 1; k /= 2)
        for (int j = k % p; j + k < N; j += 2 * k)
          for (int i = 0; i < k && i + j + k < N; ++i)
            if ((i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              a[n] = i + j;
              b[n] = i + j + k;
              ++n;
            }
  }
};
template <int N>
__device__ __forceinline__ void sort(double (&x)[N]) {
  constexpr SortNet<N> net;
#pragma unroll
  for (int t = 0; t < net.n; ++t) order(x[net.a[t]], x[net.b[t]]);
}
// list = the best N of list and other (given in reverse), both sorted
template <int N>
__device__ __forceinline__ void merge(double (&list)[N], const double (&other)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) list[i] = fmax(list[i], other[N - 1 - i]);
#pragma unroll
  for (int d = N / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & d) == 0) order(list[i], list[i + d]);
}
template <int L, int N, int X = 1>
__device__ __forceinline__ void merge_lanes(double (&list)[N]) {
  if constexpr (X < L) {
    double other[N];
#pragma unroll
    for (int i = 0; i < N; ++i) other[i] = across<X>(list[i]);
    merge<N>(list, other);
    merge_lanes<L, N, 2 * X>(list);
  }
}

// ------------------------------------------------------------------------------- memory
__device__ __forceinline__ float load_one(const void* p, int64_t i, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}
// Two numbers rounded to bf16 (to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
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
// exp(z - max) * inv; s = exp(z - max).  A row of -inf only (nothing left of it) has max = 0
// and inv = 0.
struct RowNorm {
  float max, inv;
};

template <int L, int V>
__device__ __forceinline__ float row_max(const float (&z)[V]) {
  float m = z[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, z[v]);
  return group_max<L>(m);
}

template <int L, int V>
__device__ __forceinline__ RowNorm softmax_row(const float (&z)[V], float (&s)[V]) {
  float m = row_max<L, V>(z);
  const bool none = m == -INFINITY;
  m = none ? 0.0f : m;
  float sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = exp_of(z[v] - m);
    sum += s[v];
  }
  sum = group_sum<L>(sum);
  return {m, none ? 0.0f : 1.0f / sum};
}

// ------------------------------------------------------------------------------ forward
// What the workgroups of a call with several have counted, in the workspace: [workgroup][E]
// probabilities, [workgroup][E] choices, [workgroup] live rows; before them the word in
// which the second kernel's workgroups add up the loss.
struct Parts {
  unsigned long long* word;
  float* p;
  int* n;
  int* rows;
  __device__ Parts(const RouteArgs& a, int G)
      : word((unsigned long long*)a.workspace),
        p((float*)((uint8_t*)a.workspace + kRouteWsHeader)),
        n((int*)(p + (int64_t)G * a.E)),
        rows(n + (int64_t)G * a.E) {}
};

__device__ __forceinline__ float coef_of(const RouteArgs& a, int n, int live) {
  const float rows = (float)live;
  return live ? a.balance * (float)a.E / (float)a.k * (float)n / rows / rows : 0.0f;
}

// A call of one workgroup ends with the sums over rows; the workgroups of a larger one leave
// theirs to route_sums_kernel.  32768 x 256 fp32, 8 of each row, with the loss: 15.7 us (2.2
// TB/s), then 5.9 for the sums; the networks' f64 instructions and their registers, which
// leave two or three waves a SIMD to hide the loads, bound it.  64 x 256, one workgroup: 8.5.
template <int L, int V, int KM>
__global__ void __launch_bounds__(kThreads, V == 32 ? 3 : 4)
route_kernel(RouteArgs a) {
  constexpr int RW = 64 / L, EP = L * V;
  constexpr int KP = KM > L ? KM / L : 1;             // choices that a lane writes
  __shared__ int hist[EP];
  __shared__ __attribute__((aligned(16))) float psum[kWaves * RW][EP];
  __shared__ __attribute__((aligned(16))) float bias[EP];
  __shared__ int live_rows;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % L, sub = lane / L;
  const bool sums = a.counts != nullptr;
  for (int e = tid; e < EP; e += kThreads) {
    hist[e] = 0;
    // a bias of -0 as +0: a key is then never -0, which would lie below the +0 it equals
    bias[e] = a.bias && e < a.E ? a.bias[e] + 0.0f : 0.0f;
  }
  if (tid == 0) live_rows = 0;
  __syncthreads();

  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  int nlive = 0;
  const int64_t step = (int64_t)gridDim.x * kWaves * RW;
  for (int64_t row0 = ((int64_t)blockIdx.x * kWaves + wave) * RW; row0 < a.T; row0 += step) {
    const int64_t row = row0 + sub;
    const bool in = row < a.T;
    const int64_t at = in ? row : a.T - 1;
    float z[V], s[V];
    load_row<L, V>(a, at, l, -INFINITY, z);
    const bool live = in && (!a.row_valid || a.row_valid[at] != 0);
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = live ? z[v] : -INFINITY;
    if (live && l == 0) ++nlive;

    // the best KM keys of the row, in every lane of it
    double list[KM];
    constexpr int NB = KM < V ? KM : V;               // candidates sorted at a time
#pragma unroll
    for (int b = 0; b < V / NB; ++b) {
      __builtin_amdgcn_sched_barrier(0);              // one block's candidates at a time
      double x[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int v = b * NB + i, e = 4 * ((v / 4) * L + l) + (v & 3);
        x[i] = pack_key(z[v] + bias[e], e);
      }
      sort<NB>(x);
      if (b == 0) {
#pragma unroll
        for (int i = 0; i < KM; ++i) list[i] = i < NB ? x[i < NB ? i : 0] : no_key();
      } else if constexpr (NB == KM) {
        merge<KM>(list, x);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    merge_lanes<L, KM>(list);
    __builtin_amdgcn_sched_barrier(0);

    RowNorm n{0.0f, 0.0f};
    if (!a.sigmoid) {
      n = softmax_row<L, V>(z, s);
    } else if (a.loss) {
      const Shift shift = shift_for(row_max<L, V>(z));
      float sum = 0.0f, slope;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = sigmoid(z[v], &slope, shift);
        sum += s[v];
      }
      sum = group_sum<L>(sum);
      n.inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    if (a.loss) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = __builtin_fmaf(s[v], n.inv, acc[v]);
    }

    // lane l of the row keeps the choices l, l + L, ...
    int ids[KP];
    float w[KP];
#pragma unroll
    for (int q = 0; q < KP; ++q) {
      const int j = q * L + l;
      double d = list[0];
#pragma unroll
      for (int i = 1; i < KM; ++i) d = j == i ? list[i] : d;
      ids[q] = j < a.k ? key_expert(d) : -1;
      w[q] = 0.0f;
      if (ids[q] >= 0) {
        const float zc = a.bias ? load_one(a.logits, at * a.ld + ids[q], a.bf16) : key_value(d);
        w[q] = a.sigmoid ? sigmoid(zc) : exp_of(zc - n.max) * n.inv;
        if (sums) atomicAdd(&hist[ids[q]], 1);
      }
    }
    float f = a.scale;
    if (a.normalize) {
      bool low = false;
#pragma unroll
      for (int q = 0; q < KP; ++q) low = low || (ids[q] >= 0 && w[q] < kTinyScore);
      // under softmax without a bias the largest logit is a choice's
      if ((a.bias || a.sigmoid) && any(low)) {
        low = in_row<L>(low);
        float top = -INFINITY, rest;
#pragma unroll
        for (int q = 0; q < KP; ++q)
          if (ids[q] >= 0) top = fmaxf(top, load_one(a.logits, at * a.ld + ids[q], a.bf16));
        top = group_max<L>(top);
#pragma unroll
        for (int q = 0; q < KP; ++q)
          if (low && ids[q] >= 0)
            w[q] = relative_score(a, load_one(a.logits, at * a.ld + ids[q], a.bf16), top, &rest);
      }
      // in pairs, pairs of pairs ... of the choices, whatever L is
      float part[KP];
#pragma unroll
      for (int q = 0; q < KP; ++q) part[q] = group_sum<L>(w[q]);
#pragma unroll
      for (int d = 1; d < KP; d *= 2)
#pragma unroll
        for (int q = 0; q < KP; q += 2 * d) part[q] += part[q + d];
      f = part[0] == 0.0f ? 0.0f : a.scale / part[0];
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

  // the workgroup's sums, the probabilities in the order of its rows' places
  if (l == 0) atomicAdd(&live_rows, nlive);
  if (a.loss) {
#pragma unroll
    for (int c = 0; c < V / 4; ++c)
      *(float4*)&psum[wave * RW + sub][4 * (c * L + l)] =
          make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
  }
  __syncthreads();
  const int G = (int)gridDim.x, b = blockIdx.x;
  Parts part(a, G);
  float sum = 0.0f;
  for (int e = tid; e < a.E; e += kThreads) {
    const int n = hist[e];
    float p = 0.0f;
    if (a.loss)
      for (int w = 0; w < kWaves * RW; ++w) p += psum[w][e];
    if (G > 1) {
      part.n[(int64_t)b * a.E + e] = n;
      if (a.loss) part.p[(int64_t)b * a.E + e] = p;
    } else {
      a.counts[e] = n;
      if (a.loss) {
        const float c = coef_of(a, n, live_rows);
        a.coef[e] = c;
        sum += live_rows ? c * p : 0.0f;
      }
    }
  }
  if (G > 1) {
    if (tid == 0) part.rows[b] = live_rows;
    if (tid == 0 && b == 0) *part.word = 0;
  } else if (a.loss) {
    sum = group_sum<64>(sum);
    __syncthreads();
    if (lane == 0) bias[wave] = sum;
    __syncthreads();
    if (tid == 0) *a.loss = (bias[0] + bias[1]) + (bias[2] + bias[3]);
  }
}

// Sums over the first kernel's G workgroups: a workgroup takes `cols` experts, its threads
// one of them and a slice of the G each; then the slices of a wave, then the waves, in a
// fixed order.  The workgroups' parts of the loss meet in one word: the loss is balance * E
// times sum_e (n_e / (k V)) (p_e / V), a number in [0, 1], which each adds as a multiple of
// 2^-44 together with one arrival, in one atomic addition; integers add up to the same in
// any order, and who finds all others arrived has the sum.  (To store parts, arrive and read
// them back takes three trips to memory instead of one.)
constexpr int kSumThreads = 1024, kSumMinCols = 16, kSumWaves = kSumThreads / 64;

__global__ void __launch_bounds__(kSumThreads)
route_sums_kernel(RouteArgs a, int G, int cols) {
  __shared__ int n_s[kSumThreads], live_s[kSumWaves];
  __shared__ float p_s[kSumThreads], loss_s[kSumWaves];
  const int tid = threadIdx.x, c = tid & (cols - 1), slices = kSumThreads / cols, slice = tid / cols;
  const int e = blockIdx.x * cols + c, ee = e < a.E ? e : a.E - 1;
  Parts part(a, G);
  int n = 0, live = tid < G ? part.rows[tid] : 0;
  float p = 0.0f;
  constexpr int U = 8;                     // sums in flight (without a loss p is not used)
  for (int g0 = slice; g0 < G; g0 += U * slices) {
    int nv[U];
    float pv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * slices < G ? g0 + u * slices : slice;
      nv[u] = part.n[(int64_t)g * a.E + ee];
      pv[u] = part.p[(int64_t)g * a.E + ee];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (g0 + u * slices < G) {
        n += nv[u];
        p += pv[u];
      }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) live += __shfl_xor(live, off, 64);
  for (int off = cols; off < 64; off *= 2) {
    n += __shfl_xor(n, off, 64);
    p += __shfl_xor(p, off, 64);
  }
  n_s[tid] = n;
  p_s[tid] = p;
  if ((tid & 63) == 0) live_s[tid >> 6] = live;
  __syncthreads();
  live = 0;
#pragma unroll
  for (int w = 0; w < kSumWaves; ++w) live += live_s[w];
  float sum = 0.0f;
  if (tid < cols && e < a.E) {
    const int each = cols < 64 ? 64 : cols;       // threads between two sums of an expert
    for (int w = each; w < kSumThreads; w += each) {
      n += n_s[w + tid];
      p += p_s[w + tid];
    }
    a.counts[e] = n;
    if (a.loss) {
      a.coef[e] = coef_of(a, n, live);
      const float rows = (float)live;
      sum = live ? ((float)n / ((float)a.k * rows)) * (p / rows) : 0.0f;
    }
  }
  if (!a.loss) return;
  sum = group_sum<64>(sum);
  if ((tid & 63) == 0) loss_s[tid >> 6] = sum;
  __syncthreads();
  if (tid >= 64) return;
  sum = group_sum<16>(loss_s[tid & 15]);
  if (tid != 0) return;
  constexpr int kFraction = 44, kCount = 56;
  constexpr unsigned long long kNaN = 1ull << 48;         // past any sum, 64 of them below kCount
  const unsigned long long mine =
      (1ull << kCount) | (sum != sum ? kNaN : (unsigned long long)((double)sum * (1ull << kFraction) + 0.5));
  const unsigned long long all =
      mine + __hip_atomic_fetch_add(part.word, mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if ((int)(all >> kCount) != (int)gridDim.x) return;
  const unsigned long long x = all & ((1ull << kCount) - 1);
  const float share = x >= kNaN ? __builtin_nanf("") : (float)((double)x / (1ull << kFraction));
  *a.loss = a.balance * (float)a.E * share;
}

// Experts of a workgroup of the second kernel: at most about 16 of the G sums a thread.
int sum_cols(int E, int G) {
  int cols = kSumMinCols;
  while (cols < E && cols < kSumThreads && 2 * cols * G <= 16 * kSumThreads) cols *= 2;
  return cols;
}
static_assert(kRouteMaxGrid <= kSumThreads, "one thread a workgroup's live rows");
static_assert((kRouteMaxE + kSumMinCols - 1) / kSumMinCols <= 64, "arrivals");

// ----------------------------------------------------------------------------- backward
// A row with tiny scores, its loss's part from n and us under softmax.  With q the normalized
// weights over their factor and g their gradients times it, a choice's part of dz is
// q (g - sum of g q), times 1 - s under sigmoid.
template <int L>
__device__ __forceinline__ void tiny_row(const RouteArgs& a, int64_t row, int l, float g_loss, RowNorm n,
                                         float us) {
  const int64_t at = row * a.ld;
  auto logit = [&](int e) { return load_one(a.logits, at + e, a.bf16); };
  auto of_loss = [&](int e) { return a.coef ? g_loss * a.coef[e] : 0.0f; };
  Shift shift;
  if (a.sigmoid) {
    float max = -INFINITY, sum = 0.0f, c;
    us = 0.0f;
#pragma unroll 1
    for (int e = l; e < a.E; e += L) max = fmaxf(max, logit(e));
    shift = shift_for(group_max<L>(max));
#pragma unroll 1
    for (int e = l; e < a.E; e += L) {
      const float s = sigmoid(logit(e), &c, shift);
      sum += s;
      us = __builtin_fmaf(of_loss(e), s, us);
    }
    sum = group_sum<L>(sum);
    n.inv = !a.coef || sum == 0.0f ? 0.0f : 1.0f / sum;
    us = a.coef ? group_sum<L>(us) * n.inv : 0.0f;
  }
  // f(expert, its logit, its weight's gradient) for the row's choices
  auto each = [&](auto f) {
    if (!a.grad_weights) return;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
      const int e = a.ids_in[row * a.k + j];
      if (e >= 0 && e < a.E) f(e, logit(e), a.scale * a.grad_weights[row * a.k + j]);
    }
  };
  float top = -INFINITY, total = 0.0f, dot = 0.0f, rest;
  each([&](int, float x, float) { top = fmaxf(top, x); });
  each([&](int, float x, float g) {
    const float s = relative_score(a, x, top, &rest);
    total += s;
    dot = __builtin_fmaf(g, s, dot);
  });
  const float it = total == 0.0f ? 0.0f : 1.0f / total, mean = dot * it;
#pragma unroll 1
  for (int e = l; e < a.E; e += L) {
    float dz, c;
    if (a.sigmoid) {
      sigmoid(logit(e), &c, shift);
      dz = (of_loss(e) - us) * n.inv * c;
    } else {
      dz = exp_of(logit(e) - n.max) * n.inv * (of_loss(e) - us);
    }
    each([&](int chosen, float x, float g) {
      if (chosen != e) return;
      if (a.normalize) {
        const float q = relative_score(a, x, top, &rest) * it;
        dz += q * (g - mean) * rest;
      } else {                                  // under sigmoid only
        sigmoid(x, &c);
        dz += g * c;
      }
    });
    if (a.bf16) ((uint16_t*)a.grad_logits)[row * a.ld_grad + e] = (uint16_t)pack_bf16(dz, 0.0f);
    else ((float*)a.grad_logits)[row * a.ld_grad + e] = dz;
  }
}

// dz from the weights' gradients and the loss's (coef, the same for every row).  A row's
// scores go through a row of LDS, where the lanes that keep its choices pick theirs up, and
// the choices' score gradients through another, which is zero but for them.  A wave's next
// rows are loaded before its present ones are worked on.  32768 x 256 fp32: 16.8 us, 4.1 TB/s
// (a copy of 64 MB, as much as it reads and writes, reaches 5.0, one of 256 MB 5.4); 8192 x 8
// bf16: 4.4 us, a launch's latency, 0.3 of it for the code of rows with tiny scores.
template <int L, int V>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(RouteArgs a) {
  constexpr int RW = 64 / L, EP = L * V;
  constexpr int KP = L >= kRouteMaxK ? 1 : kRouteMaxK / L;   // choices of a lane
  __shared__ __attribute__((aligned(16))) float rows_s[kWaves * RW][EP], rows_d[kWaves * RW][EP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % L, sub = lane / L;
  float* sr = rows_s[wave * RW + sub];
  float* dr = rows_d[wave * RW + sub];
  float u[V];
  const float g_loss = a.coef ? (a.grad_loss ? *a.grad_loss : 1.0f) : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = 4 * ((v / 4) * L + l) + (v & 3);
    dr[e] = 0.0f;
    u[v] = a.coef && e < a.E ? g_loss * a.coef[e] : 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * kWaves * RW;
  const int64_t first = ((int64_t)blockIdx.x * kWaves + wave) * RW;

  float z[V], gw[KP];
  int id[KP], valid;
  auto load = [&](int64_t row) {
    const int64_t at = row < a.T ? row : a.T - 1;
    load_row<L, V>(a, at, l, -INFINITY, z);
    valid = row < a.T && (!a.row_valid || a.row_valid[at] != 0);
#pragma unroll
    for (int q = 0; q < KP; ++q) {
      const int j = q * L + l;
      id[q] = -1;
      gw[q] = 0.0f;
      if (a.grad_weights && j < a.k) {
        id[q] = a.ids_in[at * a.k + j];
        gw[q] = a.grad_weights[at * a.k + j];
      }
    }
  };
  if (first < a.T) load(first + sub);
  for (int64_t row0 = first; row0 < a.T; row0 += step) {
    const int64_t row = row0 + sub;
    float x[V], s[V], c[V], g[KP];
    int chosen[KP];
    const bool live = valid;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = z[v];      // of padding whatever it holds: not used
#pragma unroll
    for (int q = 0; q < KP; ++q) {
      chosen[q] = live && id[q] >= 0 && id[q] < a.E ? id[q] : -1;
      g[q] = chosen[q] >= 0 ? a.scale * gw[q] : 0.0f;
    }
    if (row0 + step < a.T) load(row + step);

    RowNorm n{0.0f, 0.0f};
    float us = 0.0f;                              // sum of u p over the row
    bool tiny = false;                            // to be done by tiny_row
    if (a.sigmoid) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = sigmoid(x[v], &c[v]);
        sum += s[v];
        us = __builtin_fmaf(u[v], s[v], us);
      }
      sum = group_sum<L>(sum);
      tiny = live && a.coef && sum < kTinySum;
      // without the loss a NaN among the scores stays its own
      n.inv = !a.coef || sum == 0.0f ? 0.0f : 1.0f / sum;
      us = a.coef ? group_sum<L>(us) * n.inv : 0.0f;
    } else {
      n = softmax_row<L, V>(x, s);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] *= n.inv;
        us = __builtin_fmaf(u[v], s[v], us);
      }
      us = group_sum<L>(us);
    }
    float ds = 0.0f;                              // sum of D s over the chosen: 0 if normalized
    if (a.grad_weights) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q)
        *(float4*)&sr[4 * (q * L + l)] = make_float4(s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]);
      wave_lds_sync();
      float sc[KP], total = 0.0f, dot = 0.0f;
#pragma unroll
      for (int q = 0; q < KP; ++q) {
        sc[q] = chosen[q] >= 0 ? sr[chosen[q]] : 0.0f;
        total += sc[q];
        dot = __builtin_fmaf(g[q], sc[q], dot);
      }
      if (a.normalize) {
        total = group_sum<L>(total);
        dot = group_sum<L>(dot);
        const float it = total == 0.0f ? 0.0f : 1.0f / total;
        const float mean = dot * it;
#pragma unroll
        for (int q = 0; q < KP; ++q) {
          tiny = tiny || (chosen[q] >= 0 && sc[q] < kTinyScore);
          g[q] = (g[q] - mean) * it;
        }
      }
#pragma unroll
      for (int q = 0; q < KP; ++q)
        if (chosen[q] >= 0) {
          dr[chosen[q]] = g[q];
          ds = __builtin_fmaf(g[q], sc[q], ds);
        }
      ds = a.sigmoid || a.normalize ? 0.0f : group_sum<L>(ds);
      wave_lds_sync();
    }
    float dz[V];
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const float4 d = a.grad_weights ? *(const float4*)&dr[4 * (q * L + l)] : make_float4(0, 0, 0, 0);
      const float dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = 4 * q + i;
        const float r = a.sigmoid ? ((u[v] - us) * n.inv + dv[i]) * c[v] : s[v] * (u[v] + dv[i] - (us + ds));
        dz[v] = live ? r : 0.0f;
      }
    }
    if (a.grad_weights) {
      wave_lds_sync();
#pragma unroll
      for (int q = 0; q < KP; ++q)
        if (chosen[q] >= 0) dr[chosen[q]] = 0.0f;
    }
    if (row < a.T) {
      const int64_t at = row * a.ld_grad;
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const int e = 4 * (q * L + l);
        if (a.vec_grad) {
          if (e < a.E) {
            if (a.bf16)
              *(uint2*)((uint16_t*)a.grad_logits + at + e) =
                  make_uint2(pack_bf16(dz[4 * q], dz[4 * q + 1]), pack_bf16(dz[4 * q + 2], dz[4 * q + 3]));
            else
              *(float4*)((float*)a.grad_logits + at + e) =
                  make_float4(dz[4 * q], dz[4 * q + 1], dz[4 * q + 2], dz[4 * q + 3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e + i < a.E) {
              if (a.bf16) ((uint16_t*)a.grad_logits)[at + e + i] = (uint16_t)pack_bf16(dz[4 * q + i], 0.0f);
              else ((float*)a.grad_logits)[at + e + i] = dz[4 * q + i];
            }
        }
      }
    }
    if (any(tiny)) {
      wave_memory_sync();
      if (in_row<L>(tiny)) tiny_row<L>(a, row, l, g_loss, n, us);
    }
  }
}

template <int L, int V>
void launch_forward(const RouteArgs& a, int grid, hipStream_t stream) {
  const int k = a.k;
  auto* f = k <= 2   ? &route_kernel<L, V, 2>
            : k <= 4 ? &route_kernel<L, V, 4>
            : k <= 8 ? &route_kernel<L, V, 8>
                     : &route_kernel<L, V, 16>;
  hipLaunchKernelGGL(f, dim3(grid), dim3(kThreads), 0, stream, a);
  if (a.counts && grid > 1) {
    const int cols = sum_cols(a.E, grid);
    hipLaunchKernelGGL(route_sums_kernel, dim3((a.E + cols - 1) / cols), dim3(kSumThreads), 0, stream,
                       a, grid, cols);
  }
}

template <int L, int V>
void launch_backward(const RouteArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL((route_backward_kernel<L, V>), dim3(grid), dim3(kThreads), 0, stream, a);
}

int lanes_for(int64_t E, int V) {
  int L = 1;
  while (L * V < E) L *= 2;
  return L;
}

// Forward launch shape.  Few experts a lane (V = 8) spread a row over more lanes: shorter
// chains, for calls that do not fill the GPU.  Many (V = 32) leave less to merge across
// lanes: less work in all.  With `counts` under sigmoid, rows that one workgroup takes in two
// passes are left to one, which needs no second kernel (64 x 256 with counts, one call after the
// other: 12.1 us as two kernels on 16 workgroups, 8.6 as one).  Under softmax the sum over a
// row, and with it the weights' last bits, would then differ from those of a call that asks
// for no counts.
struct Shape {
  int V, L, grid;
};
Shape forward_shape(int64_t T, int64_t E, bool one_if_small) {
  Shape h;
  auto set = [&](int V) {
    h.V = V;
    h.L = lanes_for(E, V);
    if (V == 32 && h.L < 2) h.L = 2;
    const int64_t rows = (int64_t)kWaves * 64 / h.L, blocks = (T + rows - 1) / rows;
    h.grid = (int)(blocks < 1 ? 1 : blocks < kRouteMaxGrid ? blocks : kRouteMaxGrid);
  };
  set(E > 512 || T * E >= kRouteWideWork ? 32 : 8);
  if (one_if_small && h.grid > 1) {
    const Shape few = h;
    set(E > 16 ? 32 : 8);
    if (h.grid > 2) return few;
    h.grid = 1;
  }
  return h;
}

}  // namespace

int route_slots(int64_t T, int64_t E) {
  const int g = forward_shape(T, E, false).grid;
  return g > 1 ? g : 0;
}

void launch_route(const RouteArgs& a, hipStream_t stream) {
  const Shape h = forward_shape(a.T, a.E, a.sigmoid && a.counts);
  if (h.V == 32) {
    switch (h.L) {
      case 2: return launch_forward<2, 32>(a, h.grid, stream);
      case 4: return launch_forward<4, 32>(a, h.grid, stream);
      case 8: return launch_forward<8, 32>(a, h.grid, stream);
      case 16: return launch_forward<16, 32>(a, h.grid, stream);
      default: return launch_forward<32, 32>(a, h.grid, stream);
    }
  }
  switch (h.L) {
    case 1: return launch_forward<1, 8>(a, h.grid, stream);
    case 2: return launch_forward<2, 8>(a, h.grid, stream);
    case 4: return launch_forward<4, 8>(a, h.grid, stream);
    case 8: return launch_forward<8, 8>(a, h.grid, stream);
    case 16: return launch_forward<16, 8>(a, h.grid, stream);
    case 32: return launch_forward<32, 8>(a, h.grid, stream);
    default: return launch_forward<64, 8>(a, h.grid, stream);
  }
}

void launch_route_backward(const RouteArgs& a, hipStream_t stream) {
  // few experts a lane while the call does not fill the GPU (4099 x 60: 3.3 us with 4, 4.1 with
  // 8), more, and fewer steps across lanes, once it does (32768 x 256: 16.4 us with 8, 17.8
  // with 4, 20.7 with 16, whose registers leave too few waves)
  const int V = a.E > 512 ? 16 : a.E > 256 || a.T * a.E >= kRouteWideWork / 2 ? 8 : 4;
  const int L = lanes_for(a.E, V);
  const int64_t rows = (int64_t)kWaves * 64 / L, blocks = (a.T + rows - 1) / rows;
  const int grid = (int)(blocks < 1024 ? blocks : 1024);
  if (V == 16) return launch_backward<64, 16>(a, grid, stream);
  if (V == 8) {
    switch (L) {
      case 1: return launch_backward<1, 8>(a, grid, stream);
      case 2: return launch_backward<2, 8>(a, grid, stream);
      case 4: return launch_backward<4, 8>(a, grid, stream);
      case 8: return launch_backward<8, 8>(a, grid, stream);
      case 16: return launch_backward<16, 8>(a, grid, stream);
      case 32: return launch_backward<32, 8>(a, grid, stream);
      default: return launch_backward<64, 8>(a, grid, stream);
    }
  }
  switch (L) {
    case 1: return launch_backward<1, 4>(a, grid, stream);
    case 2: return launch_backward<2, 4>(a, grid, stream);
    case 4: return launch_backward<4, 4>(a, grid, stream);
    case 8: return launch_backward<8, 4>(a, grid, stream);
    case 16: return launch_backward<16, 4>(a, grid, stream);
    case 32: return launch_backward<32, 4>(a, grid, stream);
    default: return launch_backward<64, 4>(a, grid, stream);
  }
}

}  // namespace dg
