// dg_wgrad.hip -- a weight's gradient from two matrices of fp8 codes with 1x128 scales, for
// gfx950:  dW_g[n,k] = sum over the rows t of group g of (sP[t,n/128] P[t,n]) (sQ[t,k/128] Q[t,k]).
//
// The sum runs over rows, so each row's scales are inside it and no fp8 product can carry
// them: the codes become bf16 on their way to v_mfma_f32_32x32x16_bf16, which accumulates in
// fp32: P with both scales, rounded once, Q as it is (a code is a bf16 number).
//
// Both operands lie row by row, while the matrix instruction wants 8 rows of a column in a
// lane: the codes of 64 rows are copied as they are into LDS (direct copies, three such steps
// ahead) and ds_read_b64_tr_b8 turns 8 rows x 16 columns on their way to the registers.  32-byte
// pieces of an LDS row are swapped by the row's low bits, so that the 8 rows of a read lie in
// different banks.
//
// What bounds it: the matrix pipe at the clock that the power leaves it; conversions (two
// instructions for a scaled code, half a one for the others, P's once for each of two waves, Q's
// for each of four) run beside it.  16384 rows of 8 groups by (4096, 7168): 1024 to 1060 us, 0.9 PFLOP/s of
// the rows that count (a library's bf16 product of 8192^3: 1.31); without the conversions 916 us,
// without the copies 971, without the stores 1001, without the products 713 (of 1097 then).
// 1093 rows by (7168, 2048): 42 us, 0.77 PFLOP/s, 5 us of them the gradient's way to memory, in bf16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_ffn.h"
#include "dg_fp8.h"

namespace dg {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i lds_v2i;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kDeep = 64;          // rows of a step
constexpr int kStages = 4;
constexpr int kPast = 0x7FFFFF00;  // past every copy's range

// Two codes of a word as fp32.
template <int FMT, bool HI>
__device__ __forceinline__ v2f two(unsigned w) {
  return FMT == kFmtE5M2 ? __builtin_amdgcn_cvt_pk_f32_bf8((int)w, HI) : __builtin_amdgcn_cvt_pk_f32_fp8((int)w, HI);
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
  const v2b v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(unsigned, v);
}

// Eight codes times their rows' scales, and eight codes, as bf16.
template <int FMT>
__device__ __forceinline__ v8b scaled_bf16(v2i c, const v4f& s0, const v4f& s1) {
  const v2f a = two<FMT, false>(c[0]), b = two<FMT, true>(c[0]), d = two<FMT, false>(c[1]), e = two<FMT, true>(c[1]);
  const uint4 v = make_uint4(pack_bf16(a[0] * s0[0], a[1] * s0[1]), pack_bf16(b[0] * s0[2], b[1] * s0[3]),
                             pack_bf16(d[0] * s1[0], d[1] * s1[1]), pack_bf16(e[0] * s1[2], e[1] * s1[3]));
  return __builtin_bit_cast(v8b, v);
}
template <int FMT, bool HI>
__device__ __forceinline__ unsigned two_bf16(int w) {
  const v2b v = FMT == kFmtE5M2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((unsigned)w, 1.0f, HI)
                                : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)w, 1.0f, HI);
  return __builtin_bit_cast(unsigned, v);
}
template <int FMT>
__device__ __forceinline__ v8b plain_bf16(v2i c) {
  const uint4 v = make_uint4(two_bf16<FMT, false>(c[0]), two_bf16<FMT, true>(c[0]), two_bf16<FMT, false>(c[1]),
                             two_bf16<FMT, true>(c[1]));
  return __builtin_bit_cast(v8b, v);
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}
// At most `ahead` batches of PER copies in flight.
template <int PER>
__device__ __forceinline__ void wait_batches(int ahead) {
  if (ahead >= 2)
    wait_vmcnt<2 * PER>();
  else if (ahead == 1)
    wait_vmcnt<PER>();
  else
    wait_vmcnt<0>();
}
__device__ __forceinline__ void step_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);            // this wave's LDS writes are done
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_over(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// Every step-th of the 128-row blocks of a group (those whose first row names it), from the
// skip-th on; without groups, of all blocks.
// 256 of them are looked at at a time: the look waits for memory, and with it for every copy
// in flight.
template <bool GROUPED>
struct Blocks {
  const int32_t* idx;
  int g, lane;
  int end, step, skip;
  int b;                           // the blocks in masks are b .. b + 255; without groups the next
  uint64_t mask[4];
  __device__ __forceinline__ void look() {
    int lead[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = b + 64 * k + lane;
      lead[k] = idx[(int64_t)(at < end ? at : 0) * kAlignM];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mask[k] = __builtin_amdgcn_ballot_w64(b + 64 * k + lane < end && lead[k] == g);
  }
  __device__ __forceinline__ int next() {       // -1: none left
    if (!GROUPED) {
      const int at = b;
      b += step;
      return at < end ? at : -1;
    }
    for (;;) {
      while ((mask[0] | mask[1] | mask[2] | mask[3]) == 0) {
        b += 256;
        if (b >= end) return -1;
        look();
      }
      const int k = mask[0] ? 0 : mask[1] ? 1 : mask[2] ? 2 : 3;
      uint64_t m = mask[0] ? mask[0] : mask[1] ? mask[1] : mask[2] ? mask[2] : mask[3];
      const int i = 64 * k + (int)__builtin_ctzll(m);
      m &= m - 1;
      if (k == 0) mask[0] = m;
      if (k == 1) mask[1] = m;
      if (k == 2) mask[2] = m;
      if (k == 3) mask[3] = m;
      if (skip-- > 0) continue;
      skip = step - 1;
      return b + i;
    }
  }
};

// Eight elements of the gradient, added to what it holds if it accumulates.
__device__ __forceinline__ void put8(const WgradArgs& a, int64_t at, v4f lo, v4f hi) {
  if (a.bf16) {
    uint4* w = (uint4*)((uint16_t*)a.dW + at);
    if (a.accumulate) {
      const uint4 o = *w;
      lo += (v4f){__uint_as_float(o.x << 16), __uint_as_float(o.x & 0xFFFF0000u), __uint_as_float(o.y << 16),
                  __uint_as_float(o.y & 0xFFFF0000u)};
      hi += (v4f){__uint_as_float(o.z << 16), __uint_as_float(o.z & 0xFFFF0000u), __uint_as_float(o.w << 16),
                  __uint_as_float(o.w & 0xFFFF0000u)};
    }
    *w = make_uint4(pack_bf16(lo[0], lo[1]), pack_bf16(lo[2], lo[3]), pack_bf16(hi[0], hi[1]), pack_bf16(hi[2], hi[3]));
  } else {
    v4f* w = (v4f*)((float*)a.dW + at);
    if (a.accumulate) {
      lo += w[0];
      hi += w[1];
    }
    w[0] = lo;
    w[1] = hi;
  }
}

// A tile of BN columns of P by BK of Q: eight waves, 4 x 2, of BN / 4 by BK / 2.
template <int BN_, int BK_, int FP_, int FQ_>
struct WgradCfg {
  static constexpr int BN = BN_, BK = BK_, FP = FP_, FQ = FQ_;
  static constexpr int NI = BN / 128, NK = BK / 64;        // 32-column fragments a wave
  static constexpr int NB = BN / 128, KB = BK / 128;       // scale columns of P and Q
  static constexpr int KINDS = NB + KB;
  static constexpr int PC = BN / 128, QC = BK / 128;       // copies of a wave: 8 rows of both
  static constexpr int STAGE = kDeep * (BN + BK);
  static constexpr int RING = 8;                           // steps whose scales and indices are kept
  // LDS: the stages, scales as copied, their products, the rows' group indices
  static constexpr int S_OFF = kStages * STAGE;
  static constexpr int M_OFF = S_OFF + RING * KINDS * kDeep * 4;
  static constexpr int R_OFF = M_OFF + 2 * NB * KB * kDeep * 4;
  static constexpr int LDS_BYTES = R_OFF + RING * kDeep * 4;
  static_assert((BN == 128 || BN == 256) && (BK == 128 || BK == 256) && LDS_BYTES <= 160 * 1024, "tile");
};

// The 32-byte pieces of an LDS row are swapped by this.
__device__ __forceinline__ int piece_of(int width, int row) { return width == 256 ? row & 7 : (row >> 1) & 3; }

// Copies of this wave's eight rows of a step, 1 KB each, from column col0 on; rows of another
// group, and rows past the last, come as zeros.
template <int WIDTH, bool GROUPED>
__device__ __forceinline__ void copy_rows(uint8_t* lds, const uint8_t* from, int ld, int64_t left, int col0,
                                          const int32_t* idx, int g, int wave, int lane) {
  const __amdgpu_buffer_rsrc_t r = buffer_over(from, (int)(left < kDeep ? left : kDeep) * ld);
  constexpr int LANES = WIDTH / 16, ROWS = 64 / LANES;   // of a row, of a copy
#pragma unroll
  for (int it = 0; it < 8 / ROWS; ++it) {
    const int row = 8 * wave + it * ROWS + lane / LANES, c = lane % LANES;
    const int off = row * ld + col0 + (((c >> 1) ^ piece_of(WIDTH, row)) << 5) + (c & 1) * 16;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (8 * wave + it * ROWS) * WIDTH), 16,
                                             !GROUPED || idx[row] == g ? off : kPast, 0, 0, 0);
  }
}

// A column of 64 rows' scales (or their group indices).
__device__ __forceinline__ void copy_column(uint8_t* lds, const void* from, int ld, int64_t left, int col,
                                            int lane) {
  const __amdgpu_buffer_rsrc_t r = buffer_over(from, (int)(left < kDeep ? left : kDeep) * ld * 4);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, (lane * ld + col) * 4, 0, 0, 0);
}

// Where a batch of copies comes from.
struct Batch {
  const uint8_t *p, *q;          // the step's first rows
  int64_t left;                  // rows from there on
  const void* s;                 // a later step's first row of this wave's column
  int64_t left_s;
  int n, k, n0, k0, ld_s, col_s, g, wave, lane;
  bool has_column;
};

// One step: start the copies of a later one into `next` and `next_s`, then multiply the one staged
// in `cur`, whose rows' scales are `sc`.  The restrict qualifiers let the compiler see that no
// read need wait for the copies in flight; all copies and products go through this call.
template <class C, bool GROUPED>
__device__ __forceinline__ void wgrad_step(uint8_t* __restrict__ next, uint8_t* __restrict__ next_s,
                                           const uint8_t* __restrict__ cur, const float* __restrict__ sc,
                                           const int32_t* __restrict__ idx, const Batch& b, bool issue, bool compute, const int (&p_at)[C::NI],
                                           const int (&q_at)[C::NK], v16f (&acc)[C::NI][C::NK]) {
  constexpr int BN = C::BN, BK = C::BK;
  if (issue) {
    copy_rows<BN, GROUPED>(next, b.p, b.n, b.left, b.n0, idx, b.g, b.wave, b.lane);
    copy_rows<BK, GROUPED>(next + kDeep * BN, b.q, b.k, b.left, b.k0, idx, b.g, b.wave, b.lane);
    if (b.has_column) copy_column(next_s, b.s, b.ld_s, b.left_s, b.col_s, b.lane);
  }
  if (!compute) return;
  // 16 rows at a time: the next 16 are read and converted between the MFMAs of these
  constexpr int S = kDeep / 16, F = C::NI + C::NK, M = C::NI * C::NK;
  v2i raw[2][F];
  v4f s0[2], s1[2];
  v8b op[2][F];
  auto read = [&](int f, int r) {
    return f < C::NI ? __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(cur + p_at[f < C::NI ? f : 0] + r * BN))
                     : __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i*)(cur + q_at[f < C::NI ? 0 : f - C::NI] + r * BK));
  };
  auto convert = [&](int f, int s) {
    return f < C::NI ? scaled_bf16<C::FP>(raw[s & 1][f], s0[s & 1], s1[s & 1]) : plain_bf16<C::FQ>(raw[s & 1][f]);
  };
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int f = 0; f < F; ++f) raw[s][f] = read(f, 16 * s);
    s0[s] = *(const v4f*)(sc + 16 * s);
    s1[s] = *(const v4f*)(sc + 16 * s + 4);
  }
#pragma unroll
  for (int f = 0; f < F; ++f) op[0][f] = convert(f, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int s = 0; s < S; ++s) {
#pragma unroll
    for (int m = 0; m < (M > F ? M : F); ++m) {
      if (m < M) {
        const int i = m % C::NI, k = m / C::NI;
        acc[i][k] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(op[s & 1][C::NI + k], op[s & 1][i], acc[i][k], 0, 0, 0);
      }
      if (m < F && s + 1 < S) op[(s + 1) & 1][m] = convert(m, s + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (s + 2 < S) {
#pragma unroll
      for (int f = 0; f < F; ++f) raw[s & 1][f] = read(f, 16 * (s + 2));
      s0[s & 1] = *(const v4f*)(sc + 16 * (s + 2));
      s1[s & 1] = *(const v4f*)(sc + 16 * (s + 2) + 4);
    }
  }
}

template <class C, bool GROUPED>
__global__ void __launch_bounds__(512) wgrad_kernel(WgradArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  constexpr int BN = C::BN, BK = C::BK;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int tiles_n = (a.N + BN - 1) / BN, tiles_k = (a.K + BK - 1) / BK;
  const int nbn = a.N / kBlockK, nbk = a.K / kBlockK;
  // A group's consecutive tiles run on one XCD (workgroups go round them), in bands of four rows
  // of tiles, so that they read the same columns through its L2; every XCD has its share of each
  // group, whose rows may be many or few.
  const unsigned per = (unsigned)tiles_n * tiles_k;
  const unsigned gs = blockIdx.x / per;
  unsigned id = blockIdx.x - gs * per;
  if (per % 8 == 0) id = (id % 8) * (per / 8) + id / 8;
  const unsigned band = id / (4u * tiles_k), in_band = id - band * 4u * tiles_k;
  const unsigned high = min(4u, (unsigned)tiles_n - band * 4u);
  const int n0 = (int)(band * 4 + in_band % high) * BN, k0 = (int)(in_band / high) * BK;
  const int g = (int)(gs % (unsigned)a.G), split = (int)(gs / (unsigned)a.G);
  const int nblocks = (int)((a.T + kAlignM - 1) / kAlignM);

  Blocks<GROUPED> blocks;
  blocks.idx = a.group_idx;
  blocks.g = g;
  blocks.lane = lane;
  blocks.end = nblocks;
  blocks.step = a.splits;
  blocks.skip = split;
  blocks.b = GROUPED ? 0 : split;
  if (GROUPED && nblocks > 0)
    blocks.look();
  else
    blocks.mask[0] = blocks.mask[1] = blocks.mask[2] = blocks.mask[3] = 0;
  // First row of the next step, or -1: a block is two steps, the second unless it is empty.
  int64_t block_row = -1;
  auto next_step = [&]() -> int64_t {
    if (block_row >= 0 && block_row % kAlignM == 0 && block_row + kDeep < a.T) {
      block_row += kDeep;
      return block_row;
    }
    const int b = blocks.next();
    block_row = b < 0 ? -1 : (int64_t)b * kAlignM;
    return block_row;
  };
  // this wave's column, if it has one: of the scales (P's, then Q's), then the group indices
  const bool has_scales = wave < C::KINDS, of_q = wave >= C::NB, has_idx = GROUPED && wave == C::KINDS;
  const int ld_s = has_idx ? 1 : of_q ? nbk : nbn;
  const int col_s = has_idx ? 0 : of_q ? k0 / kBlockK + wave - C::NB : n0 / kBlockK + wave;
  const uint8_t* column = (const uint8_t*)(has_idx ? (const void*)a.group_idx : of_q ? a.sQ : a.sP);

  const int wn = wave & 3, wk = wave >> 2;
  const int wave_scale = (wn * C::NI * 32 / kBlockK) * C::KB + (wk * C::NK * 32 / kBlockK);
  // a lane's part of a transposing read: 8 bytes of row 8 (lane / 32) + (lane % 16) / 2
  const int half = lane >> 5, j = lane & 15, fr = 8 * half + (j >> 1), fb = ((lane >> 4) & 1) * 16 + (j & 1) * 8;
  int p_at[C::NI], q_at[C::NK];
#pragma unroll
  for (int i = 0; i < C::NI; ++i) p_at[i] = fr * BN + (((wn * C::NI + i) ^ piece_of(BN, fr)) << 5) + fb;
#pragma unroll
  for (int k = 0; k < C::NK; ++k)
    q_at[k] = kDeep * BN + fr * BK + (((wk * C::NK + k) ^ piece_of(BK, fr)) << 5) + fb;

  v16f acc[C::NI][C::NK];
#pragma unroll
  for (int i = 0; i < C::NI; ++i)
#pragma unroll
    for (int k = 0; k < C::NK; ++k)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][k][e] = 0.0f;

  // Batch x: the codes of step x, the scales of step x + 1 and the indices of step x + 3 (whose
  // codes are copied when batch x has landed); pos[i]: first row of step x + i, or -1.
  constexpr int AHEAD = kStages - 1;
  int64_t pos[AHEAD + 1];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) pos[i] = i == 0 || pos[i > 0 ? i - 1 : 0] >= 0 ? next_step() : -1;
  Batch bt;
  bt.n = a.N;
  bt.k = a.K;
  bt.n0 = n0;
  bt.k0 = k0;
  bt.ld_s = ld_s;
  bt.col_s = col_s;
  bt.g = g;
  bt.wave = wave;
  bt.lane = lane;
  bt.has_column = has_scales || has_idx;
  if (has_scales && pos[0] >= 0)
    copy_column(smem + C::S_OFF + wave * kDeep * 4, column + pos[0] * ld_s * 4, ld_s, a.T - pos[0], col_s, lane);
  if (GROUPED) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (has_idx && pos[i] >= 0)
        copy_column(smem + C::R_OFF + i * kDeep * 4, column + pos[i] * 4, 1, a.T - pos[i], 0, lane);
    wait_vmcnt<0>();
    step_barrier();
  }
  int issued = 0;
  for (int step = 1 - kStages; step < 0 || step < issued; ++step) {
    if (step >= -1) {
      // batch `step` has landed (step -1: the first scales)
      const int ahead = step < 0 ? issued : issued - step - 1;
      if (bt.has_column)
        wait_batches<C::PC + C::QC + 1>(ahead);
      else
        wait_batches<C::PC + C::QC>(ahead);
      step_barrier();                                    // and the step before has been read
      if (t < C::NB * C::KB * kDeep) {
        // products of both scales of the next step's rows, zero for rows of other groups (whose
        // codes come as zeros)
        const int ring = (step + 1) & (C::RING - 1);
        const float* s = (const float*)(smem + C::S_OFF) + ring * C::KINDS * kDeep + lane;
        const bool counts = !GROUPED || ((const int32_t*)(smem + C::R_OFF))[ring * kDeep + lane] == g;
        ((float*)(smem + C::M_OFF))[(((step + 1) & 1) * C::NB * C::KB + wave) * kDeep + lane] =
            counts ? s[wave / C::KB * kDeep] * s[(C::NB + wave % C::KB) * kDeep] : 0.0f;
      }
    }
    const bool issue = pos[0] >= 0;
    const int st = issued % kStages, ring = issued & (C::RING - 1);
    int later = 0;                                       // the column's step
    if (issue) {
      pos[AHEAD] = pos[AHEAD - 1] >= 0 ? next_step() : -1;
      bt.p = a.P + pos[0] * a.N;
      bt.q = a.Q + pos[0] * a.K;
      bt.left = a.T - pos[0];
      const int64_t at = has_idx ? pos[AHEAD] : pos[1];
      later = (issued + (has_idx ? AHEAD : 1)) & (C::RING - 1);
      bt.s = column + (at < 0 ? 0 : at) * ld_s * 4;
      bt.left_s = at < 0 ? 0 : a.T - at;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) pos[i] = pos[i + 1];
      ++issued;
    }
    wgrad_step<C, GROUPED>(
        smem + st * C::STAGE,
        smem + (has_idx ? C::R_OFF + later * kDeep * 4 : C::S_OFF + (later * C::KINDS + wave) * kDeep * 4),
        smem + (step & (kStages - 1)) * C::STAGE,
        (const float*)(smem + C::M_OFF) + ((step & 1) * C::NB * C::KB + wave_scale) * kDeep + 8 * half,
        (const int32_t*)(smem + C::R_OFF) + ring * kDeep, bt, issue, step >= 0, p_at, q_at, acc);
  }

  // lane l has column n = l % 32 and k = 8 e + 4 (l / 32) .. + 3 of e = 0 .. 3; a swap between the
  // lane halves gives it 8 consecutive k of e = 2 j + l / 32
#pragma unroll
  for (int i = 0; i < C::NI; ++i) {
    const int64_t n = n0 + 32 * (wn * C::NI + i) + (lane & 31);
#pragma unroll
    for (int k = 0; k < C::NK; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i][k][8 * j + c]),
                                                          __float_as_uint(acc[i][k][8 * j + 4 + c]), false, false);
          v[c] = __uint_as_float(s[0]);
          v[4 + c] = __uint_as_float(s[1]);
        }
        const int col = k0 + 32 * (wk * C::NK + k) + 16 * j + 8 * half;
        if (n >= a.N || col >= a.K) continue;
        const int64_t at = ((int64_t)g * a.N + n) * a.K + col;
        const v4f lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        if (a.splits > 1) {
          v4f* w = (v4f*)(a.partial + (int64_t)split * a.G * a.N * a.K + at);
          w[0] = lo;
          w[1] = hi;
        } else {
          put8(a, at, lo, hi);
        }
      }
  }
}

// The parts of a gradient added up, in order.
__global__ void __launch_bounds__(256) wgrad_sum_kernel(WgradArgs a, int64_t n8) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n8) return;
  const v4f* s = (const v4f*)a.partial + 2 * i;
  v4f lo = s[0], hi = s[1];
  for (int k = 1; k < a.splits; ++k) {
    s += 2 * n8;
    lo += s[0];
    hi += s[1];
  }
  put8(a, 8 * i, lo, hi);
}

template <class C>
void launch_tiles(const WgradArgs& a, hipStream_t stream) {
  const int64_t grid = (int64_t)((a.N + C::BN - 1) / C::BN) * ((a.K + C::BK - 1) / C::BK) * a.G * a.splits;
  if (a.group_idx)
    hipLaunchKernelGGL((wgrad_kernel<C, true>), dim3((unsigned)grid), dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((wgrad_kernel<C, false>), dim3((unsigned)grid), dim3(512), 0, stream, a);
}

template <int FP, int FQ>
void launch(const WgradArgs& a, hipStream_t stream) {
  if (a.big)
    launch_tiles<WgradCfg<256, 256, FP, FQ>>(a, stream);
  else
    launch_tiles<WgradCfg<128, 128, FP, FQ>>(a, stream);
}

}  // namespace

// Tiles of 256 x 256 (a code is converted for 4 or 2 waves' products of 64 x 128) where there are
// more than 128 of them, else of 128 x 128, which then all run at once, two a CU: 2048 rows by
// (4096, 4096), 256 tiles, 76 us against 109; by (4096, 2048), 128 tiles, 58 against 56; by (2048, 2048)
// 50 against 38.  Of groups one may have most of the rows, whose tiles then go on alone: more
// than 64 tiles a group, too (8192 rows, half of them one's, of 8 groups (4096, 2048) 173 us against
// 240, (2048, 2048) 120 against 124, (2048, 1024) 117 against 75).  Of few tiles each group's rows are
// dealt out among workgroups until the GPU has one a CU, eight blocks of 128 rows each at least if
// they are one group's: 8192 rows by (256, 256) 24 us, 249 by one workgroup a tile.
WgradPlan wgrad_plan(int64_t T, int64_t N, int64_t K, int64_t G) {
  WgradPlan p;
  const int64_t big = (N + 255) / 256 * ((K + 255) / 256);
  p.big = big > 64 && big * G > 128;
  const int64_t tiles = (p.big ? big : (N / kBlockK) * (K / kBlockK)) * G;
  const int64_t blocks = (T + kBlockK - 1) / kBlockK;
  int64_t s = tiles > 0 ? 256 / tiles : 1;
  if (s > blocks / 8) s = blocks / 8;
  p.splits = s < 1 ? 1 : (int)s;
  return p;
}

void launch_wgrad(const WgradArgs& a, hipStream_t stream) {
  if (a.p_fmt == kFmtE4M3)
    a.q_fmt == kFmtE4M3 ? launch<0, 0>(a, stream) : launch<0, 1>(a, stream);
  else
    a.q_fmt == kFmtE4M3 ? launch<1, 0>(a, stream) : launch<1, 1>(a, stream);
  if (a.splits > 1) {
    const int64_t n8 = (int64_t)a.G * a.N * a.K / 8;
    hipLaunchKernelGGL(wgrad_sum_kernel, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0, stream, a, n8);
  }
}

}  // namespace dg
