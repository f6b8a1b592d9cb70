// dg_kernels.hip -- FP8 (e4m3fn) block-scaled NT GEMM kernels for gfx950 (CDNA4): the tiled
// kernel over the machinery of dg_tile.h, the stream-K kernel for short wide problems, and
// the table of instances.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dg_internal.h"
#include "dg_tile.h"

namespace dg {
namespace {

// Split-K partials are stored bit-inverted, so that an all-zero word marks a slot not
// yet written (the workspace's partial slots start zero filled and every call leaves
// them so).  The only value whose inverse is zero, the NaN with every bit set, is first
// replaced by another NaN.
__device__ __forceinline__ v4i encode_partial(v4f v) {
  v4i u = __builtin_bit_cast(v4i, v);
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = ~(u[e] == -1 ? (int)0xFFC00000u : u[e]);
  return u;
}
__device__ __forceinline__ v4f decode_partial(v4i u) { return __builtin_bit_cast(v4f, ~u); }

// Cache policy of loads that poll for another workgroup's partials: sc1 (device
// coherent) plus the intrinsic's volatile bit, so that each poll stays inside its loop.
constexpr int kPollAux = (int)0x80000010u;

// One K-block step: start the copy of a later block into `next`, then multiply the block
// staged in `cur`.  The two stage pointers are restrict-qualified so that the compiler
// knows the reads of `cur` cannot see the copy into `next` and does not wait for it;
// every copy and every read of the K loop goes through this one call site (the
// prologue too), so they all carry the same pair of alias scopes.
template <class C>
__device__ __forceinline__ void kb_step(uint8_t* __restrict__ next, const uint8_t* __restrict__ cur,
                                        const TileCtx& cn, bool issue, int kb_next,
                                        const TileCtx& cc, bool compute,
                                        v4f (&acc)[C::TI][C::TJ]) {
  if (issue) issue_stage<C>(next, cn, kb_next);
  if (compute) compute_stage<C>(cur, cc, acc);
}

// bf16 (round-to-nearest-even) store of one wave's accumulator sub-tiles; rows at or past
// `rows` and columns at or past N are not written.
template <class C>
__device__ __forceinline__ void store_tile_bf16(const v4f (&acc)[C::TI][C::TJ], uint16_t* C_out,
                                                int N, int row0, int rows, int n0, int wm, int wn,
                                                int q, int l16) {
#pragma unroll
  for (int i = 0; i < C::TI; ++i) {
    const int ml = wm * C::WM + 16 * i + l16;
    if (ml >= rows) continue;
    uint16_t* crow = C_out + (size_t)(row0 + ml) * N;
#pragma unroll
    for (int j = 0; j < C::TJ; ++j) {
      const int n = n0 + wn * C::WN + 16 * j + 4 * q;
      const v4f v = acc[i][j];
      if (((N & 3) == 0) && n + 3 < N) {
        const uint32_t lo = bf16x2_rne(v[0], v[1]);
        const uint32_t hi = bf16x2_rne(v[2], v[3]);
        *(uint2*)(crow + n) = make_uint2(lo, hi);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < N) crow[n + e] = bf16_rne(v[e]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------
// Stream-K kernel for short, wide problems (dense, all rows in one tile: the decode
// shapes).  The (column tile, K block) iterations, tile-major, are split evenly over the
// persistent grid, so every CU streams the same share of B whatever the shape, and one
// load pipeline runs through a workgroup's whole range, across tile boundaries.
// A tile whose K blocks all fall in one workgroup's range is stored as bf16 directly.
// A tile shared by n workgroups (its contributors, consecutive in workgroup order) is
// reduced deterministically with no waiting: each contributor stores its fp32 partial in
// fragment order (one contiguous 1 KB block per 16x16 sub-tile) with device-coherent
// (sc1) stores and, once they are complete, adds one to the tile's arrival counter (a
// device-scope atomic); the contributor that finds n-1 there is the last, resets the
// counter to zero and sums the n partials in workgroup order, then stores bf16.  No
// workgroup ever waits for another, so the result does not depend on which workgroups
// run at the same time.  A workgroup holds at most two shared tiles: the first and the
// last of its range.
// Reduction of a shared stream-K tile, spread over its contributors, none of which
// depends on another making progress.  The tile's fragments are split into P parts
// (fragment f of wave w is in part (w*TI*TJ + f) % P, P = min(reducers, fragments, 32),
// the reducers being the contributors whose range ends inside the tile), and
// contributor c < P reduces part c: it polls the contributors' slots for the part
// (their stores are the signal: a written word is never zero), boundedly, sums them in
// workgroup order, stores bf16 and zeroes the slots.  Every contributor then counts its
// arrival at the tile, with the bit of the part it completed, in one 64-bit atomic add on
// the tile's record (arrivals in the high word, completed parts in the low).  The last to
// arrive knows that every partial is stored and that nobody touches the record again:
// it reduces the parts nobody completed (a contributor whose wait ran out leaves its part
// to it) and clears the record.  Each part is summed in the same order whoever reduces
// it.  All of this runs per wave: the fragments of wave w of every contributor form
// their own reduction with their own record, so the waves of a workgroup never wait for
// one another (a wave with no fragment in its part has completed it at once).
//
// This wave's fragments of the parts in `mask`, FCH fragments at a time, their partials
// from CB contributors per batch of loads in flight (polled until every word is written,
// at most `polls` times; slots past the buffer or of no fragment read zeros without
// touching memory and count as written), summed in workgroup order and stored as bf16
// (rows at or past `rows`, columns at or past N are not written).  With ZERO the slots
// are zeroed instead.  Returns false if a poll ran out (nothing is zeroed then).
template <class C, bool ZERO>
__device__ __forceinline__ bool reduce_parts(int mask, int P, int n, int g_first, int first_slot,
                                             __amdgpu_buffer_rsrc_t part_rsrc,
                                             const GemmArgs& p, int row0, int rows, int n0,
                                             int wave, int wm, int wn, int lane, int polls) {
  constexpr int NF = C::TI * C::TJ;
  constexpr int FCH = NF < 2 ? NF : 2;         // 16 loads in flight per poll
  constexpr int CB = 8;
  constexpr int WAVE_SLOT = NF * 64 * 4;                   // floats of one wave's partial
  constexpr int kPastBuffer = 0x7FFFFF00;
  const int l16 = lane & 15, q = lane >> 4;
  int f = 0;
#pragma unroll 1
  for (;;) {
    int fl[FCH];                                          // the chunk's fragments, or -1
#pragma unroll
    for (int k = 0; k < FCH; ++k) {
      while (f < NF && !((mask >> ((wave * NF + f) % P)) & 1)) ++f;
      fl[k] = f < NF ? f : -1;
      f = f < NF ? f + 1 : f;
    }
    if (fl[0] < 0) break;
    v4f sum[FCH];
#pragma unroll
    for (int k = 0; k < FCH; ++k) sum[k] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += CB) {
      // a contributor's slot for this tile: 0 if its range starts inside the tile (the
      // tile is its first), else 1 (the tile is its last): only the first contributor's
      // range can start before the tile
      int off[CB][FCH];
#pragma unroll
      for (int u = 0; u < CB; ++u) {
        const int gg = g_first + c0 + u;
        const int slot = c0 + u == 0 ? first_slot : 0;
        const int base = ((gg * 2 + slot) * C::W + wave) * WAVE_SLOT * 4;
#pragma unroll
        for (int k = 0; k < FCH; ++k) {
          off[u][k] = c0 + u < n && fl[k] >= 0 ? base + (fl[k] * 64 + lane) * 16 : kPastBuffer;
        }
      }
      if constexpr (ZERO) {
#pragma unroll
        for (int u = 0; u < CB; ++u)
#pragma unroll
          for (int k = 0; k < FCH; ++k)
            if (off[u][k] != kPastBuffer)
              __builtin_amdgcn_raw_buffer_store_b128((v4i){0, 0, 0, 0}, part_rsrc, off[u][k], 0,
                                                     16 /* sc1 */);
        continue;
      }
      // slots of no contributor or fragment read zeros: they count as written
      unsigned dead[CB][FCH];
#pragma unroll
      for (int u = 0; u < CB; ++u)
#pragma unroll
        for (int k = 0; k < FCH; ++k) dead[u][k] = off[u][k] == kPastBuffer ? ~0u : 0u;
      v4i raw[CB][FCH];
      bool ready = false;
#pragma unroll 1
      for (int poll = 0; poll < polls && !ready; ++poll) {
        if (poll > 0) __builtin_amdgcn_s_sleep(2);
#pragma unroll
        for (int u = 0; u < CB; ++u)
#pragma unroll
          for (int k = 0; k < FCH; ++k)
            raw[u][k] = __builtin_amdgcn_raw_buffer_load_b128(part_rsrc, off[u][k], 0, kPollAux);
        // the smallest word over all loads (unsigned; a dead slot counts as all ones) is
        // zero iff some slot is not written yet: min/max arithmetic, one compare per poll
        unsigned least = ~0u;
#pragma unroll
        for (int u = 0; u < CB; ++u)
#pragma unroll
          for (int k = 0; k < FCH; ++k) {
            const v4i r = raw[u][k];
            const unsigned m = min(min((unsigned)r.x, (unsigned)r.y), min((unsigned)r.z, (unsigned)r.w));
            least = min(least, max(m, dead[u][k]));
          }
        ready = __builtin_amdgcn_ballot_w64(least == 0) == 0;
      }
      if (!ready) return false;
#pragma unroll
      for (int u = 0; u < CB; ++u) {
        if (c0 + u >= n) break;
#pragma unroll
        for (int k = 0; k < FCH; ++k) sum[k] += decode_partial(raw[u][k]);
      }
    }
    if constexpr (!ZERO) {
#pragma unroll
      for (int k = 0; k < FCH; ++k) {
        if (fl[k] < 0) continue;
        const int fi = fl[k] / C::TJ, fj = fl[k] - fi * C::TJ;
        const int row = wm * C::WM + 16 * fi + l16;
        const int col = n0 + wn * C::WN + 16 * fj + 4 * q;
        if (row >= rows) continue;
        uint16_t* dst = p.C + (size_t)(row0 + row) * p.N;
        const v4f v = sum[k];
        if (((p.N & 3) == 0) && col + 3 < p.N) {
          *(uint2*)(dst + col) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (col + e < p.N) dst[col + e] = bf16_rne(v[e]);
        }
      }
    }
  }
  return true;
}

template <int KIND, class C>
__global__ void __launch_bounds__(C::NT)
gemm_fp8_stream_kernel(GemmArgs p) {
  constexpr int TI = C::TI, TJ = C::TJ, STAGES = C::STAGES;
  constexpr int FRAG_FLOATS = 64 * 4;                        // one 16x16 fp32 sub-tile
  constexpr int WAVE_SLOT = TI * TJ * FRAG_FLOATS;           // one wave's partial
  static_assert(C::W <= 8, "the workspace holds one arrival record per wave, 8 per tile");
  static_assert(C::XW == 0, "every wave of the stream kernel computes");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[STAGES * C::STAGE_BYTES];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int wm = wave / C::WAVES_N;
  const int wn = wave - wm * C::WAVES_N;
  const int q = lane >> 4;
  const int l16 = lane & 15;
  const int nkb = p.nkb;
  // masked form: the tiles under masked_m, counted on the device (the grid is sized for
  // the capacity, so some workgroups may get no iterations at all)
  MaskedPlan mp;
  int num_tiles = p.num_tiles;
  if (KIND == kMasked) {
    mp = masked_plan<C>(p, lane);
    num_tiles = mp.total;
  }
  const long W = (long)num_tiles * nkb;
  // the iterations are split over the first min(grid, W) workgroups, so that each of them
  // has at least one (the contributor arithmetic of the reduction relies on it); the
  // others have nothing to do
  const long G = W < (long)gridDim.x ? W : (long)gridDim.x;
  const long g = blockIdx.x;
  const long i_begin = g < G ? stream_start<C>(g, W, G) : 0;
  const long i_end = g < G ? stream_start<C>(g + 1, W, G) : 0;
  const int t_first = (int)udiv(i_begin, nkb);

  TileCtx cn, cc;
  cn.A = p.A;
  cn.sA = p.sA;
  cn.Bg = p.B;
  cn.sBg = p.sB;
  cn.K = p.K;
  cn.nkb = nkb;
  cn.nnb = p.nnb;
  cn.N = p.N;
  cn.a_row0 = 0;
  cn.rows = p.rows;
  cn.wave = wave;
  cn.cw = wave;
  cn.lane = lane;
  cn.wm = wm;
  cn.wn = wn;
  cn.q = q;
  cn.l16 = l16;
  cc = cn;

  // partial slots: two per workgroup (the first and the last tile of its range)
  __amdgpu_buffer_rsrc_t part_rsrc = __builtin_amdgcn_make_buffer_rsrc(
      p.partial, (short)0, (int)((size_t)G * 2 * C::W * WAVE_SLOT * 4), 0x00020000);

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};

  // Iteration bookkeeping with 32-bit counters only (no division in the loop): the copy
  // runs STAGES-1 iterations ahead of the math; relative iteration r lives in stage
  // r % STAGES for both.
  const int n_iter = (int)(i_end - i_begin);
  int tn = t_first, kbn = (int)(i_begin - (long)t_first * nkb), sn = 0;   // next copy
  int tc = tn, kbc = kbn, sc = 0, in_tile = 0;                              // next math
  MaskedCursor mn = {0, 0, 0}, mc = {0, 0, 0};      // masked form: the same two tiles
  if (KIND == kMasked && n_iter > 0) {
    mn = masked_seek<C>(mp, p.tiles_n, t_first);
    mc = mn;
  }
  int shared_tile[2] = {-1, -1};
  int seg_row0[2] = {0, 0}, seg_rows[2] = {0, 0}, seg_n0[2] = {0, 0};  // where they go
  for (int step = 1 - STAGES; step < n_iter; ++step) {
    if (step >= 0) {
      wait_stage_copies<C, STAGES - 2>(wave, min(STAGES - 2, n_iter - 1 - step));
      stage_barrier();
    }
    const bool issue = step + STAGES - 1 < n_iter;
    if (KIND == kMasked) {
      masked_tile<C>(p, mp, mn, cn);
      masked_tile<C>(p, mp, mc, cc);
    } else {
      cn.n0 = tn * C::BN;
      cn.nb_first = cn.n0 / kBlockK;
      cc.n0 = tc * C::BN;
      cc.nb_first = cc.n0 / kBlockK;
    }
    kb_step<C>(smem + sn * C::STAGE_BYTES, smem + sc * C::STAGE_BYTES, cn, issue, kbn, cc,
               step >= 0, acc);
    if (issue) {
      sn = sn + 1 == STAGES ? 0 : sn + 1;
      if (++kbn == nkb) {
        kbn = 0;
        ++tn;
        if (KIND == kMasked && step + STAGES < n_iter) masked_next<C>(mp, p.tiles_n, mn);
      }
    }
    if (step < 0) continue;
    sc = sc + 1 == STAGES ? 0 : sc + 1;
    ++in_tile;
    const bool tile_end = kbc == nkb - 1 || step == n_iter - 1;
    if (++kbc == nkb) kbc = 0;
    if (!tile_end) continue;

    // tile tc ends here for this workgroup
    if (in_tile == nkb) {
      store_tile_bf16<C>(acc, p.C, p.N, cc.a_row0, cc.rows, cc.n0, wm, wn, q, l16);
    } else {
      const int seg = tc == t_first ? 0 : 1;
      shared_tile[seg] = tc;
      seg_row0[seg] = cc.a_row0;
      seg_rows[seg] = cc.rows;
      seg_n0[seg] = cc.n0;
      const int base = (int)(((g * 2 + seg) * C::W + wave) * WAVE_SLOT) * 4;
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(encode_partial(acc[i][j]), part_rsrc,
                                                 base + ((i * TJ + j) * 64 + lane) * 16, 0,
                                                 16 /* sc1: device coherent */);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
    ++tc;
    if (KIND == kMasked && step < n_iter - 1) masked_next<C>(mp, p.tiles_n, mc);
    in_tile = 0;
  }

  // ---- hand-off of the shared tiles (see reduce_parts), wave by wave: the waves of a
  // workgroup never wait for one another and touch no LDS here.  Jobs 0 and 1: this
  // wave's own part of the last and the first shared tile; then its arrival at both;
  // jobs 2 and 3: the parts nobody completed, where this wave arrived last.
  if (shared_tile[0] < 0 && shared_tile[1] < 0) return;
  // per shared tile, once: first contributor, contributors, parts, this workgroup's
  // index among the contributors, and the first contributor's slot
  int gfv[2], nv[2], pv[2], cv[2], fsv[2];
#pragma unroll
  for (int sg = 0; sg < 2; ++sg) {
    const long x0 = (long)(shared_tile[sg] < 0 ? 0 : shared_tile[sg]) * nkb, x1 = x0 + nkb - 1;
    const long gf = udiv((x0 + 1) * G + W - 1, W) - 1;
    const long gl = udiv((x1 + 1) * G + W - 1, W) - 1;
    // the parts go to the contributors whose range ends inside the tile: the last
    // contributor's range usually goes on into the next tiles (the tile is its first,
    // stored long before), so it takes a part only when its range ends with the tile
    const int nr = (int)(gl - gf) + (stream_start<C>(gl + 1, W, G) == x1 + 1 ? 1 : 0);
    gfv[sg] = (int)gf;
    nv[sg] = (int)(gl - gf + 1);
    pv[sg] = min(nr, min(C::W * TI * TJ, 32));
    cv[sg] = (int)(g - gf);
    fsv[sg] = stream_start<C>(gf, W, G) < x0 ? 1 : 0;
  }
  bool polled = false;
  int okmask = 0, left0 = 0, left1 = 0;
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    if (k == 2) {
      // this wave's partial stores are complete before its arrival is counted: a wave
      // that polled has used loads issued after them (vmcnt retires in issue order); with
      // a zero poll bound nothing was loaded
      if (!polled || p.helper_polls == 0) wait_vmcnt<0>();
      unsigned long long before[2] = {0ull, 0ull};
#pragma unroll
      for (int sg = 0; sg < 2; ++sg) {
        const unsigned long long mine =
            (1ull << 32) | ((okmask >> sg) & 1 ? 1ull << cv[sg] : 0ull);
        if (lane == 0 && shared_tile[sg] >= 0)
          before[sg] = __hip_atomic_fetch_add(
              (unsigned long long*)p.arrivals + gfv[sg] * C::W + wave, mine, __ATOMIC_RELAXED,
              __HIP_MEMORY_SCOPE_AGENT);
      }
#pragma unroll
      for (int sg = 0; sg < 2; ++sg) {
        if (shared_tile[sg] < 0) continue;
        const int hi = __builtin_amdgcn_readlane((int)(before[sg] >> 32), 0);
        const int lo = __builtin_amdgcn_readlane((int)before[sg], 0);
        if (hi == nv[sg] - 1) {                 // the last to arrive
          const int mine_done = (okmask >> sg) & 1 ? 1 << cv[sg] : 0;
          // every part (P can be 32: no 1 << 32 on a 32-bit int)
          const unsigned all = pv[sg] >= 32 ? ~0u : (1u << pv[sg]) - 1u;
          const int left = (int)(all & ~(unsigned)(lo | mine_done));
          if (sg) left1 = left; else left0 = left;
          if (lane == 0)
            __hip_atomic_store((unsigned long long*)p.arrivals + gfv[sg] * C::W + wave, 0ull,
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
    }
    const int sg = (k & 1) ^ 1;              // the last shared tile first
    if ((sg ? shared_tile[1] : shared_tile[0]) < 0) continue;
    const int P = sg ? pv[1] : pv[0], c = sg ? cv[1] : cv[0];
    const int mask = k < 2 ? (c < P ? 1 << c : 0) : (sg ? left1 : left0);
    if (!mask) continue;
    polled = polled || k < 2;
    const int n = sg ? nv[1] : nv[0], gf = sg ? gfv[1] : gfv[0], fs = sg ? fsv[1] : fsv[0];
    const int row0 = sg ? seg_row0[1] : seg_row0[0];
    const int rows = sg ? seg_rows[1] : seg_rows[0];
    const int n0 = sg ? seg_n0[1] : seg_n0[0];
    // an owner polls at most helper_polls times; the last arrival's partials are all
    // stored, so its leftover parts never wait
    if (reduce_parts<C, false>(mask, P, n, gf, fs, part_rsrc, p, row0, rows, n0, wave, wm, wn,
                               lane, k < 2 ? p.helper_polls : kHelperPolls)) {
      reduce_parts<C, true>(mask, P, n, gf, fs, part_rsrc, p, 0, 0, 0, wave, wm, wn, lane, 0);
      if (k < 2) okmask |= 1 << sg;
    }
  }
}

template <int KIND, class C>
void launch_stream(const GemmArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_fp8_stream_kernel<KIND, C>), dim3(grid), dim3(C::NT), 0, stream, a);
}

// persistent stream grid: one workgroup per CU (at most kStreamGrid); dense calls follow
// stream_grid (128x24576x1536 on 192 workgroups shares no tile: 24.5 -> 21.8 us;
// 128x2112x7168 on 231: 14.9 -> 13.1 us); the masked form's tiles are counted on the
// device, so its grid covers the capacity
int grid_stream(const GemmArgs& a, int num_cus) {
  const long g = num_cus < kStreamGrid ? num_cus : kStreamGrid;
  if (a.masked_m) {
    const long work = (long)a.num_tiles * a.nkb;
    return (int)(work < g ? work : g);
  }
  return (int)stream_grid(a.num_tiles, a.nkb, g);
}

template <int KIND, class C>
void launch(const GemmArgs& a, int grid, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_fp8_kernel<KIND, C>), dim3(grid), dim3(C::NT), 0, stream, a);
}

// persistent grid: one workgroup per CU (the LDS budget allows no more), capped by work
int grid_persistent(const GemmArgs& a, int num_cus) {
  return a.num_tiles < num_cus ? a.num_tiles : num_cus;
}

// Tile shapes, each built for the four operand-format pairs (FA, FB).
template <int FA, int FB> using Big = Cfg<256, 256, 4, 2, 2, false, FA, FB, 4>;     // 8 waves, 64x128 each
template <int FA, int FB> using Big224 = Cfg<256, 224, 4, 2, 2, false, FA, FB, 4>;  // non-power-of-two N tile
template <int FA, int FB> using Big160 = Cfg<256, 160, 4, 2, 2, false, FA, FB, 4>;  // for N near 2048
// the contiguous form keeps more per-tile state: its 256x224 tile has no registers to
// spare for the copy waves' doubled copy set, so all of its waves copy.  Its 256x256
// tile prefetches into the L2 two K blocks ahead of the copies (K = 7168: 3-4% faster;
// the dense tiles ran 1-5% slower with it, their L2 hit rate being higher)
template <int FA, int FB> using BigC = Cfg<256, 256, 4, 2, 2, false, FA, FB, 4, 2>;
template <int FA, int FB> using Big224C = Cfg<256, 224, 4, 2, 2, false, FA, FB>;
template <int FA, int FB> using Mid = Cfg<128, 128, 2, 2, 3, false, FA, FB>;     // 4 waves, 64x64 each
// the same with four copy-only waves (register epilogue forms: dense and masked)
template <int FA, int FB> using MidS = Cfg<128, 128, 2, 2, 3, false, FA, FB, 0, 0, 4>;
template <int FA, int FB> using Small = Cfg<64, 128, 1, 4, 4, false, FA, FB>;    // 4 waves, 64x32 each
// stream-K decode instances: 8 waves (a wave's direct-to-LDS copies are issue-bound, so
// a workgroup needs eight of them to draw its share of HBM bandwidth), B non-temporal
template <int FA, int FB> using Str64 = Cfg<64, 128, 2, 4, 5, true, FA, FB>;     // 64 rows x 128 columns
template <int FA, int FB> using Str64n64 = Cfg<64, 64, 2, 4, 8, true, FA, FB>;   // 64 rows x 64 columns
template <int FA, int FB> using Str128 = Cfg<128, 128, 2, 4, 4, true, FA, FB>;   // 128 rows x 128 columns
template <int FA, int FB> using Str128n64 = Cfg<128, 64, 2, 4, 6, true, FA, FB>; // 128 rows x 64 columns
// 4-wave builds of the 128-column tiles (one wave per SIMD; per K block 64 KB of fragment
// reads from LDS instead of 96, 48 instead of 64) for ranges of 16 K blocks or more per
// workgroup: 128x7168x16384 44.0 -> 39.7 us, 64x7168x16384 34.0 -> 33.3 us; on shorter
// ranges they lose 2-7%
template <int FA, int FB> using Str128w4 = Cfg<128, 128, 2, 2, 4, true, FA, FB>;  // 64x64 per wave
template <int FA, int FB> using Str64w4 = Cfg<64, 128, 2, 2, 5, true, FA, FB>;    // 32x64 per wave

}  // namespace

#define DG_INST1(NAME, KIND, C, FA, FB)                                                   \
  Instance { NAME, KIND, C::BM, C::BN, kModeTiled, C::NT, FA, FB, grid_persistent,        \
             launch<KIND, C> }
#define DG_STREAM1(NAME, KIND, C, FA, FB)                                                  \
  Instance { NAME, KIND, C::BM, C::BN, kModeStream, C::NT, FA, FB, grid_stream,           \
             launch_stream<KIND, C> }
#define DG_INST(NAME, KIND, T)                                                             \
  DG_INST1(NAME, KIND, T<0 COMMA 0>, 0, 0), DG_INST1(NAME, KIND, T<1 COMMA 1>, 1, 1),      \
      DG_INST1(NAME, KIND, T<0 COMMA 1>, 0, 1), DG_INST1(NAME, KIND, T<1 COMMA 0>, 1, 0)
#define DG_STREAM(NAME, KIND, T)                                                           \
  DG_STREAM1(NAME, KIND, T<0 COMMA 0>, 0, 0), DG_STREAM1(NAME, KIND, T<1 COMMA 1>, 1, 1),  \
      DG_STREAM1(NAME, KIND, T<0 COMMA 1>, 0, 1), DG_STREAM1(NAME, KIND, T<1 COMMA 0>, 1, 0)
#define COMMA ,

static const Instance kInstances[] = {
    DG_INST("dense_256x256", kDense, Big),
    DG_INST("dense_256x224", kDense, Big224),
    DG_INST("dense_256x160", kDense, Big160),
    DG_INST("dense_128x128", kDense, MidS),
    DG_STREAM("dense_64x128_stream", kDense, Str64),
    DG_STREAM("dense_64x64_stream", kDense, Str64n64),
    DG_STREAM("dense_128x128_stream", kDense, Str128),
    DG_STREAM("dense_128x64_stream", kDense, Str128n64),
    DG_STREAM("dense_128x128_stream_4w", kDense, Str128w4),
    DG_STREAM("dense_64x128_stream_4w", kDense, Str64w4),
    DG_INST("contig_256x256", kContiguous, BigC),
    DG_INST("contig_256x224", kContiguous, Big224C),
    DG_INST("contig_128x128", kContiguous, Mid),
    DG_INST("masked_256x256", kMasked, Big),
    DG_INST("masked_128x128", kMasked, MidS),
    DG_INST("masked_64x128", kMasked, Small),
    DG_STREAM("masked_128x128_stream", kMasked, Str128),
    DG_STREAM("masked_128x64_stream", kMasked, Str128n64),
};

const Instance* instances(int* count) {
  *count = (int)(sizeof(kInstances) / sizeof(kInstances[0]));
  return kInstances;
}

}  // namespace dg
