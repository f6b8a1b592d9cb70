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

constexpr int kTile = 16;                 // rows of an MFMA tile
constexpr int kDownWaves = 8;
constexpr int kUpWaves = 4;

__device__ __forceinline__ f32x4 mfma(const uint4& a, const uint4& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float from_bf16(uint32_t b) { return __uint_as_float(b << 16); }

// Two fp32 numbers rounded to bf16 (to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

// Eight bf16 numbers at any element: one 16-byte access (the hardware takes those at any
// address).
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ void store8(uint16_t* p, const uint4& v, bool past_caches) {
  using u32x4 = __attribute__((ext_vector_type(4), aligned(2))) uint32_t;
  if (past_caches) __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, (u32x4*)p);
  else __builtin_memcpy(p, &v, 16);
}

// Lanes eight apart trade: the lower one's y for the upper one's x.  Its own inverse.
__device__ __forceinline__ void trade(uint4& x, uint4& y, bool upper) {
  uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int got = __builtin_amdgcn_mov_dpp((int)(upper ? a[i] : b[i]), 0x128, 0xF, 0xF, true);
    a[i] = upper ? (uint32_t)got : a[i];
    b[i] = upper ? b[i] : (uint32_t)got;
  }
  x = make_uint4(a[0], a[1], a[2], a[3]);
  y = make_uint4(b[0], b[1], b[2], b[3]);
}

// A number as the sum of two bf16 numbers, itself rounded (low half) and the rest rounded.
__device__ __forceinline__ uint32_t split_bf16(float v) {
  const uint32_t hi = pack_bf16(v, 0.0f) & 0xFFFFu;
  // the rest of an infinity (NaN) becomes a number that does not matter beside it
  const float rest = __builtin_amdgcn_fmed3f(v - from_bf16(hi), -0x1p120f, 0x1p120f);
  return hi | (pack_bf16(0.0f, rest) & 0xFFFF0000u);
}

// The adapters that M <= 64 rows from t0 name: lane l holds the id of row l % M (-1: none).
// Of Q workgroups (a power of two) on the same rows the q-th has those with id = q modulo Q
// if there are many, and q = 0 all of them where the rows are one or two runs.  next() gives
// its adapters one by one, in the order of their first rows, with the rows that are theirs.
template <int M>
struct TileAdapters {
  static constexpr uint64_t kRows = M == 64 ? ~0ull : (1ull << (M & 63)) - 1;
  int id;
  uint64_t own, none;      // rows of these adapters; rows without an adapter
  uint64_t left;           // rows whose adapter has not been given out
  __device__ __forceinline__ TileAdapters(const LoraArgs& a, int64_t t0, int lane, int q, int Q) {
    const int64_t t = t0 + (lane & (M - 1));
    const int i = t < a.T ? a.ids[t] : -1;
    id = i >= 0 && i < a.L ? i : -1;
    own = __builtin_amdgcn_ballot_w64(id >= 0) & kRows;
    none = __builtin_amdgcn_ballot_w64(id < 0 && t < a.T) & kRows;
    if (Q > 1) {
      const uint64_t ends = __builtin_amdgcn_ballot_w64(id != __shfl_down(id, 1, 64)) & (kRows >> 1);
      if (__builtin_popcountll(ends) <= 1) own = q == 0 ? own : 0;
      else own &= __builtin_amdgcn_ballot_w64((id & (Q - 1)) == q);
    }
    left = own;
  }
  __device__ __forceinline__ bool next(int* adapter, uint64_t* rows) {
    if (!left) return false;
    *adapter = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    *rows = __builtin_amdgcn_ballot_w64(id == *adapter) & kRows;
    left &= ~*rows;
    return true;
  }
};

__device__ __forceinline__ int rank_of(const LoraArgs& a, int adapter) {
  if (!a.ranks) return a.R;
  const int r = a.ranks[adapter];
  return r < 0 ? 0 : r < a.R ? r : a.R;
}

// nf pieces (64 deep, two instructions) of the products of NA row tiles with RT rank tiles.
// xp: this lane's row of each row tile; ap: its row of each rank tile.  A lane takes 32
// consecutive bytes of a piece, half for each instruction (x and A alike, so that the
// products pair up), and the four lane groups a 128-byte line.  U pieces are in flight
// while the ones before them are multiplied.
template <int U, int NA, int RT>
__device__ __forceinline__ void down_products(const uint16_t* const (&xp)[NA],
                                              const uint16_t* const (&ap)[RT], int nf,
                                              f32x4 (&acc)[NA][RT]) {
  uint4 x[2][U][NA][2], w[2][U][RT][2];
  // pieces past the last repeat it and are not multiplied
  auto load = [&](int b, int f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = (f + u < nf ? f + u : nf - 1) * 64;
#pragma unroll
      for (int m = 0; m < NA; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) x[b][u][m][i] = *(const uint4*)(xp[m] + at + 8 * i);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) w[b][u][r][i] = *(const uint4*)(ap[r] + at + 8 * i);
    }
  };
  auto multiply = [&](int b, int f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (f + u >= nf) break;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int m = 0; m < NA; ++m)
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[m][r] = mfma(x[b][u][m][i], w[b][u][r][i], acc[m][r]);
    }
  };
  if (nf > 0) load(0, 0);
  for (int f = 0; f < nf; f += 2 * U) {
    if (f + U < nf) load(1, f + U);
    multiply(0, f);
    if (f + 2 * U < nf) load(0, f + 2 * U);
    multiply(1, f + U);
  }
}

// The same for NA of the workgroup's MT row tiles, those with a bit in `tiles`; their sums
// are left in the leading acc.  Rows of other adapters are not read: their lanes repeat the
// item's first row.
template <int NA, int MT, int RT>
__device__ __forceinline__ void down_tiles(const LoraArgs& a, int64_t t0, uint64_t rows, uint32_t tiles,
                                           const uint16_t* const (&ap)[RT], int64_t k0, int l16, int nf,
                                           f32x4 (&acc)[MT][RT]) {
  const uint16_t* xp[NA];
  f32x4 sum[NA][RT];
  const int lead = __builtin_ctzll(rows);
#pragma unroll
  for (int m = 0; m < NA; ++m) {
    const int at = __builtin_ctz(tiles) * kTile + l16;
    tiles &= tiles - 1;
    xp[m] = a.x + (t0 + ((rows >> at) & 1 ? at : lead)) * a.ldx + k0;
#pragma unroll
    for (int r = 0; r < RT; ++r) sum[m][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  down_products<(NA + RT <= 2 ? 4 : NA + RT <= 4 ? 2 : 1)>(xp, ap, nf, sum);
#pragma unroll
  for (int m = 0; m < NA; ++m)
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[m][r] = sum[m][r];
}

// LDS cells for the sums of a workgroup's waves: all eight where that is little, else four,
// to which the other four add theirs.
template <int C>
constexpr int down_slots() { return C <= 4 ? 8 : 4; }

// Part s of h of those of the 16 MT rows from t0 that have a bit in `rows`, all of one
// adapter: the sum over the pieces [p0, p1) of K.  The workgroup's waves take an eighth of
// them each; their sums are added up in a fixed order.
template <int MT, int RT>
__device__ __forceinline__ void down_item(const LoraArgs& a, int64_t t0, uint64_t rows, int adapter, int s,
                                          int p0, int p1, float (*red)[MT * RT][kTile * 16]) {
  constexpr int W = down_slots<MT * RT>();
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int f0 = p0 + (p1 - p0) * wave / kDownWaves;
  const int nf = p0 + (p1 - p0) * (wave + 1) / kDownWaves - f0;
  const int64_t k0 = (int64_t)f0 * 64 + g * 16;
  const int rank = rank_of(a, adapter);
  const float scale = a.scales ? a.scales[adapter] : 1.0f;
  uint32_t tiles = 0;
#pragma unroll
  for (int m = 0; m < MT; ++m) tiles |= ((rows >> (m * kTile)) & 0xFFFF) ? 1u << m : 0u;
  f32x4 acc[MT][RT];
  // ranks past R repeat the last; what A holds past the adapter's rank is multiplied too (to
  // wait for the rank first costs more) and those sums are not used
  const uint16_t* ap[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int c = r * 16 + l16;
    ap[r] = a.A + ((int64_t)adapter * a.R + (c < a.R ? c : a.R - 1)) * a.K + k0;
  }
  const int na = __builtin_popcount(tiles);
  if (MT >= 4 && na > 3) down_tiles<MT >= 4 ? 4 : 1, MT, RT>(a, t0, rows, tiles, ap, k0, l16, nf, acc);
  else if (MT >= 4 && na > 2) down_tiles<MT >= 4 ? 3 : 1, MT, RT>(a, t0, rows, tiles, ap, k0, l16, nf, acc);
  else if (MT >= 2 && na > 1) down_tiles<MT >= 2 ? 2 : 1, MT, RT>(a, t0, rows, tiles, ap, k0, l16, nf, acc);
  else down_tiles<1, MT, RT>(a, t0, rows, tiles, ap, k0, l16, nf, acc);
  // acc[m][r][j]: row 4 g + j of the m-th of `tiles`, rank 16 r + l16; a cell holds its 16
  // rows rank by rank
  auto put = [&](int slot, bool add) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m >= na) break;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        f32x4* p = (f32x4*)&red[slot][m * RT + r][l16 * 16 + 4 * g];
        *p = add ? *p + acc[m][r] : acc[m][r];
      }
    }
  };
  if (W == 8) {
    put(wave, false);
  } else {
    if (wave >= 4) put(wave - 4, false);
    __syncthreads();
    if (wave < 4) put(wave, true);
  }
  __syncthreads();
  for (int i = tid; i < na * (RT * 64); i += 64 * kDownWaves) {
    // i: (row tile in `tiles`, four rows, rank), ranks fastest
    const int c = i % (RT * 16), four = i / (RT * 16), m = four / 4;
    uint32_t t = tiles;
    for (int x = 0; x < m; ++x) t &= t - 1;
    const int at = __builtin_ctz(t) * kTile + (four & 3) * 4;
    if (c >= a.R || !((rows >> at) & 15)) continue;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < rank) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        sum += *(const f32x4*)&red[w][m * RT + c / 16][(c & 15) * 16 + (four & 3) * 4];
    }
    float* h = a.h + s * a.h_part + (t0 + at) * a.R + c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((rows >> (at + j)) & 1) h[(int64_t)j * a.R] = sum[j] * scale;
  }
  __syncthreads();
}

// Of the row's lane and the lanes before it in its 16: whether an earlier one has the same id.
template <int D = 1>
__device__ __forceinline__ bool seen_before(int id) {
  if constexpr (D < kTile) {
    const int before = __builtin_amdgcn_update_dpp(-1, id, 0x110 + D, 0xF, 0xF, false);   // lane - D
    return (before == id) | seen_before<D + 1>(id);
  } else {
    return false;
  }
}

// Few rows: an item is the rows of one adapter in a tile of 16, whatever lies between them.
// Every workgroup finds the items from the ids, and the workgroups are dealt out to them
// evenly: S workgroups an item, a part of K each.  64 rows of 64 adapters of rank 16, K = 7168:
// 6.1 us, of which four are the dependent trips to memory (ids, then x and A); 128 rows,
// K = 1536, 8 adapters of ranks up to 64: 6.4.
template <int RT>
__global__ void __launch_bounds__(64 * kDownWaves, 2)
lora_down_rows_kernel(LoraArgs a) {
  __shared__ __attribute__((aligned(16))) float red[down_slots<RT>()][RT][kTile * 16];
  static_assert(kLoraFewRows <= 128, "two rows a lane");
  const int lane = threadIdx.x & 63;
  int id[2] = {-1, -1};
  uint64_t lead[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (a.T <= 64 * i) break;
    const int t = 64 * i + lane;
    id[i] = t < a.T ? a.ids[t] : -1;
    id[i] = id[i] >= 0 && id[i] < a.L ? id[i] : -1;
    lead[i] = __builtin_amdgcn_ballot_w64((id[i] >= 0) & (a.T == 1 || !seen_before(id[i])));
  }
  const uint32_t n0 = __builtin_popcountll(lead[0]), n = n0 + __builtin_popcountll(lead[1]);
  if (n == 0) return;
  // quotients of these sizes come out exact (halves are far from the next integer)
  const uint32_t most = (uint32_t)(((float)gridDim.x + 0.5f) * __builtin_amdgcn_rcpf((float)n));
  const uint32_t S = most < (uint32_t)a.S ? most : (uint32_t)a.S;
  const float per = __builtin_amdgcn_rcpf((float)S);
  const uint32_t item = (uint32_t)(((float)blockIdx.x + 0.5f) * per), s = blockIdx.x - item * S;
  if (item >= n) return;
  const bool second = item >= n0;
  const uint64_t heads = second ? lead[1] : lead[0];
  const int mine = second ? id[1] : id[0];
  const uint32_t before = __builtin_amdgcn_mbcnt_hi((uint32_t)(heads >> 32),
                                                    __builtin_amdgcn_mbcnt_lo((uint32_t)heads, 0));
  const int at = __builtin_ctzll(
      __builtin_amdgcn_ballot_w64(((heads >> lane) & 1) && before == item - (second ? n0 : 0)));
  const int adapter = __builtin_amdgcn_readlane(mine, at), tile = at & ~(kTile - 1);
  const uint64_t rows = (__builtin_amdgcn_ballot_w64(mine == adapter) >> tile) & 0xFFFF;
  const int64_t t0 = tile + (second ? 64 : 0);
  if (s == 0 && threadIdx.x < kTile && ((rows >> threadIdx.x) & 1)) a.parts[t0 + threadIdx.x] = (int)S;
  const int pieces = a.K / 64;
  const float share = (float)pieces * per;        // any rounding will do: part s ends where s + 1 begins
  down_item<1, RT>(a, t0, rows, adapter, (int)s, (int)((float)s * share),
                   s + 1 == S ? pieces : (int)((float)(s + 1) * share), red);
}

// Many rows: an item is a run of rows of one adapter within a tile of 16 MT.  Every workgroup
// counts the items for itself from the ids (64 rows a ballot), without a launch to plan it,
// and then knows its share of them:
//  - each item's K is divided alike, into as many parts as give no workgroup two, and it takes
//    its part or none;
//  - or the items' pieces of K, one item after the other, are dealt out evenly.  A piece is
//    counted as its loads, RT for the adapter's ranks and one for each tile of 16 that the run
//    touches, so the single rows of a mixed batch and the ends of prompts within a tile cost
//    what they cost.
// Dealing uses every workgroup, but a share that begins within an item costs a second item's
// start and sums.  It is done where it saves a workgroup kDealPays loads (and the items do not
// have all their parts already).  Of 139 batches (T 130 to 8192, K 512 to 16384, all ranks) none
// that saves 38 or less gained from it, but for one whose items are very uneven; of the 16 that
// save 70 or more all but three did.  Divided alike and dealt, in us, by the loads saved:
//     7  200 x 512 rank 8 mixed          15.4  19.5      71  8192 x 2048 rank 8, prompts    21.9  20.4
//    12  256 x 7168 rank 32, prompts     23.6  30.3      88  4096 x 7168 rank 32, prompts   32.7  28.9
//    20  3000 x 7168 rank 16, prompts    19.2  20.6     152  8192 x 4096 rank 8, prompts    29.9  24.1
//    36  200 x 2048 rank 64 mixed        34.0  40.5     485  4096 x 7168 rank 128, prompts  80.9  63.5
// An item's parts, at most a.S, are the workgroups that share it; their number goes to
// `parts` for each of its rows.  8192 x 16384 of rank 64: 82 us, x alone at 3.3 TB/s (a sum over
// 512 MB reads 3.9), A again from L2 for each row tile; 4096 x 2048 of rank 16: 10.0.
constexpr int kCounts = 256;              // blocks of rows, at most
constexpr float kDealPays = 64.0f;

__device__ __forceinline__ int row_id(const LoraArgs& a, int64_t t) { return t < a.T ? a.ids[t] : -1; }

// Rows at which a run within a tile of M rows begins, of 64 with these ids.
template <int M>
__device__ __forceinline__ uint64_t run_starts(const LoraArgs& a, int lane, int id) {
  const int before = __shfl_up(id, 1, 64);
  return __builtin_amdgcn_ballot_w64(id >= 0 && id < a.L && ((lane & (M - 1)) == 0 || before != id));
}

// The run that begins at row `at`: up to the end of its tile or the first row of another id.
template <int M>
__device__ __forceinline__ uint64_t run_rows(int id, int adapter, int at) {
  const int end = (at & ~(M - 1)) + M;
  const uint64_t from = ~0ull << at;
  const uint64_t stop = (__builtin_amdgcn_ballot_w64(id != adapter) | (end < 64 ? ~0ull << end : 0)) & from;
  return stop ? ((1ull << __builtin_ctzll(stop)) - 1) & from : from;
}

__device__ __forceinline__ int tiles_of(uint64_t rows) {
  int n = 0;
#pragma unroll
  for (int m = 0; m < 4; ++m) n += (rows >> (16 * m)) & 0xFFFF ? 1 : 0;
  return n;
}

template <int MT, int RT>
__global__ void __launch_bounds__(64 * kDownWaves, 2)
lora_down_kernel(LoraArgs a) {
  constexpr int M = MT * kTile, U = 8;
  __shared__ __attribute__((aligned(16))) float red[down_slots<MT * RT>()][MT * RT][kTile * 16];
  __shared__ uint32_t items[kCounts + 1], loads[kCounts + 1];   // before a block of `per` times 64 rows
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t chunks = (uint32_t)((a.T + 63) / 64);
  const uint32_t per = (chunks + kCounts - 1) / kCounts;
  const uint32_t blocks = (chunks + per - 1) / per;
  for (uint32_t b0 = wave; b0 < blocks; b0 += kDownWaves * U) {
    uint32_t n[U] = {}, w[U] = {};
    for (uint32_t c = 0; c < per; ++c) {
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        id[u] = row_id(a, (int64_t)((b0 + u * kDownWaves) * per + c) * 64 + lane);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t runs = __builtin_popcountll(run_starts<M>(a, lane, id[u]));
        n[u] += runs;
        w[u] += RT * runs + __builtin_popcountll(run_starts<kTile>(a, lane, id[u]));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (lane == 0 && b0 + u * kDownWaves < blocks) {
        items[b0 + u * kDownWaves] = n[u];
        loads[b0 + u * kDownWaves] = w[u];
      }
  }
  __syncthreads();
  if (wave < 2) {                         // sums before each block, of one array a wave
    uint32_t* v = wave ? loads : items;
    uint32_t before = 0;
    for (uint32_t b0 = 0; b0 < blocks; b0 += 64) {
      const uint32_t n = b0 + lane < blocks ? v[b0 + lane] : 0;
      uint32_t sum = n;
#pragma unroll
      for (int off = 1; off < 64; off *= 2) {
        const uint32_t up = __shfl_up(sum, off, 64);
        if (lane >= off) sum += up;
      }
      if (b0 + lane < blocks) v[b0 + lane] = before + sum - n;
      before += __shfl(sum, 63, 64);
    }
    if (lane == 0) v[blocks] = before;
  }
  __syncthreads();

  // an item is `span` units of c each, a workgroup's share `quota` of them
  const uint32_t G = gridDim.x, pieces = a.K / 64, count = items[blocks];
  if (count == 0) return;
  const uint32_t alike = G / count < (uint32_t)a.S ? G / count : a.S;
  // divided alike, a workgroup that has a part has every / busy loads; dealt, every / G
  const float busy = (float)(alike * count), every = (float)loads[blocks] * (float)pieces;
  const bool one = alike == (uint32_t)a.S || every * ((float)G - busy) < kDealPays * (float)G * busy;
  const uint32_t* first = one ? items : loads;
  const uint32_t span = one ? alike : pieces < 128 ? pieces : 128;
  const uint32_t all = first[blocks] * span;              // T <= kLoraRows: below 2^32
  uint32_t quota = 1;
  if (!one) {
    // no item has more than a.S parts, and each has a unit at least
    const uint32_t least = ((RT + MT) * span + a.S - 2) / (a.S - 1), even = (all + G - 1) / G;
    quota = even > least ? even : least;
  }
  // consecutive shares to the workgroups of one XCD (workgroups are dealt to the 8 XCDs in
  // turn), so that an adapter's A is read through one L2 or two
  const uint32_t wg = (blockIdx.x & 7) * (G / 8) + blockIdx.x / 8;
  const uint32_t u0 = wg * quota, u1 = u0 + quota < all ? u0 + quota : all;
  if (u0 >= all) return;
  int lo = -1;                            // the block that holds the first item
  const uint32_t w0 = u0 / span;
  for (uint32_t b0 = 0; b0 < blocks; b0 += 64)
    lo += __builtin_popcountll(
        __builtin_amdgcn_ballot_w64(b0 + lane < blocks && first[b0 + lane] <= w0));
  int64_t r0 = (int64_t)lo * per * 64;
  uint32_t begin = __builtin_amdgcn_readfirstlane(first[lo]) * span;   // where the item at hand begins
  for (; begin < u1; r0 += 64) {
    const int id = row_id(a, r0 + lane);
    uint64_t starts = run_starts<M>(a, lane, id);
    for (; starts && begin < u1; starts &= starts - 1) {
      const int at = __builtin_ctzll(starts), adapter = __builtin_amdgcn_readlane(id, at);
      const int tile = at & ~(M - 1);
      const uint64_t rows = run_rows<M>(id, adapter, at);
      const uint32_t c = one ? 1 : RT + tiles_of(rows);
      const uint32_t mine = begin;
      begin += c * span;
      if (begin <= u0) continue;
      const uint32_t x0 = u0 > mine ? (u0 - mine + c - 1) / c : 0, to = (u1 - mine + c - 1) / c;
      const uint32_t x1 = to < span ? to : span;
      if (x0 >= x1) continue;
      const uint32_t head = mine / quota;
      if (wg == head && tid < 64 && ((rows >> tid) & 1))
        a.parts[r0 + tid] = (int)((mine + c * (span - 1)) / quota - head) + 1;
      down_item<MT, RT>(a, r0 + tile, rows >> tile, adapter, (int)(wg - head), (int)(x0 * pieces / span),
                        (int)(x1 * pieces / span), red);
    }
  }
}

// out = base + h B^T for 16 MT rows and 16 CT columns a wave.  Weights are the MFMA's row
// operand and the rows of a tile its columns, so that a lane's four results are consecutive
// output columns; two products over interleaved weights give it eight, one 16-byte load of
// base (where the products' sum begins) and one store, whatever the rows' alignment.  Two
// such accesses of a lane cover 64 bytes of 16 rows each; lanes eight apart trade one of
// them, so that an access covers 128 bytes of 8 rows (a copy by rows of 64 bytes runs at 3.4
// TB/s here, by 128 at 3.95; 4096 x 7168).  h goes in as rounded + rest, RS 32-deep steps
// each, from LDS, where the workgroup has put it for its rows; an adapter's weights are loaded
// once for all its rows, those of NB adapters at a time.  Workgroup z = q takes the rows'
// adapters of its q, and q = 0 the rows without one.  4096 x 7168 of rank 16: 32.6 us, base and
// out at 3.6 TB/s; 128 x 24576 with 8 adapters of ranks up to 64: 15.8 us, 2.4 TB/s with B,
// the adapters of a tile one pair after the other.
template <int MT, int RS, int CT, int NB>
__global__ void __launch_bounds__(64 * kUpWaves, RS <= 2 ? 3 : 2)
lora_up_kernel(LoraArgs a) {
  constexpr int M = MT * kTile, HW = RS * 64 + 8;         // LDS row: rounded, rest, 16 bytes
  constexpr int W = kUpWaves, C = CT * 16;
  __shared__ __attribute__((aligned(16))) uint16_t hs[M * HW];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4, q = blockIdx.z;
  const uint32_t across = (uint32_t)((a.N + W * C - 1) / (W * C));
  // column blocks of a row tile in turn; the last rows first, where a mixed batch has its
  // single rows and the work of a tile is longest
  const uint32_t back = blockIdx.x / across, tile = gridDim.x / across - 1 - back;
  const int64_t t0 = (int64_t)tile * M;
  const int64_t n0 = ((int64_t)(blockIdx.x - back * across) * W + wave) * C;
  TileAdapters<M> ad(a, t0, lane, q, a.up_Q);
  // parts of the lanes' rows' sums (of rows without an adapter anything: not used)
  const int64_t t = t0 + (lane & (M - 1));
  const int lane_parts = a.parts[t < a.T ? t : a.T - 1];
  const uint64_t mine = ad.own | (q == 0 ? ad.none : 0);  // rows that this workgroup writes
  if (!mine) return;

  // A lane's 16-byte accesses to the rows of a tile: the i-th of pair p, two pairs together
  // where there are two (see above).  at(): row in the tile and column.
  constexpr bool kTrade = CT % 4 == 0;
  auto at = [&](int p, int* col) {
    *col = kTrade ? 64 * (p / 2) + 32 * (l16 >> 3) + 8 * g : 32 * p + 8 * g;
    return kTrade ? (l16 & 7) + 8 * (p & 1) : l16;
  };
  uint4 base[MT][CT / 2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int p = 0; p < CT / 2; ++p) {
      int col;
      const int row = m * kTile + at(p, &col);
      const int64_t n = n0 + col;
      const uint16_t* b = a.base + (t0 + row) * a.ld_base + n;
      base[m][p] = make_uint4(0, 0, 0, 0);
      if (a.base && ((mine >> row) & 1)) {
        if (n + 8 <= a.N) {
          base[m][p] = load8(b);
        } else {
          uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.N) u[e / 2] |= (uint32_t)b[e] << (16 * (e & 1));
          base[m][p] = make_uint4(u[0], u[1], u[2], u[3]);
        }
      }
    }
  }
  // weight rows of this lane: MFMA row m of product c is column 32 (c / 2) + 8 (m / 4) +
  // 4 (c % 2) + m % 4, so that result j of lane group g is column 32 (c / 2) + 8 g + 4 (c % 2) + j
  uint32_t brow[CT];                         // bytes from the adapter's B: at most 2^30
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int64_t n = n0 + 32 * (c / 2) + 8 * (l16 / 4) + 4 * (c & 1) + (l16 & 3);
    brow[c] = (uint32_t)(n < a.N ? n : a.N - 1) * (uint32_t)(a.R * 2);
  }
  uint32_t piece[RS];                        // this lane's 8 ranks of a step, within R
#pragma unroll
  for (int st = 0; st < RS; ++st) piece[st] = (4 * st + g) * 8 < a.R ? (4 * st + g) * 8 : 0;

  int adapter[NB];
  uint64_t rows[NB];
  uint4 w[NB][CT][RS];
  bool more = n0 < a.N;
  auto load_weights = [&]() {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      more = more && ad.next(&adapter[k], &rows[k]);
      if (!more) {
        rows[k] = 0;
        continue;
      }
      const uint8_t* B = (const uint8_t*)(a.B + (int64_t)adapter[k] * a.N * a.R);
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int st = 0; st < RS; ++st)
          w[k][c][st] = *(const uint4*)(B + (brow[c] + 2 * piece[st]));
    }
  };
  load_weights();

  // h of the rows, 8 ranks an item
  for (int i = tid; i < M * RS * 4; i += 64 * W) {
    const int row = i / (RS * 4), c = (i % (RS * 4)) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    const int S = __shfl(lane_parts, row, 64);
    if (((ad.own >> row) & 1) && c < a.R) {
      const float* p = a.h + (t0 + row) * a.R + c;
      for (int s0 = 0; s0 < S; s0 += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float* ps = p + (s0 + s < S ? s0 + s : S - 1) * a.h_part;
          x[s] = *(const float4*)ps;
          y[s] = *(const float4*)(ps + 4);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (s0 + s < S) {
            v[0] += x[s].x; v[1] += x[s].y; v[2] += x[s].z; v[3] += x[s].w;
            v[4] += y[s].x; v[5] += y[s].y; v[6] += y[s].z; v[7] += y[s].w;
          }
      }
    }
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = split_bf16(v[e]);
    *(uint4*)(hs + row * HW + c) =
        make_uint4((h[0] & 0xFFFFu) | (h[1] << 16), (h[2] & 0xFFFFu) | (h[3] << 16),
                   (h[4] & 0xFFFFu) | (h[5] << 16), (h[6] & 0xFFFFu) | (h[7] << 16));
    *(uint4*)(hs + row * HW + RS * 32 + c) =
        make_uint4((h[0] >> 16) | (h[1] & 0xFFFF0000u), (h[2] >> 16) | (h[3] & 0xFFFF0000u),
                   (h[4] >> 16) | (h[5] & 0xFFFF0000u), (h[6] >> 16) | (h[7] & 0xFFFF0000u));
  }
  __syncthreads();
  if (n0 >= a.N) return;

  f32x4 out[MT][CT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int p = 0; kTrade && p < CT / 2; p += 2) trade(base[m][p], base[m][p + 1], l16 >> 3);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const uint4 b = base[m][c / 2];
      const uint32_t u0 = c & 1 ? b.z : b.x, u1 = c & 1 ? b.w : b.y;
      out[m][c] = f32x4{from_bf16(u0 & 0xFFFFu), __uint_as_float(u0 & 0xFFFF0000u),
                        from_bf16(u1 & 0xFFFFu), __uint_as_float(u1 & 0xFFFF0000u)};
    }
  }
  for (; rows[0]; load_weights()) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (!rows[k]) break;
      const int rank = rank_of(a, adapter[k]);
      if (rank < a.R) {                      // what lies past the adapter's rank is not its
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int st = 0; st < RS; ++st) {
            uint32_t x[4] = {w[k][c][st].x, w[k][c][st].y, w[k][c][st].z, w[k][c][st].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = (int)piece[st] + 2 * e;
              x[e] = r >= rank ? 0u : r + 1 >= rank ? x[e] & 0xFFFFu : x[e];
            }
            w[k][c][st] = make_uint4(x[0], x[1], x[2], x[3]);
          }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint32_t r16 = (uint32_t)(rows[k] >> (m * kTile)) & 0xFFFFu;
        if (!r16) continue;
        uint4 hi[RS], lo[RS];
#pragma unroll
        for (int st = 0; st < RS; ++st) {
          const uint16_t* p = hs + (m * kTile + l16) * HW + (4 * st + g) * 8;
          hi[st] = *(const uint4*)p;
          lo[st] = *(const uint4*)(p + RS * 32);
        }
        const bool here = (r16 >> l16) & 1;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          f32x4 acc = out[m][c];
#pragma unroll
          for (int st = 0; st < RS; ++st) {
            acc = mfma(w[k][c][st], lo[st], acc);
            acc = mfma(w[k][c][st], hi[st], acc);
          }
          if (here) out[m][c] = acc;
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    uint4 u[CT / 2];
#pragma unroll
    for (int p = 0; p < CT / 2; ++p) {
      const f32x4 x = out[m][2 * p], y = out[m][2 * p + 1];
      u[p] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(y[0], y[1]),
                        pack_bf16(y[2], y[3]));
    }
#pragma unroll
    for (int p = 0; kTrade && p < CT / 2; p += 2) trade(u[p], u[p + 1], l16 >> 3);
#pragma unroll
    for (int p = 0; p < CT / 2; ++p) {
      int col;
      const int row = m * kTile + at(p, &col);
      const int64_t n = n0 + col;
      if (!((mine >> row) & 1)) continue;
      uint16_t* o = a.out + (t0 + row) * a.ld_out + n;
      if (n + 8 <= a.N) {
        store8(o, u[p], a.past_caches);
      } else {
        const uint32_t x[4] = {u[p].x, u[p].y, u[p].z, u[p].w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < a.N) o[e] = (uint16_t)(x[e / 2] >> (16 * (e & 1)));
      }
    }
  }
}

template <int MT>
void launch_down(const LoraArgs& a, hipStream_t stream) {
  const dim3 grid(a.grid), block(64 * kDownWaves);
  if (a.R <= 16) hipLaunchKernelGGL((lora_down_kernel<MT, 1>), grid, block, 0, stream, a);
  else if (a.R <= 32) hipLaunchKernelGGL((lora_down_kernel<MT, 2>), grid, block, 0, stream, a);
  else if (a.R <= 64) hipLaunchKernelGGL((lora_down_kernel<MT, 4>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((lora_down_kernel<MT == 4 ? 2 : MT, 8>), grid, block, 0, stream, a);
}

void launch_down_rows(const LoraArgs& a, hipStream_t stream) {
  const dim3 grid(a.grid), block(64 * kDownWaves);
  if (a.R <= 16) hipLaunchKernelGGL((lora_down_rows_kernel<1>), grid, block, 0, stream, a);
  else if (a.R <= 32) hipLaunchKernelGGL((lora_down_rows_kernel<2>), grid, block, 0, stream, a);
  else if (a.R <= 64) hipLaunchKernelGGL((lora_down_rows_kernel<4>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((lora_down_rows_kernel<8>), grid, block, 0, stream, a);
}

template <int MT, int RS, int CT, int NB>
void launch_up(const LoraArgs& a, hipStream_t stream) {
  const int64_t rows = MT * kTile, cols = kUpWaves * CT * 16;
  const dim3 grid((unsigned)((a.T + rows - 1) / rows * ((a.N + cols - 1) / cols)), 1, a.up_Q);
  hipLaunchKernelGGL((lora_up_kernel<MT, RS, CT, NB>), grid, dim3(64 * kUpWaves), 0, stream, a);
}

}  // namespace

void lora_plan(LoraArgs* a) {
  const int64_t T = a->T, K = a->K;
  auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
  a->h_part = T * a->R;
  // parts: a wave's first loads (down_products) take a part's pieces at once
  const int rt = a->R <= 16 ? 1 : a->R <= 32 ? 2 : a->R <= 64 ? 4 : 8;
  auto most = [&](int mt) { return cdiv(K, 512 * (mt + rt <= 2 ? 4 : mt + rt <= 4 ? 2 : 1)); };
  if (T <= kLoraFewRows) {
    a->mt = 0;
    // as many parts as 256 workgroups give the fewest items, but up to 16 only where more rows
    // read them back (128 x 7168 x 16384 of rank 64, two adapters in a mixed batch: 19.1 us,
    // 27.5 with 4 at most; a share of K for each row, with an item or not: 44.5)
    const int64_t S = cdiv(256, T) > 16 ? cdiv(256, T) : 16;
    a->S = (int)(S < most(1) ? S : most(1));
  } else {
    const int64_t rows = T < kLoraRows ? T : kLoraRows;
    int mt = a->R <= 64 ? 4 : 2;
    while (mt > 1 && cdiv(rows, mt * kTile) * cdiv(K, 512) < 256) mt /= 2;
    const int64_t S = cdiv(256, cdiv(rows, mt * kTile)) + 1;
    a->mt = mt;
    a->S = (int)(S < most(mt) ? S : most(mt) < 2 ? 2 : most(mt));
  }
  a->grid = a->mt == 0 && T * a->S < 256 ? (int)(T * a->S) : 256;
  // second kernel
  // 64 rows share an adapter's weights where they are many (R > 32), else 32: 4096 x 7168 of
  // rank 16 32.9 us with 64 rows a workgroup, 30.5 with 32; 8192 x 7168 of rank 64 79 and 81
  a->up_mt = a->R <= 32 ? (T <= 64 ? 1 : 2) : T <= 16 ? 1 : 4;
  // few rows: adapters two at a time in half the columns rather than one by one (100 x 4096 x
  // 7168, 40 adapters of rank 64: 31.8 us, 32.5 with 64 columns a wave)
  const bool few = T <= kLoraFewRows;
  a->up_ct = few ? 2 : 4;
  // Stores past the caches are faster by themselves at every size and slow whoever reads out
  // next, which shows up to 56 MiB and not from 70 on (K = 512, rank 16; alone, and with a copy
  // of out behind it, in us):
  //    28 MiB (2048 x 7168)  25.0 -> 23.0  33.5 -> 34.4     98 (7168 x 7168)   68.6 -> 62.7  104.2 -> 103.5
  //    56 (4096 x 7168)      39.4 -> 34.6  56.5 -> 58.3    112 (8192 x 7168)   63.5 -> 59.8  105.2 -> 106.0
  //    70 (5120 x 7168)      52.9 -> 47.3  75.8 -> 74.6    168 (12288 x 7168)  92.8 -> 88.8  157.5 -> 156.2
  //    84 (6144 x 7168)      58.7 -> 53.0  89.3 -> 85.7    224 (16384 x 7168) 114.6 -> 108.3 200.4 -> 198.5
  a->past_caches = T * a->N * 2 >= kLoraPastCaches;
  const int64_t up_tiles = cdiv(T, a->up_mt * kTile) * cdiv(a->N, kUpWaves * kTile * a->up_ct);
  // workgroups on the same rows: those that find nothing to do cost little beside few others
  // (128 x 24576 x 1536, ranks up to 64, 8 adapters: 22.9 us for up to 512 workgroups, 21.1 for
  // 1024, 24.9 for 2048)
  a->up_Q = 1;
  while (a->up_Q < (few ? 16 : 4) && a->up_Q < T && 2 * a->up_Q * up_tiles <= (few ? 1024 : 2048))
    a->up_Q *= 2;
}

void launch_lora(const LoraArgs& all, hipStream_t stream) {
  for (int64_t t = 0; t < all.T; t += kLoraRows) {
    LoraArgs a = all;
    a.T = all.T - t < kLoraRows ? all.T - t : kLoraRows;
    a.x += t * a.ldx;
    a.ids += t;
    if (a.base) a.base += t * a.ld_base;
    a.out += t * a.ld_out;
    a.h += t * a.R;
    if (a.parts) a.parts += t;
    if (a.mt == 0) launch_down_rows(a, stream);
    else if (a.mt == 4) launch_down<4>(a, stream);
    else if (a.mt == 2) launch_down<2>(a, stream);
    else launch_down<1>(a, stream);
    if (a.R <= 32) {
      if (a.up_mt == 1) launch_up<1, 1, 2, 4>(a, stream);
      else if (a.up_ct == 2) launch_up<2, 1, 2, 4>(a, stream);
      else launch_up<2, 1, 4, 2>(a, stream);
    } else if (a.R <= 64) {
      if (a.up_mt == 1) launch_up<1, 2, 2, 2>(a, stream);
      else if (a.up_ct == 2) launch_up<4, 2, 2, 2>(a, stream);
      else launch_up<4, 2, 4, 1>(a, stream);
    } else {
      if (a.up_mt == 1) launch_up<1, 4, 2, 1>(a, stream);
      else if (a.up_ct == 2) launch_up<4, 4, 2, 1>(a, stream);
      else launch_up<4, 4, 4, 1>(a, stream);
    }
  }
}

}  // namespace dg
