// Device helpers shared by the attention kernels: key-value (or query) tiles in LDS, the
// fragments read from them, cross-lane steps, and the workgroup -> (sequence, tile) map.
//
// Fragment layouts (v_mfma_f32_16x16x32_bf16; lane l, g = l / 16, c = l % 16):
//   A [16 rows x 32 k]  lane holds row c, k 8 g .. 8 g + 7
//   B [32 k x 16 cols]  lane holds column c, the same k
//   C [16 x 16]         lane holds column c, rows 4 g .. 4 g + 3
// The kernels compute score tiles with the tile staged in LDS as the rows and a wave's own
// rows (in registers) as the columns.  Two such C blocks, of tile rows r .. r + 15 and
// r + 16 .. r + 31, rounded to bf16, are the B operand of a second product over those 32
// tile rows with no exchange between lanes, if k index 8 g + j of that product stands for
// tile row r + 4 g + j (j < 4) or r + 16 + 4 g + j - 4 (j >= 4): a sum over k does not depend
// on how k is numbered, and the A operand, read transposed from the same tile
// (ds_read_b64_tr_b16), takes its rows in that numbering.
#pragma once

#include <hip/hip_runtime.h>

#include "attn_internal.h"
#include "gemm_common.h"

namespace ubx {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// A tile of `ROWS` rows of up to 32 DS elements in LDS.  Rows take 128 bytes (DS <= 2) or
// 256; 16-byte chunk q of row r is kept in slot q ^ swz(r).  swz makes both reads free of bank
// conflicts.  A 16-byte read is served 16 lanes at a time, lanes 0-3, 12-15 and 20-27 first
// (measured, by which pairs of lanes conflict), then 4-11, 16-19 and 28-31: of the rows that a
// row fragment reads, those with bits 2 and 3 alike at one chunk and the others at the next.
// Their 16 slots differ if rows whose swz differ in bit 0 alone are of the same kind: r and
// r ^ 12.  A transposing read serves 8 rows, two neighbouring chunks each: their swz differ
// above bit 0.
template <int DS>
struct Tile {
  static constexpr int CPR = DS <= 2 ? 8 : 16;  // chunks per row
  static constexpr int RB = 16 * CPR;           // bytes per row
  static constexpr int DB = 2 * DS;             // 16-wide blocks of a row
  __device__ static int swz(int r) {
    return CPR == 16 ? ((((r & 7) ^ ((r >> 1) & 4)) << 1) | ((r >> 3) & 1))
                     : (((((r >> 1) & 3) ^ ((r >> 2) & 2)) << 1) | ((r >> 3) & 1));
  }
};

// A wave's share of the direct-to-LDS loads of a tile of ROWS rows by NW waves: the byte
// offset of its lanes' 16-byte pieces from the tile's first row (OOB past head_dim).  The
// instructions' rows lie RPI NW apart; the swizzle repeats every 16 rows, so only the first
// P offsets are kept.
template <int DS, int ROWS, int NW>
struct TileLoad {
  using L = Tile<DS>;
  static constexpr int RPI = 64 / L::CPR;          // rows per wave instruction
  static constexpr int N = ROWS / RPI / NW;        // instructions per wave
  static constexpr int P = RPI * NW >= 16 ? 1 : 16 / (RPI * NW);
  static_assert(N >= 1 && N * RPI * NW == ROWS, "rows must divide over the waves");
  uint32_t off[P], step;

  __device__ void init(int wave, int lane, int64_t row_stride, int D) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int row = (j * NW + wave) * RPI + lane / L::CPR;
      const int chunk = (lane % L::CPR) ^ L::swz(row);
      off[j] = chunk * 8 < D ? (uint32_t)row * (uint32_t)(row_stride * 2) + chunk * 16 : OOB;
    }
    step = P * RPI * NW * (uint32_t)(row_stride * 2);  // N steps from OOB stay under 2^32
  }
  // rows [0, valid) at base; the others read as zeros
  __device__ void issue(const uint16_t* base, int64_t row_stride, int D, int valid, uint32_t lds,
                        int wave) const {
    const uint32_t bytes = valid > 0 ? (uint32_t)(min(valid, ROWS) - 1) * (uint32_t)(row_stride * 2) +
                                           (uint32_t)D * 2
                                     : 0u;
    const i32x4 rsrc = make_rsrc(base, bytes);
#pragma unroll
    for (int j = 0; j < N; ++j) dma16(rsrc, lds + (j * NW + wave) * 1024, off[j % P] + j / P * step);
  }
};

// Row fragment: rows 16 b .. 16 b + 15 of the tile, columns 32 s .. 32 s + 31.  The lane's
// chunk (4 s + g) ^ swz is that of s = 0 with bits changed by 4 s, so one address (of a tile on
// a 256-byte boundary) serves all.
template <int DS>
struct RowFrag {
  using L = Tile<DS>;
  const unsigned char* p;
  __device__ void init(const unsigned char* tile, int lane) {
    const int c = lane & 15, g = lane >> 4;
    p = tile + c * L::RB + ((g ^ L::swz(c)) * 16);
  }
  __device__ bf16x8 read(int off, int b, int s) const {
    const uint32_t at = ((uint32_t)(size_t)LDS_PTR(const unsigned char, p) + off) ^ (64 * s);
    return *LDS_PTR(const bf16x8, at + b * 16 * L::RB);
  }
};

// Transposed fragment: columns 16 d .. 16 d + 15 of the tile as the rows of an A operand,
// over tile rows 32 t .. 32 t + 31 in the numbering described above.
template <int DS>
struct ColFrag {
  using L = Tile<DS>;
  const unsigned char* p;
  __device__ void init(const unsigned char* tile, int lane) {
    const int c = lane & 15, g = lane >> 4;
    const int row = 4 * g + (c >> 2);
    p = tile + row * L::RB + ((((c >> 1) & 1) ^ L::swz(row)) * 16) + 8 * (c & 1);
  }
  __device__ bf16x8 read(int off, int t, int d) const {
    const uint32_t at = ((uint32_t)(size_t)LDS_PTR(const unsigned char, p) + off) ^ (32 * d);
    const uint32_t q = at + t * 32 * L::RB;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(i16x4, q));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(LDS_PTR(i16x4, q + 16 * L::RB));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// Max (sum) over the four lanes that share a column: lanes c, c + 16, c + 32, c + 48.
__device__ inline float col_max(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ inline float col_sum(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// 8 bf16 from two fp32 quads, round to nearest even.
__device__ inline bf16x8 pack8(f32x4 a, f32x4 b) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = static_cast<__bf16>(a[i]);
    r[4 + i] = static_cast<__bf16>(b[i]);
  }
  return r;
}

// 16 bytes of a row held in registers as a B operand: zeros past the valid rows or head_dim.
__device__ inline bf16x8 load_row8(const uint16_t* p, bool valid) {
  u32x4 v = {0, 0, 0, 0};
  if (valid) v = *GLOBAL_PTR(const u32x4, p);
  return __builtin_bit_cast(bf16x8, v);
}

// Diagonal tiles: a pair that the mask leaves out has weight 0, but the product over a tile's
// 32 rows would take 0 times its value, NaN for one that is not finite.  A workgroup whose
// diagonal tiles hold such values does its pass again with seen_product, every column computed
// by itself from the rows that the mask lets it see.  (As a branch in the one pass it would make
// the compiler copy or spill the accumulators.)
// Whether wave w of the W that share a tile of BYTES finds such a value in its share of it.
template <int BYTES, int W>
__device__ inline bool not_finite(const unsigned char* tile, int w, int lane) {
  static_assert(BYTES % (1024 * W) == 0, "a tile divides over the waves");
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < BYTES / (1024 * W); ++i) {
    const u32x4 x = *LDS_PTR(const u32x4, tile + (i * W + w) * 1024 + lane * 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) any |= (x[k] & 0x7F807F80u) + 0x00800080u;  // exponents of all ones carry
  }
  return (any & 0x80008000u) != 0;
}
// Bits of the lane's 8 elements whose tile rows (the first at `row`, in the numbering at the
// top) come no later than `at` (UP_TO) or no earlier.
template <bool UP_TO>
__device__ inline u32x4 keep_rows(int row, int at, int g) {
  u32x4 m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row + 4 * g + (i & 1) * 2 + (i >> 1) * 16;
    const bool lo = UP_TO ? r <= at : r >= at, hi = UP_TO ? r + 1 <= at : r + 1 >= at;
    m[i] = (lo ? 0xFFFFu : 0u) | (hi ? 0xFFFF0000u : 0u);
  }
  return m;
}
// acc + A B, column c of the 16 (the tile row at + c) from the rows that it sees.
template <bool UP_TO>
__device__ inline f32x4 seen_product(bf16x8 a, bf16x8 b, f32x4 acc, int row, int at, int lane) {
  f32x4 r = acc;
#pragma unroll 1
  for (int c = 0; c < 16; ++c) {
    const u32x4 x = __builtin_bit_cast(u32x4, a) & keep_rows<UP_TO>(row, at + c, lane >> 4);
    const f32x4 y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), b, acc, 0, 0, 0);
    if ((lane & 15) == c) r = y;
  }
  return r;
}

// Makes the compiler wait here for a value it loads.  It does not count the direct-to-LDS
// loads, so a wait that it left to a value's first use, inside a loop, would be one for all
// loads in flight there: the next tile's among them, in every iteration.
__device__ inline void arrived(bf16x8& x) { __asm__ volatile("" : "+v"(x)); }

// The barrier between the two phases of a step of kernels whose groups of waves work in turns:
// the later half of the groups starts one barrier late, so that while one half multiplies
// score tiles the other does its exponentials; all at once, each unit would idle in turn.
__device__ inline void phase_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// Whether any wave of the workgroup says so; through LDS that nothing is being loaded into.
template <int NW>
__device__ inline bool any_wave(bool x, unsigned char* smem, int wave, int lane) {
  int* flags = reinterpret_cast<int*>(smem);
  const bool mine = __ballot(x) != 0;
  __syncthreads();
  if (lane == 0) flags[wave] = mine;
  __syncthreads();
  int any = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) any |= flags[w];
  __syncthreads();
  return any != 0;
}

// Sum over NG groups of W waves each of the accumulators that wave w of every group holds,
// in group order, through NG W B F KB of LDS.  Group grp's x[0], x[1], ... become the sums of
// blocks grp, grp + NG, ... (of no block past B).
template <int NG, int W, int B, int F>
__device__ inline void join_groups(f32x4 (&x)[B][F], unsigned char* smem, int grp, int w, int lane) {
  f32x4* parts = reinterpret_cast<f32x4*>(smem);  // [NG][W][B][F][64]
  __syncthreads();
  f32x4* mine = parts + (grp * W + w) * B * F * 64 + lane;
#pragma unroll
  for (int d = 0; d < B; ++d)
#pragma unroll
    for (int f = 0; f < F; ++f) mine[(d * F + f) * 64] = x[d][f];
  __syncthreads();
  const f32x4* all = parts + (w * B + grp) * F * 64 + lane;
#pragma unroll
  for (int i = 0; i < (B + NG - 1) / NG; ++i) {
    if (i * NG + grp >= B) break;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      f32x4 y = all[(i * NG * F + f) * 64];
#pragma unroll
      for (int k = 1; k < NG; ++k) y += all[((k * W * B + i * NG) * F + f) * 64];
      x[i][f] = y;
    }
  }
}

// Sum over the wave's 64 lanes, the same value in all of them.
__device__ inline int wave_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);  // row_shr:8
  return __builtin_amdgcn_readlane(v, 15) + __builtin_amdgcn_readlane(v, 31) +
         __builtin_amdgcn_readlane(v, 47) + __builtin_amdgcn_readlane(v, 63);
}

// Inclusive prefix sum over the wave.
__device__ inline int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  const int a = __builtin_amdgcn_readlane(v, 15), b = __builtin_amdgcn_readlane(v, 31),
            c = __builtin_amdgcn_readlane(v, 47);
  const int row = (threadIdx.x & 63) >> 4;
  return v + (row > 0 ? a : 0) + (row > 1 ? b : 0) + (row > 2 ? c : 0);
}

// Rows of sequence i clamped to [0, T): a bad boundary reads no row outside the matrices.
__device__ inline int clamp_row(int x, int T) { return min(max(x, 0), T); }

struct SeqTile {
  int row0, len;  // the sequence's first row and its length; len 0: no tile
  int tile;       // tile of that sequence
};

// The tile of `rank` among the tiles of bm rows of all sequences.  Up to 64 sequences (one
// per lane): in the order of falling tile number, so that the tiles with the most work under
// a causal mask start first.  A level x holds the tiles number x - 1; C(x) = the tiles of
// level x and above; the rank's level is the largest x with C(x) > rank, its sequence by the
// rank's bit in a ballot.  A grid that runs at once needs no order, and more sequences do
// without: in sequence order.  `low_first` reverses the levels (tiles whose work falls with
// their number).
__device__ inline SeqTile find_tile(const Seqs& s, int bm, int rank, bool low_first) {
  const int lane = threadIdx.x & 63;
  SeqTile r{0, 0, 0};
  if (s.n <= 64) {
    const int i = min(lane, s.n);
    const int a = s.n > 0 ? clamp_row(s.cu[i], s.T) : 0;
    const int b = s.n > 0 ? clamp_row(s.cu[min(lane + 1, s.n)], s.T) : 0;
    const int len = max(b - a, 0);
    const int nt = (len + bm - 1) / bm;
    if (gridDim.x <= 256) {
      const int incl = wave_scan(nt);
      const uint64_t m = __ballot(incl > rank);
      if (m == 0) return r;
      const int at = __builtin_ctzll(m);
      r.row0 = __builtin_amdgcn_readlane(a, at);
      r.len = __builtin_amdgcn_readlane(len, at);
      r.tile = rank - __builtin_amdgcn_readlane(incl - nt, at);
      return r;
    }
    const int total = wave_sum(nt);
    if (rank >= total) return r;
    const int want = low_first ? total - 1 - rank : rank;
    int lo = 1, hi = (s.T + bm - 1) / bm;  // C(lo) > want always
    if (s.n <= 16) {
      // 64 levels at a time, one to a lane: 2 rounds up to 4096 tiles, where a bisection takes
      // a wave's sum for each of 12 (1.5 us of every workgroup, with 128 tiles)
      for (int step = hi; step > 1;) {
        step = (step + 63) / 64;
        const int x = lo + lane * step;
        int c = 0;
        for (int i = 0; i < s.n; ++i) c += max(__builtin_amdgcn_readlane(nt, i) - x + 1, 0);
        lo += (__popcll(__ballot(c > want)) - 1) * step;
      }
    } else {
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (wave_sum(max(nt - mid + 1, 0)) > want) lo = mid;
        else hi = mid - 1;
      }
    }
    int k = want - wave_sum(max(nt - lo, 0));  // index among the level's sequences
    uint64_t m = __ballot(nt >= lo);
    while (k-- > 0) m &= m - 1;
    const int at = __builtin_ctzll(m);
    r.row0 = __builtin_amdgcn_readlane(a, at);
    r.len = __builtin_amdgcn_readlane(len, at);
    r.tile = lo - 1;
    return r;
  }
  int before = 0;
  for (int c = 0; c < s.n; c += 64) {
    const int i = min(c + lane, s.n);
    const int a = clamp_row(s.cu[i], s.T), b = clamp_row(s.cu[min(c + lane + 1, s.n)], s.T);
    const int len = max(b - a, 0);
    const int nt = (len + bm - 1) / bm;
    const int total = wave_sum(nt);
    if (rank < before + total) {
      int k = rank - before;
      for (int j = 0; j < 64; ++j) {
        const int n = __builtin_amdgcn_readlane(nt, j);
        if (k < n) {
          r.row0 = __builtin_amdgcn_readlane(a, j);
          r.len = __builtin_amdgcn_readlane(len, j);
          r.tile = low_first ? k : n - 1 - k;
          return r;
        }
        k -= n;
      }
    }
    before += total;
  }
  return r;
}

// Four groups of waves on the keys shorten a call's longest rows.  Many sequences make many
// workgroups of few steps each, and then those of one group, two to a CU, are faster whatever
// the rows.  Measured, lengths within a factor of 5 but for an empty sequence and one of a single
// token, groups against one (forward; gradient, us): 4200 rows, 30 sequences, 8 heads on 8 29 and 20,
// 71 and 42; 2048 rows, 16 sequences 18 and 15, 40 and 34; 4264 rows, 12 sequences 32 and 29, 82 and
// 60; 2096 rows, 4 sequences, 8 on 1 23 and 32, 64 and 77.  n counts the call's sequences, empty ones
// too, as their lengths are on the device: where a table of many entries holds a few long sequences
// the rule is wrong (8184 rows of 4 heads on 4 in 5 sequences, one of 4677: 51 and 170 us with 5 to
// 23 entries, 81 and 196 with 24 and more).
inline bool few_sequences(int64_t n, int H) { return n * H < 96; }

// Tiles of bm rows that n sequences of T rows together can have.
inline int64_t max_tiles(int64_t T, int64_t n, int bm) { return T / bm + (n < T ? n : T); }

// Whether row t lies in no sequence: before the first or after the last.
__device__ inline int first_row(const Seqs& s) { return s.n > 0 ? clamp_row(s.cu[0], s.T) : s.T; }
__device__ inline int last_row(const Seqs& s) { return s.n > 0 ? clamp_row(s.cu[s.n], s.T) : s.T; }

}  // namespace
}  // namespace ubx
