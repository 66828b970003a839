// Attention of a tree of drafted tokens over a paged key-value cache.
//
//   row j of a sequence sees the tokens before the drafted ones and the nodes on its own path:
//   s_u = scale q . k_u,  lse = log sum_u exp(s_u),  out = sum_u exp(s_u - lse) v_u
//
// The rows of a key-value head's query heads are the columns of one product: a sequence of m
// nodes has m (n_heads / n_kv_heads) of them, in strips of COLS.  A workgroup takes one strip and
// some of the sequence's tiles of BN keys.  The lengths are on the device, so the cut is made
// there: sequence i's tiles go in k_i = ceil(tiles_i / c) equal parts, with the smallest c for
// which all strips' parts are as many workgroups as run at once, or twice as many (c no smaller
// than MIN_TILES; one part each where the strips are more than run at once).  The strips of one
// part of a sequence read the same keys at the same time, so they are neighbours on one XCD, whose
// L2 then serves all but one of them.  A strip in one part is finished by its workgroup; others leave parts (maximum,
// sum and unnormalised output, fp32) in the workspace, and attn_tree_join adds them in order.
//
// Keys and values come from their pages (a lane looks up a token, a tile ahead): bf16 by direct
// loads to LDS, E4M3 by registers that are stored there as bf16, so that all waves read their
// fragments as in attn_common.h.  RW waves take 16 QF columns each; KG groups of them take parts
// of a tile's keys, where columns are few.
//
// The softmax's reference is the maximum of the first tile that a column sees a key of, as in
// attn_prompt.hip: where a sum passes 2^60, or what is hidden from a column is not finite, the
// pass over the segment's tiles is repeated with the running maximum, column by column where it
// has to be.
//
// The nodes that a node sees are bits, set once per strip by following the parents in LDS; only
// the tiles of drafted tokens look at them.
//
// Sums and the softmax are fp32; the weights are rounded to bf16 as matrix-core operands, and each
// output once.
//
// Measured on MI355X, both kernels.  64 sequences of 100 to 16264 tokens and up to 60 nodes, 8 heads
// on 1, E4M3: 135-138 us (bf16 143), 0.63 PFLOP/s counted (86 GFLOP; 101 with the columns that fill the strips up);
// a step of 64 keys and 128 columns takes 1.95 us on each of a CU's two workgroups, as in
// attn_prompt.hip, 92 us if all had as many; the rest is parts of unequal length, 4 us before and
// 2 after a part's tiles, and 13 of the join.  One sequence of 32520 and 24 nodes, bf16: 22 us: 4 us to
// the first load's issue (lengths, cut, page ids), 1.6 and 6 for four tiles as memory delivers them,
// 2 to the end, and the join's 6.  Bound by memory: 64 of 8192 with 2 nodes 61 us (4.4 TB/s), E4M3 35.
// Not kept: ranges of equal length over the strips one after another, as attn_decode.hip deals
// its tokens (every part ends at once, but no two strips read the same keys together: 3.4 us a
// step in bf16, 157 us for the first case); the running maximum in every tile (185); E4M3 tiles
// stored beside the step before (162).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn_common.h"
#include "attn_path.h"
#include "kv_pages.h"

namespace ubx {
namespace {

constexpr int NW = 4;
constexpr int ITEMS = 512;     // workgroups that run at once: two on each CU
// Tiles of a part at least, where there are so many: the second case above takes 26.9 us with 2, 23.7
// with 4, 27.4 with 8.
constexpr int MIN_TILES = 4;
// Parts of LONG_PART tiles or more are cut again, for two rounds of workgroups: what one round
// leaves idle for want of equal parts is more than what starting another costs.  64 sequences of
// 8192, 48 nodes: 158 us with one, 146 with two; 16 of 100 to 16264, 60 nodes (parts of 10) 47 and 62.
constexpr int LONG_PART = 48, ROUNDS = 2;
constexpr float MOST = 0x1p60f;  // a lane's sum beyond which the pass is done again

struct TreeParams {
  TreeArgs a;
  float c;         // scale * log2(e) (/ k_scale)
  float v_inv;     // 1 / v_scale
  int32_t cap;     // tokens the page table can hold per sequence
  PageDiv div;     // by the page size
  int32_t at_once;  // workgroups of a key-value head that run at once
  int4* seqs;       // [n]: a sequence's first workgroup among `w` of a head, its k_i, its strips, w
  float* part;      // [ROUNDS at_once G, COLS, D]: a workgroup's output where a strip has several parts
  float2* stat;     // [ROUNDS at_once G, COLS]: maximum (base 2, scaled), sum
};

constexpr int BN = 64;         // keys of a tile: one to a lane in the lookup of their pages

template <int DS_, int QF_, int RW_, bool F8_>
struct Shape {
  static constexpr int DS = DS_, QF = QF_, RW = RW_, KG = NW / RW;
  static constexpr bool F8 = F8_;
  using L = Tile<DS>;
  static constexpr int COLS = 16 * QF * RW, TILE = BN * L::RB, STAGE = 2 * TILE;
  static constexpr int EB = F8 ? 1 : 2;
  static constexpr int PPR = F8 ? L::CPR / 2 : L::CPR;  // 16-byte pieces of a row, as loaded
  static constexpr int RPL = 64 / PPR;                  // rows of a wave's load
  static constexpr int N = BN / RPL / NW;               // loads of a wave, of keys and of values
  static constexpr int JOIN = KG > 1 ? NW * L::DB * QF * 1024 + NW * QF * 128 : 0;
  static constexpr int KV = 2 * STAGE > JOIN ? 2 * STAGE : JOIN;
  static constexpr int LDS = KV + MAX_NODES * WORDS * 8 + MAX_NODES * 4;
};

// What rows past the end and pieces past head_dim are loaded from.
__device__ const u32x4 ZEROS = {0, 0, 0, 0};

// 16 bytes per lane from its own address into LDS at lds + 16 * lane.
__device__ inline void gather16(const unsigned char* from, uint32_t lds) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory");
}

// A sequence's rows and tokens.  Not good: more nodes than MAX_NODES, fewer cached tokens than
// nodes, or more than its row of the table holds.
struct Seq {
  int row0, m, len;
  bool good;
};
__device__ inline Seq sequence(const TreeParams& p, int i) {
  Seq s;
  s.row0 = clamp_row(p.a.seqs.cu[i], p.a.seqs.T);
  s.m = max(clamp_row(p.a.seqs.cu[i + 1], p.a.seqs.T) - s.row0, 0);
  s.len = p.a.lens[i];
  s.good = s.m <= MAX_NODES && s.len >= s.m && s.len <= p.cap;
  return s;
}

// Strips and tiles of a sequence: none of one that is not good, or has no rows.
struct Work {
  int strips, tiles;
};
template <class S>
__device__ inline Work work_of(const TreeParams& p, int i) {
  if (i >= p.a.seqs.n) return Work{0, 0};
  const Seq s = sequence(p, i);
  if (!s.good || s.m == 0) return Work{0, 0};
  return Work{(s.m * (p.a.H / p.a.G) + S::COLS - 1) / S::COLS, (s.len + BN - 1) / BN};
}

constexpr int MANY = 1 << 20;  // counts past this only have to stay past it
__device__ inline int parts_for(Work w, int c) {  // strips k_i, of one sequence
  return w.strips == 0 ? 0 : (int)min((int64_t)w.strips * ((w.tiles + c - 1) / c), (int64_t)MANY);
}

// Tiles to a part, and the workgroups that makes for a head.
struct Cut {
  int c, w;
};
template <class S>
__device__ inline Cut cut_of(const TreeParams& p, Work head) {  // head: of sequence `lane`
  const int n = p.a.seqs.n, lane = threadIdx.x & 63;
  auto all = [&](int c) {
    int sum = 0;
    for (int i = 0; i < n; i += 64) sum = min(sum + wave_sum(parts_for(i == 0 ? head : work_of<S>(p, i + lane), c)), 1 << 30);
    return sum;
  };
  int most = 0;
  float tiles = 0.0f;
  for (int i = 0; i < n; i += 64) {
    const Work w = i == 0 ? head : work_of<S>(p, i + lane);
    int x = w.tiles;
    float y = (float)w.strips * (float)x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      x = max(x, __shfl_xor(x, d));
      y += __shfl_xor(y, d);
    }
    most = max(most, __builtin_amdgcn_readfirstlane(x));
    tiles += __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(y)));
  }
  Cut cut{max(most, MIN_TILES), 0};
  cut.w = all(cut.c);  // the strips
  if (cut.w >= p.at_once) return cut;
  // the smallest c that will do, for `slots` workgroups: w is at least tiles / c, and at most the
  // strips more
  auto search = [&](int slots) {
    int lo = max(MIN_TILES, (int)(tiles * 0.999f / (float)slots));
    int hi = max(lo, (int)min((float)cut.c, tiles * 1.001f / (float)(slots - cut.w) + 2.0f));
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (all(mid) <= slots) hi = mid;
      else lo = mid + 1;
    }
    return hi;
  };
  int c = search(p.at_once);
  if (c >= LONG_PART) c = search(p.at_once * ROUNDS);
  cut.c = c;
  cut.w = all(c);
  return cut;
}

// The wave's LDS writes are done, then every wave's; direct or register loads stay in flight.
__device__ inline void lds_barrier() { __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// acc + A B over 32 keys, or over 16 whose halves of the operands hold the first 4 elements.
template <bool HALF>
__device__ inline f32x4 product(bf16x8 a, bf16x8 b, f32x4 acc) {
  if (!HALF) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
  const i16x4 x = __builtin_bit_cast(i16x4, __builtin_shufflevector(a, a, 0, 1, 2, 3));
  const i16x4 y = __builtin_bit_cast(i16x4, __builtin_shufflevector(b, b, 0, 1, 2, 3));
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(x, y, acc, 0, 0, 0);
}

template <class S>
__global__ __launch_bounds__(64 * NW, 2) void attn_tree(TreeParams p) {
  constexpr int DS = S::DS, QF = S::QF, RW = S::RW, KG = S::KG, TILE = S::TILE, STAGE = S::STAGE, N = S::N;
  constexpr int COLS = S::COLS, EB = S::EB, PPR = S::PPR, RPL = S::RPL;
  constexpr bool F8 = S::F8;
  constexpr int KB = BN / KG / 16;  // blocks of 16 keys of a group
  using L = Tile<DS>;
  extern __shared__ __align__(256) unsigned char smem[];
  uint64_t* paths = reinterpret_cast<uint64_t*>(smem + S::KV);  // [MAX_NODES][WORDS]
  int* up = reinterpret_cast<int*>(paths + MAX_NODES * WORDS);  // [MAX_NODES]
  const TreeArgs& a = p.a;
  const int group = a.H / a.G;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kg = wave / RW, col = lane & 15, g = lane >> 4;

  const Work head = work_of<S>(p, lane);
  const Cut cut = cut_of<S>(p, head);
  // XCD blockIdx % 8 takes one contiguous share of the heads' workgroups
  const int xcd = blockIdx.x % NUM_XCD, place = blockIdx.x / NUM_XCD;
  const int64_t total = (int64_t)cut.w * a.G;
  const int share = (int)(total / NUM_XCD), more = (int)(total % NUM_XCD);
  if (place >= share + (xcd < more)) return;
  const int64_t self = (int64_t)xcd * share + min(xcd, more) + place;
  const int kvh = (int)(self / cut.w);
  int item = (int)(self - (int64_t)kvh * cut.w);
  // its sequence, its strip and its part
  int seq = 0, begin = 0;
  Work w{0, 0};
  for (int c = 0; c < a.seqs.n; c += 64) {
    const Work x = c == 0 ? head : work_of<S>(p, c + lane);
    const int n = parts_for(x, cut.c), incl = wave_scan(n);
    const uint64_t m = __ballot(begin + incl > item);
    if (m) {
      const int at = __builtin_ctzll(m);
      seq = c + at;
      begin += __builtin_amdgcn_readlane(incl - n, at);
      w.strips = __builtin_amdgcn_readlane(x.strips, at);
      w.tiles = __builtin_amdgcn_readlane(x.tiles, at);
      break;
    }
    begin += __builtin_amdgcn_readlane(incl, 63);
  }
  if (w.strips == 0) return;
  const int parts = (w.tiles + cut.c - 1) / cut.c;
  const int part = (item - begin) / w.strips, strip = item - begin - part * w.strips;
  if (part >= parts) return;
  const int j0 = (int)((int64_t)part * w.tiles / parts), j1 = (int)((int64_t)(part + 1) * w.tiles / parts);
  const bool alone = parts == 1;
  if (item == begin && kvh == 0 && threadIdx.x == 0) p.seqs[seq] = make_int4(begin, parts, w.strips, cut.w);
  const Seq sq = sequence(p, seq);
  const int cols = sq.m * group, past = sq.len - sq.m;
  const int32_t* pages = a.pages + (int64_t)seq * a.pages_ld;

  const unsigned char* kb = static_cast<const unsigned char*>(a.cache.k) + kvh * a.cache.hs * EB;
  const unsigned char* vb = static_cast<const unsigned char*>(a.cache.v) + kvh * a.cache.hs * EB;
  const int piece = lane % PPR;
  const uint32_t lds = lds_addr(smem);
  RowFrag<DS> kf;
  ColFrag<DS> vf;
  kf.init(smem + kg * (BN / KG) * L::RB, lane);
  vf.init(smem + TILE + kg * (BN / KG) * L::RB, lane);

  bool lost = false;  // a page that is not there
  // A lane looks up a token: the page's id, then, with the tile before in use, its place.
  int id = 0;
  auto look = [&](int j) {
    const uint32_t t = min(j * BN + lane, sq.len - 1);
    id = pages[p.div.page(t)];  // inside the row: len <= cap
  };
  look(j0);

  // the wave's columns
  bf16x8 q[QF][DS];
  int node[QF];
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int c = strip * COLS + (rw * QF + f) * 16 + col;
    const bool live = c < cols;
    node[f] = live ? c / group : 0;
    const uint16_t* row = a.q.p + (int64_t)(sq.row0 + node[f]) * a.q.rs + (kvh * group + (live ? c % group : 0)) * a.q.hs;
#pragma unroll
    for (int s = 0; s < DS; ++s) q[f][s] = load_row8(row + 32 * s + 8 * g, live && 32 * s + 8 * g < a.D);
  }
  u32x4 kreg[N], vreg[N];  // E4M3 alone
  auto fetch = [&](int j, int stage) {
    const uint32_t t = min(j * BN + lane, sq.len - 1);
    const uint32_t o = t - p.div.page(t) * (uint32_t)a.cache.page_size;
    const bool there = (uint32_t)id < (uint32_t)a.cache.n_pages;
    lost = lost || !there;
    const int64_t place = ((there ? id : 0) * a.cache.ps + o * a.cache.ts) * EB;
    const int lo = (int)(uint32_t)place, hi = (int)(place >> 32);
    const bool all = (j + 1) * BN <= sq.len && a.D == 32 * DS;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = (i * NW + wave) * RPL + lane / PPR;
      const int chunk = F8 ? piece : piece ^ L::swz(r);
      const int64_t at = (int64_t)(((uint64_t)(uint32_t)__shfl(hi, r) << 32) | (uint32_t)__shfl(lo, r)) + chunk * 16;
      const unsigned char *k = kb + at, *v = vb + at;
      if (!all && !(chunk * (16 / EB) < a.D && j * BN + r < sq.len))
        k = v = reinterpret_cast<const unsigned char*>(&ZEROS);
      if (F8) {
        kreg[i] = *GLOBAL_PTR(const u32x4, k);
        vreg[i] = *GLOBAL_PTR(const u32x4, v);
      } else {
        const uint32_t to = lds + stage + (i * NW + wave) * 1024;
        gather16(k, to);
        gather16(v, to + TILE);
      }
    }
  };
  auto keep = [&](int stage) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = (i * NW + wave) * RPL + lane / PPR;
      unsigned char* at = smem + stage + r * L::RB;
      const int s0 = ((2 * piece) ^ L::swz(r)) * 16, s1 = ((2 * piece + 1) ^ L::swz(r)) * 16;
      *LDS_PTR(u32x4, at + s0) = cvt8(kreg[i][0], kreg[i][1]);
      *LDS_PTR(u32x4, at + s1) = cvt8(kreg[i][2], kreg[i][3]);
      *LDS_PTR(u32x4, at + TILE + s0) = cvt8(vreg[i][0], vreg[i][1]);
      *LDS_PTR(u32x4, at + TILE + s1) = cvt8(vreg[i][2], vreg[i][3]);
    }
  };

  auto start = [&] {  // the first tile, whose page ids are looked up
    fetch(j0, 0);
    if (j0 + 1 < j1) look(j0 + 1);
  };
  start();

  if (j1 * BN > past) {
    for (int i = threadIdx.x; i < sq.m; i += 64 * NW) {
      const int q = a.parents[sq.row0 + i];
      up[i] = q >= 0 && q < i ? q : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < sq.m; i += 64 * NW) {
      uint64_t w[WORDS] = {};
      for (int n = i; n >= 0; n = up[n])
#pragma unroll
        for (int k = 0; k < WORDS; ++k)
          if (n >> 6 == k) w[k] |= 1ull << (n & 63);
#pragma unroll
      for (int k = 0; k < WORDS; ++k) paths[i * WORDS + k] = w[k];
    }
    __syncthreads();
  }

  f32x4 o[L::DB][QF];
  float m[QF], l[QF];
  // All tiles of the part, the first of which is being loaded.  FIXED: the reference is the first tile's maximum, and hidden
  // values are finite (0 times another would be NaN); true where that will not do.
  auto pass = [&](auto fixed) __attribute__((always_inline)) {
    constexpr bool FIXED = decltype(fixed)::value;
    bool bad = false;
#pragma unroll
    for (int f = 0; f < QF; ++f) {
      m[f] = -INFINITY;
      l[f] = 0.0f;
#pragma unroll
      for (int d = 0; d < L::DB; ++d) o[d][f] = f32x4{0, 0, 0, 0};
    }
    // DRAFTED: tiles that hold drafted tokens; FIRST: or a column's first
    auto step = [&](int j, int off, auto drafted, auto begins) __attribute__((always_inline)) {
      constexpr bool DRAFTED = decltype(drafted)::value, FIRST = decltype(begins)::value;
      f32x4 s[KB][QF];
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int f = 0; f < QF; ++f) s[b][f] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int d = 0; d < DS; ++d)
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          const bf16x8 kk = kf.read(off, b, d);
#pragma unroll
          for (int f = 0; f < QF; ++f)
            s[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[f][d], s[b][f], 0, 0, 0);
        }
      uint64_t see[QF];
      if (DRAFTED) {
        const int at = j * BN + kg * (BN / KG) - past;
#pragma unroll
        for (int f = 0; f < QF; ++f) {
          see[f] = seen_bits(paths + node[f] * WORDS, at, BN / KG);
          const uint64_t mine = see[f] >> (4 * g);
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!((mine >> (16 * b + i)) & 1)) s[b][f][i] = -INFINITY;
        }
        if (FIXED) bad = bad || not_finite<TILE, NW>(smem + off + TILE, wave, lane);
      }
      if (!FIXED || FIRST) {
#pragma unroll
        for (int f = 0; f < QF; ++f) {
          float x = s[0][f][0];
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) x = fmaxf(x, s[b][f][i]);
          x = col_max(x);
          if (FIXED) {
            // no score, though the column sees a key of the group's
            bad = bad || (m[f] == -INFINITY && x == -INFINITY && (!DRAFTED || see[f] != 0));
            m[f] = m[f] == -INFINITY ? x : m[f];
          } else {
            x = fmaxf(x, m[f]);
            const float r = exp2_(m[f] * p.c - (x == -INFINITY ? 0.0f : x * p.c));  // 0 the first time
            m[f] = x;
            l[f] *= r;
#pragma unroll
            for (int d = 0; d < L::DB; ++d) o[d][f] *= r;
          }
        }
      }
#pragma unroll
      for (int f = 0; f < QF; ++f) {
        const float base = (!FIXED || FIRST) && m[f] == -INFINITY ? 0.0f : m[f] * p.c;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[b][f][i] = exp2_(s[b][f][i] * p.c - base);
            sum[i] += s[b][f][i];
          }
        l[f] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      // products over 32 keys, or the 16 that each of four groups has
      constexpr int NT = KB > 1 ? KB / 2 : 1;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        bf16x8 pf[QF];
#pragma unroll
        for (int f = 0; f < QF; ++f) pf[f] = pack8(s[KB > 1 ? 2 * t : 0][f], s[KB > 1 ? 2 * t + 1 : 0][f]);
#pragma unroll
        for (int d = 0; d < L::DB; ++d) {
          const bf16x8 vv = KB > 1 ? vf.read(off, t, d) : vf.read_half(off, d);
#pragma unroll
          for (int f = 0; f < QF; ++f) {
            if (FIXED || !DRAFTED) {
              o[d][f] = product<KB == 1>(vv, pf[f], o[d][f]);
              continue;
            }
            // every column by itself, from the keys that it sees
            f32x4 r = o[d][f];
#pragma unroll 1
            for (int c = 0; c < 16; ++c) {
              const uint64_t w = __shfl(see[f], c) >> (32 * t + 4 * g);
              u32x4 x = __builtin_bit_cast(u32x4, vv);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t two = (uint32_t)(w >> ((i & 1) * 2 + (i >> 1) * 16));
                x[i] &= (two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u);
              }
              const f32x4 y = product<KB == 1>(__builtin_bit_cast(bf16x8, x), pf[f], o[d][f]);
              if (col == c) r = y;
            }
            o[d][f] = r;
          }
        }
      }
    };
    const int full = min(max(past / BN, j0), j1);  // tiles of tokens that every row sees
    // bf16: the next tile's direct loads are in flight while this one is used; E4M3: its
    // registers' loads are.  In both each of the two stages is written after the barrier that
    // ends its last use.
    int stage = 0;
    auto turn = [&](int j, auto drafted, auto begins) __attribute__((always_inline)) {
      if (F8) keep(stage);
      else wait_vmcnt_and_barrier<0>();
      if (j + 1 < j1) fetch(j + 1, stage ^ STAGE);
      if (j + 2 < j1) look(j + 2);
      if (F8) lds_barrier();
      step(j, stage, drafted, begins);
      stage ^= STAGE;
    };
    int j = j0;
    if (FIXED && j < full) turn(j++, std::false_type{}, std::true_type{});
    for (; j < full; ++j) turn(j, std::false_type{}, std::false_type{});
    for (; j < j1; ++j) turn(j, std::true_type{}, std::true_type{});
    if (FIXED) {
      float z = 0.0f;  // NaN if an output is not finite
#pragma unroll
      for (int f = 0; f < QF; ++f) {
        bad = bad || !(l[f] < MOST);
#pragma unroll
        for (int d = 0; d < L::DB; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) z += o[d][f][i] * 0.0f;
      }
      bad = bad || z != 0.0f;
    }
    __syncthreads();
    return bad;
  };
  if (any_wave<NW>(pass(std::true_type{}), smem, wave, lane)) {
    look(j0);
    start();
    pass(std::false_type{});
  }
  lost = __ballot(lost) != 0;

  float base[QF], sum[QF];
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    sum[f] = col_sum(l[f]);
    base[f] = m[f] == -INFINITY ? -INFINITY : m[f] * p.c;
    if (lost) sum[f] = NAN;
  }
  constexpr int MINE = (L::DB + KG - 1) / KG;  // blocks of the output that a wave writes
  if (KG > 1) {
    f32x4* parts = reinterpret_cast<f32x4*>(smem);  // [KG][RW][DB][QF][64]
    float2* stats = reinterpret_cast<float2*>(smem + NW * L::DB * QF * 1024);  // [KG][RW][QF][16]
    f32x4* mine = parts + wave * L::DB * QF * 64 + lane;
#pragma unroll
    for (int f = 0; f < QF; ++f) {
#pragma unroll
      for (int d = 0; d < L::DB; ++d) mine[(d * QF + f) * 64] = o[d][f];
      if (g == 0) stats[(wave * QF + f) * 16 + col] = make_float2(base[f], sum[f]);
    }
    __syncthreads();
    const f32x4* all = parts + (rw * L::DB + kg) * QF * 64 + lane;
#pragma unroll
    for (int f = 0; f < QF; ++f) {
      float2 x[KG];
      float top = -INFINITY, tot = 0.0f;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        x[k] = stats[((k * RW + rw) * QF + f) * 16 + col];
        top = fmaxf(top, x[k].x);
      }
      const float b = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        x[k].x = exp2_(x[k].x - b);
        tot += x[k].x * x[k].y;
      }
      base[f] = top;
      sum[f] = tot;
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        if (i * KG + kg >= L::DB) break;
        f32x4 y = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KG; ++k) y += all[((k * RW * L::DB + i * KG) * QF + f) * 64] * x[k].x;
        o[i][f] = y;
      }
    }
  }
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int c0 = (rw * QF + f) * 16 + col, c = strip * COLS + c0;
    if (c >= cols) continue;
    const int head = kvh * group + c % group;
    const int64_t row = sq.row0 + c / group;
    const float inv = sum[f] == 0.0f ? 0.0f : p.v_inv / sum[f];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int e = 16 * (i * KG + kg) + 4 * g;
      if (e >= a.D) continue;
      if (alone) {
        const f32x4 x = o[i][f] * inv;
        *reinterpret_cast<uint2*>(a.out.p + row * a.out.rs + head * a.out.hs + e) =
            make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
      } else {
        *reinterpret_cast<f32x4*>(p.part + (self * COLS + c0) * a.D + e) = o[i][f];
      }
    }
    if (g == 0 && kg == 0) {
      if (!alone) p.stat[self * COLS + c0] = make_float2(base[f], sum[f]);
      else if (a.lse) a.lse[(int64_t)head * a.seqs.T + row] = sum[f] == 0.0f ? -INFINITY : base[f] * LN2 + logf(sum[f]);
    }
  }
}

// Rows of no sequence (zeros) and of sequences that are not good (NaN), and the sum of the parts,
// in order, of strips that have several.  A workgroup takes a row's heads, half a wave each in turn
// (JW 1), or JW waves share a row and head: wave w adds parts w, w + JW, ..., eight loads
// ahead.  Lane i, of 32 or 64, holds the 4 or 2 elements from 4 i or 2 i on.
template <int JW, int COLS>
__global__ __launch_bounds__(JW > 4 ? 64 * JW : 256) void attn_tree_join(TreeParams p) {
  constexpr int WAVES = JW > 4 ? JW : 4, AHEAD = 8, LANES = JW == 1 ? 32 : 64, E = 128 / LANES;
  using Vec = float __attribute__((ext_vector_type(E)));
  __shared__ Vec red[WAVES][64];
  __shared__ float2 tops[WAVES];
  const TreeArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave % JW, T = a.seqs.T, group = a.H / a.G;
  const int row = JW == 1 ? blockIdx.x : blockIdx.x / a.H;
  // sequences that end at or before the row come first: their number is its sequence
  int seq = 0;
  for (int c = 0; c < a.seqs.n; c += 64) {
    const int i = c + lane;
    const int m = __popcll(__ballot((i < a.seqs.n ? a.seqs.cu[i + 1] : 0x7FFFFFFF) <= row));
    seq += m;
    if (m < 64) break;
  }
  Seq s{0, 0, 0, true};
  int4 in = make_int4(0, 1, 0, 0);
  if (seq < a.seqs.n) {
    s = sequence(p, seq);
    in = p.seqs[seq];  // not written, and not used, for one that is not good
  }
  const bool none = seq >= a.seqs.n || row < s.row0;
  if (!none && s.good) {
    if (in.y == 1) return;
    // (sequences that overlap, of boundaries that do not rise, may have left anything)
    if (in.x < 0 || in.y < 1 || in.z < 1 || in.w > ROUNDS * p.at_once || in.x + (int64_t)in.y * in.z > in.w) return;
  }
  const int e = lane % LANES * E;
  auto write = [&](uint16_t* out, Vec x) {
    if (e >= a.D) return;
#pragma unroll
    for (int k = 0; k < E; k += 2) *reinterpret_cast<uint32_t*>(out + e + k) = pack_bf16x2(x[k], x[k + 1]);
  };
  for (int head = JW == 1 ? 2 * wave + lane / LANES : blockIdx.x % a.H; head < a.H; head += JW == 1 ? 2 * WAVES : a.H) {
    uint16_t* out = a.out.p + (int64_t)row * a.out.rs + head * a.out.hs;
    float* lse = a.lse ? a.lse + (int64_t)head * T + row : nullptr;
    if (none || !s.good) {
      if (w == 0) {
        const float x = none ? 0.0f : NAN;
        write(out, Vec(x));
        if (e == 0 && lse) *lse = none ? -INFINITY : NAN;
      }
      continue;
    }
    const int kvh = head / group, c = (row - s.row0) * group + head - kvh * group;
    if (c / COLS >= in.z) continue;
    const int64_t first = ((int64_t)kvh * in.w + in.x + c / COLS) * COLS + c % COLS, step = (int64_t)in.z * COLS;
    float m = -INFINITY, sum = 0.0f;
    Vec x = 0.0f;
    for (int i0 = w; i0 < in.y; i0 += AHEAD * JW) {
      float2 st[AHEAD];
      Vec v[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int i = i0 + j * JW;
        const int64_t k = first + min(i, in.y - 1) * step;
        st[j] = i < in.y ? p.stat[k] : make_float2(-INFINITY, 0.0f);
        v[j] = *reinterpret_cast<const Vec*>(p.part + k * a.D + min(e, a.D - E));
      }
      float top = m;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) top = fmaxf(top, st[j].x);
      const float b = top == -INFINITY ? 0.0f : top;
      const float r = exp2_(m - b);
      m = top;
      sum *= r;
      x *= r;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (i0 + j * JW >= in.y) break;
        const float f = exp2_(st[j].x - b);
        sum += f * st[j].y;
        x += f * v[j];
      }
    }
    if (JW > 1) {
      red[wave][lane] = x;
      if (lane == 0) tops[wave] = make_float2(m, sum);
      __syncthreads();
      if (w != 0) return;
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < JW; ++k) top = fmaxf(top, tops[k].x);
      const float b = top == -INFINITY ? 0.0f : top;
      m = top;
      sum = 0.0f;
      x = 0.0f;
#pragma unroll
      for (int k = 0; k < JW; ++k) {
        const float f = exp2_(tops[k].x - b);
        sum += f * tops[k].y;
        x += f * red[k][lane];
      }
    }
    const float inv = sum == 0.0f ? 0.0f : p.v_inv / sum;
    write(out, x * inv);
    if (e == 0 && lse) *lse = sum == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) * LN2 + logf(sum);
  }
}

constexpr int MOST_COLS = 128;
int at_once(int G) { return G < ITEMS ? ITEMS / G : 1; }
int64_t part_bytes(int G, int D, int cols) { return (int64_t)ROUNDS * at_once(G) * G * cols * (8 + 4 * (int64_t)D); }

template <class S>
hipError_t run(const TreeArgs& a, hipStream_t s) {
  TreeParams p{};
  p.a = a;
  p.cap = table_cap(a.pages_per_seq, a.cache.page_size);
  p.c = a.scale * LOG2E * (S::F8 ? 1.0f / a.cache.k_scale : 1.0f);
  p.v_inv = S::F8 ? 1.0f / a.cache.v_scale : 1.0f;
  p.at_once = at_once(a.G);
  p.div = page_div((uint32_t)a.cache.page_size);
  const int64_t rows = (int64_t)ROUNDS * p.at_once * a.G * S::COLS;
  p.stat = static_cast<float2*>(a.ws);
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + rows * 8);
  p.seqs = reinterpret_cast<int4*>(p.part + rows * a.D);
  // as many workgroups as strips there can be, if those are more than run at once
  const int64_t strips = (int64_t)a.seqs.T * (a.H / a.G) / S::COLS + a.seqs.n;
  const int64_t most = (int64_t)ROUNDS * p.at_once;
  const int64_t blocks = ((strips > most ? strips : most) * a.G + NUM_XCD - 1) / NUM_XCD * NUM_XCD;
  const int64_t outputs = (int64_t)a.seqs.T * a.H;
  if (outputs > 0x7FFFFFFF || blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kernel = &attn_tree<S>;
  hipError_t e = ensure_lds_attr(reinterpret_cast<const void*>(kernel), S::LDS);
  if (e == hipSuccess && a.seqs.n > 0) e = launch_k(kernel, dim3((unsigned)blocks), dim3(64 * NW), S::LDS, s, p);
  if (e != hipSuccess || outputs == 0) return e;
  // few outputs have many parts, which more waves then share; many are a row's heads to a workgroup
  // (13 us in the first case above; 19.5 with a workgroup of a wave each, 17-19 with a wave for a head)
  if (outputs <= 512) return launch_k(&attn_tree_join<16, S::COLS>, dim3((unsigned)outputs), dim3(1024), 0, s, p);
  if (outputs <= 4096) return launch_k(&attn_tree_join<4, S::COLS>, dim3((unsigned)outputs), dim3(256), 0, s, p);
  return launch_k(&attn_tree_join<1, S::COLS>, dim3((unsigned)a.seqs.T), dim3(256), 0, s, p);
}

template <int DS, bool F8>
hipError_t choose(const TreeArgs& a, hipStream_t s) {
  // By the columns of a sequence, on average: the host knows no more.  Fewer columns to a wave or
  // workgroup read the same keys more often, more of them multiply by columns that are not there.
  const int64_t cols = a.seqs.n > 0 ? ((int64_t)a.seqs.T * (a.H / a.G) + a.seqs.n - 1) / a.seqs.n : 1;
  if (cols <= 16) return run<Shape<DS, 1, 1, F8>>(a, s);
  if (cols <= 32) return run<Shape<DS, 2, 1, F8>>(a, s);
  if (cols <= 64) return run<Shape<DS, 2, 2, F8>>(a, s);
  return run<Shape<DS, 2, 4, F8>>(a, s);
}

template <bool F8>
hipError_t by_dim(const TreeArgs& a, hipStream_t s) {
  if (a.D <= 64) return choose<2, F8>(a, s);
  if (a.D <= 96) return choose<3, F8>(a, s);
  return choose<4, F8>(a, s);
}

}  // namespace

size_t attn_tree_bytes(int32_t H, int32_t G, int32_t D, int64_t rows, int32_t n) {
  return (size_t)(part_bytes(G, D, MOST_COLS) + (int64_t)n * 16);
}

hipError_t launch_attn_tree(const TreeArgs& a, hipStream_t s) {
  return a.cache.e4m3 ? by_dim<true>(a, s) : by_dim<false>(a, s);
}

}  // namespace ubx
