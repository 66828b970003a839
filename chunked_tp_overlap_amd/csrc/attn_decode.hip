// Attention of one new token per sequence over a paged key-value cache.
//
//   s_u = scale q . k_u,  lse = log sum_u exp(s_u),  out = sum_u exp(s_u - lse) v_u
//
// HBM-bound: the keys and values of every cached token are read once and used for a few
// operations each.  The lengths are on the device and ragged, so the work is cut by them
// there: the tokens of all sequences, in units of 32 one sequence after another, are dealt in
// equal contiguous ranges over as many workgroups as run at once, so that none waits for a
// second round.  A workgroup finds its range from the lengths and walks the sequences that it
// covers.  It finishes a sequence that lies in its range whole; parts of one (maximum, sum and
// unnormalised output, fp32) go to the workspace: at most two per workgroup, that of its first
// sequence and that of its last.  attn_decode_join adds a sequence's parts in order.
//
// A wave takes 32 tokens at a time.  Scores are K q^T on matrix cores, the query heads of a
// group (up to 16) as the 16 columns: keys go from memory straight into the A fragment.
// Values pass through a wave-private LDS tile, from which transposing reads give V^T
// (attn_common.h).  The next step's keys and values are loaded into registers before the
// present ones are used, which holds 16 KB in flight for each of a CU's 8 waves throughout;
// more waves without that (12, or 16 with fewer registers) were slower (110, 137 us against
// 104 in the first case below).
//
// Measured on MI355X, both kernels, where a plain read reaches 5.3 to 6.4 TB/s (1 GiB, by the number
// of workgroups and the cache policy): 64 sequences of 1 to 8192 tokens, 4 + 4 heads of 128, bf16,
// pages of 16: 104 us (4.9 TB/s); 128 of 100 to 32520, 8 heads on 1, E4M3, pages of 64: 94 us (5.6
// TB/s).  Under a window of 4096 and 16 first tokens 64 of 1 to 16264 tokens, as the first: 97 us (4.9);
// E4M3 57 (4.1).
#include <hip/hip_runtime.h>

#include "attn_common.h"
#include "kv_pages.h"

namespace ubx {
namespace {

constexpr int NW = 4;
constexpr int STEP = 32;          // tokens a wave takes at a time
constexpr int ITEMS = 512;        // workgroups that run at once: two on each CU
constexpr int MIN_UNITS = 8;      // units of 32 tokens that a workgroup takes at least, if sequences are as long
constexpr int COLS = 16;          // query heads of a workgroup

struct DecodeParams {
  DecodeArgs a;
  float c;          // scale * log2(e) (/ k_scale)
  float v_inv;      // 1 / v_scale
  int32_t qb;       // column blocks of a group
  int32_t cap;      // tokens the page table can hold per sequence
  int32_t ranges;   // most ranges the tokens are dealt in; G qb workgroups share one
  int2* parts_of;   // [n]: a sequence's first part's row of `part`, and its number of parts
  float* part;      // [2 ranges, G qb, COLS, D]: parts of a range's first and last sequence
  float2* stat;     // [2 ranges, G qb, COLS]: maximum (base 2, scaled), sum
};

// Cached tokens of sequence i, as far as the page table reaches.
__device__ inline int kv_len(const DecodeParams& p, int i) { return clamp_len(p.a.lens[i], p.cap); }

// Units of a sequence of len tokens that its new token sees: all, or under a window `sink` of
// the first tokens and those from unit sink + gap on.  Tokens before `from` are hidden but for
// the first win.sinks.
struct Units {
  int n, sink, gap, from;
  __device__ int token(int u) const { return (u < sink ? u : u + gap) * STEP; }
};
template <bool WIN>
__device__ inline Units units(int len, Window win) {
  Units u{(len + STEP - 1) / STEP, 0, 0, 0};
  if (WIN) {
    u.from = max(len - win.size, 0);
    u.sink = min((win.sinks + STEP - 1) / STEP, u.from / STEP);
    u.gap = u.from / STEP - u.sink;
    u.n -= u.gap;
  }
  return u;
}

// Ranges for S units of n sequences.  A range takes MIN_UNITS units at least, unless sequences are shorter: each that a range
// covers costs it a chain of loads and a join of its waves, some 3 us, so that there are 4 n
// ranges if there can be.  Measured with 0, n, 2 n and 4 n: 23 sequences of up to 3 tokens, 8 heads
// on 1 35, 13, 13, 13 us; 64 of 20 to 200 29, 23, 18, 18; 160 of 50 to 500, 16 heads on 1 33, 33, 35,
// 30.
__device__ inline int ranges_of(int64_t S, int n, int most) {
  return (int)min((int64_t)most, max((S + MIN_UNITS - 1) / MIN_UNITS, min(S, 4 * (int64_t)n)));
}

// Units of sequences c + lane, up to 2^25 each: 64 of them fit 32 unsigned bits.
template <bool WIN>
__device__ inline uint32_t units_of(const DecodeParams& p, int c) {
  const int i = c + (threadIdx.x & 63);
  return i < p.a.n ? units<WIN>(kv_len(p, i), p.a.win).n : 0;
}

// head: units_of(p, 0)
template <bool WIN>
__device__ inline Deal deal_units(const DecodeParams& p, uint32_t head) {
  int64_t S = (uint32_t)wave_sum((int)head);
  for (int c = 64; c < p.a.n; c += 64) S += (uint32_t)wave_sum((int)units_of<WIN>(p, c));
  Deal d;
  d.init(S, ranges_of(S, p.a.n, p.ranges));
  return d;
}

// The sequence that holds a unit, and the units before that sequence.
template <bool WIN>
__device__ inline int find_sequence(const DecodeParams& p, uint32_t head, int64_t unit, int64_t& first) {
  int64_t before = 0;
  for (int c = 0; c < p.a.n; c += 64) {
    const uint32_t u = c == 0 ? head : units_of<WIN>(p, c);
    const uint32_t incl = (uint32_t)wave_scan((int)u);
    const uint64_t m = __ballot(before + incl > unit);
    if (m) {
      const int at = __builtin_ctzll(m);
      first = before + (uint32_t)__builtin_amdgcn_readlane((int)(incl - u), at);
      return c + at;
    }
    before += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
  return p.a.n;
}

template <int DS, bool F8>
struct Layout {
  static constexpr int EB = F8 ? 1 : 2;                                      // bytes per element
  static constexpr int KV = F8 ? (DS + 1) / 2 : DS;                          // 16-byte loads of a key row per lane
  static constexpr int VPR = F8 ? Tile<DS>::CPR / 2 : Tile<DS>::CPR;         // 16-byte pieces of a value row
  static constexpr int VI = STEP * VPR / 64;                                 // value loads per lane
};

// The 32 keys and values of a step: key row 16 b + lane % 16 of block b, and value rows
// i (64 / VPR) + lane / VPR.
template <int DS, bool F8>
struct Step {
  u32x4 k[2][Layout<DS, F8>::KV], v[Layout<DS, F8>::VI];
};

// WHOLE: pages of a multiple of 16 tokens, so that a block of 16 tokens lies in one page: its
// place is uniform over the wave, and its rows' offsets from there are the same in all steps.
// Otherwise every token's place is looked up.
// WIN: under a window (a.win).  Hidden tokens of a unit count as those past the end, and their
// pages, which may be gone, are not looked up where a block or token is hidden whole.
template <int DS, bool F8, bool WHOLE, bool WIN>
__global__ __launch_bounds__(64 * NW, DS == 2 ? 3 : 2) void attn_decode(DecodeParams p) {
  using L = Tile<DS>;
  using Y = Layout<DS, F8>;
  using S = Step<DS, F8>;
  constexpr int TILE = STEP * L::RB;
  constexpr int MERGE = NW * COLS * (32 * DS + 2) * 4;
  constexpr int SMEM = NW * TILE > MERGE ? NW * TILE : MERGE;
  constexpr int EB = Y::EB, KV = Y::KV, VPR = Y::VPR, VI = Y::VI;
  constexpr int RPI = 64 / VPR;  // value rows of a load
  __shared__ __align__(256) unsigned char smem[SMEM];
  const DecodeArgs& a = p.a;
  const int GQ = a.G * p.qb;
  const int gq = blockIdx.x % GQ, rank = blockIdx.x / GQ;
  const int kvh = gq / p.qb, group = a.H / a.G, col0 = (gq - kvh * p.qb) * COLS;
  const int cols = min(group - col0, COLS);
  const uint32_t head = units_of<WIN>(p, 0);
  const Deal deal = deal_units<WIN>(p, head);
  if (rank >= deal.W) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int64_t unit0 = deal.begin(rank), unit1 = deal.begin(rank + 1);
  const unsigned char* kb = static_cast<const unsigned char*>(a.cache.k) + kvh * a.cache.hs * EB;
  const unsigned char* vb = static_cast<const unsigned char*>(a.cache.v) + kvh * a.cache.hs * EB;
  unsigned char* tile = smem + wave * TILE;
  ColFrag<DS> vf;
  vf.init(tile, lane);
  const int pieces = a.D * EB / 16;
  const uint32_t row_bytes = (uint32_t)(a.cache.ts * EB);  // used when WHOLE only
  uint32_t kofs[KV];
  const int vpiece = lane % VPR < pieces ? lane % VPR : 0;
#pragma unroll
  for (int s = 0; s < KV; ++s) kofs[s] = (WHOLE ? col * row_bytes : 0) + (4 * s + g < pieces ? 4 * s + g : 0) * 16;
  // Lanes whose last keys' piece lies past head_dim read piece 0, which their zero queries turn
  // into NaN if it is infinite (E4M3 has no infinity): those pieces count as zeros.
  u32x4 in_key[KV];
#pragma unroll
  for (int s = 0; s < KV; ++s) {
    const uint32_t in = 4 * s + g < pieces ? 0xFFFFFFFFu : 0u;
    in_key[s] = u32x4{in, in, in, in};
  }
  const uint32_t vofs = (WHOLE ? lane / VPR * row_bytes : 0) + vpiece * 16;

  int64_t first = 0;  // units before the sequence
  int seq = find_sequence<WIN>(p, head, unit0, first);
  for (int64_t unit = unit0; unit < unit1 && seq < a.n; ++seq) {
    const int len = kv_len(p, seq);
    const Units un = units<WIN>(len, a.win);
    const int64_t last = first + un.n;  // units up to the sequence's end
    if (last == first) continue;
    const int ubegin = (int)(unit - first), uend = (int)(min(last, unit1) - first);
    const int begin = ubegin * STEP;
    const int end = WIN ? len : (int)min((int64_t)uend * STEP, (int64_t)len);
    const bool alone = unit == first && last <= unit1;
    const int64_t item = (int64_t)(2 * rank + (unit != unit0)) * GQ + gq;
    if (unit == first && gq == 0 && threadIdx.x == 0)
      p.parts_of[seq] = make_int2(2 * rank + (unit != unit0), alone ? 1 : deal.range_of(last - 1) - rank + 1);
    unit = first = last;
    const int32_t* pages = a.pages + (int64_t)seq * a.pages_ld;
    bool bad = a.lens[seq] > p.cap;

    // queries: element order of the key fragments below
    bf16x8 q[DS];
    const uint16_t* qrow = a.q.p + (int64_t)seq * a.q.rs + (kvh * group + col0 + col) * a.q.hs;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      const int e = F8 ? 64 * (s / 2) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
      q[s] = load_row8(qrow + e, col < cols && e < a.D);
    }
    f32x4 o[L::DB];
#pragma unroll
    for (int d = 0; d < L::DB; ++d) o[d] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    // The wave's steps: tokens t0 + NW STEP j .. + 31, j < n; under a window those of unit
    // ubegin + wave + NW j.
    const int t0 = begin + wave * STEP;
    const int n = WIN ? max(uend - ubegin - wave + NW - 1, 0) / NW
                      : t0 < end ? (end - t0 + NW * STEP - 1) / (NW * STEP) : 0;
    auto token_of = [&](int j) { return WIN ? un.token(ubegin + wave + j * NW) : t0 + j * (NW * STEP); };
    auto hidden = [&](int t) { return t >= end || (WIN && t < un.from && t >= a.win.sinks); };
    int64_t place = 0;  // element offset of a token in head 0, or -1
    auto look_up = [&](int t) {
      place = token_offset(t, pages[page_entry(t, a.cache.page_size, a.pages_per_seq)], a.cache.n_pages,
                           a.cache.page_size, a.cache.ps, a.cache.ts);
      bad = bad || place < 0;
      place = max(place, (int64_t)0) * EB;
    };
    // E4M3 rows pass by the caches.  Measured, passing by and not: the second case above 95 and
    // 105 us, 64 sequences of 100 to 8192 tokens, 2 heads of 64 on 2 26 and 39.  Of bf16, where
    // a row takes two lines, only some calls gain: with its values alone passing by, the first
    // case takes 99 instead of 104, but 32 sequences of 4000 to 8192, 32 heads on 1 (two
    // workgroups read each row) 59 instead of 53, 64 of 100 to 8192, 2 heads of 64 on 2 54
    // instead of 51.
    auto load = [](const unsigned char* at) {
      return F8 ? __builtin_nontemporal_load(GLOBAL_PTR(const u32x4, at)) : *GLOBAL_PTR(const u32x4, at);
    };
    auto fetch = [&](int j, S& x) {
      const int t = token_of(j);
      if (WHOLE) {
        // lane 2 i + b: block b of the i-th step from here, 32 steps at a time
        if (WIN) {
          if (j % 32 == 0) {
            const int b = token_of(min(j + (lane >> 1), n - 1)) + (lane & 1) * 16, sinks = a.win.sinks;
            look_up(b >= end || (b >= sinks && b + 16 <= un.from) ? (end - 1) / 16 * 16 : b);
          }
        } else if (j % 32 == 0) {
          look_up(min(t + (lane >> 1) * (NW * STEP) + (lane & 1) * 16, (end - 1) / 16 * 16));
        }
        const int i = j % 32 * 2;
        const int64_t at[2] = {lane_of(place, i), lane_of(place, i + 1)};
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int s = 0; s < KV; ++s) x.k[b][s] = load(kb + at[b] + kofs[s]);
#pragma unroll
        for (int i = 0; i < VI; ++i)
          x.v[i] = load(vb + at[i * RPI / 16] + (int64_t)(i * RPI % 16) * row_bytes + vofs);
      } else {
        if (WIN) look_up(hidden(t + (lane & 31)) ? end - 1 : t + (lane & 31));
        else look_up(min(t + (lane & 31), end - 1));  // past the end: the last token again
        const int lo = (int)(uint32_t)place, hi = (int)(place >> 32);
        auto row = [&](int r) {
          return (int64_t)(((uint64_t)(uint32_t)__shfl(hi, r) << 32) | (uint32_t)__shfl(lo, r));
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const unsigned char* at = kb + row(16 * b + col);
#pragma unroll
          for (int s = 0; s < KV; ++s) x.k[b][s] = load(at + kofs[s]);
        }
#pragma unroll
        for (int i = 0; i < VI; ++i)
          x.v[i] = load(vb + row(i * RPI + lane / VPR) + vofs);
      }
    };
    auto use = [&](int j, S& x) {
      const int t = token_of(j);
      f32x4 s[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
      for (int d = 0; d < DS; ++d)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const u32x4 y = x.k[b][F8 ? d / 2 : d];
          // above a head_dim of 64 only the last piece can lie past it
          const u32x4 w = F8 ? (d & 1 ? cvt8(y[2], y[3]) : cvt8(y[0], y[1])) : DS == 2 || d == DS - 1 ? y & in_key[d] : y;
          s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), q[d], s[b], 0, 0, 0);
        }
      if (t + STEP > end || (WIN && t < un.from)) {
        // rows past the end hold anything: no weight, and zeros, as 0 times anything is not 0
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (hidden(t + 16 * b + 4 * g + i)) s[b][i] = -INFINITY;
#pragma unroll
        for (int i = 0; i < VI; ++i)
          if (hidden(t + i * RPI + lane / VPR)) x.v[i] = u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < VI; ++i) {
        const int r = i * RPI + lane / VPR, piece = lane % VPR;
        if (F8) {
          const u32x4 w0 = cvt8(x.v[i][0], x.v[i][1]), w1 = cvt8(x.v[i][2], x.v[i][3]);
          *LDS_PTR(u32x4, tile + r * L::RB + (((2 * piece) ^ L::swz(r)) * 16)) = w0;
          *LDS_PTR(u32x4, tile + r * L::RB + (((2 * piece + 1) ^ L::swz(r)) * 16)) = w1;
        } else {
          *LDS_PTR(u32x4, tile + r * L::RB + ((piece ^ L::swz(r)) * 16)) = x.v[i];
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[b][i]);
      top = fmaxf(col_max(top), m);
      const float base = top == -INFINITY ? 0.0f : top * p.c;
      const float r = exp2_(m * p.c - base);
      m = top;
#pragma unroll
      for (int d = 0; d < L::DB; ++d) o[d] *= r;
      float sum = 0.0f;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[b][i] = exp2_(s[b][i] * p.c - base);
          sum += s[b][i];
        }
      l = l * r + sum;
      const bf16x8 pf = pack8(s[0], s[1]);
#pragma unroll
      for (int d = 0; d < L::DB; ++d)
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf.read(0, 0, d), pf, o[d], 0, 0, 0);
    };
    // A step's loads are in flight while the one before is used.  (The last step's are made
    // again in place of a next one's: a branch would make its wait one for all loads.)
    if (n > 0) {
      S x, y;
      fetch(0, x);
      for (int j = 0;; j += 2) {
        fetch(min(j + 1, n - 1), y);
        use(j, x);
        if (j + 1 >= n) break;
        fetch(min(j + 2, n - 1), x);
        use(j + 1, y);
        if (j + 2 >= n) break;
      }
    }
    bad = __ballot(bad) != 0;
    l = col_sum(l);
    if (bad) l = NAN;
    // join the waves: [wave][column][32 DS values, maximum, sum]
    __syncthreads();
    constexpr int ROW = 32 * DS + 2;
    float* mine = reinterpret_cast<float*>(smem) + (wave * COLS + col) * ROW;
#pragma unroll
    for (int d = 0; d < L::DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[16 * d + 4 * g + i] = o[d][i];
    if (g == 0) {
      mine[32 * DS] = m == -INFINITY ? -INFINITY : m * p.c;
      mine[32 * DS + 1] = l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < cols * a.D; i += 64 * NW) {
      const int h = i / a.D, d = i - h * a.D;
      const float* w0 = reinterpret_cast<const float*>(smem) + h * ROW;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) mm = fmaxf(mm, w0[w * COLS * ROW + 32 * DS]);
      const float b = mm == -INFINITY ? 0.0f : mm;
      float sum = 0.0f, x = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = exp2_(w0[w * COLS * ROW + 32 * DS] - b);
        sum += f * w0[w * COLS * ROW + 32 * DS + 1];
        x += f * w0[w * COLS * ROW + d];
      }
      const int head = kvh * group + col0 + h;
      if (alone) {
        const float inv = sum == 0.0f ? 0.0f : p.v_inv / sum;
        a.out.p[(int64_t)seq * a.out.rs + head * a.out.hs + d] = (uint16_t)pack_bf16x2(x * inv, 0.0f);
        if (d == 0 && a.lse)
          a.lse[(int64_t)head * a.T + seq] = sum == 0.0f ? -INFINITY : b * LN2 + logf(sum);
      } else {
        p.part[(item * COLS + h) * a.D + d] = x;
        if (d == 0) p.stat[item * COLS + h] = make_float2(mm, sum);
      }
    }
    __syncthreads();  // the next sequence's values may take the place of what was joined
  }
}

// Row and head of a workgroup: zeros for rows of no sequence or length 0; the sum of the
// parts, in order, for sequences of several ranges.  Wave w adds parts w, w + JW, ..., eight
// loads ahead (their places are known before their values); lane i holds elements 2 i, 2 i + 1.
template <int JW>
__global__ __launch_bounds__(64 * JW) void attn_decode_join(DecodeParams p) {
  __shared__ float2 red[JW][64];
  __shared__ float2 tops[JW];
  constexpr int AHEAD = 8;
  const DecodeArgs& a = p.a;
  const int head = blockIdx.x % a.H, row = blockIdx.x / a.H;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int len = row < a.n ? kv_len(p, row) : 0;
  uint16_t* out = a.out.p + (int64_t)row * a.out.rs + head * a.out.hs;
  if (len == 0) {
    if ((int)threadIdx.x < a.D / 2) *reinterpret_cast<uint32_t*>(out + 2 * threadIdx.x) = 0;
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)head * a.T + row] = -INFINITY;
    return;
  }
  const int2 parts = p.parts_of[row];
  const int count = parts.y;
  if (count == 1) return;
  const int group = a.H / a.G, kvh = head / group, hc = head - kvh * group;
  const int GQ = a.G * p.qb, gq = kvh * p.qb + hc / COLS, h = hc % COLS;
  // the first part may be its range's last sequence's, the others are their ranges' first
  auto at = [&](int i) {
    return ((int64_t)(i == 0 ? parts.x : (parts.x & ~1) + 2 * i) * GQ + gq) * COLS + h;
  };
  // the running maximum and sum of this wave's parts, as for the tokens
  float m = -INFINITY, sum = 0.0f;
  float2 x = make_float2(0.0f, 0.0f);
  for (int i0 = wave; i0 < count; i0 += AHEAD * JW) {
    float2 st[AHEAD], v[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int i = i0 + j * JW;
      const int64_t k = at(min(i, count - 1));
      st[j] = i < count ? p.stat[k] : make_float2(-INFINITY, 0.0f);
      v[j] = *reinterpret_cast<const float2*>(p.part + k * a.D + min(2 * lane, a.D - 2));
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) top = fmaxf(top, st[j].x);
    const float b = top == -INFINITY ? 0.0f : top;
    const float r = exp2_(m - b);
    m = top;
    sum *= r;
    x.x *= r;
    x.y *= r;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (i0 + j * JW >= count) break;
      const float f = exp2_(st[j].x - b);
      sum += f * st[j].y;
      x.x += f * v[j].x;
      x.y += f * v[j].y;
    }
  }
  red[wave][lane] = x;
  if (lane == 0) tops[wave] = make_float2(m, sum);
  __syncthreads();
  if (wave != 0) return;
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < JW; ++w) top = fmaxf(top, tops[w].x);
  const float b = top == -INFINITY ? 0.0f : top;
  sum = 0.0f;
  x = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < JW; ++w) {
    const float f = exp2_(tops[w].x - b);
    sum += f * tops[w].y;
    x.x += f * red[w][lane].x;
    x.y += f * red[w][lane].y;
  }
  const float inv = sum == 0.0f ? 0.0f : p.v_inv / sum;
  if (2 * lane < a.D) *reinterpret_cast<uint32_t*>(out + 2 * lane) = pack_bf16x2(x.x * inv, x.y * inv);
  if (lane == 0 && a.lse)
    a.lse[(int64_t)head * a.T + row] = sum == 0.0f ? -INFINITY : b * LN2 + logf(sum);
}

int64_t head_blocks(int32_t H, int32_t G) { return (int64_t)G * ((H / G + COLS - 1) / COLS); }
int32_t max_ranges(int64_t GQ) { return GQ < ITEMS ? (int32_t)(ITEMS / GQ) : 1; }

template <int DS, bool F8, bool WHOLE, bool WIN>
hipError_t run(const DecodeArgs& a, hipStream_t s) {
  DecodeParams p{};
  p.a = a;
  p.qb = (a.H / a.G + COLS - 1) / COLS;
  p.cap = table_cap(a.pages_per_seq, a.cache.page_size);
  p.c = a.scale * LOG2E * (F8 ? 1.0f / a.cache.k_scale : 1.0f);
  p.v_inv = F8 ? 1.0f / a.cache.v_scale : 1.0f;
  const int64_t GQ = head_blocks(a.H, a.G);
  p.ranges = max_ranges(GQ);
  const int64_t blocks = p.ranges * GQ;
  p.stat = static_cast<float2*>(a.ws);
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + 2 * blocks * COLS * 8);
  p.parts_of = reinterpret_cast<int2*>(p.part + 2 * blocks * COLS * a.D);
  if ((int64_t)a.T * a.H > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipError_t e = hipSuccess;
  if (a.n > 0) e = launch_k(&attn_decode<DS, F8, WHOLE, WIN>, dim3((unsigned)blocks), dim3(64 * NW), 0, s, p);
  if (e == hipSuccess)
    // Few rows: long sequences of many parts, so more waves share them (one sequence of 32520
    // tokens, 8 heads on 1, 127 parts: both kernels 17.1 us with 4 waves, 15.2 with 16)
    e = (int64_t)a.T * a.H <= 256
            ? launch_k(&attn_decode_join<16>, dim3((unsigned)(a.T * a.H)), dim3(1024), 0, s, p)
            : launch_k(&attn_decode_join<4>, dim3((unsigned)(a.T * a.H)), dim3(256), 0, s, p);
  return e;
}

template <int DS, bool F8>
hipError_t run_paged(const DecodeArgs& a, hipStream_t s) {
  // a block's offsets from its place take 32 bits
  const bool whole = a.cache.page_size % 16 == 0 && a.cache.ts < (1 << 26);
  if (a.win.size) return whole ? run<DS, F8, true, true>(a, s) : run<DS, F8, false, true>(a, s);
  return whole ? run<DS, F8, true, false>(a, s) : run<DS, F8, false, false>(a, s);
}

}  // namespace

size_t attn_decode_bytes(int32_t H, int32_t G, int32_t D, int32_t n) {
  const int64_t GQ = head_blocks(H, G);
  return (size_t)(2 * max_ranges(GQ) * GQ * COLS * (8 + (int64_t)D * 4) + (int64_t)n * 8);
}

hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s) {
  // E4M3 keys take two steps of a 16-byte piece each: an even number of them
  if (a.cache.e4m3) return a.D <= 64 ? run_paged<2, true>(a, s) : run_paged<4, true>(a, s);
  return a.D <= 64 ? run_paged<2, false>(a, s) : a.D <= 96 ? run_paged<3, false>(a, s) : run_paged<4, false>(a, s);
}

}  // namespace ubx
