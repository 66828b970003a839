// Gradient of causal attention within packed sequences.
//
//   P = exp(s - lse),  delta = dout . out,  dS = P (dout v^T - delta)
//   dq = scale dS k,   dk = scale dS^T q,   dv = P^T dout
//
// attn_bwd_rows leaves delta and lse log2(e) of each row in the workspace.  In attn_bwd two
// kinds of workgroups, each recomputing P from lse, take the three products' sums, so that
// every sum runs in one workgroup in a fixed order (no atomics, the same bits on every run):
//  - bwd_q owns query rows of one head and walks the key tiles, as the forward pass does.
//  - bwd_kv owns key rows of one key-value head and walks the query tiles of its heads.  With
//    few key tiles the heads of a group go to several workgroups, whose fp32 parts
//    attn_bwd_join adds in order.
//
// Measured on MI355X, all launches, calls one after another.  16264 tokens in 2 sequences, 8 heads of
// 128 on 1: 883 us, 1.08 PFLOP/s of the seven products done (five are counted); the matrix cores
// are busy 52% of the time at the 2.1 GHz that the power limit leaves.  8184 tokens in 5 sequences,
// 4 heads of 128 on 4: 170-174 us, bounded by the steps of the longest rows, as the forward pass.
// (One call at a time, under a profiler, its kernels take 187.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "attn_common.h"

namespace ubx {
namespace {

// NR waves of 32 rows each (of queries or keys), NG times: group grp takes the tiles (of keys
// or queries, ROWS rows in LDS) grp, grp + NG, ... of what the rows meet.
template <int DS_, int NR_, int NG_, int ROWS_>
struct Shape {
  static constexpr int DS = DS_, NR = NR_, NG = NG_, ROWS = ROWS_, F = 2;
  using L = Tile<DS>;
  static constexpr int NW = NR * NG, BM = 16 * F * NR, TILE = ROWS * L::RB;
  static constexpr int JOIN = NG > 1 ? NW * L::DB * F * 1024 : 0;
};

struct BwdParams {
  PromptBwdArgs a;
  float c;
  float* lse2;   // [H, T]
  float* delta;  // [H, T]
  float* part;   // [parts, 2, G, T, D] when parts > 1
  int32_t ranks;
  int32_t parts;
};

__device__ inline void dma4(i32x4 rsrc, uint32_t lds, uint32_t voffset) {
  __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(voffset),
                   "s"(rsrc)
                   : "memory");
}

// Zeros in the rows of no sequence, dealt over the workgroups of a head.
__device__ inline void fill_pad(const Heads& x, const Seqs& s, int D, int head, int rank, int ranks) {
  const int lo = first_row(s), hi = last_row(s);
  const int pad = lo + (s.T - hi);
  for (int i = rank; i < pad; i += ranks) {
    const int64_t t = i < lo ? i : hi + (i - lo);
    if ((int)threadIdx.x < D / 8)
      *GLOBAL_PTR(u32x4, x.p + t * x.rs + head * x.hs + threadIdx.x * 8) = u32x4{0, 0, 0, 0};
  }
}

__device__ inline void store4(uint16_t* p, f32x4 x) {
  uint2 w = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  *reinterpret_cast<uint2*>(p) = w;
}

// Sum over the LPR lanes (8 or 16) that share a row.
template <int LPR>
__device__ inline float row_sum(float x) {
  auto add = [&](float y) { x += y; };
  add(__int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xf, 0xf, true)));   // lane ^ 1
  add(__int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xf, 0xf, true)));   // lane ^ 2
  add(__int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xf, 0xf, true)));  // 7 - lane
  if (LPR == 16)
    add(__int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x140, 0xf, 0xf, true)));  // 15 - lane
  return x;
}

// delta and lse log2(e) of all rows, 32 of one head to a wave; what they are in rows of no
// sequence is not read.
template <int LPR>
__global__ __launch_bounds__(256) void attn_bwd_rows(BwdParams p) {
  constexpr int AT_ONCE = 64 / LPR, N = 32 / AT_ONCE;
  const PromptBwdArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t T = a.seqs.T, task = (int64_t)blockIdx.x * 4 + wave;
  const int head = (int)(task % a.H);
  const int64_t row0 = task / a.H * 32;
  if (row0 >= T) return;
  const int e = lane % LPR * 8;
  bf16x8 d[N], o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = row0 + i * AT_ONCE + lane / LPR;
    const bool in = row < T && e < a.D;
    d[i] = load_row8(a.dout.p + row * a.dout.rs + head * a.dout.hs + e, in);
    o[i] = load_row8(a.out.p + row * a.out.rs + head * a.out.hs + e, in);
  }
  if (lane < 32 && row0 + lane < T) {
    const int64_t at = head * T + row0 + lane;
    const float l = a.lse[at];
    p.lse2[at] = l == -INFINITY ? 0.0f : l * LOG2E;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) x += (float)d[i][k] * (float)o[i][k];
    x = row_sum<LPR>(x);
    const int64_t row = row0 + i * AT_ONCE + lane / LPR;
    if (lane % LPR == 0 && row < T) p.delta[head * T + row] = x;
  }
}

// What pack8 leaves of 8 values, as bf16.  P and dS are rounded to bf16 for the matrix cores, by
// up to 2^-8 of each.  The rows of few keys, in the diagonal tiles, have the largest dS, and
// those that suffer most from delta's error (out is bf16): their dS is used as two bf16 numbers,
// which takes the gradients' error from 1.53 of that of their own rounding to 1.32 (sequences of 1
// to 521 tokens; 1.47 to 1.37 with 817 to 5038) for 13.4 us instead of 12.6.
__device__ inline bf16x8 rest8(f32x4 a, f32x4 b, bf16x8 hi) {
  auto rest = [](float x, __bf16 h) {
    const float r = x - (float)h;
    return fabsf(r) < 1e38f ? r : 0.0f;  // x, or its rounding, may be infinite
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = rest(a[i], hi[i]);
    b[i] = rest(b[i], hi[4 + i]);
  }
  return pack8(a, b);
}

template <class S>
__device__ __forceinline__ void bwd_q(const BwdParams& p, int head, int rank, unsigned char* smem) {
  constexpr int DS = S::DS, QF = S::F, NG = S::NG, BN = S::ROWS, BM = S::BM, TILE = S::TILE;
  using L = Tile<DS>;
  constexpr int STAGE = NG * 2 * TILE;
  const PromptBwdArgs& a = p.a;
  fill_pad(a.dq, a.seqs, a.D, head, rank, p.ranks);
  const SeqTile st = find_tile(a.seqs, BM, rank, false);
  if (st.len == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave % S::NR, grp = wave / S::NR;
  const int col = lane & 15, g = lane >> 4;
  const int kvh = head / (a.H / a.G);
  const int q0 = st.tile * BM;
  const int wq0 = q0 + w * 16 * QF;
  const int n_keys = min(q0 + BM, st.len);
  const int tiles = (n_keys + BN - 1) / BN;
  const uint16_t* kbase = a.k.p + (int64_t)st.row0 * a.k.rs + kvh * a.k.hs;
  const uint16_t* vbase = a.v.p + (int64_t)st.row0 * a.v.rs + kvh * a.v.hs;
  TileLoad<DS, BN, S::NR> kl, vl;
  kl.init(w, lane, a.k.rs, a.D);
  vl.init(w, lane, a.v.rs, a.D);
  const uint32_t lds = lds_addr(smem) + grp * 2 * TILE;
  auto load = [&](int j, int stage) {
    kl.issue(kbase + (int64_t)j * BN * a.k.rs, a.k.rs, a.D, st.len - j * BN, lds + stage * STAGE, w);
    vl.issue(vbase + (int64_t)j * BN * a.v.rs, a.v.rs, a.D, st.len - j * BN, lds + stage * STAGE + TILE, w);
  };
  if (grp < tiles) load(grp, 0);
  bf16x8 q[QF][DS], dout[QF][DS];
  float lse2[QF], delta[QF];
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int t = wq0 + f * 16 + col;
    const bool ok = t < st.len;
    const int64_t row = st.row0 + t;
    const uint16_t* qr = a.q.p + row * a.q.rs + head * a.q.hs;
    const uint16_t* dr = a.dout.p + row * a.dout.rs + head * a.dout.hs;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      const int e = 32 * s + 8 * g;
      q[f][s] = load_row8(qr + e, ok && e < a.D);
      dout[f][s] = load_row8(dr + e, ok && e < a.D);
    }
    lse2[f] = ok ? p.lse2[(int64_t)head * a.seqs.T + row] : 0.0f;
    delta[f] = ok ? p.delta[(int64_t)head * a.seqs.T + row] : 0.0f;
  }
#pragma unroll
  for (int f = 0; f < QF; ++f)
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      arrived(q[f][s]);
      arrived(dout[f][s]);
    }
  RowFrag<DS> rf;  // of k; v's lie TILE bytes on
  ColFrag<DS> cf;
  rf.init(smem + grp * 2 * TILE, lane);
  cf.init(smem + grp * 2 * TILE, lane);
  f32x4 acc[L::DB][QF];
  const int steps = (tiles + NG - 1) / NG;
  const bool late = grp >= (NG + 1) / 2;
  // All key tiles, the first of which is being loaded; true if a diagonal one holds values that
  // are not finite, unless it is CAREFUL of them.
  auto pass = [&](auto careful) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(careful)::value;
    bool bad = false;
#pragma unroll
    for (int d = 0; d < L::DB; ++d)
#pragma unroll
      for (int f = 0; f < QF; ++f) acc[d][f] = f32x4{0, 0, 0, 0};
    if (late) phase_barrier();
    // DIAGONAL: tiles that may hold keys after one of the workgroup's queries
    auto step = [&](int i, auto diagonal) __attribute__((always_inline)) {
      constexpr bool DIAGONAL = decltype(diagonal)::value;
      const int j = i * NG + grp;
      const int stage = (i & 1) * STAGE;
      wait_vmcnt_and_barrier<0>();
      if (j + NG < tiles) load(j + NG, (i + 1) & 1);
      const bool live = NG == 1 || j < tiles;
      const int k0 = j * BN;
      if (!CAREFUL && DIAGONAL && live)
        bad = bad || not_finite<TILE, S::NR>(smem + grp * 2 * TILE + stage, w, lane);
#pragma unroll
      for (int t = 0; t < BN / 32; ++t) {
        f32x4 s[2][QF], dp[2][QF];
        if (live) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int f = 0; f < QF; ++f) {
              s[b][f] = f32x4{0, 0, 0, 0};
              dp[b][f] = f32x4{0, 0, 0, 0};
            }
#pragma unroll
          for (int d = 0; d < DS; ++d)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const bf16x8 kk = rf.read(stage, 2 * t + b, d);
              const bf16x8 vv = rf.read(stage + TILE, 2 * t + b, d);
#pragma unroll
              for (int f = 0; f < QF; ++f) {
                s[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[f][d], s[b][f], 0, 0, 0);
                dp[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, dout[f][d], dp[b][f], 0, 0, 0);
              }
            }
        }
        if (NG > 1) phase_barrier();
        if (!live) continue;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int f = 0; f < QF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[b][f][i] = exp2_(s[b][f][i] * p.c - lse2[f]) * (dp[b][f][i] - delta[f]);
        if (DIAGONAL && k0 + BN - 1 > wq0) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int f = 0; f < QF; ++f)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (k0 + t * 32 + b * 16 + 4 * g + i > wq0 + f * 16 + col) s[b][f][i] = 0.0f;
        }
        bf16x8 ds[QF], rest[QF];
#pragma unroll
        for (int f = 0; f < QF; ++f) {
          ds[f] = pack8(s[0][f], s[1][f]);
          if (DIAGONAL) rest[f] = rest8(s[0][f], s[1][f], ds[f]);
        }
        if (CAREFUL && DIAGONAL) {
#pragma unroll
          for (int d = 0; d < L::DB; ++d)
#pragma unroll
            for (int f = 0; f < QF; ++f) {
              acc[d][f] = seen_product<true>(cf.read(stage, t, d), ds[f], acc[d][f], k0 + t * 32, wq0 + f * 16, lane);
              acc[d][f] = seen_product<true>(cf.read(stage, t, d), rest[f], acc[d][f], k0 + t * 32, wq0 + f * 16, lane);
            }
          continue;
        }
#pragma unroll
        for (int d = 0; d < L::DB; ++d) {
          const bf16x8 kk = cf.read(stage, t, d);
#pragma unroll
          for (int f = 0; f < QF; ++f) {
            acc[d][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, ds[f], acc[d][f], 0, 0, 0);
            if (DIAGONAL) acc[d][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, rest[f], acc[d][f], 0, 0, 0);
          }
        }
      }
    };
    const int full = min(q0 / (BN * NG), steps);  // steps of tiles before every query
    int i = 0;
    for (; i < full; ++i) step(i, std::false_type{});
    for (; i < steps; ++i) step(i, std::true_type{});
    if (NG > 1 && !late) phase_barrier();
    return bad;
  };
  if (any_wave<S::NW>(pass(std::false_type{}), smem, wave, lane)) {
    if (grp < tiles) load(grp, 0);
    pass(std::true_type{});
  }
  if (NG > 1) join_groups<NG, S::NR>(acc, smem, grp, w, lane);
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int t = wq0 + f * 16 + col;
    if (t >= st.len) continue;
    uint16_t* out = a.dq.p + (int64_t)(st.row0 + t) * a.dq.rs + head * a.dq.hs;
#pragma unroll
    for (int i = 0; i < (L::DB + NG - 1) / NG; ++i) {
      const int e = 16 * (i * NG + grp) + 4 * g;
      if (e < a.D) store4(out + e, acc[i][f] * a.scale);
    }
  }
}

// The values stay in LDS beside the query tiles: with them in registers too, the 128
// accumulators of 32 keys left too few for the rest.
template <class S>
__device__ __forceinline__ void bwd_kv(const BwdParams& p, int gp, int rank, unsigned char* smem) {
  constexpr int DS = S::DS, KF = S::F, NG = S::NG, BQ = S::ROWS, BK = S::BM, TILE = S::TILE;
  using L = Tile<DS>;
  constexpr int SET = 2 * TILE + 2 * BQ * 4;  // q rows, dout rows, lse2, delta
  constexpr int STAGE = NG * SET;
  constexpr int V = 2 * STAGE;  // the values' place
  static_assert(BQ == 32, "one step of the second products");
  const PromptBwdArgs& a = p.a;
  const int kvh = gp / p.parts, part = gp - kvh * p.parts;
  if (part == 0) {
    fill_pad(a.dk, a.seqs, a.D, kvh, rank, p.ranks);
    fill_pad(a.dv, a.seqs, a.D, kvh, rank, p.ranks);
  }
  const SeqTile st = find_tile(a.seqs, BK, rank, true);
  if (st.len == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave % S::NR, grp = wave / S::NR;
  const int col = lane & 15, g = lane >> 4;
  const int k0 = st.tile * BK;
  const int wk0 = k0 + w * 16 * KF;
  const int heads = a.H / a.G / p.parts, head0 = kvh * (a.H / a.G) + part * heads;
  const int qt0 = k0 / BQ, qtiles = (st.len + BQ - 1) / BQ - qt0;
  const int total = heads * qtiles;
  const int64_t T = a.seqs.T;
  const uint32_t lds = lds_addr(smem);
  TileLoad<DS, BQ, S::NR> ql, dl;
  ql.init(w, lane, a.q.rs, a.D);
  dl.init(w, lane, a.dout.rs, a.D);
  // The query tiles that may hold rows before one of the workgroup's keys come first, head by
  // head, then the others: item j of the group's j = grp, grp + NG, ...
  const int edge = min(BK / BQ, qtiles);
  struct Item {
    int h, q, end;  // head, query tile, and where the head's tiles of this kind end
  };
  auto advance = [&](Item& x, int n) {
    for (; n > 0; --n)
      if (++x.q == x.end) {
        if (++x.h == heads) {
          x.h = 0;
          x.end = qtiles;
        }
        x.q = x.end == edge ? 0 : edge;
      }
  };
  Item next;  // the group's next load
  auto start = [&] {
    next = Item{0, 0, edge};
    advance(next, grp);
  };
  start();
  auto load = [&](int stage) {
    const int head = head0 + next.h, r = (qt0 + next.q) * BQ, valid = st.len - r;
    const uint32_t at = lds + stage * STAGE + grp * SET;
    const int64_t row = st.row0 + r;
    ql.issue(a.q.p + row * a.q.rs + head * a.q.hs, a.q.rs, a.D, valid, at, w);
    dl.issue(a.dout.p + row * a.dout.rs + head * a.dout.hs, a.dout.rs, a.D, valid, at + TILE, w);
    if (w < 2 && lane < BQ) {
      const float* x = (w == 0 ? p.lse2 : p.delta) + head * T + row;
      dma4(make_rsrc(x, (uint32_t)min(valid, BQ) * 4), at + 2 * TILE + w * BQ * 4, lane * 4);
    }
    advance(next, NG);
  };
  {
    TileLoad<DS, BK, S::NW> vl;
    vl.init(wave, lane, a.v.rs, a.D);
    vl.issue(a.v.p + (int64_t)(st.row0 + k0) * a.v.rs + kvh * a.v.hs, a.v.rs, a.D, st.len - k0, lds + V, wave);
  }
  if (grp < total) load(0);
  bf16x8 k[KF][DS];
#pragma unroll
  for (int f = 0; f < KF; ++f) {
    const int u = wk0 + f * 16 + col;
    const uint16_t* kr = a.k.p + (st.row0 + u) * a.k.rs + kvh * a.k.hs;
#pragma unroll
    for (int s = 0; s < DS; ++s) k[f][s] = load_row8(kr + 32 * s + 8 * g, u < st.len && 32 * s + 8 * g < a.D);
  }
#pragma unroll
  for (int f = 0; f < KF; ++f)
#pragma unroll
    for (int s = 0; s < DS; ++s) arrived(k[f][s]);
  // This wave's share of the values is in LDS: all waves read them after the first barrier, which
  // the later groups reach without a step's wait.
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  RowFrag<DS> rf;  // from the stage; the group's q lie grp SET bytes on, dout TILE further
  ColFrag<DS> cf;
  rf.init(smem, lane);
  cf.init(smem, lane);
  f32x4 dk[L::DB][KF], dv[L::DB][KF];
  const int steps = (total + NG - 1) / NG;
  const bool late = grp >= (NG + 1) / 2;
  // As in bwd_q.  A tile's rows past the sequence's end are zeros, and so are their products, but
  // not with a key or value that is not finite: then a sum is NaN, and the CAREFUL pass leaves
  // those rows out.
  auto pass = [&](auto careful) __attribute__((always_inline)) {
    constexpr bool CAREFUL = decltype(careful)::value;
    bool bad = false;
#pragma unroll
    for (int d = 0; d < L::DB; ++d)
#pragma unroll
      for (int f = 0; f < KF; ++f) dk[d][f] = dv[d][f] = f32x4{0, 0, 0, 0};
    Item now{0, 0, edge};
    advance(now, grp);
    if (late) phase_barrier();
    auto step = [&](int i, auto diagonal) __attribute__((always_inline)) {
      constexpr bool DIAGONAL = decltype(diagonal)::value;
      const int j = i * NG + grp;
      const int stage = (i & 1) * STAGE + grp * SET;
      wait_vmcnt_and_barrier<0>();
      if (j + NG < total) load((i + 1) & 1);
      const bool live = NG == 1 || j < total;
      const int q0 = (qt0 + now.q) * BQ;
      advance(now, NG);
      const float* rows = reinterpret_cast<const float*>(smem + stage + 2 * TILE);
      f32x4 s[2][KF], dp[2][KF];
      if (live) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const f32x4 nd = -*LDS_PTR(const f32x4, rows + BQ + b * 16 + 4 * g);
#pragma unroll
          for (int f = 0; f < KF; ++f) {
            s[b][f] = f32x4{0, 0, 0, 0};
            dp[b][f] = nd;
          }
        }
#pragma unroll
        for (int d = 0; d < DS; ++d) {
          bf16x8 v[KF];
#pragma unroll
          for (int f = 0; f < KF; ++f) v[f] = rf.read(V, w * KF + f, d);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const bf16x8 qq = rf.read(stage, b, d);
            const bf16x8 dd = rf.read(stage + TILE, b, d);
#pragma unroll
            for (int f = 0; f < KF; ++f) {
              s[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qq, k[f][d], s[b][f], 0, 0, 0);
              dp[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dd, v[f], dp[b][f], 0, 0, 0);
            }
          }
        }
      }
      if (NG > 1) phase_barrier();
      if (!live) return;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const f32x4 l2 = *LDS_PTR(const f32x4, rows + b * 16 + 4 * g);
#pragma unroll
        for (int f = 0; f < KF; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[b][f][i] = exp2_(s[b][f][i] * p.c - l2[i]);
            dp[b][f][i] *= s[b][f][i];
          }
      }
      if (DIAGONAL && q0 < wk0 + 16 * KF - 1) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int f = 0; f < KF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (wk0 + f * 16 + col > q0 + b * 16 + 4 * g + i) s[b][f][i] = dp[b][f][i] = 0.0f;
      }
      if (CAREFUL && q0 + BQ > st.len) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int f = 0; f < KF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (q0 + b * 16 + 4 * g + i >= st.len) s[b][f][i] = dp[b][f][i] = 0.0f;
      }
      bf16x8 pf[KF], ds[KF], rest[KF];
#pragma unroll
      for (int f = 0; f < KF; ++f) {
        pf[f] = pack8(s[0][f], s[1][f]);
        ds[f] = pack8(dp[0][f], dp[1][f]);
        if (DIAGONAL) rest[f] = rest8(dp[0][f], dp[1][f], ds[f]);
      }
      if (!CAREFUL && DIAGONAL)
        bad = bad || not_finite<2 * TILE, S::NR>(smem + stage, w, lane);
      if (CAREFUL && DIAGONAL) {
#pragma unroll
        for (int d = 0; d < L::DB; ++d)
#pragma unroll
          for (int f = 0; f < KF; ++f) {
            dv[d][f] = seen_product<false>(cf.read(stage + TILE, 0, d), pf[f], dv[d][f], q0, wk0 + f * 16, lane);
            dk[d][f] = seen_product<false>(cf.read(stage, 0, d), ds[f], dk[d][f], q0, wk0 + f * 16, lane);
            dk[d][f] = seen_product<false>(cf.read(stage, 0, d), rest[f], dk[d][f], q0, wk0 + f * 16, lane);
          }
        return;
      }
#pragma unroll
      for (int d = 0; d < L::DB; ++d) {
        const bf16x8 dd = cf.read(stage + TILE, 0, d);
        const bf16x8 qq = cf.read(stage, 0, d);
#pragma unroll
        for (int f = 0; f < KF; ++f) {
          dv[d][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(dd, pf[f], dv[d][f], 0, 0, 0);
          dk[d][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qq, ds[f], dk[d][f], 0, 0, 0);
          if (DIAGONAL) dk[d][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qq, rest[f], dk[d][f], 0, 0, 0);
        }
      }
    };
    const int first = min((heads * edge + NG - 1) / NG, steps);  // steps with tiles of the first kind
    int i = 0;
    for (; i < first; ++i) step(i, std::true_type{});
    for (; i < steps; ++i) step(i, std::false_type{});
    if (NG > 1 && !late) phase_barrier();
    if (!CAREFUL && st.len % BQ != 0) {
      float z = 0.0f;  // NaN if a sum is not finite
#pragma unroll
      for (int d = 0; d < L::DB; ++d)
#pragma unroll
        for (int f = 0; f < KF; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i) z += dk[d][f][i] * 0.0f + dv[d][f][i] * 0.0f;
      bad = bad || z != 0.0f;
    }
    return bad;
  };
  if (any_wave<S::NW>(pass(std::false_type{}), smem, wave, lane)) {
    start();
    if (grp < total) load(0);
    pass(std::true_type{});
  }
  if (NG > 1) {
    join_groups<NG, S::NR>(dk, smem, grp, w, lane);
    join_groups<NG, S::NR>(dv, smem, grp, w, lane);
  }
#pragma unroll
  for (int f = 0; f < KF; ++f) {
    const int u = wk0 + f * 16 + col;
    if (u >= st.len) continue;
    const int64_t row = st.row0 + u;
    if (p.parts == 1) {
      uint16_t* ok = a.dk.p + row * a.dk.rs + kvh * a.dk.hs;
      uint16_t* ov = a.dv.p + row * a.dv.rs + kvh * a.dv.hs;
#pragma unroll
      for (int i = 0; i < (L::DB + NG - 1) / NG; ++i) {
        const int e = 16 * (i * NG + grp) + 4 * g;
        if (e < a.D) {
          store4(ok + e, dk[i][f] * a.scale);
          store4(ov + e, dv[i][f]);
        }
      }
    } else {
      float* ok = p.part + (((int64_t)(part * 2) * a.G + kvh) * T + row) * a.D;
      float* ov = ok + (int64_t)a.G * T * a.D;
#pragma unroll
      for (int i = 0; i < (L::DB + NG - 1) / NG; ++i) {
        const int e = 16 * (i * NG + grp) + 4 * g;
        if (e < a.D) {
          *reinterpret_cast<f32x4*>(ok + e) = dk[i][f];
          *reinterpret_cast<f32x4*>(ov + e) = dv[i][f];
        }
      }
    }
  }
}

// Both kinds in one launch, each by falling work, so that the second starts where the last and
// longest of the first still run.  Measured on an earlier version of the two, 8184 rows of 4 heads on
// 4 in 5 sequences: 190 us, where a launch for each took 84 and 125; rank by rank in turns 230.
template <class SQ, class SK>
__global__ __launch_bounds__(64 * SQ::NW, 2) void attn_bwd(BwdParams p) {
  extern __shared__ __align__(256) unsigned char smem[];
  const int H = p.a.H, GP = p.a.G * p.parts, b = blockIdx.x, kv = p.ranks * GP;
  if (b < kv) bwd_kv<SK>(p, b % GP, b / GP, smem);
  else bwd_q<SQ>(p, (b - kv) % H, (b - kv) / H, smem);
}

// dk and dv from their parts, in part order; 8 elements per thread.
__global__ __launch_bounds__(256) void attn_bwd_join(BwdParams p) {
  const PromptBwdArgs& a = p.a;
  const int vec = a.D / 8;
  const int lo = first_row(a.seqs), hi = last_row(a.seqs);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = (int64_t)a.seqs.T * vec;
  if (i >= per * a.G * 2) return;
  const int which = (int)(i / (per * a.G));
  const int64_t r = i - which * per * a.G;
  const int kvh = (int)(r / per);
  const int64_t row = (r - kvh * per) / vec;
  const int e = (int)(r % vec) * 8;
  if (row < lo || row >= hi) return;
  const int64_t step = (int64_t)a.G * a.seqs.T * a.D;
  const float* x = p.part + which * step + ((int64_t)kvh * a.seqs.T + row) * a.D + e;
  f32x4 s0 = *reinterpret_cast<const f32x4*>(x), s1 = *reinterpret_cast<const f32x4*>(x + 4);
  for (int k = 1; k < p.parts; ++k) {
    x += 2 * step;
    s0 += *reinterpret_cast<const f32x4*>(x);
    s1 += *reinterpret_cast<const f32x4*>(x + 4);
  }
  const Heads& o = which ? a.dv : a.dk;
  const float scale = which ? 1.0f : a.scale;
  u32x4 w;
  w[0] = pack_bf16x2(s0[0] * scale, s0[1] * scale);
  w[1] = pack_bf16x2(s0[2] * scale, s0[3] * scale);
  w[2] = pack_bf16x2(s1[0] * scale, s1[1] * scale);
  w[3] = pack_bf16x2(s1[2] * scale, s1[3] * scale);
  *GLOBAL_PTR(u32x4, o.p + row * o.rs + kvh * o.hs + e) = w;
}

constexpr int64_t align256(int64_t x) { return (x + 255) / 256 * 256; }

// Calls of few rows times heads take 64 rows and four groups of waves per workgroup, for the
// reason given in attn_prompt.hip.  Measured on an earlier version of both (the second case takes
// 170-174 now), the gradient alone, groups against one: 8184 rows of 4 heads on 4, 2 sequences 187 and
// 195 us, 5 sequences 161 and 196; 5120 of 8 on 1 (2) 151 and 134, of 8 on 8 (8) 115 and 99.
constexpr int64_t GROUPED_BELOW = 36 * 1024;
bool grouped(int H, int64_t rows, int64_t n) { return rows * H < GROUPED_BELOW && few_sequences(n, H); }

// Parts a group's heads are split into, until the key-value workgroups make one round (of 512,
// or of 256 of four groups): fewer leave much of the chip idle (half a round: 306 us against 252
// for 8184 rows of 8 heads on 1), more only write more parts (4096 rows: 105 us with two rounds
// against 92).
int bwd_parts(int H, int G, int64_t rows, bool small) {
  const int group = H / G;
  const int64_t tiles = small ? (rows + 63) / 64 * G : (rows + 127) / 128 * G;
  int parts = 1;
  while (parts < group && tiles * parts < (small ? 256 : 512)) {
    ++parts;
    while (group % parts) ++parts;
  }
  return parts;
}

template <class SQ, class SK>
hipError_t run(const PromptBwdArgs& a, hipStream_t s) {
  static_assert(SQ::BM == SK::BM && SQ::NW == SK::NW, "one count of tiles, one of waves");
  constexpr int DS = SQ::DS;
  const int64_t T = a.seqs.T;
  BwdParams p{};
  p.a = a;
  p.c = a.scale * LOG2E;
  p.parts = bwd_parts(a.H, a.G, T, SK::NG > 1);
  unsigned char* w = static_cast<unsigned char*>(a.ws);
  const int64_t stat = align256((int64_t)a.H * T * 4);
  p.lse2 = reinterpret_cast<float*>(w);
  p.delta = reinterpret_cast<float*>(w + stat);
  p.part = reinterpret_cast<float*>(w + 2 * stat);
  const int64_t ranks = max_tiles(T, a.seqs.n, SQ::BM) + (a.seqs.n == 0);
  const int64_t blocks = ranks * (a.H + a.G * p.parts);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  p.ranks = (int32_t)ranks;
  constexpr int lds_q = std::max(2 * SQ::NG * 2 * SQ::TILE, SQ::JOIN);
  constexpr int lds_kv = std::max(2 * SK::NG * (2 * SK::TILE + 2 * SK::ROWS * 4) + SK::BM * Tile<DS>::RB,
                                  SK::JOIN);
  constexpr int lds = std::max(lds_q, lds_kv);
  auto kernel = &attn_bwd<SQ, SK>;
  hipError_t e = ensure_lds_attr(reinterpret_cast<const void*>(kernel), lds);
  if (e == hipSuccess && T > 0) {
    auto rows = DS <= 2 ? &attn_bwd_rows<8> : &attn_bwd_rows<16>;
    e = launch_k(rows, dim3((unsigned)(((T + 31) / 32 * a.H + 3) / 4)), dim3(256), 0, s, p);
  }
  if (e == hipSuccess) e = launch_k(kernel, dim3((unsigned)blocks), dim3(64 * SQ::NW), lds, s, p);
  if (e == hipSuccess && p.parts > 1) {
    const int64_t blocks = (2 * a.G * T * (a.D / 8) + 255) / 256;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    e = launch_k(&attn_bwd_join, dim3((unsigned)blocks), dim3(256), 0, s, p);
  }
  return e;
}

template <int DS>
hipError_t choose(const PromptBwdArgs& a, hipStream_t s) {
  if (grouped(a.H, a.seqs.T, a.seqs.n)) return run<Shape<DS, 2, 4, 32>, Shape<DS, 2, 4, 32>>(a, s);
  return run<Shape<DS, 4, 1, 64>, Shape<DS, 4, 1, 32>>(a, s);
}

}  // namespace

size_t attn_prompt_bwd_need(int32_t H, int32_t G, int32_t D, int64_t rows) {
  const int parts = bwd_parts(H, G, rows, false);  // groups take no more
  return static_cast<size_t>(2 * align256((int64_t)H * rows * 4) +
                             (parts > 1 ? (int64_t)parts * 2 * G * rows * D * 4 : 0));
}

size_t attn_prompt_bwd_bytes(int32_t H, int32_t G, int32_t D, int64_t rows) {
  // the parts fall in steps as rows grow, so fewer rows can need more: each row count up to
  // `rows` is covered by the last one with the same number of key tiles
  size_t most = attn_prompt_bwd_need(H, G, D, rows);
  for (int64_t t = 1; t <= 2048 && t * 64 < rows; ++t)
    most = std::max(most, attn_prompt_bwd_need(H, G, D, t * 64));
  return most;
}

hipError_t launch_attn_prompt_bwd(const PromptBwdArgs& a, hipStream_t s) {
  if (a.D <= 64) return choose<2>(a, s);
  if (a.D <= 96) return choose<3>(a, s);
  return choose<4>(a, s);
}

}  // namespace ubx
