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
//
// Under a window both kinds walk the tiles that their rows and keys meet (attn_window.h), and the
// first tokens that stay visible get further workgroups, whose sums attn_bwd_sinks adds.  Measured,
// 16264 tokens in 2 sequences, 8 heads on 1, a window of 2048 and 4 first tokens: 455-485 us (cards
// differ), 0.86-0.92 PFLOP/s of the seven products done; 8184 tokens in 5, 4 heads on 4, 512 and
// none: 58-63 us.
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
  float* sink_part;      // [slots, 2, G parts, MAX_SINKS, D], see SinkSlots
  int32_t slots, chunk;  // slots: 0 without first tokens that stay visible
};

constexpr int MAX_SINKS = UB_ATTN_MAX_SINKS;

__device__ inline int seq_len(const Seqs& s, int i) {
  return i < s.n ? max(clamp_row(s.cu[i + 1], s.T) - clamp_row(s.cu[i], s.T), 0) : 0;
}

// Slots of the sequences that start before row `row`.
__device__ inline int slots_before(const BwdParams& p, int row, int BK) {
  const Seqs& s = p.a.seqs;
  int sum = 0;
  for (int c = 0; c < s.n; c += 64) {
    const int i = c + (threadIdx.x & 63);
    if (i < s.n && clamp_row(s.cu[i], s.T) < row) sum += sink_slots(seq_len(s, i), BK, p.a.win, p.chunk).count;
  }
  return wave_sum(sum);
}

// The sequence of slot `slot` and the slot's number there (0: the first workgroup's); len 0: none.
__device__ inline SeqTile find_slot(const BwdParams& p, int slot, int BK) {
  const Seqs& s = p.a.seqs;
  SeqTile r{0, 0, 0};
  int before = 0;
  for (int c = 0; c < s.n; c += 64) {
    const int i = c + (threadIdx.x & 63);
    const int len = seq_len(s, i);
    const int n = i < s.n ? sink_slots(len, BK, p.a.win, p.chunk).count : 0;
    const int incl = wave_scan(n);
    const uint64_t m = __ballot(before + incl > slot);
    if (m) {
      const int at = __builtin_ctzll(m);
      r.row0 = __builtin_amdgcn_readlane(clamp_row(s.cu[min(i, s.n)], s.T), at);
      r.len = __builtin_amdgcn_readlane(len, at);
      r.tile = slot - before - __builtin_amdgcn_readlane(incl - n, at);
      if (r.tile < 0 || r.tile >= __builtin_amdgcn_readlane(n, at)) r.tile = 0;
      return r;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return r;
}

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

// Under a window, rows of up to FEW keys (a narrow window's, or the first of a sequence) get delta
// from its definition, the sum of P dP over them.  From out, rounded to bf16, it is off by much of
// the dS of a row of few keys: the error of dq and dk was 2.5, 2.0 and 1.5 times that of their own
// rounding with 2, 3 and 8 keys, and is 1.0 with this.  8 rows of one head to a wave; a row's keys
// are read 16 bytes to a lane, 4 at a time (neighbouring rows' are the same ones).  The gradient
// of 8184 rows, 4 heads on 4, takes 52 us with 2 keys, 55 with 8 and 50 with 17 (64 if FEW were 16,
// where the error is 1.3 without it); 2.5 of the last are the first rows'.  Lane i < 8 has where
// row0 + i's sequence starts (past the row: none) and the row's lse log2(e).
constexpr int FEW = 8, FEW_ROWS = 8;  // keys; rows of a wave
template <int LPR>
__device__ inline void bwd_delta_few(const BwdParams& p, int head, int64_t row0, int64_t end, int start, float lse2) {
  constexpr int AT_ONCE = 64 / LPR, N = FEW_ROWS / AT_ONCE, AHEAD = 4;
  const PromptBwdArgs& a = p.a;
  const int lane = threadIdx.x & 63, kvh = head / (a.H / a.G), e = lane % LPR * 8;
  const int window = a.win.size, keys = window + a.win.sinks, most = min(keys, FEW);
  auto dot = [](bf16x8 x, bf16x8 y) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += (float)x[k] * (float)y[k];
    return row_sum<LPR>(s);
  };
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = i * AT_ONCE + lane / LPR;
    const int64_t row = row0 + r;
    const int64_t first = __shfl(start, r);
    const float l2 = __shfl(lse2, r);
    const bool in = row < end && first <= row, mine = in && e < a.D;
    const int64_t t = row - first;
    const bf16x8 q = load_row8(a.q.p + row * a.q.rs + head * a.q.hs + e, mine);
    const bf16x8 d = load_row8(a.dout.p + row * a.dout.rs + head * a.dout.hs + e, mine);
    float delta = 0.0f;
#pragma unroll 1
    for (int j0 = 0; j0 < most; j0 += AHEAD) {
      bf16x8 k[AHEAD], v[AHEAD];
      bool sees[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int i = j0 + j;
        const int64_t u = i < window ? t - i : i - window;  // the window's keys, then the first tokens before it
        sees[j] = in && i < keys && u >= 0 && (i < window || u <= t - window);
        const int64_t at = first + u;
        k[j] = load_row8(a.k.p + at * a.k.rs + kvh * a.k.hs + e, sees[j] && e < a.D);
        v[j] = load_row8(a.v.p + at * a.v.rs + kvh * a.v.hs + e, sees[j] && e < a.D);
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const float s = dot(q, k[j]), dp = dot(d, v[j]);
        delta += sees[j] ? exp2_(s * p.c - l2) * dp : 0.0f;
      }
    }
    if (lane % LPR == 0 && row < end) p.delta[head * a.seqs.T + row] = delta;
  }
}

// delta and lse log2(e) of all rows, 32 of one head to a wave; what they are in rows of no
// sequence is not read.  Under a window the first waves, which take longer, have the first rows of
// one sequence each, in one head, and the others leave those rows' delta to them.
template <int LPR, bool WIN>
__global__ __launch_bounds__(256) void attn_bwd_rows(BwdParams p) {
  constexpr int AT_ONCE = 64 / LPR, N = 32 / AT_ONCE;
  const PromptBwdArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t T = a.seqs.T, task = (int64_t)blockIdx.x * 4 + wave;
  const int head = (int)(task % a.H);
  const int64_t row0 = (task / a.H - (WIN ? a.seqs.n : 0)) * 32;
  if (row0 >= T) return;
  if constexpr (WIN) {
    const int64_t seq = task / a.H;
    if (seq < a.seqs.n) {
      const int64_t first = max(a.seqs.cu[seq], 0), end = min(min((int64_t)a.seqs.cu[seq + 1], T), first + FEW);
      float lse2 = 0.0f;
      if (lane < FEW_ROWS && first + lane < end) {
        const float l = a.lse[head * T + first + lane];
        lse2 = l == -INFINITY ? 0.0f : l * LOG2E;
      }
      bwd_delta_few<LPR>(p, head, first, end, (int)first, lse2);
      return;
    }
  }
  // lane l: where sequence c + l starts and its first FEW rows end, from row0 on, in the wave's 32
  auto starts = [&](int c, int& from, int& to) {
    const int l = min(c + lane, a.seqs.n - 1);
    const int64_t start = max(a.seqs.cu[l], 0), end = min((int64_t)a.seqs.cu[l + 1], start + FEW);
    from = (int)min(max(start - row0, (int64_t)0), (int64_t)32);
    to = (int)min(max(end - row0, (int64_t)0), (int64_t)32);
  };
  int from = 0, to = 0;
  if (WIN && a.seqs.n > 0) starts(0, from, to);
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
  unsigned first_rows = 0;  // bit i: row0 + i is one of the first FEW of its sequence
  if constexpr (WIN) {
    for (int c = 0; c < a.seqs.n; c += 64) {
      if (c) starts(c, from, to);
      for (uint64_t m = __ballot(from < to); m; m &= m - 1) {
        const int l = __ffsll((unsigned long long)m) - 1;
        first_rows |= (unsigned)((1ull << __shfl(to, l)) - (1ull << __shfl(from, l)));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float x = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) x += (float)d[i][k] * (float)o[i][k];
    x = row_sum<LPR>(x);
    const int64_t row = row0 + i * AT_ONCE + lane / LPR;
    const bool left = first_rows >> (row - row0) & 1;
    if (lane % LPR == 0 && row < T && !left) p.delta[head * T + row] = x;
  }
}

// The same under a window of up to FEW keys, first tokens included.
template <int LPR>
__global__ __launch_bounds__(256) void attn_bwd_rows_few(BwdParams p) {
  const PromptBwdArgs& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t T = a.seqs.T, task = (int64_t)blockIdx.x * 4 + wave;
  const int head = (int)(task % a.H);
  const int64_t row0 = task / a.H * FEW_ROWS;
  if (row0 >= T) return;
  // where the rows' sequences start.  Sequences that end at or before the row come first
  int seq = 0;
  for (int c = 0; c < a.seqs.n; c += 64) {
    const int end = c + lane < a.seqs.n ? a.seqs.cu[c + lane + 1] : 0x7FFFFFFF;
    int more = 0;
#pragma unroll
    for (int j = 0; j < FEW_ROWS; ++j) {
      const int m = __popcll(__ballot(end <= row0 + j));
      seq += lane == j ? m : 0;
      more |= m == 64;
    }
    if (!more) break;
  }
  const bool rows = lane < FEW_ROWS;
  const int start = rows && seq < a.seqs.n ? max(a.seqs.cu[seq], 0) : 0x7FFFFFFF;
  float lse2 = 0.0f;
  if (rows && row0 + lane < T) {
    const int64_t at = head * T + row0 + lane;
    const float l = a.lse[at];
    lse2 = l == -INFINITY ? 0.0f : l * LOG2E;
    p.lse2[at] = lse2;
  }
  bwd_delta_few<LPR>(p, head, row0, T, start, lse2);
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

template <class S, bool WIN>
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
  const KeyTiles kt = WIN ? key_tiles(q0, BM, BN, n_keys, a.win) : KeyTiles{};
  const int tiles = WIN ? kt.tiles : (n_keys + BN - 1) / BN;
  const uint16_t* kbase = a.k.p + (int64_t)st.row0 * a.k.rs + kvh * a.k.hs;
  const uint16_t* vbase = a.v.p + (int64_t)st.row0 * a.v.rs + kvh * a.v.hs;
  TileLoad<DS, BN, S::NR> kl, vl;
  kl.init(w, lane, a.k.rs, a.D);
  vl.init(w, lane, a.v.rs, a.D);
  const uint32_t lds = lds_addr(smem) + grp * 2 * TILE;
  auto load = [&](int i, int stage) {
    const int j = WIN ? kt.at(i) : i;
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
  auto product = [&](bf16x8 x, bf16x8 y, f32x4 z, int row, int at) {
    return WIN ? seen_product<true>(x, y, z, row, at, lane, a.win) : seen_product<true>(x, y, z, row, at, lane);
  };
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
    // DIAGONAL: tiles that may hold keys that one of the workgroup's queries does not see
    auto step = [&](int i, auto diagonal) __attribute__((always_inline)) {
      constexpr bool DIAGONAL = decltype(diagonal)::value;
      const int j = i * NG + grp;
      const int stage = (i & 1) * STAGE;
      wait_vmcnt_and_barrier<0>();
      if (j + NG < tiles) load(j + NG, (i + 1) & 1);
      const bool live = NG == 1 || j < tiles;
      const int k0 = (WIN ? kt.at(j) : j) * BN;
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
        if (DIAGONAL && (k0 + BN - 1 > wq0 || (WIN && k0 <= wq0 + 16 * QF - 1 - a.win.size))) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int f = 0; f < QF; ++f)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = k0 + t * 32 + b * 16 + 4 * g + i, row = wq0 + f * 16 + col;
                if (WIN ? !seen(key, row, a.win) : key > row) s[b][f][i] = 0.0f;
              }
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
              acc[d][f] = product(cf.read(stage, t, d), ds[f], acc[d][f], k0 + t * 32, wq0 + f * 16);
              acc[d][f] = product(cf.read(stage, t, d), rest[f], acc[d][f], k0 + t * 32, wq0 + f * 16);
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
    // steps of tiles before every query
    const int full = WIN ? (q0 / BN - kt.first + kt.sink) / NG : min(q0 / (BN * NG), steps);
    int i = 0;
    if (WIN) {
      const int head = min((kt.head + NG - 1) / NG, steps);
      for (; i < head; ++i) step(i, std::true_type{});
    }
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
// WIN, with `slot` >= 0: a chunk of rows beyond a sequence's first workgroup's, for the first tokens
// alone.
template <class S, bool WIN>
__device__ __forceinline__ void bwd_kv(const BwdParams& p, int gp, int rank, int slot, unsigned char* smem) {
  constexpr int DS = S::DS, KF = S::F, NG = S::NG, BQ = S::ROWS, BK = S::BM, TILE = S::TILE;
  using L = Tile<DS>;
  constexpr int SET = 2 * TILE + 2 * BQ * 4;  // q rows, dout rows, lse2, delta
  constexpr int STAGE = NG * SET;
  constexpr int V = 2 * STAGE;  // the values' place
  static_assert(BQ == 32, "one step of the second products");
  const PromptBwdArgs& a = p.a;
  const int kvh = gp / p.parts, part = gp - kvh * p.parts;
  if (part == 0 && slot < 0) {
    fill_pad(a.dk, a.seqs, a.D, kvh, rank, p.ranks);
    fill_pad(a.dv, a.seqs, a.D, kvh, rank, p.ranks);
  }
  SeqTile st;
  if (WIN && slot >= 0) {
    st = find_slot(p, slot, BK);
    if (st.tile == 0) return;  // the first workgroup's, or none
  } else {
    st = find_tile(a.seqs, BK, rank, true);
  }
  if (st.len == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wave % S::NR, grp = wave / S::NR;
  const int col = lane & 15, g = lane >> 4;
  const bool sinks = WIN && slot >= 0;
  const int k0 = sinks ? 0 : st.tile * BK;
  const int wk0 = k0 + w * 16 * KF;
  const int heads = a.H / a.G / p.parts, head0 = kvh * (a.H / a.G) + part * heads;
  // query tiles: from the first key's row to the last row that sees one of the keys
  SinkSlots span{};  // of a sequence's first keys
  QueryTiles qt;
  if (!WIN) {
    qt = query_tiles(k0, BK, BQ, st.len, Window{0, 0});
  } else {
    if (k0 == 0 && a.win.sinks > 0) span = sink_slots(st.len, BK, a.win, p.chunk);
    qt = query_tiles(k0, BK, BQ, k0 == 0 && a.win.sinks > 0 ? span.rows : window_end(k0, BK, st.len, a.win), a.win);
    if (sinks) {  // all of them may hold rows that do not see the keys after the first tokens
      qt.qt0 = (span.rows + (st.tile - 1) * p.chunk) / BQ;
      qt.n = (min(span.rows + st.tile * p.chunk, st.len) + BQ - 1) / BQ - qt.qt0;
      qt.diag = qt.tail = qt.edge = qt.n;
    }
  }
  const int qt0 = qt.qt0, qtiles = qt.n, edge = qt.edge;
  const int total = heads * qtiles;
  const int64_t T = a.seqs.T;
  const uint32_t lds = lds_addr(smem);
  TileLoad<DS, BQ, S::NR> ql, dl;
  ql.init(w, lane, a.q.rs, a.D);
  dl.init(w, lane, a.dout.rs, a.D);
  // The query tiles that may hold rows before one of the workgroup's keys come first, head by
  // head, then the others: item j of the group's j = grp, grp + NG, ...  Under a window those that
  // may hold rows which do not see one of the keys any more are of the first kind.
  auto tile_of = [&](int q) { return WIN ? qt.at(q) : q; };
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
    const int head = head0 + next.h, r = (qt0 + tile_of(next.q)) * BQ, valid = st.len - r;
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
  auto product = [&](bf16x8 x, bf16x8 y, f32x4 z, int row, int at) {
    return WIN ? seen_product<false>(x, y, z, row, at, lane, a.win) : seen_product<false>(x, y, z, row, at, lane);
  };
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
      bool live = NG == 1 || j < total;
      if (WIN && sinks && wk0 >= a.win.sinks) live = false;  // none of the wave's keys
      const int q0 = (qt0 + tile_of(now.q)) * BQ;
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
      if (DIAGONAL && (q0 < wk0 + 16 * KF - 1 || (WIN && wk0 <= q0 + BQ - 1 - a.win.size))) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int f = 0; f < KF; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = wk0 + f * 16 + col, row = q0 + b * 16 + 4 * g + i;
              if (WIN ? !seen(key, row, a.win) : key > row) s[b][f][i] = dp[b][f][i] = 0.0f;
            }
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
            dv[d][f] = product(cf.read(stage + TILE, 0, d), pf[f], dv[d][f], q0, wk0 + f * 16);
            dk[d][f] = product(cf.read(stage, 0, d), ds[f], dk[d][f], q0, wk0 + f * 16);
            dk[d][f] = product(cf.read(stage, 0, d), rest[f], dk[d][f], q0, wk0 + f * 16);
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
  // Sequences that overlap, of boundaries that do not rise, can ask for more slots than there are.
  const int own_slot = WIN && span.count > 0 && !sinks ? slots_before(p, st.row0, BK) : slot;
  const bool to_slot = WIN && span.count > 0 && own_slot >= 0 && own_slot < p.slots;
#pragma unroll
  for (int f = 0; f < KF; ++f) {
    const int u = wk0 + f * 16 + col;
    if (u >= st.len) continue;
    const int64_t row = st.row0 + u;
    if (to_slot && u < a.win.sinks) {
      float* ok = p.sink_part + (((int64_t)own_slot * 2 * a.G * p.parts + gp) * MAX_SINKS + u) * a.D;
      float* ov = ok + (int64_t)a.G * p.parts * MAX_SINKS * a.D;
#pragma unroll
      for (int i = 0; i < (L::DB + NG - 1) / NG; ++i) {
        const int e = 16 * (i * NG + grp) + 4 * g;
        if (e < a.D) {
          *reinterpret_cast<f32x4*>(ok + e) = dk[i][f];
          *reinterpret_cast<f32x4*>(ov + e) = dv[i][f];
        }
      }
    } else if (sinks) {
      continue;
    } else if (p.parts == 1) {
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
template <class SQ, class SK, bool WIN>
__global__ __launch_bounds__(64 * SQ::NW, 2) void attn_bwd(BwdParams p) {
  extern __shared__ __align__(256) unsigned char smem[];
  const int H = p.a.H, GP = p.a.G * p.parts, kv = (p.ranks + p.slots) * GP;
  const int b = blockIdx.x;
  if (b < kv) {
    const int rank = b / GP - p.slots;
    bwd_kv<SK, WIN>(p, b % GP, rank, rank < 0 ? b / GP : -1, smem);
  } else {
    bwd_q<SQ, WIN>(p, (b - kv) % H, (b - kv) / H, smem);
  }
}

// dk and dv of a sequence's first tokens from their slots, in order; blockIdx: sequence, head, and
// dk or dv.
template <int BK>
__global__ __launch_bounds__(256) void attn_bwd_sinks(BwdParams p) {
  const PromptBwdArgs& a = p.a;
  const int which = blockIdx.x & 1, kvh = (blockIdx.x >> 1) % a.G, i = (blockIdx.x >> 1) / a.G;
  const int len = seq_len(a.seqs, i);
  const int count = sink_slots(len, BK, a.win, p.chunk).count;
  if (count == 0) return;
  const int row0 = clamp_row(a.seqs.cu[i], a.seqs.T);
  const int64_t slot = slots_before(p, row0, BK);
  if (slot < 0 || slot + count > p.slots) return;
  const int64_t GP = a.G * p.parts, step = MAX_SINKS * a.D;
  constexpr int AHEAD = 8;
  const int vec = a.D / 4;
  const Heads& o = which ? a.dv : a.dk;
  for (int j = threadIdx.x; j < a.win.sinks * vec; j += 256) {
    const int u = j / vec, e = (j - u * vec) * 4;
    const float* at = p.sink_part + (slot * 2 * GP + which * GP + kvh * p.parts) * step + u * a.D + e;
    f32x4 x = {0, 0, 0, 0};
    const int n = count * p.parts;  // slot by slot, part by part, AHEAD loads at a time
    for (int c0 = 0; c0 < n; c0 += AHEAD) {
      f32x4 y[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int c = min(c0 + i, n - 1);
        y[i] = *reinterpret_cast<const f32x4*>(at + (c / p.parts * 2 * GP + c % p.parts) * step);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (c0 + i < n) x += y[i];
    }
    store4(o.p + (int64_t)(row0 + u) * o.rs + kvh * o.hs + e, x * (which ? 1.0f : a.scale));
  }
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
// Under a window, with two kinds of workgroups for a tile and head.  Measured, the gradient alone,
// groups against one, windows of 64, 512 and 2048: 2000 rows of 4 heads on 4 in one sequence (124
// tiles) 22 and 27 us, 29 and 45; 4096 (256) 36 and 31, 48 and 48, 81 and 104; 8184 (508) 66 and
// 36, 89 and 58, 161 and 122.
bool window_grouped(int H, int64_t rows, int64_t n, Window win) {
  const int64_t tiles = window_tiles(rows, n, H);
  return tiles <= 140 || (tiles <= 270 && win.size >= 1024);
}

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

int64_t slot_bytes(int G, int parts, int D) { return (int64_t)2 * G * parts * MAX_SINKS * D * 4; }

template <class SQ, class SK, bool WIN>
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
  if (WIN && a.win.sinks > 0) {
    p.chunk = sink_chunk(a.win);
    p.slots = (int32_t)std::min<int64_t>(max_slots(T, p.chunk), T / p.chunk + 2 * (int64_t)a.seqs.n);
    p.sink_part = p.part + (p.parts > 1 ? (int64_t)p.parts * 2 * a.G * T * a.D : 0);
  }
  const int64_t blocks = ranks * (a.H + a.G * p.parts) + (int64_t)p.slots * a.G * p.parts;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  p.ranks = (int32_t)ranks;
  constexpr int lds_q = std::max(2 * SQ::NG * 2 * SQ::TILE, SQ::JOIN);
  constexpr int lds_kv = std::max(2 * SK::NG * (2 * SK::TILE + 2 * SK::ROWS * 4) + SK::BM * Tile<DS>::RB,
                                  SK::JOIN);
  constexpr int lds = std::max(lds_q, lds_kv);
  auto kernel = &attn_bwd<SQ, SK, WIN>;
  hipError_t e = ensure_lds_attr(reinterpret_cast<const void*>(kernel), lds);
  if (e == hipSuccess && T > 0) {
    constexpr int LPR = DS <= 2 ? 8 : 16;
    auto rows = &attn_bwd_rows<LPR, WIN>;
    int of_wave = 32;
    int64_t first_rows = WIN ? a.seqs.n : 0;
    if (WIN && a.win.size + a.win.sinks <= FEW) {
      rows = &attn_bwd_rows_few<LPR>;
      of_wave = FEW_ROWS;
      first_rows = 0;
    }
    const int64_t blocks = (((T + of_wave - 1) / of_wave + first_rows) * a.H + 3) / 4;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    e = launch_k(rows, dim3((unsigned)blocks), dim3(256), 0, s, p);
  }
  if (e == hipSuccess) e = launch_k(kernel, dim3((unsigned)blocks), dim3(64 * SQ::NW), lds, s, p);
  if (e == hipSuccess && p.parts > 1) {
    const int64_t blocks = (2 * a.G * T * (a.D / 8) + 255) / 256;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    e = launch_k(&attn_bwd_join, dim3((unsigned)blocks), dim3(256), 0, s, p);
  }
  if (WIN && e == hipSuccess && p.slots > 0) {
    const int64_t blocks = 2 * (int64_t)a.G * a.seqs.n;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (blocks > 0) e = launch_k(&attn_bwd_sinks<SK::BM>, dim3((unsigned)blocks), dim3(256), 0, s, p);
  }
  return e;
}

template <int DS, bool WIN>
hipError_t choose(const PromptBwdArgs& a, hipStream_t s) {
  if (WIN ? window_grouped(a.H, a.seqs.T, a.seqs.n, a.win) : grouped(a.H, a.seqs.T, a.seqs.n))
    return run<Shape<DS, 2, 4, 32>, Shape<DS, 2, 4, 32>, WIN>(a, s);
  return run<Shape<DS, 4, 1, 64>, Shape<DS, 4, 1, 32>, WIN>(a, s);
}

template <bool WIN>
hipError_t by_dim(const PromptBwdArgs& a, hipStream_t s) {
  if (a.D <= 64) return choose<2, WIN>(a, s);
  if (a.D <= 96) return choose<3, WIN>(a, s);
  return choose<4, WIN>(a, s);
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

size_t attn_prompt_bwd_sink_bytes(int32_t H, int32_t G, int32_t D, int64_t rows) {
  // a call has at most H / G parts
  return static_cast<size_t>(max_slots(rows, MIN_CHUNK) * slot_bytes(G, H / G, D));
}

hipError_t launch_attn_prompt_bwd(const PromptBwdArgs& a, hipStream_t s) {
  return a.win.size ? by_dim<true>(a, s) : by_dim<false>(a, s);
}

}  // namespace ubx
