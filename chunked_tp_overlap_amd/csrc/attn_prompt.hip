// Causal attention within packed sequences, on gfx950 matrix cores.
//
//   s = scale q k^T (u <= t),  lse = log sum_u exp(s),  out = sum_u exp(s - lse) v
//
// One pass over the keys in base 2: with c = scale log2(e), p = exp2(c s - c m).  The reference
// m is the maximum of the row's first tile, not a running one: p then can exceed 1, which costs
// fp32 and bf16 nothing up to very large ratios, and no tile needs maxima, a rescaling of the
// output or an exchange between lanes.  Where a sum passes 2^60, or an output is not finite, the
// workgroup repeats its pass with the running maximum, which has no such limit: for scores that
// pass the first tile's by 41 and more.
//
// A workgroup owns BM query rows of one head.  A wave keeps 32 of them (as columns of the score
// tiles, see attn_common.h), their fp32 output [head_dim x rows] and sums in registers; the
// waves of a group share the key and value tiles that direct-to-LDS loads bring in,
// double-buffered.  Long calls: one group of four waves, two workgroups to a CU.  Short ones: four
// groups of two waves, which take the key tiles in turn and join their outputs at the end.
//
// Measured on MI355X.  One sequence of 24392 tokens, 8 heads of 128 on 1: 1.02 ms, 1.19 PFLOP/s;
// a bf16 library product of 8192^3 reaches 1.27.  The matrix cores are busy 59% of the time at
// the 1.9 GHz that the power limit leaves.  8184 tokens, the longest sequence 4677, 4 heads of 128
// on 4: 50 us.  The last rows of that sequence alone take 44: 37 steps of 128 keys, 0.95 us each,
// and 6 us before and after them.  A step is some 1900 cycles; by count, its matrix instructions
// take 1024 of each SIMD and its 128 KB of fragment reads and 64 KB of loads pass through LDS.  What
// is left is the chain of a step: barrier, scores, exponentials, products, with two waves to a
// SIMD to cover it.  Measured, the kernel in one trace 57.4 us: without loads after the first 55;
// more waves of 16 rows each 57.3; two such workgroups to a CU 62; the product with the values one
// step late, beside the next scores, 68.
//
// Rows past a sequence's end (of any input) are never read: their loads fall outside the
// buffer resource and give zeros.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "attn_common.h"

namespace ubx {
namespace {

// A lane's sum with the first tile's reference beyond which the pass is done again.
constexpr float MOST = 0x1p60f;

struct PromptParams {
  PromptArgs a;
  float c;  // scale * log2(e)
  int32_t ranks;
};

// Zeros and -inf in the rows of no sequence, dealt over the workgroups of a head.
__device__ inline void fill_pad(const PromptArgs& a, int head, int rank, int ranks) {
  const int lo = first_row(a.seqs), hi = last_row(a.seqs), T = a.seqs.T;
  const int pad = lo + (T - hi);
  const int vec = a.D / 8;
  for (int i = rank; i < pad; i += ranks) {
    const int64_t t = i < lo ? i : hi + (i - lo);
    if ((int)threadIdx.x < vec)
      *GLOBAL_PTR(u32x4, a.out.p + t * a.out.rs + head * a.out.hs + threadIdx.x * 8) = u32x4{0, 0, 0, 0};
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)head * T + t] = -INFINITY;
  }
}

// RW waves of 16 QF rows each, KG times: group kg of RW waves takes the key tiles (BN rows)
// kg, kg + KG, ...
template <int DS_, int QF_, int RW_, int KG_, int BN_>
struct Shape {
  static constexpr int DS = DS_, QF = QF_, RW = RW_, KG = KG_, BN = BN_;
  using L = Tile<DS>;
  static constexpr int NW = RW * KG, BM = 16 * QF * RW, TILE = BN * L::RB;
  static constexpr int STAGE = KG * 2 * TILE;                 // the groups' key and value tiles
  static constexpr int PART = L::DB * QF * 64 * 16;           // a wave's output, for the join
  static constexpr int STAT = NW * QF * 16 * 8;
  static constexpr int LDS = KG == 1 || 2 * STAGE > NW * PART + STAT ? 2 * STAGE : NW * PART + STAT;
};

template <class S>
__global__ __launch_bounds__(64 * S::NW, 2) void attn_prompt(PromptParams p) {
  constexpr int DS = S::DS, QF = S::QF, KG = S::KG, BN = S::BN, BM = S::BM, TILE = S::TILE;
  using L = Tile<DS>;
  constexpr int KB = BN / 16;
  extern __shared__ __align__(256) unsigned char smem[];
  const PromptArgs& a = p.a;
  const int head = blockIdx.x % a.H, rank = blockIdx.x / a.H;
  fill_pad(a, head, rank, p.ranks);
  const SeqTile st = find_tile(a.seqs, BM, rank, false);
  if (st.len == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % S::RW, kg = wave / S::RW;
  const int col = lane & 15, g = lane >> 4;
  const int kvh = head / (a.H / a.G);
  const int q0 = st.tile * BM;
  const int wq0 = q0 + rw * 16 * QF;  // the wave's first query
  const int n_keys = min(q0 + BM, st.len);
  const int tiles = (n_keys + BN - 1) / BN;
  const uint16_t* kbase = a.k.p + (int64_t)st.row0 * a.k.rs + kvh * a.k.hs;
  const uint16_t* vbase = a.v.p + (int64_t)st.row0 * a.v.rs + kvh * a.v.hs;

  TileLoad<DS, BN, S::RW> kl, vl;
  kl.init(rw, lane, a.k.rs, a.D);
  vl.init(rw, lane, a.v.rs, a.D);
  const uint32_t lds = lds_addr(smem) + kg * 2 * TILE;
  auto load = [&](int j, int stage) {  // rows past the sequence's end read as zeros
    kl.issue(kbase + (int64_t)j * BN * a.k.rs, a.k.rs, a.D, st.len - j * BN, lds + stage * S::STAGE, rw);
    vl.issue(vbase + (int64_t)j * BN * a.v.rs, a.v.rs, a.D, st.len - j * BN, lds + stage * S::STAGE + TILE, rw);
  };
  if (kg < tiles) load(kg, 0);
  bf16x8 q[QF][DS];
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int t = wq0 + f * 16 + col;
    const uint16_t* row = a.q.p + (int64_t)(st.row0 + t) * a.q.rs + head * a.q.hs;
#pragma unroll
    for (int s = 0; s < DS; ++s) q[f][s] = load_row8(row + 32 * s + 8 * g, t < st.len && 32 * s + 8 * g < a.D);
  }
#pragma unroll
  for (int f = 0; f < QF; ++f)
#pragma unroll
    for (int s = 0; s < DS; ++s) arrived(q[f][s]);

  RowFrag<DS> kf;
  ColFrag<DS> vf;
  kf.init(smem + kg * 2 * TILE, lane);
  vf.init(smem + kg * 2 * TILE + TILE, lane);
  f32x4 o[L::DB][QF];
  float m[QF], l[QF];  // a row's reference and sum
  const int steps = (tiles + KG - 1) / KG;
  const bool late = kg >= (KG + 1) / 2;
  // All key tiles, the first of which is being loaded.  FIXED: the reference is the first
  // tile's maximum, and values are finite; true where that will not do.
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
    if (late) phase_barrier();
    // DIAGONAL: tiles that may hold keys after one of the workgroup's queries
    auto step = [&](int i, auto diagonal) __attribute__((always_inline)) {
      constexpr bool DIAGONAL = decltype(diagonal)::value;
      const int j = i * KG + kg;
      const int stage = (i & 1) * S::STAGE;
      wait_vmcnt_and_barrier<0>();
      if (j + KG < tiles) load(j + KG, (i + 1) & 1);
      const int k0 = j * BN;
      const bool live = KG == 1 || j < tiles;
      f32x4 s[KB][QF];
      if (live) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int f = 0; f < QF; ++f) s[b][f] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < DS; ++d)
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            const bf16x8 kk = kf.read(stage, b, d);
#pragma unroll
            for (int f = 0; f < QF; ++f)
              s[b][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kk, q[f][d], s[b][f], 0, 0, 0);
          }
        if (DIAGONAL && k0 + BN - 1 > wq0) {
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int f = 0; f < QF; ++f)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (k0 + b * 16 + 4 * g + i > wq0 + f * 16 + col) s[b][f][i] = -INFINITY;
        }
        if (!FIXED || i == 0) {
#pragma unroll
          for (int f = 0; f < QF; ++f) {
            float x = s[0][f][0];
#pragma unroll
            for (int b = 0; b < KB; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i) x = fmaxf(x, s[b][f][i]);
            x = col_max(x);
            if (FIXED) {
              // no score, though a key of the tile is not after the query
              bad = bad || (x == -INFINITY && wq0 + f * 16 + col >= k0);
              m[f] = x == -INFINITY ? 0.0f : x;
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
      }
      if (KG > 1) phase_barrier();
      if (!live) return;
#pragma unroll
      for (int f = 0; f < QF; ++f) {
        const float base = !FIXED && m[f] == -INFINITY ? 0.0f : m[f] * p.c;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // short sums, so that a long row's l loses little
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[b][f][i] = exp2_(s[b][f][i] * p.c - base);
            sum[i] += s[b][f][i];
          }
        l[f] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      bf16x8 pf[KB / 2][QF];
#pragma unroll
      for (int t = 0; t < KB / 2; ++t)
#pragma unroll
        for (int f = 0; f < QF; ++f) pf[t][f] = pack8(s[2 * t][f], s[2 * t + 1][f]);
      if (FIXED && DIAGONAL)
        bad = bad || not_finite<TILE, S::RW>(smem + stage + kg * 2 * TILE + TILE, rw, lane);
      if (!FIXED && DIAGONAL) {
#pragma unroll
        for (int t = 0; t < KB / 2; ++t)
#pragma unroll
          for (int d = 0; d < L::DB; ++d)
#pragma unroll
            for (int f = 0; f < QF; ++f)
              o[d][f] = seen_product<true>(vf.read(stage, t, d), pf[t][f], o[d][f], k0 + 32 * t, wq0 + f * 16, lane);
        return;
      }
#pragma unroll
      for (int t = 0; t < KB / 2; ++t)
#pragma unroll
        for (int d = 0; d < L::DB; ++d) {
          const bf16x8 vv = vf.read(stage, t, d);
#pragma unroll
          for (int f = 0; f < QF; ++f)
            o[d][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, pf[t][f], o[d][f], 0, 0, 0);
        }
    };
    const int full = min(q0 / (BN * KG), steps);  // steps of tiles before every query
    int i = 0;
    for (; i < full; ++i) step(i, std::false_type{});
    for (; i < steps; ++i) step(i, std::true_type{});
    if (KG > 1 && !late) phase_barrier();
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
    return bad;
  };
  if (any_wave<S::NW>(pass(std::true_type{}), smem, wave, lane)) {
    if (kg < tiles) load(kg, 0);
    pass(std::false_type{});
  }
  constexpr int MINE = (L::DB + KG - 1) / KG;  // blocks of the output that a wave writes
  float base[QF], sum[QF];
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    sum[f] = col_sum(l[f]);
    base[f] = sum[f] == 0.0f ? -INFINITY : m[f] * p.c;
  }
  if (KG > 1) {
    // Join of the groups: all outputs and statistics through LDS; group kg joins blocks kg,
    // kg + KG, ... of the columns.
    __syncthreads();
    f32x4* parts = reinterpret_cast<f32x4*>(smem);  // [KG][RW][DB][QF][64]
    float2* stats = reinterpret_cast<float2*>(smem + S::NW * S::PART);  // [KG][RW][QF][16]
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
      float top = -INFINITY, total = 0.0f;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        x[k] = stats[((k * S::RW + rw) * QF + f) * 16 + col];
        top = fmaxf(top, x[k].x);
      }
      const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        x[k].x = exp2_(x[k].x - ref);
        total += x[k].x * x[k].y;
      }
      base[f] = top;
      sum[f] = total;
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        if (i * KG + kg >= L::DB) break;
        f32x4 y = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KG; ++k) y += all[((k * S::RW * L::DB + i * KG) * QF + f) * 64] * x[k].x;
        o[i][f] = y;
      }
    }
  }
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int t = wq0 + f * 16 + col;
    const float inv = sum[f] > 0.0f ? 1.0f / sum[f] : (sum[f] == 0.0f ? 0.0f : sum[f]);
    if (t >= st.len) continue;
    const int64_t row = st.row0 + t;
    uint16_t* out = a.out.p + row * a.out.rs + head * a.out.hs;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int e = 16 * (i * KG + kg) + 4 * g;
      if (e < a.D) {
        const f32x4 x = o[i][f] * inv;
        uint2 w = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        *reinterpret_cast<uint2*>(out + e) = w;
      }
    }
    if (g == 0 && kg == 0 && a.lse)
      a.lse[(int64_t)head * a.seqs.T + row] = sum[f] == 0.0f ? -INFINITY : base[f] * LN2 + logf(sum[f]);
  }
}

template <class S>
hipError_t run(const PromptArgs& a, hipStream_t s) {
  const int64_t ranks = max_tiles(a.seqs.T, a.seqs.n, S::BM) + (a.seqs.n == 0);
  if (ranks * a.H > 0x7FFFFFFF) return hipErrorInvalidValue;
  PromptParams p{a, a.scale * LOG2E, (int32_t)ranks};
  auto kernel = &attn_prompt<S>;
  hipError_t e = ensure_lds_attr(reinterpret_cast<const void*>(kernel), S::LDS);
  if (e != hipSuccess) return e;
  return launch_k(kernel, dim3((unsigned)(ranks * a.H)), dim3(64 * S::NW), S::LDS, s, p);
}

template <int DS>
hipError_t choose(const PromptArgs& a, hipStream_t s) {
  // A workgroup of 128 rows at the end of a sequence takes about 65536 / (rows heads) times as
  // long as the whole call would on evenly loaded CUs.  64 rows and four groups of waves on the
  // keys take a quarter, but their tiles serve half the rows: 0.6 of the rate.  Measured, groups
  // against one: 4096 rows of 8 heads on 8 (8 sequences) 33 and 37 us, 8184 of 4 on 4 (2) 55 and
  // 76; 5120 of 8 on 1 (2) 57 and 55, of 8 on 8 (8) 41 and 43; 6144 of 8 on 1 70 and 65, on 8
  // 53 and 49.
  if ((int64_t)a.seqs.T * a.H < 44 * 1024 && few_sequences(a.seqs.n, a.H)) return run<Shape<DS, 2, 2, 4, 32>>(a, s);
  return run<Shape<DS, 2, 4, 1, 64>>(a, s);
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t s) {
  if (a.D <= 64) return choose<2>(a, s);
  if (a.D <= 96) return choose<3>(a, s);
  return choose<4>(a, s);
}

}  // namespace ubx
