// Causal attention within packed sequences, on gfx950 matrix cores.
//
//   s = scale q k^T (u <= t),  lse = log sum_u exp(s),  out = sum_u exp(s - lse) v
//
// One pass over the keys with the running maximum m and sum l of the softmax, in base 2:
// with c = scale log2(e), p = exp2(c s - c m).  A workgroup owns BM query rows of one head;
// each of its 4 waves keeps its rows (as columns of the score tiles, see attn_common.h),
// their fp32 output [head_dim x rows] and statistics in registers, and all waves share the
// 64-row key and value tiles that direct-to-LDS loads bring in, double-buffered.  A score
// column lives in four lanes, so its maximum costs two lane swaps and its rescaling factor
// is a per-lane scalar.
//
// Rows past a sequence's end (of any input) are never read: their loads fall outside the
// buffer resource and give zeros.
#include <hip/hip_runtime.h>

#include "attn_common.h"

namespace ubx {
namespace {

constexpr int NW = 4;
constexpr int BN = 64;

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

template <int DS, int QF>
__global__ __launch_bounds__(64 * NW, 2) void attn_prompt(PromptParams p) {
  using L = Tile<DS>;
  constexpr int BM = 16 * QF * NW;
  constexpr int KB = BN / 16;
  constexpr int TILE = BN * L::RB;
  extern __shared__ unsigned char smem[];
  const PromptArgs& a = p.a;
  const int head = blockIdx.x % a.H, rank = blockIdx.x / a.H;
  fill_pad(a, head, rank, p.ranks);
  const SeqTile st = find_tile(a.seqs, BM, rank, false);
  if (st.len == 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int kvh = head / (a.H / a.G);
  const int q0 = st.tile * BM;
  const int wq0 = q0 + wave * 16 * QF;  // the wave's first query
  const int n_keys = min(q0 + BM, st.len);
  const int tiles = (n_keys + BN - 1) / BN;
  const uint16_t* kbase = a.k.p + (int64_t)st.row0 * a.k.rs + kvh * a.k.hs;
  const uint16_t* vbase = a.v.p + (int64_t)st.row0 * a.v.rs + kvh * a.v.hs;

  TileLoad<DS, BN, NW> kl, vl;
  kl.init(wave, lane, a.k.rs, a.D);
  vl.init(wave, lane, a.v.rs, a.D);
  const uint32_t lds = lds_addr(smem);
  auto load = [&](int j, int stage) {
    kl.issue(kbase + (int64_t)j * BN * a.k.rs, a.k.rs, a.D, st.len - j * BN, lds + stage * 2 * TILE, wave);
    vl.issue(vbase + (int64_t)j * BN * a.v.rs, a.v.rs, a.D, st.len - j * BN, lds + stage * 2 * TILE + TILE,
             wave);
  };
  bf16x8 q[QF][DS];
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int t = wq0 + f * 16 + col;
    const uint16_t* row = a.q.p + (int64_t)(st.row0 + t) * a.q.rs + head * a.q.hs;
#pragma unroll
    for (int s = 0; s < DS; ++s) q[f][s] = load_row8(row + 32 * s + 8 * g, t < st.len && 32 * s + 8 * g < a.D);
  }
  load(0, 0);

  RowFrag<DS> kf;
  ColFrag<DS> vf;
  kf.init(smem, lane);
  vf.init(smem + TILE, lane);
  f32x4 o[L::DB][QF];
  float m[QF], l[QF];
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    m[f] = -INFINITY;
    l[f] = 0.0f;
#pragma unroll
    for (int d = 0; d < L::DB; ++d) o[d][f] = f32x4{0, 0, 0, 0};
  }
  for (int j = 0; j < tiles; ++j) {
    const int stage = (j & 1) * 2 * TILE;
    wait_vmcnt_and_barrier<0>();
    if (j + 1 < tiles) load(j + 1, (j + 1) & 1);
    const int k0 = j * BN;
    if (k0 > wq0 + 16 * QF - 1) continue;  // all keys after the wave's queries
    f32x4 s[KB][QF];
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
    if (k0 + BN - 1 > wq0) {  // the diagonal: keys after the query
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int f = 0; f < QF; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k0 + b * 16 + 4 * g + i > wq0 + f * 16 + col) s[b][f][i] = -INFINITY;
    }
#pragma unroll
    for (int f = 0; f < QF; ++f) {
      float x = s[0][f][0];
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) x = fmaxf(x, s[b][f][i]);
      x = fmaxf(col_max(x), m[f]);
      const float base = x == -INFINITY ? 0.0f : x * p.c;
      const float r = exp2_(m[f] * p.c - base);  // 0 the first time
      m[f] = x;
      l[f] *= r;
#pragma unroll
      for (int d = 0; d < L::DB; ++d) o[d][f] *= r;
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[b][f][i] = exp2_(s[b][f][i] * p.c - base);
          l[f] += s[b][f][i];
        }
    }
#pragma unroll
    for (int t = 0; t < KB / 2; ++t) {
      bf16x8 pf[QF];
#pragma unroll
      for (int f = 0; f < QF; ++f) pf[f] = pack8(s[2 * t][f], s[2 * t + 1][f]);
#pragma unroll
      for (int d = 0; d < L::DB; ++d) {
        const bf16x8 vv = vf.read(stage, t, d);
#pragma unroll
        for (int f = 0; f < QF; ++f)
          o[d][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv, pf[f], o[d][f], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int f = 0; f < QF; ++f) {
    const int t = wq0 + f * 16 + col;
    const float sum = col_sum(l[f]);
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
    if (t >= st.len) continue;
    const int64_t row = st.row0 + t;
    uint16_t* out = a.out.p + row * a.out.rs + head * a.out.hs;
#pragma unroll
    for (int d = 0; d < L::DB; ++d) {
      const int e = 16 * d + 4 * g;
      if (e < a.D) {
        const f32x4 x = o[d][f] * inv;
        uint2 w = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        *reinterpret_cast<uint2*>(out + e) = w;
      }
    }
    if (g == 0 && a.lse)
      a.lse[(int64_t)head * a.seqs.T + row] = sum == 0.0f ? -INFINITY : m[f] * p.c * LN2 + logf(sum);
  }
}

template <int DS, int QF>
hipError_t run(const PromptArgs& a, hipStream_t s) {
  constexpr int lds = 4 * BN * Tile<DS>::RB;
  const int64_t ranks = max_tiles(a.seqs.T, a.seqs.n, 16 * QF * NW) + (a.seqs.n == 0);
  if (ranks * a.H > 0x7FFFFFFF) return hipErrorInvalidValue;
  PromptParams p{a, a.scale * LOG2E, (int32_t)ranks};
  auto kernel = &attn_prompt<DS, QF>;
  hipError_t e = ensure_lds_attr(reinterpret_cast<const void*>(kernel), lds);
  if (e != hipSuccess) return e;
  return launch_k(kernel, dim3((unsigned)(ranks * a.H)), dim3(64 * NW), lds, s, p);
}

}  // namespace

hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t s) {
  if (a.D <= 64) return run<2, 2>(a, s);
  if (a.D <= 96) return run<3, 2>(a, s);
  return run<4, 2>(a, s);
}

}  // namespace ubx
