// Attention of one new token per sequence over a paged key-value cache.
//
//   s_u = scale q . k_u,  lse = log sum_u exp(s_u),  out = sum_u exp(s_u - lse) v_u
//
// HBM-bound: the keys and values of every cached token are read once and used for a few
// operations each.  The lengths are on the device and ragged, so the work is cut by them
// there: chunks of C tokens, C from the total length, so that about ITEMS workgroups have
// equal work whatever the raggedness; every workgroup finds its own chunk from the lengths.
// A sequence of one chunk is finished by its workgroup; the parts of the others (maximum,
// sum and unnormalised output, fp32) go to the workspace and attn_decode_join adds them in
// order.
//
// A wave takes 32 tokens at a time.  Scores are K q^T on matrix cores, the query heads of a
// group (up to 16) as the 16 columns: keys go from memory straight into the A fragment.
// Values pass through a wave-private LDS tile, from which transposing reads give V^T
// (attn_common.h).
#include <hip/hip_runtime.h>

#include "attn_common.h"
#include "kv_pages.h"

namespace ubx {
namespace {

constexpr int NW = 4;
constexpr int STEP = 32;          // tokens a wave takes at a time
constexpr int MIN_CHUNK = NW * STEP;
constexpr int ITEMS = 1024;       // workgroups the total length is cut for
constexpr int COLS = 16;          // query heads of a workgroup

struct DecodeParams {
  DecodeArgs a;
  float c;          // scale * log2(e) (/ k_scale)
  float v_inv;      // 1 / v_scale
  int32_t qb;       // column blocks of a group
  int32_t cap;      // tokens the page table can hold per sequence
  float* part;      // [items, COLS, D]
  float2* stat;     // [items, COLS]: maximum (base 2, scaled), sum
};

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

// Cached tokens of sequence i, as far as the page table reaches.
__device__ inline int kv_len(const DecodeParams& p, int i) { return clamp_len(p.a.lens[i], p.cap); }

// Tokens of a chunk, from the total length and the workgroups that share a token.
__device__ inline int chunk_tokens(const DecodeParams& p) {
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  for (int i = lane; i < p.a.n; i += 64) total += kv_len(p, i);
  for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
  const int64_t want = (total * p.a.G * p.qb + ITEMS - 1) / ITEMS;
  const int64_t c = (want + MIN_CHUNK - 1) / MIN_CHUNK * MIN_CHUNK;
  return (int)min(max(c, (int64_t)MIN_CHUNK), (int64_t)1 << 30);
}

struct Chunk {
  int seq, len, index, count;  // sequence, its length, chunk of it, its chunks
  int first;                   // number of the sequence's first chunk among all
};

// Chunk `rank` of all sequences' chunks; false past the last.
__device__ inline bool find_chunk(const DecodeParams& p, int C, int rank, Chunk& r) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int c = 0; c < p.a.n; c += 64) {
    const int len = c + lane < p.a.n ? kv_len(p, c + lane) : 0;
    const int nc = (int)(((int64_t)len + C - 1) / C);
    const int incl = wave_scan(nc);
    const uint64_t m = __ballot(before + incl > rank);
    if (m) {
      const int at = __builtin_ctzll(m);
      r.seq = c + at;
      r.len = __builtin_amdgcn_readlane(len, at);
      r.count = __builtin_amdgcn_readlane(nc, at);
      r.first = before + __builtin_amdgcn_readlane(incl, at) - r.count;
      r.index = rank - r.first;
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

__device__ inline uint32_t cvt2(uint32_t w, bool high) {
  const auto r = high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                      : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
  return __builtin_bit_cast(uint32_t, r);
}

// 8 E4M3 codes -> 8 bf16 (exact).
__device__ inline u32x4 cvt8(uint32_t a, uint32_t b) {
  return u32x4{cvt2(a, false), cvt2(a, true), cvt2(b, false), cvt2(b, true)};
}

template <int DS, bool F8>
__global__ __launch_bounds__(64 * NW, 2) void attn_decode(DecodeParams p) {
  using L = Tile<DS>;
  constexpr int TILE = STEP * L::RB;
  constexpr int MERGE = NW * COLS * (32 * DS + 2) * 4;
  constexpr int SMEM = NW * TILE > MERGE ? NW * TILE : MERGE;
  __shared__ __align__(16) unsigned char smem[SMEM];
  const DecodeArgs& a = p.a;
  const int GQ = a.G * p.qb;
  const int gq = blockIdx.x % GQ, rank = blockIdx.x / GQ;
  const int kvh = gq / p.qb, group = a.H / a.G, col0 = (gq - kvh * p.qb) * COLS;
  const int cols = min(group - col0, COLS);
  const int C = chunk_tokens(p);
  Chunk ch;
  if (!find_chunk(p, C, rank, ch)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int begin = ch.index * C, end = min(ch.len, begin + C);
  const int32_t* pages = a.pages + (int64_t)ch.seq * a.pages_ld;
  bool bad = a.lens[ch.seq] > p.cap;

  // queries: element order of the key fragments below
  bf16x8 q[DS];
  const uint16_t* qrow = a.q.p + (int64_t)ch.seq * a.q.rs + (kvh * group + col0 + col) * a.q.hs;
#pragma unroll
  for (int s = 0; s < DS; ++s) {
    const int e = F8 ? 64 * (s / 2) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
    q[s] = load_row8(qrow + e, col < cols && e < a.D);
  }
  constexpr int EB = F8 ? 1 : 2;             // bytes per element
  constexpr int KV = F8 ? (DS + 1) / 2 : DS; // 16-byte loads of a key row per lane group
  constexpr int VPR = F8 ? L::CPR / 2 : L::CPR;  // 16-byte pieces of a value row
  constexpr int VI = STEP * VPR / 64;        // value loads per lane
  const unsigned char* kb = static_cast<const unsigned char*>(a.cache.k) + kvh * a.cache.hs * EB;
  const unsigned char* vb = static_cast<const unsigned char*>(a.cache.v) + kvh * a.cache.hs * EB;
  unsigned char* tile = smem + wave * TILE;
  ColFrag<DS> vf;
  vf.init(tile, lane);
  const int pieces = a.D * EB / 16;

  f32x4 o[L::DB];
#pragma unroll
  for (int d = 0; d < L::DB; ++d) o[d] = f32x4{0, 0, 0, 0};
  float m = -INFINITY, l = 0.0f;
  for (int t0 = begin + wave * STEP; t0 < end; t0 += NW * STEP) {
    // byte offset of token t0 + lane % 32 in head 0; positions past the end repeat the last
    const int pos = min(t0 + (lane & 31), end - 1);
    const int64_t at = token_offset(pos, pages[page_entry(pos, a.cache.page_size, a.pages_per_seq)],
                                    a.cache.n_pages, a.cache.page_size, a.cache.ps, a.cache.ts);
    bad = bad || __ballot(at < 0) != 0;
    const int64_t off = max(at, (int64_t)0) * EB;
    const int off_lo = (int)(uint32_t)off, off_hi = (int)(off >> 32);
    auto row_off = [&](int r) {
      const uint32_t x = (uint32_t)__shfl(off_lo, r);
      return (int64_t)(((uint64_t)(uint32_t)__shfl(off_hi, r) << 32) | x);
    };
    u32x4 k[2][KV], v[VI];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const unsigned char* row = kb + row_off(16 * b + col);
#pragma unroll
      for (int s = 0; s < KV; ++s) {
        const int piece = 4 * s + g;
        k[b][s] = *GLOBAL_PTR(const u32x4, row + (piece < pieces ? piece : 0) * 16);
      }
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      const int r = i * (64 / VPR) + lane / VPR, piece = lane % VPR;
      v[i] = *GLOBAL_PTR(const u32x4, vb + row_off(r) + (piece < pieces ? piece : 0) * 16);
    }
    f32x4 s[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int d = 0; d < DS; ++d)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const u32x4 w = F8 ? (d & 1 ? cvt8(k[b][d / 2][2], k[b][d / 2][3]) : cvt8(k[b][d / 2][0], k[b][d / 2][1]))
                           : k[b][F8 ? 0 : d];
        s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), q[d], s[b], 0, 0, 0);
      }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
      const int r = i * (64 / VPR) + lane / VPR, piece = lane % VPR;
      if (F8) {
        const u32x4 w0 = cvt8(v[i][0], v[i][1]), w1 = cvt8(v[i][2], v[i][3]);
        *LDS_PTR(u32x4, tile + r * L::RB + (((2 * piece) ^ L::swz(r)) * 16)) = w0;
        *LDS_PTR(u32x4, tile + r * L::RB + (((2 * piece + 1) ^ L::swz(r)) * 16)) = w1;
      } else {
        *LDS_PTR(u32x4, tile + r * L::RB + ((piece ^ L::swz(r)) * 16)) = v[i];
      }
    }
    float x = -INFINITY;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t0 + 16 * b + 4 * g + i >= end) s[b][i] = -INFINITY;
        x = fmaxf(x, s[b][i]);
      }
    x = fmaxf(col_max(x), m);
    const float base = x == -INFINITY ? 0.0f : x * p.c;
    const float r = exp2_(m * p.c - base);
    m = x;
    l *= r;
#pragma unroll
    for (int d = 0; d < L::DB; ++d) o[d] *= r;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[b][i] = exp2_(s[b][i] * p.c - base);
        l += s[b][i];
      }
    const bf16x8 pf = pack8(s[0], s[1]);
#pragma unroll
    for (int d = 0; d < L::DB; ++d)
      o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf.read(0, 0, d), pf, o[d], 0, 0, 0);
  }
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
  const bool alone = ch.count == 1;
  const int64_t item = (int64_t)(ch.first + ch.index) * GQ + gq;
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
      a.out.p[(int64_t)ch.seq * a.out.rs + head * a.out.hs + d] = (uint16_t)pack_bf16x2(x * inv, 0.0f);
      if (d == 0 && a.lse)
        a.lse[(int64_t)head * a.T + ch.seq] = sum == 0.0f ? -INFINITY : b * LN2 + logf(sum);
    } else {
      p.part[(item * COLS + h) * a.D + d] = x;
      if (d == 0) p.stat[item * COLS + h] = make_float2(mm, sum);
    }
  }
}

// Row and head of a workgroup: zeros for rows of no sequence or length 0; the sum of the
// parts, in order, for sequences of several chunks.
__global__ __launch_bounds__(256) void attn_decode_join(DecodeParams p) {
  __shared__ float red[256 * 4 + 8];
  const DecodeArgs& a = p.a;
  const int head = blockIdx.x % a.H, row = blockIdx.x / a.H;
  const int len = row < a.n ? kv_len(p, row) : 0;
  uint16_t* out = a.out.p + (int64_t)row * a.out.rs + head * a.out.hs;
  if (len == 0) {
    if ((int)threadIdx.x < a.D) out[threadIdx.x] = 0;
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)head * a.T + row] = -INFINITY;
    return;
  }
  const int C = chunk_tokens(p);
  const int count = (len + C - 1) / C;
  if (count == 1) return;
  int first = 0;
  const int lane = threadIdx.x & 63;
  for (int i = lane; i < row; i += 64) first += (int)(((int64_t)kv_len(p, i) + C - 1) / C);
  first = wave_sum(first);
  const int group = a.H / a.G, kvh = head / group, hc = head - kvh * group;
  const int GQ = a.G * p.qb;
  const int64_t item0 = (int64_t)first * GQ + kvh * p.qb + hc / COLS;
  const int h = hc % COLS;
  auto at = [&](int i) { return (item0 + (int64_t)i * GQ) * COLS + h; };
  float mm = -INFINITY;
  for (int i = lane; i < count; i += 64) mm = fmaxf(mm, p.stat[at(i)].x);
  for (int d = 1; d < 64; d *= 2) mm = fmaxf(mm, __shfl_xor(mm, d));
  const float b = mm == -INFINITY ? 0.0f : mm;
  float sum = 0.0f;
  for (int i = lane; i < count; i += 64) {
    const float2 st = p.stat[at(i)];
    sum += exp2_(st.x - b) * st.y;
  }
  for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
  const int vec = a.D / 4, groups = 256 / vec;
  const int w = threadIdx.x / vec, e = (threadIdx.x - w * vec) * 4;
  f32x4 x = {0, 0, 0, 0};
  if (w < groups)
    for (int i = w; i < count; i += groups)
      x += *reinterpret_cast<const f32x4*>(p.part + at(i) * a.D + e) * exp2_(p.stat[at(i)].x - b);
  *reinterpret_cast<f32x4*>(red + threadIdx.x * 4) = x;
  __syncthreads();
  if (w == 0) {
    for (int k = 1; k < groups; ++k) x += *reinterpret_cast<const f32x4*>(red + (k * vec) * 4 + e);
    const float inv = sum == 0.0f ? 0.0f : p.v_inv / sum;
    x *= inv;
    uint2 o = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    *reinterpret_cast<uint2*>(out + e) = o;
    if (threadIdx.x == 0 && a.lse)
      a.lse[(int64_t)head * a.T + row] = sum == 0.0f ? -INFINITY : b * LN2 + logf(sum);
  }
}

int64_t item_count(int32_t H, int32_t G, int32_t n) {
  const int64_t qb = (H / G + COLS - 1) / COLS;
  // sum of ceil(len / C) over the sequences, times the G qb workgroups that share a chunk
  return ITEMS + (int64_t)n * G * qb;
}

template <int DS, bool F8>
hipError_t run(const DecodeArgs& a, hipStream_t s) {
  DecodeParams p{};
  p.a = a;
  p.qb = (a.H / a.G + COLS - 1) / COLS;
  p.cap = table_cap(a.pages_per_seq, a.cache.page_size);
  p.c = a.scale * LOG2E * (F8 ? 1.0f / a.cache.k_scale : 1.0f);
  p.v_inv = F8 ? 1.0f / a.cache.v_scale : 1.0f;
  const int64_t items = item_count(a.H, a.G, a.n);
  p.stat = static_cast<float2*>(a.ws);
  p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.ws) + items * COLS * 8);
  const int64_t GQ = (int64_t)a.G * p.qb;
  const int64_t blocks = (items + GQ - 1) / GQ * GQ;
  if (blocks > 0x7FFFFFFF || (int64_t)a.T * a.H > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipError_t e = hipSuccess;
  if (a.n > 0) e = launch_k(&attn_decode<DS, F8>, dim3((unsigned)blocks), dim3(64 * NW), 0, s, p);
  if (e == hipSuccess)
    e = launch_k(&attn_decode_join, dim3((unsigned)(a.T * a.H)), dim3(256), 0, s, p);
  return e;
}

}  // namespace

size_t attn_decode_bytes(int32_t H, int32_t G, int32_t D, int32_t n) {
  return (size_t)(item_count(H, G, n) * COLS * (8 + (int64_t)D * 4));
}

hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s) {
  // E4M3 keys take two steps of a 16-byte piece each: an even number of them
  if (a.cache.e4m3) return a.D <= 64 ? run<2, true>(a, s) : run<4, true>(a, s);
  return a.D <= 64 ? run<2, false>(a, s) : a.D <= 96 ? run<3, false>(a, s) : run<4, false>(a, s);
}

}  // namespace ubx
