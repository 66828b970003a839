// Position rotation of q and k and the append of k and v to a paged key-value cache.
//
//   angle = pos * inv_freq[m];  (a, b) -> (a cos - b sin, b cos + a sin)
//
// pos is the token's place in its sequence, or (drafted trees) past_lens and an offset of its own;
// the place says where it is stored.
//
// HBM-bound: each of the token's (H + 2 G) D bf16 values is read once, each output written
// once; the arithmetic per element is a few operations.  What would cost is the angle: far
// positions need its reduction in 64 bits, pos * inv_freq / (2 pi) less its nearest integer,
// and a precise sine and cosine.  A workgroup therefore computes the (cos, sin) pairs of its
// tokens once into LDS, where all their heads read them.  The same pass looks up each
// token's sequence (a ballot over 64 boundaries at a time: one load's latency instead of a
// binary search's chain) and its cache slot, a token to a lane.
//
// Items: a rotary item is 8 pairs (two 16-byte vectors of one head), a copy item is one
// 16-byte vector (elements past rotary_dim, and v).  Items come in five sections (rotated q,
// rotated k, the rest of q, the rest of k, v), each numbered token by token and head by
// head; a wave takes 64 items of one section at a time, so that its lanes do the same work:
// with sections mixed in a wave every wave ran the E4M3 conversion's instructions.  The next
// items are loaded before the present ones are finished, the first ones before the lookup.
//
// Stores to the cache do not pass through the L2 (it is read by later calls, the decode steps
// above all), nor do q_out and k_out where they are larger than it: with inputs that no cache
// holds, 32520 tokens of 8 + 1 heads to an E4M3 cache take 29.0 us (5.4 TB/s, a copy's rate)
// instead of 37.2, and with ub_attn_prompt after it 612 instead of 610.  Smaller outputs the next
// call finds there: 8184 tokens of 4 + 4 heads took 12.9 us, with ub_attn_prompt 73, where past the
// L2 they took 12.5 and 74.5.
#include <hip/hip_runtime.h>

#include "attn_internal.h"
#include "gemm_common.h"
#include "kv_pages.h"

namespace ubx {
namespace {

constexpr int THREADS = 256;
constexpr int WAVES = THREADS / 64;
constexpr int MAX_TOKENS = 8;   // tokens of a workgroup
constexpr int MAX_HALF = UB_ATTN_MAX_HEAD_DIM / 2;
constexpr int64_t L2_BYTES = 32 << 20;  // the XCDs' together
enum { ROT_Q, ROT_K, REST_Q, REST_K, VALUES, SECTIONS };

struct Section {
  int32_t n;         // items per token
  int32_t per;       // items per head
  float inv_n;       // 1 / n
  uint32_t per_inv;  // ceil(2^32 / per)
  int32_t task_end;  // waves' tasks of this section and the ones before
};

struct AppendParams {
  AppendArgs a;
  int32_t tokens;  // tokens of a workgroup
  Section s[SECTIONS];
};

struct Token {
  int64_t slot;  // element offset of the token's slot in head 0 of the cache, or -1
  int64_t pos;   // for the rotation
  int32_t live;  // belongs to a sequence
};

__device__ inline float lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ inline float hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// E4M3 codes of 4 values: the rule of e4m3.h by the hardware's conversion, which rounds to
// nearest even but neither saturates (so values past 448 are cut first; NaN passes) nor keeps
// a NaN's sign (so the signs are put in from the values).
__device__ inline uint32_t e4m3x4(const float* x, float scale) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = x[i] * scale;
    if (fabsf(y[i]) > 448.0f) y[i] = copysignf(448.0f, y[i]);
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
  // top bytes of the four values
  const uint32_t tops = __builtin_amdgcn_perm(__float_as_uint(y[1]), __float_as_uint(y[0]), 0x0C0C0703u) |
                        __builtin_amdgcn_perm(__float_as_uint(y[3]), __float_as_uint(y[2]), 0x07030C0Cu);
  return ((uint32_t)w & 0x7F7F7F7Fu) | (tops & 0x80808080u);
}

// 8 values to a cache slot: bf16, or E4M3 codes of x * scale.
__device__ inline void store_cache(const KvCache& c, void* base, int64_t off, const float* x,
                                   float scale) {
  if (c.e4m3) {
    uint2 o = make_uint2(e4m3x4(x, scale), e4m3x4(x + 4, scale));
    __builtin_nontemporal_store(__builtin_bit_cast(uint64_t, o),
                                GLOBAL_PTR(uint64_t, static_cast<uint8_t*>(base) + off));
  } else {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    __builtin_nontemporal_store(o, GLOBAL_PTR(u32x4, static_cast<uint16_t*>(base) + off));
  }
}

template <bool PAST_L2>
__device__ inline void store_bf16(uint16_t* p, const float* x) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  if (PAST_L2) __builtin_nontemporal_store(o, GLOBAL_PTR(u32x4, p));
  else *GLOBAL_PTR(u32x4, p) = o;
}

__device__ inline void unpack(u32x4 v, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo(v[i]);
    x[2 * i + 1] = hi(v[i]);
  }
}

// Place of pair 8 k + u among a token's: two pairs in 16 bytes, those that lanes read together
// (of the items k of a head) side by side.
__device__ inline int at_pair(int k, int u) { return ((u >> 1) * (MAX_HALF / 8) + k) * 2 + (u & 1); }

// A lane's item of a wave's task, loaded.
struct Item {
  int sec;     // the wave's section
  bool valid;
  int j, head, e0, e1;  // token of the workgroup, head, first elements of its vectors
  u32x4 x, y;
};

__device__ inline Item load_item(const AppendParams& p, int task, int t0, int nt, int lane) {
  const AppendArgs& a = p.a;
  Item w;
  w.sec = 0;
  int base = 0;
#pragma unroll
  for (int i = 0; i + 1 < SECTIONS; ++i)
    if (task >= p.s[i].task_end) {
      w.sec = i + 1;
      base = p.s[i].task_end;
    }
  const Section s = p.s[w.sec];
  const int i = (task - base) * 64 + lane;
  // i / n: both under 2^24, so the product is off by less than one
  w.j = (int)((float)i * s.inv_n);
  int it = i - w.j * s.n;
  if (it < 0) {
    --w.j;
    it += s.n;
  } else if (it >= s.n) {
    ++w.j;
    it -= s.n;
  }
  w.valid = task < p.s[SECTIONS - 1].task_end && w.j < nt;
  w.head = s.per == 1 ? it : (int)__umulhi((uint32_t)it, s.per_inv);
  const int c = (it - w.head * s.per) * 8;
  const bool rot = w.sec <= ROT_K, inter = a.interleaved != 0;
  w.e0 = rot ? (inter ? 2 * c : c) : (w.sec == VALUES ? c : a.rotary + c);
  w.e1 = inter ? w.e0 + 8 : w.e0 + a.rotary / 2;
  w.x = w.y = u32x4{0, 0, 0, 0};
  if (w.valid) {
    const Heads& src = w.sec == VALUES ? a.v : (w.sec == ROT_Q || w.sec == REST_Q) ? a.q : a.k;
    const uint16_t* in = src.p + (int64_t)(t0 + w.j) * src.rs + w.head * src.hs;
    w.x = *GLOBAL_PTR(const u32x4, in + w.e0);
    if (rot) w.y = *GLOBAL_PTR(const u32x4, in + w.e1);
  }
  return w;
}

// 64 registers, for 8 waves per SIMD: 37.2 us in the second case above, 39.4 with 66 and 7.
template <bool PAST_L2>
__global__ __launch_bounds__(THREADS, 8) void kv_append(AppendParams p) {
  __shared__ Token tok[MAX_TOKENS];
  __shared__ float2 rot[MAX_TOKENS][MAX_HALF];
  const AppendArgs& a = p.a;
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, a.seqs.T - t0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tasks = p.s[SECTIONS - 1].task_end;
  Item w = load_item(p, wave, t0, nt, lane);
  const int half = a.rotary / 2;
  const float freq = lane < half ? a.inv_freq[lane] : 0.0f;
  if (wave == 0) {
    // lane j: token j of the workgroup.  Sequences that end at or before its row come first:
    // their number is its sequence
    int seq = 0;
    for (int c = 0; c < a.seqs.n; c += 64) {
      const int i = c + lane;
      const int end = i < a.seqs.n ? a.seqs.cu[i + 1] : 0x7FFFFFFF;
      int more = 0;
      for (int j = 0; j < nt; ++j) {
        const int m = __popcll(__ballot(end <= t0 + j));
        seq += lane == j ? m : 0;
        more |= m == 64;
      }
      if (!more) break;
    }
    if (lane < nt) {
      const int t = t0 + lane;
      Token k{-1, 0, 0};
      if (seq < a.seqs.n) {
        const int start = a.seqs.cu[seq];
        const int past = a.past ? a.past[seq] : 0;
        if (start >= 0 && start <= t) {
          const int64_t pos = (int64_t)past + (t - start);
          k.live = 1;
          k.pos = pos;
          if (a.offsets) k.pos = (int64_t)past + a.offsets[t];
          const int e = a.cache.k ? page_entry(pos, a.cache.page_size, a.pages_per_seq) : -1;
          if (e >= 0)
            k.slot = token_offset(pos, a.pages[(int64_t)seq * a.pages_ld + e], a.cache.n_pages,
                                  a.cache.page_size, a.cache.ps, a.cache.ts);
        }
      }
      tok[lane] = k;
    }
  }
  __syncthreads();
  for (int j = wave; j < nt; j += WAVES) {
    if (lane >= half) break;
    // revolutions, reduced in 64 bits; the product pos * inv_freq, of a position below 2^29 and a
    // 24-bit significand, is exact there
    double r = (double)tok[j].pos * (double)freq * 0.15915494309189533577;
    r -= rint(r);
    float s, c;
    sincospif(2.0f * (float)r, &s, &c);
    rot[j][at_pair(lane >> 3, lane & 7)] = make_float2(c, s);
  }
  __syncthreads();
  for (int task = wave; task < tasks; task += WAVES) {
    const Item next = load_item(p, task + WAVES, t0, nt, lane);
    if (w.valid) {
      const Token k = tok[w.j];
      const int64_t t = t0 + w.j;
      float x[8], y[8];
      unpack(k.live ? w.x : u32x4{0, 0, 0, 0}, x);
      const bool is_q = w.sec == ROT_Q || w.sec == REST_Q;
      const Heads& dst = is_q ? a.q_out : a.k_out;
      const bool slot = !is_q && k.slot >= 0;
      const int64_t off = k.slot + w.head * a.cache.hs;
      void* const cache = w.sec == VALUES ? a.cache.v : a.cache.k;
      const float scale = w.sec == VALUES ? a.cache.v_scale : a.cache.k_scale;
      if (w.sec <= ROT_K) {
        unpack(k.live ? w.y : u32x4{0, 0, 0, 0}, y);
        if (a.interleaved) {
          const float2* r = rot[w.j];
          const int k = w.e0 >> 4;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 c0 = r[at_pair(k, u)], c1 = r[at_pair(k, 4 + u)];
            const float p0 = x[2 * u], p1 = x[2 * u + 1], r0 = y[2 * u], r1 = y[2 * u + 1];
            x[2 * u] = p0 * c0.x - p1 * c0.y;
            x[2 * u + 1] = p1 * c0.x + p0 * c0.y;
            y[2 * u] = r0 * c1.x - r1 * c1.y;
            y[2 * u + 1] = r1 * c1.x + r0 * c1.y;
          }
        } else {
          const float2* r = rot[w.j];
          const int k = w.e0 >> 3;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float2 c = r[at_pair(k, u)];
            const float p0 = x[u], p1 = y[u];
            x[u] = p0 * c.x - p1 * c.y;
            y[u] = p1 * c.x + p0 * c.y;
          }
        }
        if (dst.p) store_bf16<PAST_L2>(dst.p + t * dst.rs + w.head * dst.hs + w.e1, y);
        if (slot) store_cache(a.cache, cache, off + w.e1, y, scale);
      }
      if (dst.p && w.sec != VALUES) store_bf16<PAST_L2>(dst.p + t * dst.rs + w.head * dst.hs + w.e0, x);
      if (slot) store_cache(a.cache, cache, off + w.e0, x, scale);
    }
    w = next;
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t s) {
  AppendParams p{};
  p.a = a;
  const int qh = a.q.p ? a.H : 0, kh = a.k.p ? a.G : 0, vh = a.cache.k ? a.G : 0;
  const int pairs = a.rotary / 16, rest = (a.D - a.rotary) / 8;
  const int heads[SECTIONS] = {qh, kh, qh, kh, vh};
  const int per[SECTIONS] = {pairs, pairs, rest, rest, a.D / 8};
  int most = 0;
  for (int i = 0; i < SECTIONS; ++i) {
    Section& x = p.s[i];
    x.n = heads[i] * per[i];
    x.per = per[i] > 0 ? per[i] : 1;
    x.inv_n = x.n > 0 ? 1.0f / (float)x.n : 0.0f;
    x.per_inv = x.per > 1 ? (uint32_t)(((uint64_t(1) << 32) + x.per - 1) / x.per) : 0;
    if (x.n > most) most = x.n;
  }
  if (a.seqs.T <= 0 || most == 0) return hipSuccess;
  // One token per workgroup of a small call starts soonest; more share the angles' and the
  // lookup's time.  2048 workgroups run at once, and past that 8 tokens serve best.  Measured with
  // 4 and 8 tokens: 8184 tokens (4 + 4 heads, bf16 cache) 11.9 and 12.9 us, 4096 11.8 with
  // 2 and 13.2 with 4; 32520 (8 + 1 heads, E4M3) 32.9 and 29.0, with 16 30.4.  An item's number stays
  // under 2^24.
  int tokens = (a.seqs.T + 2047) / 2048;
  if (tokens > MAX_TOKENS) tokens = MAX_TOKENS;
  if (tokens * (int64_t)most + 64 * (WAVES + 1) >= (1 << 24)) tokens = 1;
  p.tokens = tokens;
  int end = 0;
  for (int i = 0; i < SECTIONS; ++i) {
    end += (int)(((int64_t)p.s[i].n * tokens + 63) / 64);
    p.s[i].task_end = end;
  }
  const int blocks = (a.seqs.T + tokens - 1) / tokens;
  const int64_t out = (int64_t)a.seqs.T * ((a.q_out.p ? a.H : 0) + (a.k_out.p ? a.G : 0)) * a.D * 2;
  return launch_k(out > L2_BYTES ? &kv_append<true> : &kv_append<false>, dim3(blocks), dim3(THREADS), 0, s, p);
}

}  // namespace ubx
