// Position rotation of q and k and the append of k and v to a paged key-value cache.
//
//   angle = pos * inv_freq[m];  (a, b) -> (a cos - b sin, b cos + a sin)
//
// HBM-bound: each of the token's (H + 2 G) D bf16 values is read once, each output written
// once; the arithmetic per element is a few operations.  What would cost is the angle: far
// positions need its reduction in 64 bits, pos * inv_freq / (2 pi) less its nearest integer,
// and a precise sine and cosine.  A workgroup therefore computes the (cos, sin) pairs of its
// tokens once into LDS, where all their heads read them.  The same pass looks up each
// token's sequence (a ballot over 64 boundaries at a time: one load's latency instead of a
// binary search's chain) and its cache slot.
//
// Items: a rotary item is 8 pairs (two 16-byte vectors of one head), a copy item is one
// 16-byte vector (elements past rotary_dim, and v).  Items of one token are numbered head by
// head, so that neighbouring threads take neighbouring addresses.
#include <hip/hip_runtime.h>

#include "attn_internal.h"
#include "e4m3.h"
#include "gemm_common.h"
#include "kv_pages.h"

namespace ubx {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 8;  // tokens of a workgroup
constexpr int MAX_HALF = UB_ATTN_MAX_HEAD_DIM / 2;

struct AppendParams {
  AppendArgs a;
  int32_t tokens;      // tokens of a workgroup
  int32_t rot_per_head, copy_per_head, v_per_head;  // items
  int32_t n_rot, n_copy, n_items;                   // per token
  int32_t qh;                                       // query heads handled (0 without q)
};

struct Token {
  int64_t slot;  // element offset of the token's slot in head 0 of the cache, or -1
  int64_t pos;
  int32_t live;  // belongs to a sequence
};

__device__ inline float lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ inline float hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// 8 values to a cache slot: bf16, or E4M3 codes of x * scale.
__device__ inline void store_cache(const KvCache& c, void* base, int64_t off, const float* x,
                                   float scale) {
  if (c.e4m3) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i / 4] |= e4m3(x[i] * scale) << (8 * (i % 4));
    uint2 o = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + off) = o;
  } else {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(base) + off) = o;
  }
}

__device__ inline void store_bf16(uint16_t* p, const float* x) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<u32x4*>(p) = o;
}

__device__ inline void unpack(u32x4 v, float* x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo(v[i]);
    x[2 * i + 1] = hi(v[i]);
  }
}

__global__ __launch_bounds__(THREADS) void kv_append(AppendParams p) {
  __shared__ Token tok[MAX_TOKENS];
  __shared__ float2 rot[MAX_TOKENS][MAX_HALF];
  const AppendArgs& a = p.a;
  const int t0 = blockIdx.x * p.tokens;
  const int nt = min(p.tokens, a.seqs.T - t0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int j = wave; j < nt; j += THREADS / 64) {
    const int t = t0 + j;
    // sequences that end at or before row t come first: their number is t's sequence
    int seq = 0;
    for (int c = 0; c < a.seqs.n; c += 64) {
      const int i = c + lane;
      const int m = __popcll(__ballot(i < a.seqs.n && a.seqs.cu[min(i + 1, a.seqs.n)] <= t));
      seq += m;
      if (m < 64) break;
    }
    if (lane == 0) {
      Token k{-1, 0, 0};
      if (seq < a.seqs.n) {
        const int start = a.seqs.cu[seq];
        if (start >= 0 && start <= t) {
          const int64_t pos = (int64_t)(a.past ? a.past[seq] : 0) + (t - start);
          k.live = 1;
          k.pos = pos;
          const int e = a.cache.k ? page_entry(pos, a.cache.page_size, a.pages_per_seq) : -1;
          if (e >= 0)
            k.slot = token_offset(pos, a.pages[(int64_t)seq * a.pages_ld + e], a.cache.n_pages,
                                  a.cache.page_size, a.cache.ps, a.cache.ts);
        }
      }
      tok[j] = k;
    }
  }
  __syncthreads();
  const int half = a.rotary / 2;
  for (int i = threadIdx.x; i < nt * half; i += THREADS) {
    const int j = i / half, m = i - j * half;
    // revolutions, reduced in 64 bits; the product pos * inv_freq is exact there
    double r = (double)tok[j].pos * (double)a.inv_freq[m] * 0.15915494309189533577;
    r -= rint(r);
    float s, c;
    sincospif(2.0f * (float)r, &s, &c);
    rot[j][m] = make_float2(c, s);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nt * p.n_items; i += THREADS) {
    const int j = i / p.n_items;
    int it = i - j * p.n_items;
    const int64_t t = t0 + j;
    const Token k = tok[j];
    float x[8], y[8];
    if (it < p.n_rot) {
      const int head = it / p.rot_per_head, m = (it - head * p.rot_per_head) * 8;
      const bool is_q = head < p.qh;
      const int hh = is_q ? head : head - p.qh;
      const Heads& src = is_q ? a.q : a.k;
      const Heads& dst = is_q ? a.q_out : a.k_out;
      const int e0 = a.interleaved ? 2 * m : m, e1 = a.interleaved ? 2 * m + 8 : m + half;
      const uint16_t* in = src.p + t * src.rs + hh * src.hs;
      if (k.live) {
        unpack(*reinterpret_cast<const u32x4*>(in + e0), x);
        unpack(*reinterpret_cast<const u32x4*>(in + e1), y);
        if (a.interleaved) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 c0 = rot[j][m + u], c1 = rot[j][m + 4 + u];
            const float p0 = x[2 * u], p1 = x[2 * u + 1], r0 = y[2 * u], r1 = y[2 * u + 1];
            x[2 * u] = p0 * c0.x - p1 * c0.y;
            x[2 * u + 1] = p1 * c0.x + p0 * c0.y;
            y[2 * u] = r0 * c1.x - r1 * c1.y;
            y[2 * u + 1] = r1 * c1.x + r0 * c1.y;
          }
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const float2 c = rot[j][m + u];
            const float p0 = x[u], p1 = y[u];
            x[u] = p0 * c.x - p1 * c.y;
            y[u] = p1 * c.x + p0 * c.y;
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) x[u] = y[u] = 0.0f;
      }
      if (dst.p) {
        uint16_t* o = dst.p + t * dst.rs + hh * dst.hs;
        store_bf16(o + e0, x);
        store_bf16(o + e1, y);
      }
      if (!is_q && k.slot >= 0) {
        const int64_t off = k.slot + hh * a.cache.hs;
        store_cache(a.cache, a.cache.k, off + e0, x, a.cache.k_scale);
        store_cache(a.cache, a.cache.k, off + e1, y, a.cache.k_scale);
      }
      continue;
    }
    it -= p.n_rot;
    const bool is_v = it >= p.n_copy;
    if (is_v) it -= p.n_copy;
    const int per = is_v ? p.v_per_head : p.copy_per_head;
    const int head = it / per, e = (is_v ? 0 : a.rotary) + (it - head * per) * 8;
    const bool is_q = !is_v && head < p.qh;
    const int hh = is_v || is_q ? head : head - p.qh;
    const Heads& src = is_v ? a.v : is_q ? a.q : a.k;
    const Heads& dst = is_q ? a.q_out : a.k_out;
    if (k.live) {
      unpack(*reinterpret_cast<const u32x4*>(src.p + t * src.rs + hh * src.hs + e), x);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = 0.0f;
    }
    if (!is_v && dst.p) store_bf16(dst.p + t * dst.rs + hh * dst.hs + e, x);
    if (!is_q && k.slot >= 0)
      store_cache(a.cache, is_v ? a.cache.v : a.cache.k, k.slot + hh * a.cache.hs + e, x,
                  is_v ? a.cache.v_scale : a.cache.k_scale);
  }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs& a, hipStream_t s) {
  AppendParams p{};
  p.a = a;
  p.qh = a.q.p ? a.H : 0;
  const int kh = a.k.p ? a.G : 0;
  p.rot_per_head = a.rotary / 16;
  p.copy_per_head = (a.D - a.rotary) / 8;
  p.v_per_head = a.D / 8;
  p.n_rot = (p.qh + kh) * p.rot_per_head;
  p.n_copy = (p.qh + kh) * p.copy_per_head;
  p.n_items = p.n_rot + p.n_copy + (a.cache.k ? a.G * p.v_per_head : 0);
  if (a.seqs.T <= 0 || p.n_items == 0) return hipSuccess;
  // Few tokens: one per workgroup, for latency.  Many: 8, so that the angles' cost is shared
  // by more threads and fewer workgroups start.
  p.tokens = a.seqs.T <= 1024 ? 1 : MAX_TOKENS;
  const int blocks = (a.seqs.T + p.tokens - 1) / p.tokens;
  return launch_k(&kv_append, dim3(blocks), dim3(THREADS), 0, s, p);
}

}  // namespace ubx
