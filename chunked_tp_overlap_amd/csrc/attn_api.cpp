// C ABI of the attention calls: argument checks, then one launcher each (include/ub.h).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <string>

#include <rocprofiler-sdk-roctx/roctx.h>

#include "attn_internal.h"

namespace {

struct TraceRange {
  explicit TraceRange(const char* name) { roctxRangePushA(name); }
  ~TraceRange() { roctxRangePop(); }
  TraceRange(const TraceRange&) = delete;
  TraceRange& operator=(const TraceRange&) = delete;
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxRowStride = int64_t(1) << 22;
constexpr int64_t kMaxRows = int64_t(1) << 30;

// The first error of a call's checks.  A message names the argument.
struct Checks {
  ub_handle_t h;
  ub_status_t st = UB_OK;
  void bad(ub_status_t s, const std::string& m) {
    if (st == UB_OK) st = ubx::ctx_fail(h, s, m);
  }
  void need(bool ok, const char* m) {
    if (!ok) bad(UB_ERR_INVALID_ARG, m);
  }
};

const char* cfg_error(const ub_attn_cfg_t* c, ub_status_t* st) {
  *st = UB_ERR_INVALID_ARG;
  if (!c) return "cfg is NULL";
  if (c->n_heads < 1 || c->n_kv_heads < 1 || c->n_heads % c->n_kv_heads != 0 || c->n_heads > 65536)
    return "n_kv_heads must divide n_heads (both >= 1, n_heads <= 65536)";
  if (c->head_dim < 8 || c->head_dim % 8 != 0) return "head_dim must be a positive multiple of 8";
  if (c->rotary_dim < 0 || c->rotary_dim > c->head_dim || c->rotary_dim % 16 != 0)
    return "rotary_dim must be a multiple of 16 in [0, head_dim]";
  if (c->rope_interleaved != 0 && c->rope_interleaved != 1) return "rope_interleaved must be 0 or 1";
  if (!std::isfinite(c->softmax_scale) || !(c->softmax_scale > 0.0f))
    return "softmax_scale must be finite and > 0";
  if (c->head_dim > UB_ATTN_MAX_HEAD_DIM) {
    *st = UB_ERR_UNSUPPORTED;
    return "head_dim above UB_ATTN_MAX_HEAD_DIM";
  }
  return nullptr;
}

void check_cfg(Checks& c, const ub_attn_cfg_t* cfg) {
  ub_status_t st = UB_OK;
  const char* m = cfg_error(cfg, &st);
  if (m) c.bad(st, m);
}

// x as the launchers take it; an absent optional matrix has p == nullptr.
ubx::Heads heads(Checks& c, const char* name, const ub_heads_t* x, int32_t n, int64_t T,
                 const ub_attn_cfg_t* cfg, bool optional = false) {
  if (c.st != UB_OK || (!x && optional)) return ubx::Heads{};
  const std::string s(name);
  if (!x || !x->ptr) {
    c.bad(UB_ERR_INVALID_ARG, s + " is NULL");
    return ubx::Heads{};
  }
  const int64_t hs = x->head_stride ? x->head_stride : cfg->head_dim;
  if (!aligned16(x->ptr)) c.bad(UB_ERR_INVALID_ARG, s + " must be 16-byte aligned");
  if (x->row_stride % 8 != 0 || x->row_stride < cfg->head_dim || x->row_stride >= kMaxRowStride)
    c.bad(UB_ERR_INVALID_ARG, s + ": row_stride must be a multiple of 8, >= head_dim and < 2^22");
  if (hs % 8 != 0 || hs < 0 || hs > (int64_t(1) << 40) || (n > 1 && hs < cfg->head_dim))
    c.bad(UB_ERR_INVALID_ARG, s + ": head_stride must be a multiple of 8 and >= head_dim");
  if (c.st == UB_OK && x->rows < T)
    c.bad(UB_ERR_BUFFER_TOO_SMALL, s + " holds " + std::to_string(x->rows) + " rows, the active shape has " +
                                       std::to_string(T));
  return ubx::Heads{static_cast<uint16_t*>(x->ptr), x->row_stride, hs};
}

ubx::Seqs seqs(Checks& c, const int32_t* cu, int32_t n, int64_t T) {
  c.need(n >= 0, "n_seqs must be >= 0");
  c.need(cu != nullptr, "cu_seqlens is NULL");
  if (c.st == UB_OK && T > kMaxRows) c.bad(UB_ERR_UNSUPPORTED, "more than 2^30 active rows");
  return ubx::Seqs{cu, n, static_cast<int32_t>(T)};
}

ubx::KvCache cache(Checks& c, const ub_kv_cache_t* x, const int32_t* table, int64_t ld,
                   int32_t per_seq, int32_t n, const ub_attn_cfg_t* cfg) {
  if (c.st != UB_OK) return ubx::KvCache{};
  if (!x || !x->k || !x->v) {
    c.bad(UB_ERR_INVALID_ARG, "cache (k and v) is NULL");
    return ubx::KvCache{};
  }
  if (x->dtype != UB_DTYPE_BF16 && x->dtype != UB_DTYPE_FP8_E4M3)
    c.bad(UB_ERR_DTYPE, "key-value caches are bf16 or fp8 E4M3");
  const bool f8 = x->dtype == UB_DTYPE_FP8_E4M3;
  const int64_t unit = f8 ? 16 : 8;
  c.need(aligned16(x->k) && aligned16(x->v), "cache k and v must be 16-byte aligned");
  c.need(x->page_stride % unit == 0 && x->head_stride % unit == 0 && x->token_stride % unit == 0,
         "cache strides must be multiples of 16 bytes");
  c.need(x->page_stride >= 0 && x->head_stride >= 0 && x->token_stride >= 0, "cache strides must be >= 0");
  c.need(!f8 || cfg->head_dim % 16 == 0, "an E4M3 cache needs head_dim to be a multiple of 16");
  c.need(x->n_pages >= 1 && x->n_pages <= INT32_MAX, "cache n_pages must be in [1, 2^31)");
  c.need(x->page_size >= 1, "cache page_size must be >= 1");
  if (f8)
    c.need(std::isfinite(x->k_scale) && x->k_scale > 0.0f && std::isfinite(x->v_scale) && x->v_scale > 0.0f,
           "k_scale and v_scale must be finite and > 0");
  c.need(n == 0 || table != nullptr, "page_table is NULL");
  c.need(per_seq >= 1 && ld >= per_seq, "pages_per_seq must be >= 1 and pages_ld >= pages_per_seq");
  return ubx::KvCache{x->k, x->v, x->page_stride, x->head_stride, x->token_stride,
                      static_cast<int32_t>(x->n_pages), x->page_size, f8,
                      f8 ? x->k_scale : 1.0f, f8 ? x->v_scale : 1.0f};
}

void workspace(Checks& c, const void* ws, size_t have, size_t need) {
  if (need == 0 || c.st != UB_OK) return;
  c.need(ws != nullptr && aligned16(ws), "workspace must be non-NULL and 16-byte aligned");
  if (c.st == UB_OK && have < need)
    c.bad(UB_ERR_BUFFER_TOO_SMALL,
          "workspace of " + std::to_string(have) + " bytes, " + std::to_string(need) + " needed");
}

ub_status_t launched(ub_handle_t h, hipError_t e, const char* what) {
  if (e == hipSuccess) return UB_OK;
  if (e == hipErrorInvalidValue)
    return ubx::ctx_fail(h, UB_ERR_UNSUPPORTED, std::string(what) + ": more workgroups than a launch holds");
  return ubx::ctx_fail(h, UB_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

// No C++ exception crosses the ABI (messages allocate).
template <class F>
ub_status_t guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return UB_ERR_HIP;
  }
}

}  // namespace

extern "C" {

UB_API ub_status_t ub_attn_required_bytes(ub_attn_op_t op, const ub_attn_cfg_t* cfg, int64_t rows,
                                          int32_t n_seqs, size_t* bytes) {
  ub_status_t st = UB_OK;
  if (cfg_error(cfg, &st)) return st;
  if (!bytes || rows < 0 || rows > kMaxRows || n_seqs < 0) return UB_ERR_INVALID_ARG;
  switch (op) {
    case UB_ATTN_PROMPT:
      *bytes = 0;
      return UB_OK;
    case UB_ATTN_PROMPT_BWD:
      *bytes = ubx::attn_prompt_bwd_bytes(cfg->n_heads, cfg->n_kv_heads, cfg->head_dim, rows);
      return UB_OK;
    case UB_ATTN_DECODE:
      *bytes = ubx::attn_decode_bytes(cfg->n_heads, cfg->n_kv_heads, cfg->head_dim, n_seqs);
      return UB_OK;
    default:
      return UB_ERR_INVALID_ARG;
  }
}

UB_API ub_status_t ub_kv_append(ub_handle_t h, const ub_heads_t* q, const ub_heads_t* k,
                                const ub_heads_t* v, const ub_heads_t* q_out,
                                const ub_heads_t* k_out, const float* inv_freq,
                                const int32_t* cu_seqlens, const int32_t* past_lens,
                                int32_t n_seqs, const ub_kv_cache_t* kv,
                                const int32_t* page_table, int64_t pages_ld,
                                int32_t pages_per_seq, const ub_attn_cfg_t* cfg,
                                ub_stream_t stream) {
  const TraceRange range("ub_kv_append");
  if (!h) return UB_ERR_NOT_INITIALIZED;
  return guarded([&] {
    Checks c{h};
    check_cfg(c, cfg);
    if (c.st != UB_OK) return c.st;
    const int64_t T = ubx::ctx_rows(h);
    ubx::AppendArgs a{};
    a.H = cfg->n_heads;
    a.G = cfg->n_kv_heads;
    a.D = cfg->head_dim;
    a.rotary = cfg->rotary_dim;
    a.interleaved = cfg->rope_interleaved;
    c.need((q == nullptr) == (q_out == nullptr), "q and q_out must both be given, or neither");
    c.need(k != nullptr || (!kv && !k_out), "k is NULL");
    c.need(v != nullptr || !kv, "v is NULL");
    a.q = heads(c, "q", q, a.H, T, cfg, true);
    a.q_out = heads(c, "q_out", q_out, a.H, T, cfg, true);
    if (kv || k_out) a.k = heads(c, "k", k, a.G, T, cfg);
    a.k_out = heads(c, "k_out", k_out, a.G, T, cfg, true);
    if (kv) a.v = heads(c, "v", v, a.G, T, cfg);
    a.seqs = seqs(c, cu_seqlens, n_seqs, T);
    c.need(a.rotary == 0 || inv_freq != nullptr, "inv_freq is NULL");
    a.inv_freq = inv_freq;
    a.past = past_lens;
    if (kv) a.cache = cache(c, kv, page_table, pages_ld, pages_per_seq, n_seqs, cfg);
    a.pages = page_table;
    a.pages_ld = pages_ld;
    a.pages_per_seq = pages_per_seq;
    if (c.st != UB_OK) return c.st;
    ub_status_t st = ubx::ctx_bind(h);
    if (st != UB_OK) return st;
    return launched(h, ubx::launch_kv_append(a, static_cast<hipStream_t>(stream)), "ub_kv_append");
  });
}

UB_API ub_status_t ub_attn_prompt(ub_handle_t h, const ub_heads_t* q, const ub_heads_t* k,
                                  const ub_heads_t* v, const ub_heads_t* out, float* lse,
                                  const int32_t* cu_seqlens, int32_t n_seqs,
                                  const ub_attn_cfg_t* cfg, void* ws, size_t ws_bytes,
                                  ub_stream_t stream) {
  const TraceRange range("ub_attn_prompt");
  if (!h) return UB_ERR_NOT_INITIALIZED;
  (void)ws;
  (void)ws_bytes;
  return guarded([&] {
    Checks c{h};
    check_cfg(c, cfg);
    if (c.st != UB_OK) return c.st;
    const int64_t T = ubx::ctx_rows(h);
    ubx::PromptArgs a{};
    a.H = cfg->n_heads;
    a.G = cfg->n_kv_heads;
    a.D = cfg->head_dim;
    a.scale = cfg->softmax_scale;
    a.q = heads(c, "q", q, a.H, T, cfg);
    a.k = heads(c, "k", k, a.G, T, cfg);
    a.v = heads(c, "v", v, a.G, T, cfg);
    a.out = heads(c, "out", out, a.H, T, cfg);
    a.lse = lse;
    a.seqs = seqs(c, cu_seqlens, n_seqs, T);
    if (c.st != UB_OK) return c.st;
    ub_status_t st = ubx::ctx_bind(h);
    if (st != UB_OK) return st;
    return launched(h, ubx::launch_attn_prompt(a, static_cast<hipStream_t>(stream)), "ub_attn_prompt");
  });
}

UB_API ub_status_t ub_attn_prompt_bwd(ub_handle_t h, const ub_heads_t* dout, const ub_heads_t* q,
                                      const ub_heads_t* k, const ub_heads_t* v,
                                      const ub_heads_t* out, const float* lse,
                                      const ub_heads_t* dq, const ub_heads_t* dk,
                                      const ub_heads_t* dv, const int32_t* cu_seqlens,
                                      int32_t n_seqs, const ub_attn_cfg_t* cfg, void* ws,
                                      size_t ws_bytes, ub_stream_t stream) {
  const TraceRange range("ub_attn_prompt_bwd");
  if (!h) return UB_ERR_NOT_INITIALIZED;
  return guarded([&] {
    Checks c{h};
    check_cfg(c, cfg);
    if (c.st != UB_OK) return c.st;
    const int64_t T = ubx::ctx_rows(h);
    ubx::PromptBwdArgs a{};
    a.H = cfg->n_heads;
    a.G = cfg->n_kv_heads;
    a.D = cfg->head_dim;
    a.scale = cfg->softmax_scale;
    a.dout = heads(c, "dout", dout, a.H, T, cfg);
    a.q = heads(c, "q", q, a.H, T, cfg);
    a.k = heads(c, "k", k, a.G, T, cfg);
    a.v = heads(c, "v", v, a.G, T, cfg);
    a.out = heads(c, "out", out, a.H, T, cfg);
    a.dq = heads(c, "dq", dq, a.H, T, cfg);
    a.dk = heads(c, "dk", dk, a.G, T, cfg);
    a.dv = heads(c, "dv", dv, a.G, T, cfg);
    c.need(lse != nullptr, "lse is NULL");
    a.lse = lse;
    a.seqs = seqs(c, cu_seqlens, n_seqs, T);
    if (c.st == UB_OK) workspace(c, ws, ws_bytes, ubx::attn_prompt_bwd_need(a.H, a.G, a.D, T));
    a.ws = ws;
    if (c.st != UB_OK) return c.st;
    ub_status_t st = ubx::ctx_bind(h);
    if (st != UB_OK) return st;
    return launched(h, ubx::launch_attn_prompt_bwd(a, static_cast<hipStream_t>(stream)),
                    "ub_attn_prompt_bwd");
  });
}

UB_API ub_status_t ub_attn_decode(ub_handle_t h, const ub_heads_t* q, const ub_kv_cache_t* kv,
                                  const int32_t* page_table, int64_t pages_ld,
                                  int32_t pages_per_seq, const int32_t* kv_lens, int32_t n_seqs,
                                  const ub_heads_t* out, float* lse, const ub_attn_cfg_t* cfg,
                                  void* ws, size_t ws_bytes, ub_stream_t stream) {
  const TraceRange range("ub_attn_decode");
  if (!h) return UB_ERR_NOT_INITIALIZED;
  return guarded([&] {
    Checks c{h};
    check_cfg(c, cfg);
    if (c.st != UB_OK) return c.st;
    const int64_t T = ubx::ctx_rows(h);
    ubx::DecodeArgs a{};
    a.H = cfg->n_heads;
    a.G = cfg->n_kv_heads;
    a.D = cfg->head_dim;
    a.scale = cfg->softmax_scale;
    a.q = heads(c, "q", q, a.H, T, cfg);
    a.out = heads(c, "out", out, a.H, T, cfg);
    a.lse = lse;
    c.need(n_seqs >= 0 && n_seqs <= T, "n_seqs must be in [0, T]: one row of q per sequence");
    c.need(n_seqs == 0 || kv_lens != nullptr, "kv_lens is NULL");
    if (c.st == UB_OK && T > kMaxRows) c.bad(UB_ERR_UNSUPPORTED, "more than 2^30 active rows");
    a.cache = cache(c, kv, page_table, pages_ld, pages_per_seq, n_seqs, cfg);
    a.pages = page_table;
    a.pages_ld = pages_ld;
    a.pages_per_seq = pages_per_seq;
    a.lens = kv_lens;
    a.n = n_seqs;
    a.T = static_cast<int32_t>(T);
    if (c.st == UB_OK) workspace(c, ws, ws_bytes, ubx::attn_decode_bytes(a.H, a.G, a.D, n_seqs));
    a.ws = ws;
    if (c.st != UB_OK) return c.st;
    ub_status_t st = ubx::ctx_bind(h);
    if (st != UB_OK) return st;
    return launched(h, ubx::launch_attn_decode(a, static_cast<hipStream_t>(stream)), "ub_attn_decode");
  });
}

}  // extern "C"
