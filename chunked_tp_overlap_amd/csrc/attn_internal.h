// Internal contracts of the attention calls: what attn_api.cpp (argument checks) passes to
// the launchers in kv_append.hip, attn_prompt.hip, attn_prompt_bwd.hip and attn_decode.hip,
// and what it uses of a handle.
#pragma once

#include <string>

#include "ub_internal.h"

namespace ubx {

// ---- the handle, from ub_api.cpp ----------------------------------------------------------
// Records a message for ub_last_error and returns `st`.
ub_status_t ctx_fail(ub_handle_t h, ub_status_t st, const std::string& message);
// Binds the handle to the current device (as every work-issuing call does).
ub_status_t ctx_bind(ub_handle_t h);
int64_t ctx_rows(ub_handle_t h);  // the active T

// ---- launches -----------------------------------------------------------------------------
// A [rows, heads, dim] matrix: strides in elements, head stride resolved.
struct Heads {
  uint16_t* p;
  int64_t rs, hs;
};

struct KvCache {
  void* k;
  void* v;
  int64_t ps, hs, ts;  // page, head and token strides, elements
  int32_t n_pages;
  int32_t page_size;
  int32_t e4m3;
  float k_scale, v_scale;
};

struct Seqs {
  const int32_t* cu;
  int32_t n;
  int32_t T;
};

struct AppendArgs {
  Heads q, k, v, q_out, k_out;  // p == nullptr: absent
  const float* inv_freq;
  Seqs seqs;
  const int32_t* past;
  KvCache cache;  // k == nullptr: no append
  const int32_t* pages;
  int64_t pages_ld;
  int32_t pages_per_seq;
  int32_t H, G, D, rotary;
  int32_t interleaved;
};
hipError_t launch_kv_append(const AppendArgs& a, hipStream_t s);

struct PromptArgs {
  Heads q, k, v, out;
  float* lse;
  Seqs seqs;
  int32_t H, G, D;
  float scale;
};
hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t s);

struct PromptBwdArgs {
  Heads dout, q, k, v, out, dq, dk, dv;
  const float* lse;
  Seqs seqs;
  int32_t H, G, D;
  float scale;
  void* ws;
};
// Workspace of a call with `rows` rows, and the most any call with up to `rows` rows needs.
size_t attn_prompt_bwd_need(int32_t H, int32_t G, int32_t D, int64_t rows);
size_t attn_prompt_bwd_bytes(int32_t H, int32_t G, int32_t D, int64_t rows);
hipError_t launch_attn_prompt_bwd(const PromptBwdArgs& a, hipStream_t s);

struct DecodeArgs {
  Heads q, out;
  float* lse;
  KvCache cache;
  const int32_t* pages;
  int64_t pages_ld;
  int32_t pages_per_seq;
  const int32_t* lens;
  int32_t n, T;
  int32_t H, G, D;
  float scale;
  void* ws;
};
size_t attn_decode_bytes(int32_t H, int32_t G, int32_t D, int32_t n);
hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s);

}  // namespace ubx
