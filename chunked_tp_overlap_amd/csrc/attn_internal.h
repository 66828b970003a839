// Internal contracts of the attention calls: what attn_api.cpp (argument checks) passes to
// the launchers in kv_append.hip, attn_prompt.hip, attn_prompt_bwd.hip, attn_decode.hip, attn_tree.hip
// and kv_manage.hip, and what it uses of a handle.
#pragma once

#include <string>

#include "attn_window.h"
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
  const int32_t* offsets;  // a row's position for the rotation, from past; nullptr: its place
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
  Window win;
};
hipError_t launch_attn_prompt(const PromptArgs& a, hipStream_t s);

struct PromptBwdArgs {
  Heads dout, q, k, v, out, dq, dk, dv;
  const float* lse;
  Seqs seqs;
  int32_t H, G, D;
  float scale;
  void* ws;
  Window win;
};
// Workspace of a call with `rows` rows, and the most any call with up to `rows` rows needs.
size_t attn_prompt_bwd_need(int32_t H, int32_t G, int32_t D, int64_t rows);
size_t attn_prompt_bwd_bytes(int32_t H, int32_t G, int32_t D, int64_t rows);
// What first tokens that stay visible add to it, whatever the window.
size_t attn_prompt_bwd_sink_bytes(int32_t H, int32_t G, int32_t D, int64_t rows);
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
  Window win;
};
size_t attn_decode_bytes(int32_t H, int32_t G, int32_t D, int32_t n);
hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s);

// The page operations (kv_manage.hip).  A table of n rows of `per` entries, ld apart.
struct Table {
  int32_t* p;
  int64_t ld;
  int32_t per, n;
};
struct ForkArgs {
  int32_t* refs;
  int32_t n_pages, page;
  Table in, out;
  const int32_t* lens;
  const int32_t* parents;
  int32_t* lens_out;
};
hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t s);

struct ResizeArgs {
  int32_t* refs;
  int32_t n_pages, page;
  Table table;
  const int32_t* lens;
  const int32_t* new_lens;
  int32_t* lens_out;
  int32_t* copies;  // [n, 3]
  Window win;       // size 0: none
  void* ws;
};
size_t kv_resize_bytes(int32_t n);
hipError_t launch_kv_resize(const ResizeArgs& a, hipStream_t s);

hipError_t launch_kv_copy_pages(const KvCache& c, int32_t G, int32_t D, const int32_t* copies, int32_t n,
                                hipStream_t s);

struct CompactArgs {
  KvCache cache;
  const int32_t* pages;
  int64_t pages_ld;
  int32_t pages_per_seq;
  const int32_t* lens;
  const int32_t* kept;
  int64_t kept_ld;
  int32_t most;  // entries of a row of `kept`
  const int32_t* kept_lens;
  int32_t* lens_out;
  int32_t n, G, D;
};
hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t s);

struct TreeArgs {
  Heads q, out;
  float* lse;
  KvCache cache;
  const int32_t* pages;
  int64_t pages_ld;
  int32_t pages_per_seq;
  const int32_t* lens;
  const int32_t* parents;
  Seqs seqs;
  int32_t H, G, D;
  float scale;
  void* ws;
};
size_t attn_tree_bytes(int32_t H, int32_t G, int32_t D, int64_t rows, int32_t n);
hipError_t launch_attn_tree(const TreeArgs& a, hipStream_t s);

}  // namespace ubx
