// Where a token lives in a paged cache.  Lengths, positions and page ids come from device
// memory that the host never reads, so this is where a bad one is kept inside the caller's
// buffers (tests/cpp/kv_pages_check.cpp runs it on the CPU).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ubx {

// Tokens of a sequence that its row of the page table can hold, of a length that may be
// anything.  cap = min(pages_per_seq * page_size, 2^30 - 1).
__host__ __device__ inline int clamp_len(int len, int cap) {
  return len < 0 ? 0 : (len < cap ? len : cap);
}
__host__ __device__ inline int table_cap(int pages_per_seq, int page_size) {
  const int64_t c = (int64_t)pages_per_seq * page_size;
  return (int)(c < 0x3FFFFFFF ? c : 0x3FFFFFFF);
}

// Entry of a sequence's row of the page table for position pos (P: int or int64_t), or -1
// outside it.
template <class P>
__host__ __device__ inline int page_entry(P pos, int page_size, int pages_per_seq) {
  if (pos < 0) return -1;
  const P e = pos / page_size;
  return e < pages_per_seq ? (int)e : -1;
}

// Element offset, in head 0, of token pos of a sequence whose table entry for it holds `id`;
// -1 if there is no such page.
template <class P>
__host__ __device__ inline int64_t token_offset(P pos, int id, int n_pages, int page_size,
                                                int64_t page_stride, int64_t token_stride) {
  if (pos < 0 || id < 0 || id >= n_pages) return -1;
  return id * page_stride + (pos % page_size) * token_stride;
}

}  // namespace ubx
