// What rows see under a sliding window, as tiles and as workgroups: plain arithmetic, which
// tests/cpp/attn_window_check.cpp runs on the CPU.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ub.h"

namespace ubx {

// A row at position t of its sequence sees u <= t with t - u < size, or u < sinks; size 0: all
// u <= t.
struct Window {
  int32_t size, sinks;
};
constexpr int32_t kMaxWindow = 1 << 30;  // no row's distance reaches it

__host__ __device__ inline bool seen(int key, int row, Window win) {
  return key <= row && (key > row - win.size || key < win.sinks);
}

__host__ __device__ inline int smaller(int a, int b) { return a < b ? a : b; }
__host__ __device__ inline int larger(int a, int b) { return a > b ? a : b; }

// The key tiles of BN keys that rows q0 .. q0 + BM - 1 see, as one list: `sink` tiles of the
// first tokens, then those from `first` on.  Of `tiles` in all, the first `head` hold keys
// that the window hides from one of the rows.
struct KeyTiles {
  int sink, first, head, tiles;
  __host__ __device__ int at(int j) const { return j < sink ? j : j - sink + first; }
};
__host__ __device__ inline KeyTiles key_tiles(int q0, int BM, int BN, int n_keys, Window win) {
  KeyTiles k;
  k.first = larger(q0 - win.size + 1, 0) / BN;
  k.sink = smaller((win.sinks + BN - 1) / BN, k.first);
  k.tiles = k.sink + (n_keys + BN - 1) / BN - k.first;
  k.head = smaller(k.sink + (larger(q0 + BM - win.size, 0) + BN - 1) / BN - k.first, k.tiles);
  return k;
}

// The query tiles of BQ rows with rows that see one of keys k0 .. k0 + BK - 1: `n` from tile qt0 on,
// up to row `last`.  The first `diag` of them may hold rows before one of the keys, those from
// `tail` on rows that do not see one any more.  They are numbered with the `edge` tiles of both
// kinds first.
struct QueryTiles {
  int qt0, n, diag, tail, edge;
  __host__ __device__ int at(int q) const { return q < diag ? q : q < edge ? q - diag + tail : q - edge + diag; }
};
__host__ __device__ inline QueryTiles query_tiles(int k0, int BK, int BQ, int last, Window win) {
  QueryTiles q;
  q.qt0 = k0 / BQ;
  q.n = (last + BQ - 1) / BQ - q.qt0;
  q.diag = smaller(BK / BQ, q.n);
  q.tail = win.size == 0 ? q.n : smaller(larger((int)(((int64_t)k0 + win.size) / BQ) - q.qt0, q.diag), q.n);
  q.edge = q.diag + q.n - q.tail;
  return q;
}
// The last row, and one more, that sees one of keys k0 .. k0 + BK - 1 through the window.
__host__ __device__ inline int window_end(int k0, int BK, int len, Window win) {
  const int64_t e = (int64_t)k0 + BK - 1 + win.size;
  return e < len ? (int)e : len;
}

// The first tokens that stay visible are seen by all later rows: the workgroup of a sequence's
// first keys would walk all of it where every other walks a window's rows.  It takes the rows up
// to `rows`, as far as its other keys are seen, and further workgroups take `chunk` rows each.
// Their sums for the first tokens go to slots of the workspace, one for the first workgroup and
// one for each of the others, the sequences' one after another, and are added in order.  Where
// what is left is no longer than MIN_CHUNK the first workgroup takes it all.
constexpr int MIN_CHUNK = 512;
struct SinkSlots {
  int rows;   // of a sequence's first workgroup, all or a multiple of 32
  int count;  // slots of the sequence: 0 or 1 + chunks
};
__host__ __device__ inline SinkSlots sink_slots(int len, int BK, Window win, int chunk) {
  SinkSlots s;
  s.rows = smaller((BK - 1 + win.size + 31) / 32 * 32, len);
  s.count = 0;
  if (len - s.rows <= MIN_CHUNK) s.rows = len;
  else s.count = 1 + (len - s.rows + chunk - 1) / chunk;
  return s;
}
// Rows of a chunk: as many as another workgroup of one window takes.
inline int sink_chunk(Window win) {
  const int rows = (win.size + 31) / 32 * 32;
  return rows < MIN_CHUNK ? MIN_CHUNK : rows < (1 << 20) ? rows : 1 << 20;
}
// Slots that sequences of T rows together can take: each of them has more than MIN_CHUNK rows left.
inline int64_t max_slots(int64_t T, int64_t chunk) { return T / chunk + 2 * (T / MIN_CHUNK); }

}  // namespace ubx
