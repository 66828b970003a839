// attn_window.h on the CPU: the tiles that a windowed call walks hold every pair that is seen, those
// it does not mask nothing else, and the slots of first tokens stay inside their workspace.
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>

#include "attn_window.h"
#include "kv_pages.h"

using namespace ubx;

int main() {
  std::mt19937_64 rng(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (uint64_t)(hi - lo + 1)); };
  long checks = 0;
  const int sizes[] = {1, 2, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 500, 1000, kMaxWindow};
  for (int r = 0; r < 6000; ++r) {
    const Window win{r % 3 ? sizes[rng() % 15] : pick(1, 1500), r % 2 ? 0 : pick(0, UB_ATTN_MAX_SINKS)};
    const int len = r % 5 ? pick(1, 900) : pick(1, 6000);
    const int BM = r % 2 ? 64 : 128, BN = r % 4 < 2 ? 32 : 64, BQ = 32;
    // rows' keys
    const int q0 = pick(0, (len - 1) / BM) * BM, n_keys = std::min(q0 + BM, len);
    const KeyTiles k = key_tiles(q0, BM, BN, n_keys, win);
    std::vector<char> listed((n_keys + BN - 1) / BN, 0);
    if (k.tiles < 1 || k.head < 0 || k.head > k.tiles || k.sink < 0) return 1;
    const int full = q0 / BN - k.first + k.sink;
    for (int j = 0; j < k.tiles; ++j) {
      const int t = k.at(j);
      if (t < 0 || t >= (int)listed.size() || listed[t]) return 2;
      listed[t] = 1;
      if (j >= k.head && j < full)
        for (int row : {q0, n_keys - 1})
          for (int key : {t * BN, t * BN + BN - 1})
            if (!seen(key, row, win)) return 3;
    }
    for (int i = 0; i < 60; ++i) {
      const int row = pick(q0, n_keys - 1);
      const int key = i % 3 ? pick(0, row) : std::min(row, pick(0, UB_ATTN_MAX_SINKS));
      if (seen(key, row, win) && !listed[key / BN]) return 4;
      ++checks;
    }
    // keys' rows
    const int BK = BM, chunk = sink_chunk(win);
    const int k0 = pick(0, (len - 1) / BK) * BK, k1 = std::min(k0 + BK, len);
    const bool first = k0 == 0 && win.sinks > 0;
    const SinkSlots s = sink_slots(len, BK, win, chunk);
    const QueryTiles q = query_tiles(k0, BK, BQ, first ? s.rows : window_end(k0, BK, len, win), win);
    std::vector<int> by((len + BQ - 1) / BQ, 0);
    if (q.n < 1 || q.edge < 0 || q.edge > q.n) return 5;
    for (int j = 0; j < q.n; ++j) {
      const int t = q.qt0 + q.at(j);
      if (t < 0 || t >= (int)by.size() || by[t]) return 6;
      by[t] = 1;
      if (j >= q.edge)
        for (int row : {t * BQ, std::min(t * BQ + BQ, len) - 1})
          for (int key : {k0, k1 - 1})
            if (!seen(key, row, win) && !(first && s.count == 0 && key < win.sinks)) return 7;
    }
    if (first && s.count > 0) {
      if (s.rows % 32 || s.rows >= len) return 8;
      for (int c = 1; c < s.count; ++c) {
        const int a = s.rows + (c - 1) * chunk, b = std::min(s.rows + c * chunk, len);
        if (a >= b) return 9;
        for (int t = a / BQ; t < (b + BQ - 1) / BQ; ++t) {
          if (by[t]) return 10;
          by[t] = 2;
        }
      }
    }
    for (int i = 0; i < 60; ++i) {
      const int key = i % 3 ? pick(k0, k1 - 1) : std::min(k1 - 1, k0 + pick(0, UB_ATTN_MAX_SINKS));
      const int row = pick(key, len - 1);
      if (!seen(key, row, win)) continue;
      const int t = by[row / BQ];
      if (t == 0 || (t == 2 && key >= win.sinks)) {
        // a first token outside the first keys' tile has no workgroup for its later rows
        return 11;
      }
      ++checks;
    }
  }
  // slots of any sequences of T rows together
  for (int r = 0; r < 20000; ++r) {
    const Window win{sizes[rng() % 15], pick(1, UB_ATTN_MAX_SINKS)};
    const int BK = r % 2 ? 64 : 128, chunk = sink_chunk(win), T = pick(1, 40000);
    int64_t slots = 0, n = 0;
    for (int left = T; left > 0; ++n) {
      const int len = std::min(left, r % 3 ? pick(1, 3000) : pick(500, 800));
      slots += sink_slots(len, BK, win, chunk).count;
      left -= len;
    }
    if (slots > max_slots(T, chunk) || slots > T / chunk + 2 * n) return 12;
    if (max_slots(T, chunk) > max_slots(T, MIN_CHUNK)) return 13;
    ++checks;
  }
  // the page of a token
  for (int r = 0; r < 40000; ++r) {
    const uint32_t size = r < 700 ? 1 + r : r < 731 ? 1u << (r - 700) : 1 + (uint32_t)(rng() % 0x7FFFFFFF);
    const PageDiv d = page_div(size);
    for (int i = 0; i < 12; ++i) {
      const int64_t q = (int64_t)(rng() % ((1u << 30) / size + 1)) * size + (i % 3 - 1);
      const uint32_t t = (uint32_t)std::min<int64_t>(std::max<int64_t>(i < 9 ? q : (int64_t)(rng() % (1u << 30)), 0), (1 << 30) - 1);
      if (d.page(t) != t / size) return 14;
      ++checks;
    }
  }
  std::printf("ok %ld\n", checks);
  return 0;
}
