// kv_pages.h on the CPU: whatever lengths, positions and page ids say, a table entry read is
// inside the table's row and a token's offset inside the cache.
#include <climits>
#include <cstdio>
#include <random>

#include "kv_pages.h"

int main() {
  std::mt19937_64 rng(5);
  long checks = 0;
  const int odd[] = {INT_MIN, INT_MIN + 1, -1000000, -1, 0, 1, 2, 1 << 20, 0x3FFFFFFE, INT_MAX - 1, INT_MAX};
  for (int r = 0; r < 20000; ++r) {
    const int page = 1 + (int)(rng() % (r % 2 ? 200 : 4)), per_seq = 1 + (int)(rng() % (r % 3 ? 50 : 1 << 22));
    const int n_pages = 1 + (int)(rng() % (r % 5 ? 64 : INT_MAX - 1));
    const int64_t ts = 8 * (int64_t)(1 + rng() % 4096), ps = ts * page + 8 * (int64_t)(rng() % 64);
    const int cap = ubx::table_cap(per_seq, page);
    for (int len : odd) {
      const int c = ubx::clamp_len(len, cap);
      if (c < 0 || (int64_t)c > (int64_t)per_seq * page || (len >= 0 && len <= cap && c != len)) return 1;
      if (c > 0 && ubx::page_entry(c - 1, page, per_seq) < 0) return 2;
      ++checks;
    }
    for (int i = 0; i < 32; ++i) {
      const int64_t pos = i < 11 ? (int64_t)odd[i] + odd[rng() % 11] : (int64_t)(rng() % ((uint64_t)per_seq * page + 3));
      const int e = ubx::page_entry(pos, page, per_seq);
      if (e < -1 || e >= per_seq) return 3;
      if ((e >= 0) != (pos >= 0 && pos < (int64_t)per_seq * page)) return 4;
      const int id = i % 3 ? (int)(rng() % n_pages) : odd[rng() % 11];
      const int64_t off = ubx::token_offset(pos, id, n_pages, page, ps, ts);
      const bool good = pos >= 0 && id >= 0 && id < n_pages;
      if (good != (off >= 0)) return 5;
      if (good && (off / ps != id || off % ps != pos % page * ts)) return 6;
      ++checks;
    }
  }
  std::printf("ok %ld\n", checks);
  return 0;
}
