// attn_path.h on the CPU: the bits of a group's keys are those of the tokens before the tree and of the
// nodes on the row's path, key by key, and nothing beyond the group's keys.
#include <cstdio>
#include <random>
#include <vector>

#include "attn_path.h"

using namespace ubx;

int main() {
  std::mt19937_64 rng(11);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (uint64_t)(hi - lo + 1)); };
  long checks = 0;
  for (int r = 0; r < 3000; ++r) {
    const int m = r % 3 ? pick(1, 60) : pick(1, MAX_NODES);
    std::vector<int> up(m);
    for (int i = 0; i < m; ++i) up[i] = r % 4 == 0 ? -1 : r % 4 == 1 ? i - 1 : pick(-1, i - 1);
    for (int c = 0; c < 40; ++c) {
      const int node = pick(0, m - 1), n = 16 << (c % 3);
      uint64_t path[WORDS] = {};
      std::vector<char> on(m, 0);
      for (int i = node; i >= 0; i = up[i]) {
        on[i] = 1;
        path[i / 64] |= 1ull << (i % 64);
      }
      const int at = c % 2 ? pick(-130, m + 130) : pick(-64, 64);
      const uint64_t got = seen_bits(path, at, n);
      for (int i = 0; i < 64; ++i) {
        const int key = at + i;
        const bool sees = i < n && (key < 0 || (key < m && on[key]));
        if (((got >> i) & 1) != sees) return 1;
        ++checks;
      }
    }
  }
  std::printf("ok %ld\n", checks);
  return 0;
}
