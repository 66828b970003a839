// The nodes that a drafted token sees, as bits: plain arithmetic, which
// tests/cpp/attn_path_check.cpp runs on the CPU.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ub.h"

namespace ubx {

constexpr int MAX_NODES = UB_ATTN_MAX_TREE;
constexpr int WORDS = MAX_NODES / 64;

// Bits of the n <= 64 keys from key `at` after the first drafted one (before it, if negative) that
// a node with these path bits sees; none past them.
__host__ __device__ inline uint64_t seen_bits(const uint64_t* path, int at, int n) {
  const uint64_t keys = n < 64 ? (1ull << n) - 1 : ~0ull;
  if (at <= -64) return keys;
  if (at < 0) return ((path[0] << -at) | ((1ull << -at) - 1)) & keys;
  const int w = at >> 6, s = at & 63;
  if (w >= WORDS) return 0;
  uint64_t x = path[w] >> s;
  if (s && w + 1 < WORDS) x |= path[w + 1] << (64 - s);
  return x & keys;
}

}  // namespace ubx
