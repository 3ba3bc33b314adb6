// How much work one launch may have (host code).
#pragma once

#include <stdint.h>

namespace mi355moe {

// A launch has fewer than 2^32 threads along a dimension of its grid: the runtime launches more than
// that modulo 2^32, without an error.
constexpr int64_t most_blocks(int threads) { return (int64_t)0xFFFFFFFF / threads; }

// Items that one launch takes at most, where an item has `units` units of work and a workgroup of
// `threads` threads takes `per_block` of them.
constexpr int64_t most_items(int threads, int64_t per_block, int64_t units) {
  return most_blocks(threads) * per_block / units;
}

}  // namespace mi355moe
