// Test-only queries (host code): how much work one launch is given.
#include <stdint.h>

#include "../../mxfp8_mxfp4_experts_amd/csrc/grid.h"

extern "C" {

int64_t probe_most_blocks(int threads) { return mi355moe::most_blocks(threads); }

int64_t probe_most_items(int threads, int64_t per_block, int64_t units) {
  return mi355moe::most_items(threads, per_block, units);
}

}  // extern "C"
