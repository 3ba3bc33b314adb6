// Test-only queries (host code): which kernel the sizes of a dense product
// choose, so that the tests can say that they run every one of them.
#include <stdint.h>

#include "../../mxfp8_mxfp4_experts_amd/csrc/dense_pick.h"

using namespace mi355moe;

extern "C" {

// Kb: bytes of K.  out: variant (-1: the direct kernel), splits of K, the
// variant's tile height and width (0), the direct kernel's Q, and its steps of K.
void probe_dense_pick(int M, int N, int64_t Kb, int32_t* out) {
  const Pick k = pick(M, N, Kb);
  const int stages = (int)((Kb + kStageK - 1) / kStageK), per = (stages + k.splits - 1) / k.splits;
  const int q = direct_q(M, N, Kb), step = 64 * q * kDirectWaves;
  out[0] = k.variant;
  out[1] = (stages + per - 1) / per;
  out[2] = k.variant < 0 ? 0 : kVariants[k.variant].bm;
  out[3] = k.variant < 0 ? 0 : kVariants[k.variant].bn;
  out[4] = q;
  out[5] = (int32_t)((Kb + step - 1) / step);
}

int probe_num_variants(void) { return kNumVariants; }

// Q of the one launch that quantises and multiplies, 0: two launches.
int probe_fused_q(int M, int N, int K) { return fused_q(M, N, K); }

}  // extern "C"
