// Test-only queries (host code): which kernel the sizes of a block-scaled FP8
// product choose, so that the tests can say that they run every one of them.
#include <stdint.h>

#include "../../mxfp8_mxfp4_experts_amd/csrc/fp8_pick.h"

using namespace mi355moe;

extern "C" {

// out: variant (-1: the direct kernel), splits of K, the variant's tile height and width (0), the
// direct kernel's Q, and its steps of K.
void probe_fp8_pick(int M, int N, int K, int32_t* out) {
  const Fp8Pick k = fp8_pick(M, N, K);
  const int stages = (K + 127) / 128, per = (stages + k.splits - 1) / k.splits;
  const int q = fp8_direct_q(M, N, K), step = 128 * q * kFp8Waves;
  out[0] = k.variant;
  out[1] = (stages + per - 1) / per;
  out[2] = k.variant < 0 ? 0 : kFp8Variants[k.variant].bm;
  out[3] = k.variant < 0 ? 0 : kFp8Variants[k.variant].bn;
  out[4] = q;
  out[5] = (K + step - 1) / step;
}

int probe_fp8_variants(void) { return kFp8NumVariants; }

// Q of the one launch that quantises and multiplies, 0: two launches.
int probe_fp8_raw(int M, int N, int K) { return fp8_raw(M, N, K); }

// The variant of a grouped product.
int probe_fp8_grouped(int R, int E, int N, int K) { return fp8_pick_grouped(R, E, N, K); }

}  // extern "C"
