// Types shared by the block-scaled FP8 product kernels (fp8.hip says what they compute).
#pragma once

#include "common.h"
#include "fc_common.h"
#include "launch.h"

namespace mi355moe {

constexpr int kScaleBlock = 128;   // elements of K, and output columns, that share a scale

// One 16x16x128 product of E4M3 operands (no block scales), from zero.  The weights are the first
// operand: lane (g, l) holds output columns 4 g .. 4 g + 3 of token l.  An operand is K [16 g,
// 16 g + 16) and [64 + 16 g, 64 + 16 g + 16) of its row.
__device__ __forceinline__ v4f mfma_fp8(v4i b_lo, v4i b_hi, v4i a_lo, v4i a_hi) {
  const v8i b = {b_lo[0], b_lo[1], b_lo[2], b_lo[3], b_hi[0], b_hi[1], b_hi[2], b_hi[3]};
  const v8i a = {a_lo[0], a_lo[1], a_lo[2], a_lo[3], a_hi[0], a_hi[1], a_hi[2], a_hi[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0,
                                                          0, 0, 0, 0);
}

// Columns n .. n + 3 of output row m, as one store at element alignment unless the row ends.
__device__ __forceinline__ void fp8_store(const Fp8Params& p, v4f s, int64_t m, int n) {
  typedef uint32_t any2 __attribute__((ext_vector_type(2), aligned(2)));
  if (n >= p.N) return;
  uint16_t* o = p.out + m * p.ld_out + n;
  const any2 h = {f32x2_to_bf16x2(s[0], s[1]), f32x2_to_bf16x2(s[2], s[3])};
  if (n + 4 <= p.N) {
    *reinterpret_cast<any2*>(o) = h;
  } else {
    const uint64_t h4 = ((uint64_t)h[1] << 32) | h[0];
    for (int j = 0; j < 3 && n + j < p.N; ++j) o[j] = (uint16_t)(h4 >> (16 * j));
  }
}

}  // namespace mi355moe
