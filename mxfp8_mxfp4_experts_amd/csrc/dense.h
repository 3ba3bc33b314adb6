// Types shared by the dense product kernels: the two matrix instructions
// behind one interface and the epilogue.
#pragma once

#include "common.h"
#include "launch.h"

namespace mi355moe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

struct DenseI8 {
  using Acc = v4i;
  using Elem = int;
  static constexpr bool kInt = true;
  static __device__ __forceinline__ Acc mfma(v4i a, v4i b, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};
struct DenseBf16 {
  using Acc = v4f;
  using Elem = float;
  static constexpr bool kInt = false;
  static __device__ __forceinline__ Acc mfma(v4i a, v4i b, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
  }
};

// The scales of token m and output columns n .. n + 3 (INT8).
struct DenseScales {
  float x, w[4];
};
template <class T>
__device__ __forceinline__ DenseScales dense_scales(const DenseParams& p, int m, int n) {
  DenseScales s{1.0f, {1.0f, 1.0f, 1.0f, 1.0f}};
  if constexpr (T::kInt) {
    s.x = p.sx[min(m, p.M - 1)];
#pragma unroll
    for (int j = 0; j < 4; ++j) s.w[j] = p.sw[min(n + j, p.N - 1)];
  }
  return s;
}

// Token m's four sums for output columns n .. n + 3 (n a multiple of 4):
// scaled (INT8: one rounding per factor, the int32 sum's conversion
// included), rounded to the output type and stored, as one vector where the
// row's place and the column count allow it.
template <class T>
__device__ __forceinline__ void dense_store(const DenseParams& p, typename T::Acc s,
                                            const DenseScales& sc, int m, int n) {
  if (m >= p.M || n >= p.N) return;
  float f[4];
  const bool whole = n + 4 <= p.N;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = (float)s[j];
    if constexpr (T::kInt) f[j] = f[j] * sc.x * sc.w[j];
  }
  const int64_t at = (int64_t)m * p.ld_out + n;
  if (p.out_f32) {
    float* o = static_cast<float*>(p.out) + at;
    if (whole && p.out_vec) {
      *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
      for (int j = 0; j < 4 && n + j < p.N; ++j) o[j] = f[j];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(p.out) + at;
    const uint2 h = make_uint2(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]));
    if (whole && p.out_vec) {
      *reinterpret_cast<uint2*>(o) = h;
    } else {
      const uint64_t h4 = ((uint64_t)h.y << 32) | h.x;
      for (int j = 0; j < 4 && n + j < p.N; ++j) o[j] = (uint16_t)(h4 >> (16 * j));
    }
  }
}

}  // namespace mi355moe
