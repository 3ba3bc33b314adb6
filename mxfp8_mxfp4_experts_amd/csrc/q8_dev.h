// Rows in 8 bits: device functions shared by the norm (norm.hip) and the
// few-token integer products (dense.hip).
#pragma once

#include "common.h"
#include "fc_common.h"   // e4m3x4_scaled
#include "route_dev.h"   // wave_max_u32

namespace mi355moe {

// A barrier after LDS writes that leaves global loads and stores under way (the
// compiler's own barrier waits for them all).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  asm volatile("s_barrier" ::: "memory");
}

constexpr float kMinScale = 1.17549435e-38f;   // 2^-126: 1 / s stays finite

// Wavefront sum, uniform result: inclusive scans within 16-lane rows (row_shr
// 1, 2, 4, 8), then row_bcast 15 and 31 carry the rows' sums up to lane 63.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf,
                                                        false));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0x111, 0xf>(v);
  v = add_dpp<0x112, 0xf>(v);
  v = add_dpp<0x114, 0xf>(v);
  v = add_dpp<0x118, 0xf>(v);
  v = add_dpp<0x142, 0xa>(v);
  v = add_dpp<0x143, 0xc>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]),
                    f32x2_to_bf16x2(f[4], f[5]), f32x2_to_bf16x2(f[6], f[7]));
}

// Bits of the largest |value| of 8 bf16 (as a float's; a NaN counts as the
// largest).
__device__ __forceinline__ uint32_t absmax8_bits(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (w[i] << 16) & 0x7FFFFFFFu, hi = w[i] & 0x7FFF0000u;
    top = top > lo ? top : lo;
    top = top > hi ? top : hi;
  }
  return top;
}

// A row's scale and its reciprocal; for a row that holds an infinity or a NaN
// the scale is NaN and every code 0 (inv 0, odd set).
struct Int8Scale {
  float scale, inv;
  bool odd;
};
__device__ __forceinline__ Int8Scale int8_scale(float amax) {
  Int8Scale s;
  s.odd = !(amax <= 3.402823466e38f);
  const float v = fmaxf(amax / 127.0f, kMinScale);
  s.inv = 1.0f / v;
  s.scale = s.odd ? __uint_as_float(0x7FC00000u) : v;
  return s;
}

// Whole numbers of [-127, 127] of 8 values.  Adding 1.5 * 2^23 rounds to the
// nearest whole number, ties to even, and leaves it in the low bits (two's
// complement), so a byte is picked out without a conversion.
__device__ __forceinline__ uint2 int8x8(const float (&f)[8], const Int8Scale& s) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = fminf(fmaxf(f[i] * s.inv, -127.0f), 127.0f);
    w[i] = __float_as_uint(r + 12582912.0f);
  }
  uint32_t q[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __builtin_amdgcn_perm(w[4 * h + 1], w[4 * h], 0x0C0C0400u);
    const uint32_t b = __builtin_amdgcn_perm(w[4 * h + 3], w[4 * h + 2], 0x04000C0Cu);
    q[h] = s.odd ? 0u : (a | b);
  }
  return make_uint2(q[0], q[1]);
}

// MXFP8 codes of a lane's 8 values and its 32-element group's scale byte;
// the group is four consecutive lanes.
__device__ __forceinline__ uint2 mxfp8x8(const float (&f)[8], uint32_t& scale) {
  float amax = 0.0f;
  uint32_t odd = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(f[i]);
    amax = a > amax ? a : amax;   // NaN compares false: ignored
    odd |= (__float_as_uint(f[i]) & 0x7F800000u) == 0x7F800000u;
  }
  amax = fmaxf(amax, __shfl_xor(amax, 1));
  amax = fmaxf(amax, __shfl_xor(amax, 2));
  odd |= __shfl_xor(odd, 1);
  odd |= __shfl_xor(odd, 2);
  const int e = mx8_exponent(amax);
  scale = (uint32_t)(e + 127);
  uint32_t lo = 0, hi = 0;
  if (!odd && e > -127) {
    const float s2 = __uint_as_float((uint32_t)(e + 127) << 23);
    lo = e4m3x4_scaled(f[0], f[1], f[2], f[3], s2);
    hi = e4m3x4_scaled(f[4], f[5], f[6], f[7], s2);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) lo |= e4m3_encode(ldexpf(f[i], -e)) << (8 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) hi |= e4m3_encode(ldexpf(f[4 + i], -e)) << (8 * i);
  }
  return make_uint2(lo, hi);
}

}  // namespace mi355moe
