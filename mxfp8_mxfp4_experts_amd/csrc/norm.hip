// Residual addition + root-mean-square norm + 8-bit output, and the 8-bit
// integer quantisation of plain rows.
//
//   h = x + r (float32; stored as bf16),   rstd = 1 / sqrt(mean(h^2) + eps),
//   y = (h * w) * rstd (float32; stored as bf16 if wanted), and y in 8 bits:
//   MXFP8 with the rule of moe_quant_mxfp8, or INT8 with one float scale per
//   row, s = max(absmax / 127, 2^-126), q = rint(y * (1 / s)).
//
// The norm and the 8-bit rounding start from the float32 sum, not from its
// bf16 copy: y is rounded once on its way to each output.
//
// One workgroup per row, one pass: the row stays in registers between the
// reduction and the outputs.  Rounding is monotone, so the largest |y| is the
// largest |h * w| times rstd exactly, and the sum of squares and the absolute
// maximum are reduced together with one barrier.
//
// Memory bounds it at many rows (8192 x 7168 with a residual and MXFP8: 530 MB in
// 92.9 us, 5.7 TB/s; INT8 quantisation alone 176 MB in 31 us), the chain of load,
// reduction and stores at few (one row 3.3 us).  Rows narrower than 512 leave
// lanes idle, 48 of 64 at 128 (65536 x 128: 77 MB in 21.5 us, 3.5 TB/s).
#include "common.h"
#include "launch.h"
#include "q8_dev.h"

namespace mi355moe {

namespace {

// A piece of h, past the caches: what comes next reads y and the 8-bit output,
// h only the next block.  (Stored so as well, those two made the norm of 8192 x
// 7168 5 us faster, and the INT8 product of 256 tokens after it 4 us slower.)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_past(uint16_t* row, int c, const uint4& v) {
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(row) + c);
}

// One row per workgroup, P 8-element pieces per thread (piece tid + i *
// blockDim).  NORM false: y = x (the 8-bit quantisation alone).
template <int P, int Q8, bool NORM>
__global__ __launch_bounds__(1024) void norm_kernel(NormParams p) {
  __shared__ float sum_s[16];
  __shared__ uint32_t max_s[16];
  const int tid = threadIdx.x, n = p.H / 8;
  const int64_t row = blockIdx.x;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.ld_x);
  const uint4* r = reinterpret_cast<const uint4*>(p.res + (p.res ? row * p.ld_res : 0));
  const uint4* w = reinterpret_cast<const uint4*>(p.weight);

  uint4 xv[P], rv[P], wv[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = tid + i * (int)blockDim.x;
    if (c < n) {
      xv[i] = x[c];
      if (NORM && p.res) rv[i] = r[c];
      if (NORM) wv[i] = w[c];
    }
  }
  float f[P][8];
  float sum = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = tid + i * (int)blockDim.x;
    if (c >= n) continue;
    unpack8(xv[i], f[i]);
    if constexpr (NORM) {
      if (p.res) {
        float g[8];
        unpack8(rv[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] += g[j];
      }
      if (p.h) store_past(p.h + row * p.ld_h, c, pack8(f[i]));
      float g[8];
      unpack8(wv[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum += f[i][j] * f[i][j];
        f[i][j] *= g[j];
      }
    }
    if constexpr (Q8 == MOE_Q8_INT8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = __float_as_uint(f[i][j]) & 0x7FFFFFFFu;
        top = a > top ? a : top;
      }
    }
  }
  // Every wavefront adds the wavefronts' sums in the same order.
  const int wave = tid >> 6, n_waves = (int)blockDim.x >> 6;
  if constexpr (NORM) sum = wave_sum(sum);
  if constexpr (Q8 == MOE_Q8_INT8) top = wave_max_u32(top);   // a NaN's bits are the largest: not hidden
  if ((tid & 63) == 0) {
    if constexpr (NORM) sum_s[wave] = sum;
    if constexpr (Q8 == MOE_Q8_INT8) max_s[wave] = top;
  }
  lds_barrier();
  sum = 0.0f;
  top = 0;
  for (int i = 0; i < n_waves; ++i) {
    if constexpr (NORM) sum += sum_s[i];
    if constexpr (Q8 == MOE_Q8_INT8) top = max_s[i] > top ? max_s[i] : top;
  }
  const float rstd = NORM ? 1.0f / sqrtf(sum / (float)p.H + p.eps) : 1.0f;
  Int8Scale s8;
  if constexpr (Q8 == MOE_Q8_INT8) {
    s8 = int8_scale(NORM ? __uint_as_float(top) * rstd : __uint_as_float(top));
    if (tid == 0) reinterpret_cast<float*>(p.xs)[row] = s8.scale;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = tid + i * (int)blockDim.x;
    const bool in = c < n;   // alike for the four lanes of a 32-element group
    if (!in) continue;
    if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] *= rstd;
      if (p.y) reinterpret_cast<uint4*>(p.y + row * p.ld_y)[c] = pack8(f[i]);
    }
    if constexpr (Q8 == MOE_Q8_INT8) {
      reinterpret_cast<uint2*>(p.xq + row * p.ld_q)[c] = int8x8(f[i], s8);
    }
    if constexpr (Q8 == MOE_Q8_MXFP8) {
      uint32_t scale;
      const uint2 q = mxfp8x8(f[i], scale);
      reinterpret_cast<uint2*>(p.xq + row * p.ld_q)[c] = q;
      if ((c & 3) == 0) p.xs[row * (p.H / 32) + c / 4] = (uint8_t)scale;
    }
  }
}

template <int P>
hipError_t launch_p(const NormParams& p, int q8, bool norm, int threads, hipStream_t stream) {
  const dim3 grid(p.T), block(threads);
  if (!norm)
    hipLaunchKernelGGL((norm_kernel<P, MOE_Q8_INT8, false>), grid, block, 0, stream, p);
  else if (q8 == MOE_Q8_NONE)
    hipLaunchKernelGGL((norm_kernel<P, MOE_Q8_NONE, true>), grid, block, 0, stream, p);
  else if (q8 == MOE_Q8_MXFP8)
    hipLaunchKernelGGL((norm_kernel<P, MOE_Q8_MXFP8, true>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((norm_kernel<P, MOE_Q8_INT8, true>), grid, block, 0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormParams& p, int q8, bool norm, hipStream_t stream) {
  const int pieces = p.H / 8;
  // Two pieces per thread where that leaves at least two wavefronts (8192 rows of
  // 7168, before the stores went past the L2: norm 100.6 us with one piece, 96.6
  // with two, 99.1 with four; INT8 alone 41.2, 32.3, 32.1), four for rows past
  // 16384.
  const int per = pieces <= 64 ? 1 : pieces <= 2048 ? 2 : 4;   // H <= kMaxNormH = 32768
  const int threads = ((pieces + per - 1) / per + 63) / 64 * 64;
  if (per == 1) return launch_p<1>(p, q8, norm, threads, stream);
  if (per == 2) return launch_p<2>(p, q8, norm, threads, stream);
  return launch_p<4>(p, q8, norm, threads, stream);
}

}  // namespace mi355moe
