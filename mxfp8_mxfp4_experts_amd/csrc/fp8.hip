// Products of E4M3 codes with a float scale for each block of 128:
//   out[m, n] = bf16( sum over blocks b of 128 along K of
//               (sa[b, m] * sb[n / 128, b]) * sum_{k in b} a[m, k] w[n, k] ),
// the blocks' sums by the matrix unit, scaled and added in float.  Dense (one weight), and
// grouped: rows [offs[e], offs[e + 1]) of the output take weight e, and their tokens stand in
// that order too or are found through sorted_route.  And the tokens' quantisation.
#include "common.h"
#include "fp8.h"
#include "launch.h"
#include "q8_dev.h"

namespace mi355moe {

namespace {

// Codes of a lane's 8 values and the scale of their 128-element block (16 neighbouring lanes):
// s = max(amax / 448, 2^-126), code = e4m3(x * (1 / s)); a block with an infinity or a NaN gets
// s = NaN and codes 0.
__device__ __forceinline__ float fp8_scale(float amax, float& inv) {
  const float v = fmaxf(amax / 448.0f, kMinScale);
  const bool odd = !(amax <= 3.402823466e38f);
  inv = odd ? 0.0f : 1.0f / v;
  return odd ? __uint_as_float(0x7FC00000u) : v;
}
__device__ __forceinline__ uint2 fp8x8(const float (&f)[8], float inv, bool odd) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = odd ? 0.0f : fminf(fmaxf(f[i] * inv, -448.0f), 448.0f);
  return make_uint2(e4m3x4_scaled(q[0], q[1], q[2], q[3], 1.0f),
                    e4m3x4_scaled(q[4], q[5], q[6], q[7], 1.0f));
}

// Eight elements per lane; 16 lanes share a block of 128.
__global__ __launch_bounds__(256) void quant_fp8_kernel(const uint16_t* __restrict__ x,
                                                        int64_t ld_x, int T, int H,
                                                        uint8_t* __restrict__ xq, int64_t ld_q,
                                                        float* __restrict__ xs, int64_t ld_s) {
  const int KB = (H + kScaleBlock - 1) / kScaleBlock;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = at / (16 * KB);
  if (t >= T) return;                     // alike for a block's 16 lanes
  const int c = (int)(at - t * (16 * KB)), k = 8 * c;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (k < H) v = *reinterpret_cast<const uint4*>(x + t * ld_x + k);
  uint32_t top = absmax8_bits(v);         // a NaN counts as the largest
#pragma unroll
  for (int i = 1; i < 16; i <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, i));
  float inv, f[8];
  const float s = fp8_scale(__uint_as_float(top), inv);
  unpack8(v, f);
  if (k < H) *reinterpret_cast<uint2*>(xq + t * ld_q + k) = fp8x8(f, inv, !(s == s));
  if ((c & 15) == 0) xs[(c >> 4) * ld_s + t] = s;
}

// 16 bytes at k of a row of K bytes, zeros past its end (the load itself is unconditional).
__device__ __forceinline__ v4i load_piece(const uint8_t* row, int k, int K) {
  v4i v = *reinterpret_cast<const v4i*>(row + min(k, K - 16));
  if (k >= K) v = v4i{0, 0, 0, 0};
  return v;
}

// Few rows per weight: a workgroup of four wavefronts takes 16 output columns of up to 16 rows,
// each wavefront every fourth block of K; their sums are added through LDS in wavefront order.
__global__ __launch_bounds__(256) void fp8_direct_kernel(Fp8Params p) {
  __shared__ v4f red_s[4][64];
  __shared__ int count_s[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int cols = (p.N + 15) / 16;
  const int64_t slot = blockIdx.x / cols;
  const int n0 = 16 * (int)(blockIdx.x - slot * cols);
  int64_t m0 = 16 * slot, m1 = p.M;
  const uint8_t* b = p.b;
  const float* sb = p.sb;
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock, NB = (p.N + kScaleBlock - 1) / kScaleBlock;
  if (p.offs) {
    // Slot = output row: its expert is the number of experts that end at or before it.  The
    // workgroup has work where the row is the first of 16 of its expert.
    int n = 0;
    for (int e = tid; e < p.E; e += 256) n += (int64_t)p.offs[e + 1] <= slot;
    n = (int)wave_sum((float)n);
    if (lane == 0) count_s[wave] = n;
    __syncthreads();
    const int e = count_s[0] + count_s[1] + count_s[2] + count_s[3];
    if (e >= p.E) return;
    const int first = max(p.offs[e], 0);
    if (slot < first || (slot - first) % 16 != 0) return;
    m0 = slot;
    m1 = min(p.offs[e + 1], p.M);
    if (m1 <= slot) return;   // offsets out of order
    b += (int64_t)e * p.N * p.K;
    sb += (int64_t)e * NB * KB;
  }
  const int64_t m = m0 + l < m1 ? m0 + l : m1 - 1;
  int64_t row = m;
  if (p.route) row = min(max(p.route[m] / p.top_k, 0), p.a_rows - 1);
  const uint8_t* ap = p.a + row * p.ld_a;
  const uint8_t* bp = b + (int64_t)min(n0 + l, p.N - 1) * p.K;
  const float* sbp = sb + (int64_t)(n0 / kScaleBlock) * KB;
  v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
  for (int kb = wave; kb < KB; kb += 4) {
    const int k = kScaleBlock * kb + 16 * g;
    const v4f s = mfma_fp8(load_piece(bp, k, p.K), load_piece(bp, k + 64, p.K),
                           load_piece(ap, k, p.K), load_piece(ap, k + 64, p.K));
    const float f = p.sa[kb * p.ld_sa + row] * sbp[kb];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(s[i], f, acc[i]);
  }
  red_s[wave][lane] = acc;
  __syncthreads();
  if (wave == 0 && m0 + l < m1) {
    const v4f s = ((red_s[0][lane] + red_s[1][lane]) + red_s[2][lane]) + red_s[3][lane];
    fp8_store(p, s, m0 + l, n0 + 4 * g);
  }
}

}  // namespace

hipError_t launch_quant_fp8(const uint16_t* x, int64_t ld_x, int T, int H, uint8_t* xq,
                            int64_t ld_q, float* xs, int64_t ld_s, hipStream_t stream) {
  const int64_t lanes = (int64_t)T * 16 * ((H + kScaleBlock - 1) / kScaleBlock);
  const int64_t blocks = (lanes + 255) / 256;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(quant_fp8_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, x, ld_x, T, H,
                     xq, ld_q, xs, ld_s);
  return hipGetLastError();
}

size_t fp8_workspace(int, int) { return 0; }

hipError_t launch_fp8(const Fp8Params& p, hipStream_t stream) {
  const int64_t slots = p.offs ? p.M : (p.M + 15) / 16;
  const int64_t blocks = slots * ((p.N + 15) / 16);
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(fp8_direct_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mi355moe
