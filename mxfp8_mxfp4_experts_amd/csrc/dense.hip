// Dense products C = A B^T with both operands contiguous along K:
//   INT8: C[m, n] = (sum_k a[m, k] b[n, k]) * sx[m] * sw[n], the sum exact in
//         int32; bf16 or float32 out;
//   BF16: C[m, n] = sum_k a[m, k] b[n, k] in float32; float32 out.
//
// Both matrix instructions take 16 bytes of each operand per lane and give a
// 16x16 tile (v_mfma_i32_16x16x64_i8, v_mfma_f32_16x16x32_bf16), so the
// kernels move bytes along K and do not care which type they carry.  The
// weight fragment is the first operand: a lane then holds four neighbouring
// output columns of one token.
#include "common.h"
#include "dense.h"
#include "launch.h"

namespace mi355moe {

namespace {

// Few rows: no operand is used twice enough to pay for LDS.  A workgroup owns
// 16 output columns and 16 MI tokens; its W wavefronts split K (64 bytes in
// turn, so together they read runs of 64 W bytes of each weight row), each
// feeding the matrix unit straight from global loads, and the partial tiles
// are added through LDS in wavefront order.
template <class T, int MI, int W>
__global__ __launch_bounds__(64 * W) void dense_direct_kernel(DenseParams p) {
  using Acc = typename T::Acc;
  __shared__ Acc red_s[W][MI][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MI;
  const uint8_t* bp = p.b + (int64_t)min(n0 + r, p.N - 1) * p.ld_b + 16 * g;
  const uint8_t* ap[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
    ap[i] = p.a + (int64_t)min(m0 + 16 * i + r, p.M - 1) * p.ld_a + 16 * g;
  Acc acc[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) acc[i] = Acc{0, 0, 0, 0};
  const int Kb = p.Kb;
#pragma unroll 4
  for (int k = 64 * wave; k < Kb; k += 64 * W) {
    const bool in = k + 16 * g < Kb;   // K is whole 16-byte pieces
    const v4i zero{0, 0, 0, 0};
    const v4i b = in ? *reinterpret_cast<const v4i*>(bp + k) : zero;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const v4i a = in ? *reinterpret_cast<const v4i*>(ap[i] + k) : zero;
      acc[i] = T::mfma(b, a, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) red_s[wave][i][lane] = acc[i];
  __syncthreads();
  for (int j = threadIdx.x; j < 64 * MI; j += 64 * W) {
    const int i = j >> 6, l = j & 63;
    Acc s = red_s[0][i][l];
#pragma unroll
    for (int w = 1; w < W; ++w) s += red_s[w][i][l];
    dense_store<T>(p, s, m0 + 16 * i + (l & 15), n0 + 4 * (l >> 4));
  }
}

template <class T, int MI, int W>
hipError_t direct(const DenseParams& p, hipStream_t stream) {
  const dim3 grid((p.N + 15) / 16, (p.M + 16 * MI - 1) / (16 * MI));
  hipLaunchKernelGGL((dense_direct_kernel<T, MI, W>), grid, dim3(64 * W), 0, stream, p);
  return hipGetLastError();
}

template <class T>
hipError_t launch(const DenseParams& p, hipStream_t stream) {
  if (p.M <= 16) return direct<T, 1, 16>(p, stream);
  return direct<T, 4, 4>(p, stream);
}

}  // namespace

size_t dense_workspace(bool, int, int, int64_t) { return 0; }

hipError_t launch_dense(bool i8, const DenseParams& p, hipStream_t stream) {
  return i8 ? launch<DenseI8>(p, stream) : launch<DenseBf16>(p, stream);
}

}  // namespace mi355moe
