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
#include "dense_tile.h"
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

// The tiled kernel's variants, widest tile first: what one stage takes with at
// most one workgroup per CU and with two, and what a workgroup takes besides
// (first loads, epilogue), in ns on 256 CUs; fitted to sweeps over M = 32 ..
// 8192 at K = 7168 (INT8, N = 3584) and H = 7168 (BF16, N = 896).
struct Variant {
  int bm, bn, per_cu;
  float one, two, fixed;
};
constexpr Variant kVariants[] = {
    {256, 224, 1, 1360, 0, 10500}, {128, 224, 1, 850, 0, 3500}, {128, 128, 1, 500, 0, 3000},
    {128, 128, 2, 720, 930, 3000}, {64, 128, 2, 290, 550, 2000}, {64, 64, 2, 170, 340, 1500},
    {32, 64, 2, 110, 225, 1500},   {32, 32, 2, 80, 123, 1500},
};
constexpr int kNumVariants = sizeof(kVariants) / sizeof(kVariants[0]);
constexpr int kCus = 256;
constexpr int kMaxSplits = 16;
constexpr int kDirectRows = 16;

struct Pick {
  int variant;   // -1: the direct kernel
  int splits;
};

// The variant and split of K with the least estimated time: whole rounds of
// workgroups at their stage time, plus, with K split, the partial sums'
// way through memory (4 bytes/ps) and a second launch.
Pick pick(int M, int N, int64_t Kb) {
  if (M <= kDirectRows) return {-1, 1};
  const int stages = (int)((Kb + kStageK - 1) / kStageK);
  Pick best{-1, 1};
  float least = 0;
  for (int v = 0; v < kNumVariants; ++v) {
    const Variant& c = kVariants[v];
    const int64_t tiles = (int64_t)((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (int s = 1; s <= kMaxSplits && s <= stages; ++s) {
      // Splits are for launches that leave CUs idle.
      if (s > 1 && (tiles * s > 2 * kCus || stages / s < 4)) break;
      const int per = (stages + s - 1) / s;
      const int64_t wgs = tiles * s, full = wgs / (kCus * c.per_cu), rest = wgs % (kCus * c.per_cu);
      const float whole = per * (c.per_cu == 2 ? c.two : c.one) + c.fixed;
      float t = full * whole;
      if (rest) t += rest <= kCus ? per * c.one + c.fixed : whole;
      if (s > 1) t += 2500.0f + (float)s * M * N * 8 / 4000.0f;
      if (best.variant < 0 || t < least) {
        least = t;
        best = {v, s};
      }
    }
  }
  return best;
}

template <class T>
hipError_t launch(const DenseParams& p, hipStream_t stream) {
  const Pick k = pick(p.M, p.N, p.Kb);
  // The tiled kernel reaches a tile's rows by 31-bit offsets; rows further
  // apart than that take the direct kernel, whose addresses are 64-bit.
  const int64_t ld = p.ld_a > p.ld_b ? p.ld_a : p.ld_b;
  if (k.variant < 0 || 256 * ld + p.Kb >= (int64_t)1 << 31)
    return p.M <= kDirectRows ? direct<T, 1, 16>(p, stream) : direct<T, 4, 4>(p, stream);
  switch (k.variant) {
    case 0: return dense_tile_launch<T, 2, 2, 8, 7, 2, 1>(p, k.splits, stream);
    case 1: return dense_tile_launch<T, 2, 2, 4, 7, 3, 1>(p, k.splits, stream);
    case 2: return dense_tile_launch<T, 2, 2, 4, 4, 4, 1>(p, k.splits, stream);
    case 3: return dense_tile_launch<T, 2, 2, 4, 4, 2, 2>(p, k.splits, stream);
    case 4: return dense_tile_launch<T, 2, 2, 2, 4, 3, 2>(p, k.splits, stream);
    case 5: return dense_tile_launch<T, 2, 2, 2, 2, 4, 2>(p, k.splits, stream);
    case 6: return dense_tile_launch<T, 2, 2, 1, 2, 6, 2>(p, k.splits, stream);
    default: return dense_tile_launch<T, 2, 2, 1, 1, 8, 2>(p, k.splits, stream);
  }
}

}  // namespace

size_t dense_workspace(int M, int N, int64_t Kb) {
  if (M <= 0) return 0;
  const Pick k = pick(M, N, Kb);
  if (k.variant < 0 || k.splits == 1) return 0;
  return (size_t)k.splits * M * ((N + 3) / 4 * 4) * 4;
}

hipError_t launch_dense(bool i8, const DenseParams& p, hipStream_t stream) {
  return i8 ? launch<DenseI8>(p, stream) : launch<DenseBf16>(p, stream);
}

}  // namespace mi355moe
