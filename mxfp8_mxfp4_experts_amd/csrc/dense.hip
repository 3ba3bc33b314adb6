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
#include "dense_pick.h"
#include "dense_tile.h"
#include "launch.h"
#include "q8_dev.h"

namespace mi355moe {

namespace {

// Few rows: no operand is used twice enough to pay for LDS, and the weights' one
// way from memory bounds the product (INT8 1 x 3584 x 7168: 25.7 MB in 7.2 - 8.0 us,
// 3.2 - 3.6 TB/s with the launch; BF16 8 x 896 x 7168: 5.7 - 6.1 us, the chain of
// load, products and join).  A workgroup of W
// wavefronts owns 16 / Q output columns and 16 / Q tokens and splits K over its
// wavefronts, each feeding the matrix unit straight from global loads, with the
// loads of several steps in flight; the partial tiles are added through LDS in
// wavefront order.
//
// Q: a 16x16 tile of 16 columns x 16 tokens is mostly empty for one to eight
// tokens, and N / 16 workgroups are too few to draw on the whole chip's
// bandwidth.  With Q > 1 the tile's rows are (column, kq) and its columns
// (token, kq), where kq < Q says which of Q neighbouring 64-byte pieces of K
// the row or column carries: the products with equal kq on both sides are the
// sums wanted, the others are not read.  So a workgroup covers 16 / Q columns at
// Q times the length of K per step, and a launch has Q times the workgroups.
template <class T, int Q>
struct DirectGeom {
  static constexpr int kCols = 16 / Q;              // output columns, and tokens
  static constexpr int kStep = 64 * Q * kDirectWaves;   // bytes of K per step
};

// Adds the wavefronts' tiles and stores the workgroup's outputs.
template <class T, int Q>
__device__ __forceinline__ void direct_finish(const DenseParams& p, typename T::Acc acc, int m0,
                                              int n0, typename T::Acc* red_s) {
  using Acc = typename T::Acc;
  using E = typename T::Elem;
  constexpr int C = 16 / Q;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tid = threadIdx.x;
  red_s[64 * wave + lane] = acc;
  __syncthreads();
  if constexpr (Q == 1) {
    if (tid < 64) {
      Acc s = red_s[lane];
#pragma unroll
      for (int w = 1; w < kDirectWaves; ++w) s += red_s[64 * w + lane];
      const int m = m0 + (lane & 15), n = n0 + 4 * (lane >> 4);
      dense_store<T>(p, s, dense_scales<T>(p, m, n), m, n);
    }
  } else {
    // Entry e of a wavefront's tile: lane e / 4, element e % 4 -- row 4 (lane / 16)
    // + e % 4, column lane % 16.  One thread per output: its Q entries on the
    // diagonal, wavefront by wavefront.
    const E* red = reinterpret_cast<const E*>(red_s);
    if (tid < C * C) {
      const int c = tid % C, m = tid / C;
      E s = 0;
#pragma unroll
      for (int kq = 0; kq < Q; ++kq) {
        const int row = c * Q + kq, col = m * Q + kq;
        const int e = 4 * (16 * (row >> 2) + col) + (row & 3);
#pragma unroll
        for (int w = 0; w < kDirectWaves; ++w) s += red[256 * w + e];
      }
      if (m0 + m < p.M && n0 + c < p.N) {
        float f = (float)s;
        if constexpr (T::kInt) f = f * p.sx[m0 + m] * p.sw[n0 + c];
        const int64_t at = (int64_t)(m0 + m) * p.ld_out + n0 + c;
        if (p.out_f32)
          static_cast<float*>(p.out)[at] = f;
        else
          static_cast<uint16_t*>(p.out)[at] = (uint16_t)f32x2_to_bf16x2(f, 0.0f);
      }
    }
  }
}

// 16 bytes at k of a row of Kb bytes, zeros past its end.  The load itself is
// unconditional (of the row's last piece there): loads under a condition would
// make the compiler wait for all loads before any is used.
__device__ __forceinline__ v4i load_piece(const uint8_t* row, int k, int Kb) {
  v4i v = *reinterpret_cast<const v4i*>(row + min(k, Kb - 16));
  if (k >= Kb) v = v4i{0, 0, 0, 0};
  return v;
}

// kHalf steps' loads at once, twice; MORE: K is longer than that.  Short rows take
// the small batches, whose registers let two workgroups share a CU.
template <class T, int Q, int kHalf, bool MORE>
__global__ __launch_bounds__(64 * kDirectWaves) void dense_direct_kernel(DenseParams p) {
  using Acc = typename T::Acc;
  using G = DirectGeom<T, Q>;
  __shared__ Acc red_s[64 * kDirectWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (lane & 15) / Q, kq = lane % Q, g = lane >> 4;
  const int n0 = blockIdx.x * G::kCols, m0 = blockIdx.y * G::kCols;
  const int k0 = 64 * (Q * wave + kq) + 16 * g;    // K is whole 16-byte pieces
  const uint8_t* bp = p.b + (int64_t)min(n0 + c, p.N - 1) * p.ld_b;
  const uint8_t* ap = p.a + (int64_t)min(m0 + c, p.M - 1) * p.ld_a;
  Acc acc{0, 0, 0, 0};
  // With MORE the halves take turns: one's matrix instructions while the other is
  // on its way.
  struct Batch {
    v4i a[kHalf], b[kHalf];
  } one, two;
  auto load = [&](Batch& s, int k) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i) {
      s.b[i] = load_piece(bp, k0 + k + i * G::kStep, p.Kb);
      s.a[i] = load_piece(ap, k0 + k + i * G::kStep, p.Kb);
    }
  };
  auto use = [&](const Batch& s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i) acc = T::mfma(s.b[i], s.a[i], acc);
  };
  load(one, 0);
  load(two, kHalf * G::kStep);
  if constexpr (!MORE) {
    use(one);
    use(two);
  } else {
    for (int k = 0; k < p.Kb; k += 2 * kHalf * G::kStep) {
      use(one);
      load(one, k + 2 * kHalf * G::kStep);
      use(two);
      load(two, k + 3 * kHalf * G::kStep);
    }
  }
  direct_finish<T, Q>(p, acc, m0, n0, red_s);
}

// INT8 with bf16 tokens, in one launch: the workgroup quantises its tokens (16 / Q,
// with the rule of moe_quant_int8) into LDS while its first weight loads are on
// their way.  kUnits: units of 512 elements per wavefront.
template <int Q, int kBatch, int kUnits>
__global__ __launch_bounds__(64 * kDirectWaves) void dense_direct_quant_kernel(
    DenseParams p, const uint16_t* __restrict__ x, int64_t ld_x) {
  using T = DenseI8;
  using G = DirectGeom<T, Q>;
  extern __shared__ __attribute__((aligned(16))) uint8_t tok_s[];   // [tokens][K + 16]
  __shared__ v4i red_s[64 * kDirectWaves];
  __shared__ uint32_t max_s[kUnits * kDirectWaves];
  __shared__ float sx_s[16 / Q];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = (lane & 15) / Q, kq = lane % Q, g = lane >> 4;
  const int n0 = blockIdx.x * G::kCols, m0 = blockIdx.y * G::kCols;
  const int M = min(p.M - m0, G::kCols);
  const int K = p.Kb, pieces = K / 8, row_s = K + 16, units = (pieces + 63) / 64;
  x += m0 * ld_x;
  const int k0 = 64 * (Q * wave + kq) + 16 * g;
  const uint8_t* bp = p.b + (int64_t)min(n0 + c, p.N - 1) * p.ld_b;
  const v4i zero{0, 0, 0, 0};
  // Units of 512 elements of a token: wavefront w takes units w, w + 16, ..., all
  // their loads at once -- before the weights', since loads come back in order --
  // and leaves each unit's absolute maximum (as bits: a NaN counts as the
  // largest).
  uint4 xv[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = wave + kDirectWaves * i, m = u / units, q = 64 * (u - m * units) + lane;
    // Past the last piece or token the last one again: no other maximum.
    xv[i] = reinterpret_cast<const uint4*>(x + min(m, M - 1) * ld_x)[min(q, pieces - 1)];
  }
  asm volatile("" ::: "memory");
  v4i b[kBatch];
#pragma unroll
  for (int i = 0; i < kBatch; ++i) b[i] = load_piece(bp, k0 + i * G::kStep, K);
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    if (wave + kDirectWaves * i >= M * units) break;   // uniform
    const uint32_t top = wave_max_u32(absmax8_bits(xv[i]));
    if (lane == 0) max_s[wave + kDirectWaves * i] = top;
  }
  lds_barrier();
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int u = wave + kDirectWaves * i, m = u / units, q = 64 * (u - m * units) + lane;
    if (m >= M) break;
    uint32_t top = 0;
    for (int j = 0; j < units; ++j) top = max(top, max_s[m * units + j]);
    const Int8Scale s = int8_scale(__uint_as_float(top));
    if (q == 0) sx_s[m] = s.scale;
    if (q < pieces) {
      float f[8];
      unpack8(xv[i], f);
      *reinterpret_cast<uint2*>(tok_s + m * row_s + 8 * q) = int8x8(f, s);
    }
  }
  lds_barrier();

  const uint8_t* ap = tok_s + min(c, M - 1) * row_s;
  v4i acc = zero;
  for (int k = 0; k < K; k += kBatch * G::kStep) {
    v4i next[kBatch];
    if (k + kBatch * G::kStep < K) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        next[i] = load_piece(bp, k0 + k + (kBatch + i) * G::kStep, K);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      acc = T::mfma(b[i], load_piece(ap, k0 + k + i * G::kStep, K), acc);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) b[i] = next[i];
  }
  p.sx = sx_s;
  p.M = M;
  p.out = static_cast<uint8_t*>(p.out) + m0 * p.ld_out * (p.out_f32 ? 4 : 2);
  direct_finish<T, Q>(p, acc, 0, n0, red_s);
}

template <class T, int Q>
hipError_t direct(const DenseParams& p, hipStream_t stream) {
  constexpr int C = 16 / Q;
  const dim3 grid((p.N + C - 1) / C, (p.M + C - 1) / C);
  const dim3 block(64 * kDirectWaves);
  const int steps = (p.Kb + DirectGeom<T, Q>::kStep - 1) / DirectGeom<T, Q>::kStep;
  if (steps <= 2)
    hipLaunchKernelGGL((dense_direct_kernel<T, Q, 1, false>), grid, block, 0, stream, p);
  else if (steps <= 4)
    hipLaunchKernelGGL((dense_direct_kernel<T, Q, 2, false>), grid, block, 0, stream, p);
  else if (steps <= 8)
    hipLaunchKernelGGL((dense_direct_kernel<T, Q, 4, false>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((dense_direct_kernel<T, Q, 4, true>), grid, block, 0, stream, p);
  return hipGetLastError();
}
template <class T>
hipError_t direct(const DenseParams& p, hipStream_t stream) {
  switch (direct_q(p.M, p.N, p.Kb)) {
    case 1: return direct<T, 1>(p, stream);
    case 2: return direct<T, 2>(p, stream);
    default: return direct<T, 4>(p, stream);
  }
}

template <int Q, int kBatch>
hipError_t direct_quant(const DenseParams& p, const uint16_t* x, int64_t ld_x,
                        hipStream_t stream) {
  constexpr int C = 16 / Q;
  const dim3 grid((p.N + C - 1) / C, (p.M + C - 1) / C), block(64 * kDirectWaves);
  const int tokens = p.M < C ? p.M : C;
  const size_t lds = (size_t)tokens * (p.Kb + 16);
  // One unit per wavefront reaches K = 8192, where batches of 4 are for more than 2048 Q and of 8
  // for more than 4096 Q.
  if constexpr (kBatch == 2 || kBatch * Q < 16) {
    if (tokens * ((p.Kb + 511) / 512) <= kDirectWaves) {
      hipLaunchKernelGGL((dense_direct_quant_kernel<Q, kBatch, 1>), grid, block, lds, stream, p, x,
                         ld_x);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((dense_direct_quant_kernel<Q, kBatch, kFusedUnits>), grid, block, lds, stream,
                     p, x, ld_x);
  return hipGetLastError();
}
template <int Q>
hipError_t direct_quant(const DenseParams& p, const uint16_t* x, int64_t ld_x,
                        hipStream_t stream) {
  const int steps = (p.Kb + DirectGeom<DenseI8, Q>::kStep - 1) / DirectGeom<DenseI8, Q>::kStep;
  if (steps <= 2) return direct_quant<Q, 2>(p, x, ld_x, stream);
  if (steps <= 4) return direct_quant<Q, 4>(p, x, ld_x, stream);
  return direct_quant<Q, 8>(p, x, ld_x, stream);
}

template <class T>
hipError_t launch(const DenseParams& p, hipStream_t stream) {
  const Pick k = pick(p.M, p.N, p.Kb);
  // The tiled kernel reaches a tile's rows by 31-bit offsets; rows further
  // apart than that take the direct kernel, whose addresses are 64-bit.
  const int64_t ld = p.ld_a > p.ld_b ? p.ld_a : p.ld_b;
  if (k.variant < 0 || 256 * ld + p.Kb >= (int64_t)1 << 31)
    return direct<T>(p, stream);
  switch (k.variant) {
    case 0: return dense_tile_launch<T, 2, 2, 8, 7, 2, 1>(p, k.splits, stream);
    case 1: return dense_tile_launch<T, 2, 2, 4, 7, 3, 1>(p, k.splits, stream);
    case 2: return dense_tile_launch<T, 4, 2, 2, 4, 4, 2>(p, k.splits, stream);
    case 3: return dense_tile_launch<T, 2, 2, 2, 4, 3, 2>(p, k.splits, stream);
    case 4: return dense_tile_launch<T, 2, 2, 3, 2, 3, 2>(p, k.splits, stream);
    case 5: return dense_tile_launch<T, 4, 2, 1, 2, 4, 4>(p, k.splits, stream);
    case 6: return dense_tile_launch<T, 2, 2, 2, 2, 4, 2>(p, k.splits, stream);
    case 7: return dense_tile_launch<T, 2, 2, 1, 2, 6, 2>(p, k.splits, stream);
    default: return dense_tile_launch<T, 2, 2, 1, 1, 8, 2>(p, k.splits, stream);
  }
}

}  // namespace

size_t dense_workspace(int M, int N) { return sizeof(float) * (size_t)most_partials(M, N); }

int dense_fused_q(int M, int N, int K) { return fused_q(M, N, K); }

hipError_t launch_dense_quant(int q, const DenseParams& p, const uint16_t* x,
                              int64_t ld_x, hipStream_t stream) {
  switch (q) {
    case 1: return direct_quant<1>(p, x, ld_x, stream);
    case 2: return direct_quant<2>(p, x, ld_x, stream);
    default: return direct_quant<4>(p, x, ld_x, stream);
  }
}

hipError_t launch_dense(bool i8, const DenseParams& p, hipStream_t stream) {
  return i8 ? launch<DenseI8>(p, stream) : launch<DenseBf16>(p, stream);
}

}  // namespace mi355moe
