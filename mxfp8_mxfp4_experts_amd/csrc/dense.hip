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
#include "q8_dev.h"

namespace mi355moe {

namespace {

// Few rows: no operand is used twice enough to pay for LDS, and the weights' one
// way from memory bounds the product (INT8 1 x 3584 x 7168: 25.7 MB in 7.3 us, 3.5
// TB/s with the launch; BF16 8 x 896 x 7168: 5.0 us, the chain of load, products
// and join).  A workgroup of W
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
constexpr int kDirectWaves = 16;
constexpr int kFusedUnits = 4;         // units of 512 elements a wavefront quantises

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

// Estimated time of the direct kernel past its launch, in ns.  A workgroup reads
// its columns and its tokens, a CU about 90 bytes/ns where a load instruction
// takes whole 128-byte lines (Q of 2 or 4) and 51 where it takes half lines; first
// loads and the join take half a microsecond, longer with more sums per output;
// the chip reads its weights at about 5600 bytes/ns.  (Router product of 32
// tokens, 896 x 7168: 14.9 us with Q = 1, 9.5 with 2; INT8 16 x 3584 x 7168: 8.7 us
// with 1, 11.2 with 2.)
constexpr int kCus = 256;
float direct_ns(int q, int M, int N, int64_t Kb) {
  const int c = 16 / q;
  const int64_t wgs = (int64_t)((N + c - 1) / c) * ((M + c - 1) / c);
  const float bytes = (float)(c + (M < c ? M : c)) * Kb;
  const float one = q == 1 ? bytes / 51.0f + 530.0f : bytes / 90.0f + (q == 2 ? 490.0f : 850.0f);
  const float per_cu = (float)((wgs + kCus - 1) / kCus) * one;
  const float chip = (float)N * Kb / 5600.0f;
  return per_cu > chip ? per_cu : chip;
}
// The Q of least estimated time.
int direct_q(int M, int N, int64_t Kb) {
  int best = 1;
  for (int q = 2; q <= 4; q *= 2)
    if (direct_ns(q, M, N, Kb) < direct_ns(best, M, N, Kb)) best = q;
  return best;
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
  if (tokens * ((p.Kb + 511) / 512) <= kDirectWaves)
    hipLaunchKernelGGL((dense_direct_quant_kernel<Q, kBatch, 1>), grid, block, lds, stream, p, x,
                       ld_x);
  else
    hipLaunchKernelGGL((dense_direct_quant_kernel<Q, kBatch, kFusedUnits>), grid, block, lds,
                       stream, p, x, ld_x);
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

// The tiled kernel's variants, widest tile first: what one stage takes with at
// most one workgroup per CU and with two, and what a workgroup takes besides
// (first loads, epilogue), in ns on 256 CUs.  These and the other times of the
// estimate are fitted to every variant and split of 618 products of both types (M
// 17 .. 8192, N 8 .. 3584, K bytes 128 .. 14336, log-uniform): what `pick` takes
// is 1.3% slower than the best of them in the mean, 27% at worst.  64 x 64 tiles
// come with eight wavefronts, which take short K and two workgroups per CU 1 to 4%
// faster, and with four, which take long K in one round faster (INT8 256 x 3584 x
// 7168: 14.0 against 14.7 us).
struct Variant {
  int bm, bn, per_cu;
  float one, two, fixed;
};
constexpr Variant kVariants[] = {
    {256, 224, 1, 1400, 0, 11000}, {128, 224, 1, 760, 0, 3300}, {128, 128, 1, 440, 0, 2100},
    {64, 128, 2, 270, 560, 1500},  {96, 64, 2, 210, 470, 1700}, {64, 64, 2, 170, 310, 1100},
    {64, 64, 2, 165, 320, 1220},   {32, 64, 2, 100, 230, 1100}, {32, 32, 2, 85, 170, 1000},
};
constexpr int kNumVariants = sizeof(kVariants) / sizeof(kVariants[0]);
constexpr int kMaxSplits = 16;
constexpr int kDirectRows = 16;        // up to here always the direct kernel
constexpr int kDirectMost = 512;       // up to here the direct kernel if it is estimated faster
constexpr int kFusedBytes = 44 << 10;  // a workgroup's codes in LDS, next to 16 KB of partial tiles

// Most partial sums (4 bytes each) that a product of these sizes may use: grows
// with M, so a workspace for M rows serves every smaller M.
constexpr int64_t kMostPartials = 1 << 22;
int64_t most_partials(int M, int N) {
  const int64_t all = (int64_t)kMaxSplits * M * ((N + 3) / 4 * 4);
  return all < kMostPartials ? all : kMostPartials;
}

struct Pick {
  int variant;   // -1: the direct kernel
  int splits;
  float ns;      // estimated
};

// The kernel, variant and split of K with the least estimated time: whole rounds
// of workgroups at their stage time, 2 us of launch, plus, with K split, a second
// launch and the partial sums' way through the caches (11 bytes/ps).
Pick pick(int M, int N, int64_t Kb) {
  Pick best{-1, 1, 3.4e38f};
  if (M <= kDirectMost) best.ns = 1900.0f + direct_ns(direct_q(M, N, Kb), M, N, Kb);
  if (M <= kDirectRows) return best;
  const int stages = (int)((Kb + kStageK - 1) / kStageK);
  const float join = (float)M * N * 8 / 11000.0f;
  const int64_t sums = (int64_t)M * ((N + 3) / 4 * 4);
  // Splits are for launches that leave CUs idle; each has four stages at least.
  int most = kMaxSplits < stages / 4 ? kMaxSplits : stages / 4;
  while (most > 1 && most * sums > most_partials(M, N)) --most;
  for (int v = 0; v < kNumVariants; ++v) {
    const Variant& c = kVariants[v];
    const int64_t tiles = (int64_t)((M + c.bm - 1) / c.bm) * ((N + c.bn - 1) / c.bn);
    for (int s = 1; s == 1 || (s <= most && tiles * s <= 2 * kCus); ++s) {
      const int per = (stages + s - 1) / s, at_once = kCus * c.per_cu;
      const int64_t wgs = tiles * s;
      const int rest = (int)(wgs & (at_once - 1));   // a power of two
      const float whole = per * (c.per_cu == 2 ? c.two : c.one) + c.fixed;
      float t = 2000.0f + (float)(wgs >> (7 + c.per_cu)) * whole;
      if (rest) t += rest <= kCus ? per * c.one + c.fixed : whole;
      if (s > 1) t += 1700.0f + s * join;
      if (t < best.ns) best = {v, s, t};
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

// One launch that quantises every workgroup's tokens anew, or two?  The estimate
// of the one (fitted as those above, to 258 products of 1 .. 1024 tokens, 160 of
// them faster in one launch: 64 x 512 x 512 4.2 against 6.0 us, 256 x 240 x 736 5.2
// against 5.6, 28 x 2889 x 1104 8.2 against 6.6) against the other's with 2.7 us
// for the quantisation, and half a microsecond because a second launch costs the
// host 3.5 us.  On 128 other products the choice is 1.3% slower than the better.
int dense_fused_q(int M, int N, int K) {
  float least = 0.0f;
  int best = 0;
  for (int q = 1; q <= 4; q *= 2) {
    const int c = 16 / q, tokens = M < c ? M : c, units = tokens * ((K + 511) / 512);
    if (units > kFusedUnits * kDirectWaves || tokens * (K + 16) > kFusedBytes) continue;
    if (M > 65535 * c) continue;   // the grid's second dimension
    const int64_t wgs = (int64_t)((N + c - 1) / c) * ((M + c - 1) / c);
    const float first = units > kDirectWaves ? 2100.0f : 1200.0f;
    const float one = (float)(c + 2 * tokens) * K / 60.0f + first;
    const float per_cu = (float)((wgs + kCus - 1) / kCus) * one, chip = (float)N * K / 5600.0f;
    const float t = per_cu > chip ? per_cu : chip;
    if (!best || t < least) {
      least = t;
      best = q;
    }
  }
  return best && least <= pick(M, N, K).ns + 500.0f ? best : 0;
}

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
