// Products of E4M3 codes with a float scale for each block of 128:
//   out[m, n] = bf16( sum over blocks b of 128 along K of
//               (sa[b, m] * sb[n / 128, b]) * sum_{k in b} a[m, k] w[n, k] ),
// the blocks' sums by the matrix unit, scaled and added in float.  Dense (one weight), and
// grouped: rows [offs[e], offs[e + 1]) of the output take weight e, and their tokens stand in
// that order too or are found through sorted_route.  And the tokens' quantisation.
#include "common.h"
#include "fp8.h"
#include "fp8_pick.h"
#include "fp8_tile.h"
#include "grid.h"
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

// Eight elements per lane; 16 lanes share a block of 128.  A wavefront takes kUnits units of 512
// elements of a row, units in a row's order, its loads all at once.
constexpr int kQuantUnits = 2;
__global__ __launch_bounds__(256) void quant_fp8_kernel(const uint16_t* __restrict__ x,
                                                        int64_t ld_x, int T, int H, int per_row,
                                                        uint8_t* __restrict__ xq, int64_t ld_q,
                                                        float* __restrict__ xs, int64_t ld_s) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const uint32_t first = (blockIdx.x * 4u + wave) * kQuantUnits;
  uint4 v[kQuantUnits];
  int64_t t[kQuantUnits];
  int k[kQuantUnits];
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    const uint32_t u = first + i;
    t[i] = u / (uint32_t)per_row;
    k[i] = 512 * (int)(u - (uint32_t)t[i] * (uint32_t)per_row) + 8 * lane;
    v[i] = make_uint4(0, 0, 0, 0);
    if (t[i] < T && k[i] < H) v[i] = *reinterpret_cast<const uint4*>(x + t[i] * ld_x + k[i]);
  }
#pragma unroll
  for (int i = 0; i < kQuantUnits; ++i) {
    if (t[i] >= T) return;                  // alike for the wavefront
    uint32_t top = absmax8_bits(v[i]);      // a NaN counts as the largest
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    float inv, f[8];
    const float s = fp8_scale(__uint_as_float(top), inv);
    unpack8(v[i], f);
    if (k[i] < H) {
      *reinterpret_cast<uint2*>(xq + t[i] * ld_q + k[i]) = fp8x8(f, inv, !(s == s));
      if (lane % 16 == 0) xs[(k[i] / kScaleBlock) * ld_s + t[i]] = s;
    }
  }
}

// 16 bytes at k of a row of K bytes, zeros past its end (the load itself is unconditional).
__device__ __forceinline__ v4i load_piece(const uint8_t* row, int k, int K) {
  v4i v = *reinterpret_cast<const v4i*>(row + min(k, K - 16));
  if (k >= K) v = v4i{0, 0, 0, 0};
  return v;
}

// Few tokens, dense: a workgroup of 16 wavefronts owns 16 / Q output columns and 16 / Q tokens and
// splits K over its wavefronts, each feeding the matrix unit from global loads, with the loads of
// several steps in flight; the partial tiles are added through LDS in wavefront order.
//
// Q: with Q > 1 a tile's rows are (column, kq) and its columns (token, kq), where kq < Q says
// which of Q neighbouring blocks of K the row or column carries; the products with equal kq on
// both sides are the sums wanted, the others are not read.  So a tile that few tokens would leave
// mostly empty takes Q blocks of K, and a launch has Q times the workgroups.
// Adds the wavefronts' tiles and stores the workgroup's outputs.
template <int Q>
__device__ __forceinline__ void direct_finish(const Fp8Params& p, v4f acc, int64_t m0, int n0,
                                              v4f* red_s) {
  constexpr int C = 16 / Q;
  const int tid = threadIdx.x, lane = tid & 63;
  red_s[tid] = acc;
  __syncthreads();
  if constexpr (Q == 1) {
    if (tid < 64) {
      v4f s = red_s[lane];
#pragma unroll
      for (int w = 1; w < kFp8Waves; ++w) s += red_s[64 * w + lane];
      if (m0 + (lane & 15) < p.M) fp8_store(p, s, m0 + (lane & 15), n0 + 4 * (lane >> 4));
    }
  } else {
    // Entry e of a wavefront's tile: lane e / 4, element e % 4 -- row 4 (lane / 16) + e % 4, column
    // lane % 16.  One thread per output: its Q entries on the diagonal, wavefront by wavefront.
    const float* red = reinterpret_cast<const float*>(red_s);
    if (tid < C * C) {
      const int col = tid % C, m = tid / C;
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        const int rr = col * Q + k, cc = m * Q + k;
        const int e = 4 * (16 * (rr >> 2) + cc) + (rr & 3);
#pragma unroll
        for (int w = 0; w < kFp8Waves; ++w) s += red[256 * w + e];
      }
      if (m0 + m < p.M && n0 + col < p.N)
        p.out[(m0 + m) * p.ld_out + n0 + col] = (uint16_t)f32x2_to_bf16x2(s, 0.0f);
    }
  }
}

template <int Q, int B>
__global__ __launch_bounds__(64 * kFp8Waves) void fp8_direct_kernel(Fp8Params p) {
  constexpr int C = 16 / Q;
  __shared__ v4f red_s[64 * kFp8Waves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (lane & 15) / Q, kq = lane % Q, g = lane >> 4;
  const int cols = (p.N + C - 1) / C;
  const int64_t m0 = (int64_t)(blockIdx.x / cols) * C;
  const int n0 = (int)(blockIdx.x % cols) * C;
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock;
  const int64_t row = min(m0 + c, (int64_t)p.M - 1);
  const uint8_t* bp = p.b + (int64_t)min(n0 + c, p.N - 1) * p.K;
  const uint8_t* ap = p.a + row * p.ld_a;
  const float* sap = p.sa + row;
  const float* sbp = p.sb + (int64_t)(n0 / kScaleBlock) * KB;
  v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
  for (int base = 0; base < KB; base += kFp8Waves * Q * B) {
    v4i b[B][2], a[B][2];
    float s[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int kb = base + Q * (wave + kFp8Waves * i) + kq, k = kScaleBlock * kb + 16 * g;
      b[i][0] = load_piece(bp, k, p.K);
      b[i][1] = load_piece(bp, k + 64, p.K);
      a[i][0] = load_piece(ap, k, p.K);
      a[i][1] = load_piece(ap, k + 64, p.K);
      // Blocks past the end have no part, whatever scale is read for them.
      const float f = sap[min(kb, KB - 1) * p.ld_sa] * sbp[min(kb, KB - 1)];
      s[i] = kb < KB ? f : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const v4f t = mfma_fp8(b[i][0], b[i][1], a[i][0], a[i][1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(t[e], s[i], acc[e]);
    }
  }
  direct_finish<Q>(p, acc, m0, n0, red_s);
}

// The same from bf16 tokens, in one launch: the workgroup quantises its tokens (16 / Q at most)
// into LDS while its first weight loads are on their way.  U: pieces of 8 elements per thread.
template <int Q, int B, int U>
__global__ __launch_bounds__(64 * kFp8Waves) void fp8_direct_raw_kernel(
    Fp8Params p, const uint16_t* __restrict__ x, int64_t ld_x) {
  constexpr int C = 16 / Q;
  extern __shared__ __attribute__((aligned(16))) uint8_t tok_s[];   // codes, then scales
  __shared__ v4f red_s[64 * kFp8Waves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = (lane & 15) / Q, kq = lane % Q, g = lane >> 4;
  const int cols = (p.N + C - 1) / C;
  const int64_t m0 = (int64_t)(blockIdx.x / cols) * C;
  const int n0 = (int)(blockIdx.x % cols) * C;
  const int M = (int)min((int64_t)C, p.M - m0);
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock, per_row = 16 * KB;
  const int row_s = kScaleBlock * KB + 16;
  float* const scale_s = reinterpret_cast<float*>(tok_s + M * row_s);
  const uint8_t* bp = p.b + (int64_t)min(n0 + c, p.N - 1) * p.K;
  // Tokens before weights: loads come back in order.
  uint4 xv[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int at = tid + 64 * kFp8Waves * i, m = at / per_row, k = 8 * (at - m * per_row);
    xv[i] = *reinterpret_cast<const uint4*>(x + (m0 + min(m, M - 1)) * ld_x + min(k, p.K - 8));
    if (k >= p.K) xv[i] = make_uint4(0, 0, 0, 0);
  }
  asm volatile("" ::: "memory");
  auto block = [&](int i) { return Q * (wave + kFp8Waves * i) + kq; };
  v4i b[B][2];
#pragma unroll
  for (int i = 0; i < B; ++i) {
    b[i][0] = load_piece(bp, kScaleBlock * block(i) + 16 * g, p.K);
    b[i][1] = load_piece(bp, kScaleBlock * block(i) + 16 * g + 64, p.K);
  }
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int at = tid + 64 * kFp8Waves * i, m = at / per_row, q = at - m * per_row;
    // A block is 16 neighbouring lanes, all of them with a token or none.
    uint32_t top = absmax8_bits(xv[i]);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    float inv, f[8];
    const float s = fp8_scale(__uint_as_float(top), inv);
    unpack8(xv[i], f);
    if (m < M) {
      *reinterpret_cast<uint2*>(tok_s + m * row_s + 8 * q) = fp8x8(f, inv, !(s == s));
      if (q % 16 == 0) scale_s[m * KB + q / 16] = s;
    }
  }
  lds_barrier();
  const uint8_t* ap = tok_s + min(c, M - 1) * row_s;
  const float* sap = scale_s + min(c, M - 1) * KB;
  const float* sbp = p.sb + (int64_t)(n0 / kScaleBlock) * KB;
  v4f acc{0.0f, 0.0f, 0.0f, 0.0f};
  for (int base = 0; base < KB; base += kFp8Waves * Q * B) {
    const int after = base + kFp8Waves * Q * B;
    v4i next[B][2];
    if (after < KB) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        next[i][0] = load_piece(bp, kScaleBlock * (after + block(i)) + 16 * g, p.K);
        next[i][1] = load_piece(bp, kScaleBlock * (after + block(i)) + 16 * g + 64, p.K);
      }
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int kb = base + block(i), at = min(kb, KB - 1);
      const v4i lo = *reinterpret_cast<const v4i*>(ap + kScaleBlock * at + 16 * g);
      const v4i hi = *reinterpret_cast<const v4i*>(ap + kScaleBlock * at + 16 * g + 64);
      const float f = kb < KB ? sap[at] * sbp[at] : 0.0f;
      const v4f t = mfma_fp8(b[i][0], b[i][1], lo, hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = fmaf(t[e], f, acc[e]);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      b[i][0] = next[i][0];
      b[i][1] = next[i][1];
    }
  }
  direct_finish<Q>(p, acc, m0, n0, red_s);
}

template <int Q>
int direct_steps(const Fp8Params& p) {
  return (p.K + kScaleBlock * Q * kFp8Waves - 1) / (kScaleBlock * Q * kFp8Waves);
}
// More tokens than a launch takes go in several.
template <int Q>
hipError_t direct(Fp8Params p, hipStream_t stream) {
  constexpr int C = 16 / Q;
  const int steps = direct_steps<Q>(p), cols = (p.N + C - 1) / C;
  const dim3 block(64 * kFp8Waves);
  const int64_t most = C * most_items(64 * kFp8Waves, 1, cols);
  for (int64_t left = p.M; left > 0; left -= p.M) {
    p.M = (int)(left < most ? left : most);
    const dim3 grid((unsigned)((p.M + C - 1) / C * (int64_t)cols));
    if (steps == 1)
      hipLaunchKernelGGL((fp8_direct_kernel<Q, 1>), grid, block, 0, stream, p);
    else if (steps == 2)
      hipLaunchKernelGGL((fp8_direct_kernel<Q, 2>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((fp8_direct_kernel<Q, 4>), grid, block, 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    p.a += p.M * p.ld_a;
    p.sa += p.M;
    p.out += p.M * p.ld_out;
  }
  return hipSuccess;
}

template <int Q, int U>
hipError_t direct_raw(const Fp8Params& p, const uint16_t* x, int64_t ld_x, hipStream_t stream) {
  constexpr int C = 16 / Q;
  const int64_t blocks = (int64_t)((p.M + C - 1) / C) * ((p.N + C - 1) / C);
  // (fp8_raw takes this kernel for a sixtieth of that at most.)
  if (blocks > most_blocks(64 * kFp8Waves)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(64 * kFp8Waves);
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock, M = p.M < C ? p.M : C;
  const size_t lds = (size_t)M * (kScaleBlock * KB + 16 + 4 * KB);
  const int steps = direct_steps<Q>(p);
  if (steps == 1)
    hipLaunchKernelGGL((fp8_direct_raw_kernel<Q, 1, U>), grid, block, lds, stream, p, x, ld_x);
  else if (steps == 2)
    hipLaunchKernelGGL((fp8_direct_raw_kernel<Q, 2, U>), grid, block, lds, stream, p, x, ld_x);
  else
    hipLaunchKernelGGL((fp8_direct_raw_kernel<Q, 4, U>), grid, block, lds, stream, p, x, ld_x);
  return hipGetLastError();
}
template <int Q>
hipError_t direct_raw(const Fp8Params& p, const uint16_t* x, int64_t ld_x, hipStream_t stream) {
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock, M = p.M < 16 / Q ? p.M : 16 / Q;
  return M * KB <= 4 * kFp8Waves ? direct_raw<Q, 1>(p, x, ld_x, stream)
                                 : direct_raw<Q, kRawPieces>(p, x, ld_x, stream);
}

// The simple form, for tokens that 31-bit offsets do not reach: grouped, a wavefront takes tiles of 16
// rows of an expert and kFarCols columns in turn, from global loads; the bytes from the caches to the
// CUs bound it.  (300000 tokens x 8 of 28 experts, 3584 x 7168: 528 ms; 299000 tokens, which the tiled
// kernel reaches, 63.)
constexpr int kFarRows = 16, kFarBlocks = 4, kFarCols = 16 * kFarBlocks;
constexpr int kFarMost = 1 << 18;   // workgroups, which walk over the tiles
__global__ __launch_bounds__(64) void fp8_far_kernel(Fp8Params p) {
  const int lane = threadIdx.x, l = lane & 15, g = lane >> 4, per = (p.E + 63) / 64;
  const int cols = (p.N + kFarCols - 1) / kFarCols;
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock, NB = (p.N + kScaleBlock - 1) / kScaleBlock;
  const Fp8Count c = fp8_count<kFarRows>(p, per);
  const int64_t items = (int64_t)max(__builtin_amdgcn_readlane(c.upto, 63), 0) * cols;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int slot = (int)(it / cols), n0 = (int)(it - (int64_t)slot * cols) * kFarCols;
    const Fp8Found f = fp8_find<kFarRows>(p, per, c, slot);
    const uint32_t in = (uint32_t)slot - (uint32_t)f.before;
    // (As in fp8_grouped_kernel, offsets that overlap may give what is no tile of its expert.)
    if (in >= (uint32_t)fp8_tiles_of<kFarRows>({f.first, f.end})) continue;
    const int64_t m = f.first + (int64_t)in * kFarRows + l, own = m < f.end ? m : f.end - 1;
    int64_t row = own;
    if (p.route) row = min(max(p.route[own] / p.top_k, 0), p.a_rows - 1);
    const uint8_t* ap = p.a + row * p.ld_a;
    const uint8_t* bp[kFarBlocks];
#pragma unroll
    for (int j = 0; j < kFarBlocks; ++j)
      bp[j] = p.b + ((int64_t)f.e * p.N + min(n0 + 16 * j + l, p.N - 1)) * p.K;
    const float* sbp = p.sb + ((int64_t)f.e * NB + n0 / kScaleBlock) * KB;
    v4f acc[kFarBlocks];
#pragma unroll
    for (int j = 0; j < kFarBlocks; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = 0; kb < KB; ++kb) {
      const int k = kScaleBlock * kb + 16 * g;
      const v4i lo = load_piece(ap, k, p.K), hi = load_piece(ap, k + 64, p.K);
      const float s = p.sa[kb * p.ld_sa + row] * sbp[kb];
#pragma unroll
      for (int j = 0; j < kFarBlocks; ++j) {
        const v4f t = mfma_fp8(load_piece(bp[j], k, p.K), load_piece(bp[j], k + 64, p.K), lo, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(t[i], s, acc[j][i]);
      }
    }
    if (m < f.end) {
#pragma unroll
      for (int j = 0; j < kFarBlocks; ++j) fp8_store(p, acc[j], m, n0 + 16 * j + 4 * g);
    }
  }
}

}  // namespace

hipError_t launch_quant_fp8(const uint16_t* x, int64_t ld_x, int T, int H, uint8_t* xq,
                            int64_t ld_q, float* xs, int64_t ld_s, hipStream_t stream) {
  // More tokens than a launch takes go in several (2^27 units of 512 elements in each).
  const int per_row = (H + 511) / 512, per_block = 4 * kQuantUnits;
  const int64_t most = most_items(256, per_block, per_row);
  for (int64_t t = 0; t < T; t += most) {
    const int n = (int)(T - t < most ? T - t : most);
    const int64_t blocks = ((int64_t)n * per_row + per_block - 1) / per_block;
    hipLaunchKernelGGL(quant_fp8_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, x + t * ld_x,
                       ld_x, n, H, per_row, xq + t * ld_q, ld_q, xs + t, ld_s);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

size_t fp8_workspace(int M, int N, int K) {
  return fp8_may_split(M, K) ? sizeof(float) * (size_t)most_partials(M, N) : 0;
}

int fp8_raw_q(int M, int N, int K) { return fp8_raw(M, N, K); }

hipError_t launch_fp8_raw(int q, const Fp8Params& p, const uint16_t* x, int64_t ld_x,
                          hipStream_t stream) {
  switch (q) {
    case 1: return direct_raw<1>(p, x, ld_x, stream);
    case 2: return direct_raw<2>(p, x, ld_x, stream);
    default: return direct_raw<4>(p, x, ld_x, stream);
  }
}

hipError_t launch_fp8(const Fp8Params& p, hipStream_t stream) {
  // The tiled kernel reaches a tile's tokens and all scales by 31-bit offsets; tokens and scales
  // further apart take kernels whose addresses are 64-bit.
  const int64_t KB = (p.K + kScaleBlock - 1) / kScaleBlock, limit = (int64_t)1 << 31;
  const bool near = (p.route ? p.a_rows : 256) * p.ld_a + p.K < limit && 4 * KB * p.ld_sa < limit;
  if (p.offs) {
    if (!near) {
      const int64_t tiles = ((int64_t)p.M / kFarRows + (p.E < p.M ? p.E : p.M)) *
                            ((p.N + kFarCols - 1) / kFarCols);
      const unsigned blocks = (unsigned)(tiles < kFarMost ? tiles : kFarMost);
      hipLaunchKernelGGL(fp8_far_kernel, dim3(blocks), dim3(64), 0, stream, p);
      return hipGetLastError();
    }
    switch (fp8_pick_grouped(p.M, p.E, p.N, p.K)) {
      case 0: return fp8_grouped_launch<4, 2, 4, 8, 2>(p, stream);
      case 1: return fp8_grouped_launch<2, 2, 4, 4, 2>(p, stream);
      case 2: return fp8_grouped_launch<2, 2, 2, 4, 3>(p, stream);
      case 3: return fp8_grouped_launch<2, 2, 2, 2, 4>(p, stream);
      default: return fp8_grouped_launch<2, 2, 1, 2, 4>(p, stream);
    }
  }
  const Fp8Pick k = fp8_pick(p.M, p.N, p.K);
  if (k.variant >= 0 && near) {
    switch (k.variant) {
      case 0: return fp8_tile_launch<4, 2, 4, 8, 2>(p, k.splits, stream);
      case 1: return fp8_tile_launch<2, 2, 4, 4, 2>(p, k.splits, stream);
      case 2: return fp8_tile_launch<2, 2, 2, 4, 3>(p, k.splits, stream);
      case 3: return fp8_tile_launch<2, 2, 2, 2, 4>(p, k.splits, stream);
      default: return fp8_tile_launch<2, 2, 1, 2, 4>(p, k.splits, stream);
    }
  }
  switch (fp8_direct_q(p.M, p.N, p.K)) {
    case 1: return direct<1>(p, stream);
    case 2: return direct<2>(p, stream);
    default: return direct<4>(p, stream);
  }
}

}  // namespace mi355moe
