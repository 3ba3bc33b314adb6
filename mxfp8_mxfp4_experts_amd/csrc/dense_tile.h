// The tiled dense product kernel (see dense.hip for what it computes).
//
// A workgroup of WM x WN wavefronts (tokens x output columns) computes a
// 16 MI WM x 16 NI WN tile of C, each wavefront MI x NI accumulators of 16x16.
// K advances in stages of 128 bytes per row (one cache line), read by direct
// global-to-LDS loads into a ring of NBUF stages.  A stage is two
// matrix-instruction steps of 64 bytes:
//
//   step 0: the MFMAs of the first half, while the second half's operands
//           come from LDS;
//   wait for the own loads of the next stage, barrier: every wavefront has
//           now read all of this stage, so its buffer is free, and the next
//           stage is complete;
//   step 1: the MFMAs of the second half, while the loads of the stage NBUF
//           ahead go into the freed buffer and the next stage's first operands
//           come from LDS.
//
// So there is one barrier per stage, and the matrix unit has operands in
// registers on both sides of it.  LDS rows are 128 bytes with their 16-byte
// chunks XOR-swizzled by the row's low three bits: the eight lanes that LDS
// serves together read eight different bank groups, and the direct loads,
// whose LDS side is lane order, get the same order from their addresses.
//
// Rows past M or N, chunks past K and stages past the last are loads beyond
// the buffer's end: they bring zeros, touch no memory and still count.
//
// Measured (least and median of 60 launches under a trace, which the large ones
// feel): INT8 8192 x 3584 x 7168 in 256 x 224 tiles 176 - 188 us (2.2 - 2.4 POP/s;
// the matrix unit is busy 58% of the cycles at a clock that the power limit holds
// at 2.0 GHz); BF16 8192 x 896 x 7168 in 128 x 224 tiles 110 - 118 us, 100 in calls
// back to back (1.06 PFLOP/s; what bounds it is open: 1.3 GB out of the L2s is 51
// bytes/ns per CU, less than smaller tiles draw); INT8 256 x 3584 x 7168 in 64 x 64
// tiles 14.3 - 15.9 us; BF16 256 x 896 x 7168 with K in four 9.6 - 10.0 us and its
// join 2.2 - 2.7: the latter two take 60 - 85 bytes/ns per CU from L2, which bounds
// them.
#pragma once

#include "dense.h"
#include "dense_pick.h"

namespace mi355moe {

constexpr uint32_t kPastEnd = 0x80000000u;      // beyond every buffer (they are below 2^31 bytes)

typedef __attribute__((address_space(3))) uint8_t dense_lds_t;
typedef __attribute__((address_space(3))) v4i dense_lds_v4i;

// How a launch is cut: tiles, and K over `splits` workgroups.
struct DenseCut {
  int tiles_m, tiles_n, splits, stages_per_split;
};

template <class T, int WM, int WN, int MI, int NI, int NBUF>
__device__ __forceinline__ void dense_tile_body(const DenseParams& p, const DenseCut& cut) {
  using Acc = typename T::Acc;
  constexpr int W = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  // 1 KB loads (8 rows) per wavefront and stage; where a tile's rows do not
  // share out evenly the last loads bring zeros into rows that nobody reads.
  constexpr int PA = (BM / 8 + W - 1) / W, PB = (BN / 8 + W - 1) / W;
  constexpr int kOffB = PA * W * 1024, kStage = kOffB + PB * W * 1024;
  constexpr int kLoads = PA + PB, kReads = MI + NI;
  static_assert((NBUF - 1) * kLoads < 64, "vmcnt");
  constexpr int kScales = NBUF * kStage;           // then the tile's scales: BM, BN floats
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kScales + (T::kInt ? 4 * (BM + BN) : 0)];
  dense_lds_t* const lds_base = (dense_lds_t*)lds;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int r = lane & 15, g = lane >> 4;

  // Tile and split of this workgroup.  Workgroups go to the 8 XCDs in turn; each
  // XCD takes a contiguous range of them, split by split, a split's tiles in
  // blocks of up to 8 tile rows walked column by column, so what is in flight on
  // one XCD shares a range of K and rows of A and B in its L2 (BF16 256 x 896 x
  // 7168: 10.8 us with the splits spread over the XCDs, 9.6 so).
  const int n_tiles = cut.tiles_m * cut.tiles_n;
  int tile, split = 0;
  {
    const int n = n_tiles * cut.splits, b = blockIdx.x, x = b & 7, q = n >> 3, rest = n & 7;
    tile = x * q + min(x, rest) + (b >> 3);
    if (cut.splits > 1) {
      split = tile / n_tiles;
      tile -= split * n_tiles;
    }
  }
  const int blk = tile / (8 * cut.tiles_n);
  const int rows_in = min(8, cut.tiles_m - 8 * blk);
  const int in_blk = tile - blk * 8 * cut.tiles_n;
  const int tn = in_blk / rows_in, tm = 8 * blk + in_blk - tn * rows_in;
  const int m0 = tm * BM, n0 = tn * BN;
  const int s0 = split * cut.stages_per_split;
  const int n_all = (p.Kb + kStageK - 1) / kStageK;
  const int s1 = min(n_all, s0 + cut.stages_per_split);
  const int k_end = min(p.Kb, s1 * kStageK);

  const int rows_a = min(BM, p.M - m0), rows_b = min(BN, p.N - n0);
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.a) + (int64_t)m0 * p.ld_a, 0,
      (uint32_t)((rows_a - 1) * p.ld_a + p.Kb), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.b) + (int64_t)n0 * p.ld_b, 0,
      (uint32_t)((rows_b - 1) * p.ld_b + p.Kb), 0x00020000);

  // Load q of a stage: 8 rows x 128 bytes.  Row and chunk of this lane; the
  // chunk is the same for every q.
  const int lrow = lane >> 3, chunk = (lane & 7) ^ lrow;
  uint32_t va[PA], vb[PB];
#pragma unroll
  for (int q = 0; q < PA; ++q) {
    const int row = 8 * (PA * wave + q) + lrow;
    va[q] = row < rows_a ? (uint32_t)(row * p.ld_a) + 16 * chunk : kPastEnd;
  }
#pragma unroll
  for (int q = 0; q < PB; ++q) {
    const int row = 8 * (PB * wave + q) + lrow;
    vb[q] = row < rows_b ? (uint32_t)(row * p.ld_b) + 16 * chunk : kPastEnd;
  }
  auto in_k = [&](int s) { return kStageK * s + 16 * chunk < k_end; };
  // The scalar offset stays inside the buffer also past the last stage, so that
  // what lies beyond the end is told by the lane's offset alone.
  auto issue = [&](int q, int s, int buf, bool in) __attribute__((always_inline)) {
    uint8_t* base = lds + buf * kStage;
    s = min(s, n_all - 1);
    if (q < PA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, base + 1024 * (PA * wave + q), 16,
                                               in ? va[q] : kPastEnd, kStageK * s, 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, base + kOffB + 1024 * (PB * wave + q - PA), 16, in ? vb[q - PA] : kPastEnd,
          kStageK * s, 0, 0);
  };

  // The epilogue's scales, fetched before the loop so that their way from memory
  // is not at the end: into registers where there is room, else into LDS (the
  // loop's barriers lie between these writes and the epilogue's reads).
  const int m_w = m0 + 16 * MI * wm + r, n_w = n0 + 16 * NI * wn + 4 * g;
  constexpr bool kEarly = MI * NI <= 16;
  float* const scales = reinterpret_cast<float*>(lds + kScales);
  float sx[MI], sw[NI][4];
  if constexpr (T::kInt && kEarly) {
#pragma unroll
    for (int i = 0; i < MI; ++i) sx[i] = p.sx[min(m_w + 16 * i, p.M - 1)];
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) sw[j][e] = p.sw[min(n_w + 16 * j + e, p.N - 1)];
  }
  if constexpr (T::kInt && !kEarly) {
    for (int i = threadIdx.x; i < BM + BN; i += 64 * W)
      scales[i] = i < BM ? p.sx[min(m0 + i, p.M - 1)] : p.sw[min(n0 + i - BM, p.N - 1)];
  }
  auto scales_of = [&](int j) __attribute__((always_inline)) {
    if constexpr (T::kInt && !kEarly) {
      const float4 v = *reinterpret_cast<const float4*>(scales + BM + 16 * NI * wn + 16 * j + 4 * g);
      sw[j][0] = v.x;
      sw[j][1] = v.y;
      sw[j][2] = v.z;
      sw[j][3] = v.w;
    }
  };

  Acc acc[MI][NI];
  auto value = [&](int i, int j, int e) __attribute__((always_inline)) {
    float f = (float)acc[i][j][e];
    if constexpr (T::kInt) f = f * sx[i] * sw[j][e];
    return f;
  };
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      acc[i][j] = Acc{0, 0, 0, 0};
      asm volatile("" : "+a"(acc[i][j]));   // accumulation registers from the start
    }
  v4i fa[2][MI], fb[2][NI];
  // LDS offsets of this lane's operands within a stage; step 1 flips bit 6.
  const int oa = (16 * MI * wm + r) * kStageK + 16 * (g ^ (r & 7));
  const int ob = kOffB + (16 * NI * wn + r) * kStageK + 16 * (g ^ (r & 7));
  auto stage = [&](int buf) __attribute__((always_inline)) {
    int off = buf * kStage;
    asm volatile("" : "+s"(off));    // opaque: keeps the reads from being moved across stages
    return static_cast<const dense_lds_t*>(lds_base) + off;
  };
  auto read = [&](const dense_lds_t* S, int kk, int q) __attribute__((always_inline)) {
    if (q < NI)
      fb[kk][q] = *reinterpret_cast<const dense_lds_v4i*>(S + (ob ^ (64 * kk)) + 2048 * q);
    else
      fa[kk][q - NI] =
          *reinterpret_cast<const dense_lds_v4i*>(S + (oa ^ (64 * kk)) + 2048 * (q - NI));
  };
  auto mfmas = [&](int kk) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = T::mfma(fb[kk][j], fa[kk][i], acc[i][j]);
  };

#pragma unroll
  for (int b = 0; b < NBUF; ++b) {
#pragma unroll
    for (int q = 0; q < kLoads; ++q) issue(q, s0 + b, b, in_k(s0 + b));
    asm volatile("" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NBUF - 1) * kLoads) : "memory");
  asm volatile("s_barrier" ::: "memory");
  {
    const dense_lds_t* S = stage(0);
#pragma unroll
    for (int q = 0; q < kReads; ++q) read(S, 0, q);
  }
  int buf = 0;
  for (int s = s0; s < s1; ++s) {
    const dense_lds_t* S = stage(buf);
#pragma unroll
    for (int q = 0; q < kReads; ++q) read(S, 1, q);
    mfmas(0);
    // one LDS read after every second MFMA, the rest of the MFMAs cover the last reads
#pragma unroll
    for (int q = 0; q < kReads; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, MI * NI >= 2 * kReads ? 2 : 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);   // the wait stays behind the step's MFMAs
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 2) * kLoads) : "memory");
    asm volatile("s_barrier" ::: "memory");
    const int nbuf = buf + 1 == NBUF ? 0 : buf + 1;
    const dense_lds_t* S1 = stage(nbuf);
    const bool in = in_k(s + NBUF);
#pragma unroll
    for (int q = 0; q < (kLoads > kReads ? kLoads : kReads); ++q) {
      if (q < kLoads) issue(q, s + NBUF, buf, in);
      if (q < kReads) read(S1, 0, q);
    }
    mfmas(1);
#pragma unroll
    for (int q = 0; q < (kLoads > kReads ? kLoads : kReads); ++q) {
      if (q < kLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      if (q < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, MI * NI >= 2 * kReads ? 2 : 1, 0);
    }
    asm volatile("" ::: "memory");
    buf = nbuf;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the loads past the last stage

  if (cut.splits > 1) {
    // Partial sums [split][M][N rounded up to 4].
    const int64_t ldp = (p.N + 3) & ~3;
    Acc* part = static_cast<Acc*>(p.partial) + (int64_t)split * p.M * (ldp / 4);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int m = m_w + 16 * i, n = n_w + 16 * j;
        if (m < p.M && n < p.N) part[(m * ldp + n) / 4] = acc[i][j];
      }
    return;
  }
  if constexpr (T::kInt && !kEarly) {
#pragma unroll
    for (int i = 0; i < MI; ++i) sx[i] = scales[16 * MI * wm + r + 16 * i];
  }
  if (m0 + BM <= p.M && n0 + BN <= p.N && p.out_vec) {
    // A whole tile: one address per row block, no checks.
    if (p.out_f32) {
      float* o = static_cast<float*>(p.out) + (int64_t)m_w * p.ld_out + n_w;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        scales_of(j);
#pragma unroll
        for (int i = 0; i < MI; ++i)
          *reinterpret_cast<float4*>(o + 16 * i * p.ld_out + 16 * j) =
              make_float4(value(i, j, 0), value(i, j, 1), value(i, j, 2), value(i, j, 3));
      }
    } else {
      uint16_t* o = static_cast<uint16_t*>(p.out) + (int64_t)m_w * p.ld_out + n_w;
      auto pack = [&](int i, int j) __attribute__((always_inline)) {
        return make_uint2(f32x2_to_bf16x2(value(i, j, 0), value(i, j, 1)),
                          f32x2_to_bf16x2(value(i, j, 2), value(i, j, 3)));
      };
      // Two column blocks at a time: swapping the odd 16-lane rows of the first
      // with the even rows of the second leaves every lane 8 neighbouring
      // columns, block j in the even rows and j + 1 in the odd ones -- 64 bytes
      // of a token's row per store instead of 32.
      int j = 0;
      if constexpr (NI > 1) {
        if ((p.ld_out & 7) == 0) {
          uint16_t* o2 = o - 4 * g + 16 * (g & 1) + 8 * (g >> 1);
#pragma unroll
          for (; j + 1 < NI; j += 2) {
            scales_of(j);
            scales_of(j + 1);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
              const uint2 u = pack(i, j), v = pack(i, j + 1);
              const auto x = __builtin_amdgcn_permlane16_swap(u.x, v.x, false, false);
              const auto y = __builtin_amdgcn_permlane16_swap(u.y, v.y, false, false);
              *reinterpret_cast<uint4*>(o2 + 16 * i * p.ld_out + 16 * j) =
                  make_uint4(x[0], y[0], x[1], y[1]);
            }
          }
        }
      }
#pragma unroll
      for (int jj = 0; jj < NI; ++jj) {
        if (jj < j) continue;
        scales_of(jj);
#pragma unroll
        for (int i = 0; i < MI; ++i)
          *reinterpret_cast<uint2*>(o + 16 * i * p.ld_out + 16 * jj) = pack(i, jj);
      }
    }
    return;
  }
  // A tile at an edge, or rows that take no vector stores: through LDS (each
  // wavefront its own part, 16 rows at a time), so that a store instruction
  // writes neighbouring elements of a row.
  asm volatile("s_barrier" ::: "memory");   // the ring is no longer read
  constexpr int kRow = 16 * NI + 4;         // floats; the pad spreads the rows over the banks
  static_assert(W * 16 * kRow * 4 <= NBUF * kStage, "epilogue rows fit in the ring");
  float* rows = reinterpret_cast<float*>(lds) + wave * 16 * kRow;
  const int m_b = m0 + 16 * MI * wm, n_b = n0 + 16 * NI * wn;
  // A store instruction covers kRows rows (narrow tiles) or 64 columns of one.
  constexpr int kRows = NI < 4 ? 4 / NI : 1, kColSteps = (16 * NI + 63) / 64;
  const int row0 = NI < 4 ? lane / (16 * NI) : 0, col0 = NI < 4 ? lane % (16 * NI) : lane;
#pragma unroll
  for (int j = 0; j < NI; ++j) scales_of(j);
  for (int i = 0; i < MI; ++i) {
    v4f f[NI];
#pragma unroll
    for (int ii = 0; ii < MI; ++ii)
      if (ii == i) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) f[j][e] = value(ii, j, e);
      }
#pragma unroll
    for (int j = 0; j < NI; ++j)
      *reinterpret_cast<v4f*>(rows + r * kRow + 16 * j + 4 * g) = f[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 4
    for (int row = row0; row < 16; row += kRows) {
      const int m = m_b + 16 * i + row;
      if (m >= p.M) continue;
      const int64_t o = (int64_t)m * p.ld_out + n_b;
#pragma unroll
      for (int c = 0; c < kColSteps; ++c) {
        const int col = col0 + 64 * c;
        if (col < 16 * NI && n_b + col < p.N) {
          const float v = rows[row * kRow + col];
          if (p.out_f32)
            static_cast<float*>(p.out)[o + col] = v;
          else
            static_cast<uint16_t*>(p.out)[o + col] = (uint16_t)f32x2_to_bf16x2(v, 0.0f);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

template <class T, int WM, int WN, int MI, int NI, int NBUF, int WPE>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void dense_tile_kernel(DenseParams p, DenseCut cut) {
  dense_tile_body<T, WM, WN, MI, NI, NBUF>(p, cut);
}

// The splits' partial sums, added in split order.
template <class T>
__global__ __launch_bounds__(256) void dense_join_kernel(DenseParams p, int splits) {
  using Acc = typename T::Acc;
  const int per_row = (p.N + 3) / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t total = (int64_t)p.M * per_row;
  if (at >= total) return;
  const int m = (int)(at / per_row), n = 4 * (int)(at - (int64_t)m * per_row);
  const DenseScales sc = dense_scales<T>(p, m, n);
  const Acc* part = static_cast<const Acc*>(p.partial) + at;
  Acc s = part[0];
#pragma unroll 4
  for (int z = 1; z < splits; ++z) s += part[z * total];
  dense_store<T>(p, s, sc, m, n);
}

template <class T, int WM, int WN, int MI, int NI, int NBUF, int WPE>
hipError_t dense_tile_launch(const DenseParams& p, int splits, hipStream_t stream) {
  DenseCut cut;
  constexpr int BM = 16 * MI * WM, BN = 16 * NI * WN;
  cut.tiles_m = (p.M + BM - 1) / BM;
  cut.tiles_n = (p.N + BN - 1) / BN;
  const int n_all = (p.Kb + kStageK - 1) / kStageK;
  cut.stages_per_split = (n_all + splits - 1) / splits;
  cut.splits = (n_all + cut.stages_per_split - 1) / cut.stages_per_split;
  hipLaunchKernelGGL((dense_tile_kernel<T, WM, WN, MI, NI, NBUF, WPE>),
                     dim3(cut.tiles_m * cut.tiles_n * cut.splits), dim3(64 * WM * WN), 0, stream,
                     p, cut);
  if (cut.splits > 1) {
    const int64_t pieces = (int64_t)p.M * ((p.N + 3) / 4);
    hipLaunchKernelGGL((dense_join_kernel<T>), dim3((unsigned)((pieces + 255) / 256)), dim3(256),
                       0, stream, p, cut.splits);
  }
  return hipGetLastError();
}

}  // namespace mi355moe
