// The tiled block-scaled FP8 product (fp8.hip says what it computes).
//
// A workgroup of WM x WN wavefronts (tokens x output columns) computes a
// 16 MI WM x 16 NI WN tile, each wavefront MI x NI accumulators of 16x16.  K advances in stages
// of 128 bytes per row: one cache line, one scale block, one v_mfma_f32_16x16x128_f8f6f4 per
// accumulator, which starts from zero; the vector unit adds its result times the block's scale
// to the running sum, while the matrix unit works on the next column of accumulators.  Such a
// product takes the matrix unit 32 clocks and an issue slot of the vector unit half of that; its
// four multiply-adds just fit beside it, each further vector instruction costs 4 clocks.  So the
// sums are vector registers (to move them costs more than to add), and a wavefront has at most
// MI * NI = 32 of them, two wavefronts to a SIMD.
//
// Stages come by direct global-to-LDS loads into a ring of NBUF, the tokens' scales in a ring of
// their own, four stages at a time (4 bytes per token, ordered so that a lane reads its MI scales
// at once); the weight's scales of 64 stages sit in one register, a lane each.  From there a
// small tile's operands go to registers a whole stage ahead of their products (kFull), a large
// tile's column by column, with a barrier where the tokens' and where the weights' buffer is read
// to its end: it is loaded anew from there on.
//
// LDS rows are 128 bytes with their 16-byte chunks XOR-swizzled by the row's low three bits.
// Rows past the tile's last, chunks past K and stages past the last are loads beyond the buffer's
// end: they bring zeros and touch no memory.
//
// What bounds it (back to back in a graph; a traced dispatch reads up to 10% longer): 8192 x 3584 x
// 7168 in 256 x 256 tiles 178 .. 189 us, 2.2 .. 2.4 POP/s, the matrix unit (224 us with 128 x 128
// tiles, 340 with 64 x 64); 256 x 3584 x 7168 in 64 x 64 tiles 17.7 us, 205 MB from the L2s to the CUs
// at 60 .. 70 bytes/ns per CU (19.1 with 64 x 128 tiles and K in two, 21.3 with 128 x 128 in four).
// Deeper rings, two stages per barrier, weights laid out by K and prefetches into L2 gained
// nothing; with 224 columns a tile, a wavefront's columns meet two scales and each product needs
// a multiplication more, which took what the better fit of 3584 columns gave.
#pragma once

#include "fp8.h"
#include "fp8_pick.h"

namespace mi355moe {

constexpr uint32_t kFp8PastEnd = 0x80000000u;   // beyond every buffer (they are below 2^31 bytes)

typedef __attribute__((address_space(3))) uint8_t fp8_lds_t;
typedef __attribute__((address_space(3))) v4i fp8_lds_v4i;

// How a launch is cut: output columns in tiles_n; dense: rows in tiles_m, K over `splits`
// workgroups; grouped: the rows' tiles are counted on the GPU and shared out over the grid.
struct Fp8Cut {
  int tiles_m, tiles_n, splits, stages_per_split;
};

// One tile: rows [m0, m1) (at most BM), columns from n0, stages [s0, s1).
struct Fp8Tile {
  int64_t m0, m1;
  int n0, s0, s1, split, expert;
};

template <int WM, int WN, int MI, int NI, int NBUF>
struct Fp8Geom {
  static constexpr int W = WM * WN, BM = 16 * MI * WM, BN = 16 * NI * WN;
  // 1 KB loads (8 rows) per wavefront and stage.
  static constexpr int PA = BM / 8 / W, PB = BN / 8 / W;
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0, "loads share out evenly");
  // The tokens' scales come for kGroup stages at a time, 64 of them a load (a load per wavefront
  // in every stage took 11% of a 64 x 64 product's time); where the loads do not share out evenly the
  // last ones are done twice.
  static constexpr int kGroup = 4, kTokS = kGroup * BM / 64, PS = (kTokS + W - 1) / W;
  // Rings: NBUF stages of tokens, NBUF of weights, 3 groups of scales.
  static constexpr int kStageA = BM * 128, kStageB = BN * 128;
  static constexpr int kOffB = NBUF * kStageA, kOffS = kOffB + NBUF * kStageB;
  static constexpr int kScales = 3 * kGroup;
  static constexpr int kLds = kOffS + kScales * BM * 4;
  // Room for two stages' operands in registers.
  static constexpr bool kFull = 16 * (MI + NI) + 4 * MI * NI <= 144;
};

template <int WM, int WN, int MI, int NI, int NBUF, bool GROUPED>
__device__ __forceinline__ void fp8_tile_body(const Fp8Params& p, const Fp8Cut& cut,
                                              const Fp8Tile& t, uint8_t* lds) {
  using G = Fp8Geom<WM, WN, MI, NI, NBUF>;
  constexpr int BM = G::BM, BN = G::BN, PA = G::PA, PB = G::PB, PS = G::PS;
  static_assert((NBUF - 1) * (PA + PB) < 64, "vmcnt");
  static_assert(kScaleBlock % (16 * NI) == 0, "a wavefront's columns share their scales");
  fp8_lds_t* const lds_base = (fp8_lds_t*)lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // Wavefronts of the same tokens side by side: they are on different SIMDs, and of 8 the second
  // four have the tile's second half of tokens, so a tile of half its rows leaves no SIMD idle.
  const int wm = wave / WN, wn = wave % WN;
  const int r = lane & 15, g = lane >> 4;
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock;
  const int k_end = min(p.K, t.s1 * kScaleBlock);
  const int rows_a = (int)min((int64_t)BM, t.m1 - t.m0), rows_b = min(BN, p.N - t.n0);
  const bool gather = GROUPED && p.route != nullptr;

  const uint8_t* const a0 = gather ? p.a : p.a + t.m0 * p.ld_a;
  const uint32_t a_bytes =
      gather ? (uint32_t)((int64_t)(p.a_rows - 1) * p.ld_a + p.K)
             : (uint32_t)((int64_t)(rows_a - 1) * p.ld_a + p.K);
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a0), 0, a_bytes, 0x00020000);
  const uint8_t* const b0 = p.b + ((int64_t)t.expert * p.N + t.n0) * p.K;
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(b0), 0, (uint32_t)((int64_t)(rows_b - 1) * p.K + p.K), 0x00020000);
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(p.sa), 0, (uint32_t)(((int64_t)(KB - 1) * p.ld_sa + p.a_rows) * 4),
      0x00020000);

  // Row (of the tokens) that tile row i reads.
  auto token = [&](int i) __attribute__((always_inline)) {
    const int64_t m = t.m0 + min(i, rows_a - 1);
    if (!gather) return (int)m;
    return min(max(p.route[m] / p.top_k, 0), p.a_rows - 1);
  };
  const int lrow = lane >> 3, chunk = (lane & 7) ^ lrow;
  uint32_t va[PA], vb[PB], vs[PS];
#pragma unroll
  for (int q = 0; q < PA; ++q) {
    const int row = 8 * (PA * wave + q) + lrow;
    const int64_t at = gather ? (int64_t)token(row) : row;
    va[q] = row < rows_a ? (uint32_t)(at * p.ld_a) + 16 * chunk : kFp8PastEnd;
  }
#pragma unroll
  for (int q = 0; q < PB; ++q) {
    const int row = 8 * (PB * wave + q) + lrow;
    vb[q] = row < rows_b ? (uint32_t)(row * p.K) + 16 * chunk : kFp8PastEnd;
  }
#pragma unroll
  for (int q = 0; q < PS; ++q) {
    // Place 16 MI w + MI r + i of a stage's scales holds row 16 MI w + 16 i + r.
    const int at = (64 * min(PS * wave + q, G::kTokS - 1) + lane) % BM;
    const int w = at / (16 * MI), rem = at - 16 * MI * w;
    vs[q] = 4 * (uint32_t)token(16 * MI * w + 16 * (rem % MI) + rem / MI);
  }
  // Scales of the stages from s on, into the group's place in the ring.
  auto issue_s = [&](int s, int group) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < PS; ++q) {
      const int at = 64 * min(PS * wave + q, G::kTokS - 1);
      const int kb = min(s + (at + lane) / BM, KB - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, lds + G::kOffS + 4 * (BM * G::kGroup * group + at), 4,
          vs[q] + (uint32_t)kb * (uint32_t)(4 * p.ld_sa), 0, 0, 0);
    }
  };
  // From the stage that K ends in on, lanes past the end load beyond their buffer, for good (a
  // select per load and stage would cost as much as the products leave of the vector unit).
  const int s_last = p.K % kScaleBlock != 0 && t.s1 == KB ? KB - 1 : t.s1;
  auto cut_off = [&](int s) __attribute__((always_inline)) {
    if (s < s_last) return;
    const bool in = kScaleBlock * s + 16 * chunk < k_end;
#pragma unroll
    for (int q = 0; q < PA; ++q) va[q] = in ? va[q] : kFp8PastEnd;
#pragma unroll
    for (int q = 0; q < PB; ++q) vb[q] = in ? vb[q] : kFp8PastEnd;
  };
  auto issue_a = [&](int q, int s, int buf) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        ra, lds + buf * G::kStageA + 1024 * (PA * wave + q), 16, va[q],
        kScaleBlock * min(s, KB - 1), 0, 0);
  };
  auto issue_b = [&](int q, int s, int buf) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rb, lds + G::kOffB + buf * G::kStageB + 1024 * (PB * wave + q), 16, vb[q],
        kScaleBlock * min(s, KB - 1), 0, 0);
  };

  // The weight's scales: lane l has those of stage (s0 + 64 n) + l.
  const int n_wave = t.n0 + 16 * NI * wn;
  const int n_blocks = (p.N + kScaleBlock - 1) / kScaleBlock;
  float vsb;
  auto load_sb = [&](int s) __attribute__((always_inline)) {
    vsb = p.sb[((int64_t)t.expert * n_blocks + min(n_wave / kScaleBlock, n_blocks - 1)) * KB +
               min(s + lane, KB - 1)];
  };
  load_sb(t.s0);

  v4f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int oa = (16 * MI * wm + r) * kScaleBlock + 16 * (g ^ (r & 7));
  const int ob = G::kOffB + (16 * NI * wn + r) * kScaleBlock + 16 * (g ^ (r & 7));
  const int os = G::kOffS + 4 * MI * (16 * wm + r);
  auto at_lds = [&](int off) __attribute__((always_inline)) {
    asm volatile("" : "+s"(off));    // opaque: keeps the reads from being moved across stages
    return static_cast<const fp8_lds_t*>(lds_base) + off;
  };
  struct Op {
    v4i lo, hi;
  };
  auto read_a = [&](const fp8_lds_t* S, int i) __attribute__((always_inline)) {
    return Op{*reinterpret_cast<const fp8_lds_v4i*>(S + oa + 2048 * i),
              *reinterpret_cast<const fp8_lds_v4i*>(S + (oa ^ 64) + 2048 * i)};
  };
  auto read_b = [&](const fp8_lds_t* S, int j) __attribute__((always_inline)) {
    return Op{*reinterpret_cast<const fp8_lds_v4i*>(S + ob + 2048 * j),
              *reinterpret_cast<const fp8_lds_v4i*>(S + (ob ^ 64) + 2048 * j)};
  };
  typedef float vMI __attribute__((ext_vector_type(MI < 2 ? 2 : MI)));
  typedef __attribute__((address_space(3))) float lds_f;
  auto read_s = [&](const fp8_lds_t* S, float (&sa)[MI]) __attribute__((always_inline)) {
    if constexpr (MI == 1) {
      sa[0] = *reinterpret_cast<const lds_f*>(S + os);
    } else {
      typedef __attribute__((address_space(3))) vMI lds_vMI;
      const vMI v = *reinterpret_cast<const lds_vMI*>(S + os);
#pragma unroll
      for (int i = 0; i < MI; ++i) sa[i] = v[i];
    }
  };

  issue_s(t.s0, 0);
  issue_s(t.s0 + G::kGroup, 1);
#pragma unroll
  for (int v = 0; v < NBUF; ++v) {
    cut_off(t.s0 + v);
#pragma unroll
    for (int q = 0; q < PA; ++q) issue_a(q, t.s0 + v, v);
#pragma unroll
    for (int q = 0; q < PB; ++q) issue_b(q, t.s0 + v, v);
    asm volatile("" ::: "memory");
  }
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NBUF - 1) * (PA + PB)) : "memory");
  asm volatile("s_barrier" ::: "memory");
  // A column's products are added behind the next column's, the last column's behind the next
  // stage's first; `f` is then what they are scaled by.
  v4f prod[MI];
  float f[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    prod[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    f[i] = 0.0f;
  }
  auto add = [&](int i, int j) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(prod[i][e], f[i], acc[i][j][e]);
  };
  int buf = 0;
  int place = 0;                    // of this stage's scales in their ring
  auto next_place = [&]() { place = place + 1 == G::kScales ? 0 : place + 1; };
  // Every kGroup stages the scales of the group after the next: they are older than the loads
  // that the barriers before their use wait for.
  auto more_scales = [&](int s, int at) __attribute__((always_inline)) {
    if (at % G::kGroup == 0) {
      const int group = place / G::kGroup + 2;
      issue_s(s + 2 * G::kGroup, group >= 3 ? group - 3 : group);
    }
  };
  static_assert(NBUF <= G::kGroup + 1, "scales are loaded early enough");
  if constexpr (G::kFull) {
    // Two sets of a whole stage's operands in registers: one is multiplied while the other comes
    // from LDS.  A stage's buffer is free as soon as all wavefronts have read it, a stage before
    // its products, and neither LDS nor the barrier is waited for behind them.
    struct Set {
      Op a[MI], b[NI];
      float s[MI];
    } one, two;
    auto read_set = [&](const fp8_lds_t* A, const fp8_lds_t* B, const fp8_lds_t* C, Set& o)
        __attribute__((always_inline)) {
      o.b[0] = read_b(B, 0);
#pragma unroll
      for (int i = 0; i < MI; ++i) o.a[i] = read_a(A, i);
#pragma unroll
      for (int j = 1; j < NI; ++j) o.b[j] = read_b(B, j);
      read_s(C, o.s);
    };
    auto step = [&](int s, int at, const Set& o, Set& next) __attribute__((always_inline)) {
      const float sb = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vsb), at));
      const int nbuf = buf + 1 == NBUF ? 0 : buf + 1;
      cut_off(s + NBUF);
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 2) * (PA + PB)) : "memory");
      asm volatile("s_barrier" ::: "memory");
      more_scales(s, at);
      next_place();
      read_set(at_lds(nbuf * G::kStageA), at_lds(nbuf * G::kStageB), at_lds(place * BM * 4), next);
#pragma unroll
      for (int q = 0; q < PA; ++q) issue_a(q, s + NBUF, buf);
#pragma unroll
      for (int q = 0; q < PB; ++q) issue_b(q, s + NBUF, buf);
#pragma unroll
      for (int j = 0; j < NI; ++j) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          add(i, (j + NI - 1) % NI);
          if (j == 0) f[i] = o.s[i] * sb;
          prod[i] = mfma_fp8(o.b[j].lo, o.b[j].hi, o.a[i].lo, o.a[i].hi);
        }
      }
#pragma unroll
      for (int q = 0; q < MI * NI; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
      }
      asm volatile("" ::: "memory");
      buf = nbuf;
    };
    read_set(at_lds(0), at_lds(0), at_lds(0), one);
    // 64 stages at a time: see below.
    for (int c0 = t.s0; c0 < t.s1; c0 += 64) {
      if (c0 > t.s0) load_sb(c0);
      asm volatile("" : "+v"(vsb));
      const int n = min(t.s1 - c0, 64);
#pragma unroll 1
      for (int at = 0; at + 1 < n; at += 2) {
        step(c0 + at, at, one, two);
        step(c0 + at + 1, at + 1, two, one);
      }
      if (n & 1) step(c0 + n - 1, n - 1, one, two);   // the last of all: 64 is even
    }
  } else {
    // Weight operands in registers: the current column's and the next two, in a ring that comes out
    // even with the columns.
    constexpr int F = 4;
    static_assert(NI % F == 0, "a stage's first column is in the ring's first place");
    Op fa[MI], fb[F];
    float fs[MI];                     // the tokens' scales
    {
      const fp8_lds_t *A = at_lds(0), *B = at_lds(0);
      fb[0] = read_b(B, 0);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = read_a(A, i);
      read_s(at_lds(0), fs);
    }
    // Barrier JB is before the last two columns: by then their operands are in registers, so this
    // stage's weights are no longer needed in LDS, and the next stage is complete.  The tokens'
    // operands are in registers from the stage's start, so where there are columns enough a barrier
    // of their own, JA, frees the tokens' buffer almost a stage earlier: their loads and the
    // weights' then take turns, and each has about a stage's time to come.
    constexpr int JB = NI - 2;
    constexpr int JA = NI == 8 ? 1 : JB;
    constexpr int kBehind = JA < JB ? PA : 0;   // loads behind those that JB waits for
    if (16 * MI * wm >= rows_a) {
      // A wavefront without rows only loads its share: the matrix unit is left to the others.
      // (16384 x 3584 x 3584 in 28 experts, 585 rows each: 255 -> 241 us.)
      for (int s = t.s0; s < t.s1; ++s) {
        const int next = buf + 1 == NBUF ? 0 : buf + 1;
        cut_off(s + NBUF);
        if constexpr (JA < JB) {
          asm volatile("s_barrier" ::: "memory");
          more_scales(s, s - t.s0);
#pragma unroll
          for (int q = 0; q < PA; ++q) issue_a(q, s + NBUF, buf);
        }
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 2) * (PA + PB) + kBehind)
                     : "memory");
        asm volatile("s_barrier" ::: "memory");
        if constexpr (JA == JB) {
          more_scales(s, s - t.s0);
#pragma unroll
          for (int q = 0; q < PA; ++q) issue_a(q, s + NBUF, buf);
        }
#pragma unroll
        for (int q = 0; q < PB; ++q) issue_b(q, s + NBUF, buf);
        next_place();
        buf = next;
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      return;
    }
    // 64 stages at a time: the scales' register is loaded between them only, else the compiler
    // would wait for all loads in every stage before it reads a lane of it.
    for (int c0 = t.s0; c0 < t.s1; c0 += 64) {
      if (c0 > t.s0) load_sb(c0);
      asm volatile("" : "+v"(vsb));
      const int c1 = min(t.s1, c0 + 64);
#pragma unroll 1
      for (int s = c0; s < c1; ++s) {
        const float sb = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(vsb), s - c0));
        const int next = buf + 1 == NBUF ? 0 : buf + 1;
        const fp8_lds_t* B = at_lds(buf * G::kStageB);
        const fp8_lds_t* A1 = at_lds(next * G::kStageA);
        const fp8_lds_t* B1 = at_lds(next * G::kStageB);
        cut_off(s + NBUF);
        fb[1] = read_b(B, 1);
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          if (j == JA && JA < JB) {
#pragma unroll
            for (int q = 0; q < JA * MI; ++q) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_barrier" ::: "memory");
            more_scales(s, s - c0);
#pragma unroll
            for (int q = 0; q < PA; ++q) issue_a(q, s + NBUF, buf);
          }
          if (j == JB) {
            // So far: a share of the loads, the LDS reads and the sums behind every product.
#pragma unroll
            for (int q = 0; q < (JA < JB ? JB - JA : JB) * MI; ++q) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NBUF - 2) * (PA + PB) + kBehind)
                         : "memory");
            asm volatile("s_barrier" ::: "memory");
            if constexpr (JA == JB) {
              more_scales(s, s - c0);
#pragma unroll
              for (int q = 0; q < PA; ++q) issue_a(q, s + NBUF, buf);
            }
#pragma unroll
            for (int q = 0; q < PB; ++q) issue_b(q, s + NBUF, buf);
          }
          // Column j + 2's operand, or the next stage's first.
          if (j + 2 < NI)
            fb[(j + 2) % F] = read_b(B, j + 2);
          else if (j == NI - 1)
            fb[0] = read_b(B1, 0);
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            add(i, (j + NI - 1) % NI);
            if (j == 0) f[i] = fs[i] * sb;
            prod[i] = mfma_fp8(fb[j % F].lo, fb[j % F].hi, fa[i].lo, fa[i].hi);
            if (j == NI - 1) fa[i] = read_a(A1, i);
          }
        }
        next_place();
        read_s(at_lds(place * BM * 4), fs);
        // From the barrier on: the loads too.
#pragma unroll
        for (int q = 0; q < (NI - JB - 1) * MI; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        }
#pragma unroll
        for (int q = 0; q < MI; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        }
        asm volatile("" ::: "memory");
        buf = next;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i) add(i, NI - 1);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the loads past the last stage

  const int64_t m_w = t.m0 + 16 * MI * wm + r;
  const int n_w = n_wave + 4 * g;
  if (!GROUPED && cut.splits > 1) {
    // Partial sums [split][M][N rounded up to 4].
    const int64_t ldp = (p.N + 3) & ~3;
    v4f* part = static_cast<v4f*>(p.partial) + (int64_t)t.split * p.M * (ldp / 4);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int64_t m = m_w + 16 * i;
        const int n = n_w + 16 * j;
        if (m < t.m1 && n < p.N) part[(m * ldp + n) / 4] = acc[i][j];
      }
    return;
  }
  // Rows may start at any element: 8- and 16-byte stores at element alignment.
  typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t any2 __attribute__((ext_vector_type(2), aligned(2)));
  if (t.n0 + BN <= p.N) {
    // Whole columns: 8 bytes per lane, or 16 after a swap between lane rows (two column blocks
    // at a time: each lane then has 8 neighbouring columns, 64 bytes of a row per store).
    auto pack = [&](int i, int j) __attribute__((always_inline)) {
      return make_uint2(f32x2_to_bf16x2(acc[i][j][0], acc[i][j][1]),
                        f32x2_to_bf16x2(acc[i][j][2], acc[i][j][3]));
    };
    static_assert(NI % 2 == 0, "columns in pairs of blocks");
    auto pieces = [&](int i, int j) __attribute__((always_inline)) {
      const uint2 u = pack(i, j), v = pack(i, j + 1);
      const auto x = __builtin_amdgcn_permlane16_swap(u.x, v.x, false, false);
      const auto y = __builtin_amdgcn_permlane16_swap(u.y, v.y, false, false);
      return any4{x[0], y[0], x[1], y[1]};
    };
    uint16_t* o2 = p.out + m_w * p.ld_out + n_wave + 16 * (g & 1) + 8 * (g >> 1);
    if ((p.ld_out & 1) == 0) {
#pragma unroll
      for (int j = 0; j < NI; j += 2)
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const any4 v = pieces(i, j);
          if (m_w + 16 * i < t.m1) *reinterpret_cast<any4*>(o2 + 16 * i * p.ld_out + 16 * j) = v;
        }
      return;
    }
    // Every other row starts between two dwords (the first one on 16 bytes), where a 16-byte store
    // takes several times as long (8192 x 3585 x 1024: 60 us instead of 41).  There a lane stores
    // the 8 columns from its second on, the last of them from the lane with the columns after its
    // own; the first column is stored by itself, and the last lane's columns where they are.
    const bool odd = (m_w & 1) != 0;
    const int after = r + 16 * (g == 0 ? 2 : g == 2 ? 1 : g == 1 ? 3 : 0);
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      any4 v = pieces(i, 0);
#pragma unroll
      for (int j = 0; j < NI; j += 2) {
        any4 next = v;
        if (j + 2 < NI) next = pieces(i, j + 2);
        const uint32_t more = (uint32_t)__shfl((int)(g == 0 ? next[0] : v[0]), after);
        const bool shift = odd && (g != 3 || j + 2 < NI);
        uint16_t* o = o2 + 16 * i * p.ld_out + 16 * j;
        if (m_w + 16 * i < t.m1) {
          if (odd && g == 0 && j == 0) *o = (uint16_t)v[0];
          if (shift)
            v = any4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16,
                     v[3] >> 16 | more << 16};
          *reinterpret_cast<any4*>(o + shift) = v;
        }
        v = next;
      }
    }
    return;
  }
  // A tile at the columns' edge: four columns at a time, the last ones one by one.
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    if (m_w + 16 * i >= t.m1) continue;
    uint16_t* o = p.out + (m_w + 16 * i) * p.ld_out + n_w;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const uint32_t lo = f32x2_to_bf16x2(acc[i][j][0], acc[i][j][1]);
      const uint32_t hi = f32x2_to_bf16x2(acc[i][j][2], acc[i][j][3]);
      const int n = n_w + 16 * j;
      if (n + 4 <= p.N) {
        *reinterpret_cast<any2*>(o + 16 * j) = any2{lo, hi};
      } else {
        const uint64_t h = ((uint64_t)hi << 32) | lo;
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (n + e < p.N) o[16 * j + e] = (uint16_t)(h >> (16 * e));
      }
    }
  }
}

template <int WM, int WN, int MI, int NI, int NBUF>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
void fp8_tile_kernel(Fp8Params p, Fp8Cut cut) {
  using G = Fp8Geom<WM, WN, MI, NI, NBUF>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[G::kLds];
  // Workgroups go to the 8 XCDs in turn; each XCD takes a contiguous range, split by split, a
  // split's tiles in blocks of up to 8 tile rows walked column by column.
  const int n_tiles = cut.tiles_m * cut.tiles_n;
  const int n = n_tiles * cut.splits, b = blockIdx.x, x = b & 7, q = n >> 3, rest = n & 7;
  int tile = x * q + min(x, rest) + (b >> 3), split = 0;
  if (cut.splits > 1) {
    split = tile / n_tiles;
    tile -= split * n_tiles;
  }
  const int blk = tile / (8 * cut.tiles_n);
  const int rows_in = min(8, cut.tiles_m - 8 * blk);
  const int in_blk = tile - blk * 8 * cut.tiles_n;
  const int tn = in_blk / rows_in, tm = 8 * blk + in_blk - tn * rows_in;
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock;
  const int s0 = split * cut.stages_per_split;
  const int64_t m0 = (int64_t)tm * G::BM;
  fp8_tile_body<WM, WN, MI, NI, NBUF, false>(
      p, cut,
      Fp8Tile{m0, min((int64_t)p.M, m0 + G::BM), tn * G::BN, s0,
              min(KB, s0 + cut.stages_per_split), split, 0},
      lds);
}

// The output rows of an expert.  Offsets out of order are an empty expert.
struct Fp8Span {
  int first, end;
};
__device__ __forceinline__ Fp8Span fp8_span(const Fp8Params& p, int e) {
  if (e >= p.E) return {0, 0};
  const int first = max(p.offs[e], 0);
  return {first, max(min(p.offs[e + 1], p.M), first)};
}
__device__ __forceinline__ int fp8_wave_scan(int v) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(v, d);
    if (lane >= d) v += y;
  }
  return v;
}

// The tiles of BM rows of all experts, expert by expert, as a wavefront counts them: its lanes each a
// run of `per` experts.
struct Fp8Count {
  Fp8Span span;      // of the run's first expert
  int own, upto;     // the run's tiles, and with those of all runs before it
};
template <int BM>
__device__ __forceinline__ int fp8_tiles_of(Fp8Span s) {
  return (s.end - s.first + BM - 1) / BM;
}
template <int BM>
__device__ __forceinline__ Fp8Count fp8_count(const Fp8Params& p, int per) {
  const int lane = threadIdx.x & 63;
  Fp8Count c;
  c.span = fp8_span(p, lane * per);
  c.own = fp8_tiles_of<BM>(c.span);
  for (int i = 1; i < per; ++i) c.own += fp8_tiles_of<BM>(fp8_span(p, lane * per + i));
  c.upto = fp8_wave_scan(c.own);
  return c;
}
// The expert of tile `slot` of these (below the last lane's `upto`), its rows and the tiles before
// its first: the run with the tile is looked at expert by expert (up to 64 experts: one load of
// offsets and no more).
struct Fp8Found {
  int e, first, end, before;
};
template <int BM>
__device__ __forceinline__ Fp8Found fp8_find(const Fp8Params& p, int per, Fp8Count c, int slot) {
  const int lane = threadIdx.x & 63;
  Fp8Found f;
  f.e = __ffsll((long long)__ballot(c.upto > slot)) - 1;
  f.before = __builtin_amdgcn_readlane(c.upto - c.own, f.e);
  int at = f.e;                      // the lane that has the expert's rows
  if (per > 1) {
    c.span = lane < per ? fp8_span(p, f.e * per + lane) : Fp8Span{0, 0};
    c.own = fp8_tiles_of<BM>(c.span);
    c.upto = f.before + fp8_wave_scan(c.own);
    at = __ffsll((long long)__ballot(c.upto > slot)) - 1;
    f.before = __builtin_amdgcn_readlane(c.upto - c.own, at);
    f.e = f.e * per + at;
  }
  f.first = __builtin_amdgcn_readlane(c.span.first, at);
  f.end = __builtin_amdgcn_readlane(c.span.end, at);
  return f;
}

// Grouped: a workgroup for every tile that there can be; it counts the experts' tiles to find its
// own, or that there is none left for it.  Each XCD takes a contiguous range of the tiles, an
// expert's column by column, so that what runs at once on an XCD shares weights and tokens.
// (Workgroups that stay and take tile after tile were slower, in an earlier form of this kernel: 16384
// x 3584 x 3584 in 32 experts 316 us against 278, in 28 359 against 288: nothing covers a tile's first
// loads and its stores.  All experts' whole tiles first and the last, shorter ones of each after them: in 28 experts 269 against 241, since an
// expert's tiles then no longer share its weights.)
template <int WM, int WN, int MI, int NI, int NBUF>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2)))
void fp8_grouped_kernel(Fp8Params p, Fp8Cut cut) {
  using G = Fp8Geom<WM, WN, MI, NI, NBUF>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[G::kLds];
  const int per = (p.E + 63) / 64;
  const Fp8Count c = fp8_count<G::BM>(p, per);
  // (Offsets that overlap may count more tiles than the grid has, or than 31 bits hold: what then
  // is no tile of its expert is left out below.)
  const uint32_t items = (uint32_t)min(
      (int64_t)max(__builtin_amdgcn_readlane(c.upto, 63), 0) * cut.tiles_n, (int64_t)0x7FFFFFFF);
  const uint32_t x = blockIdx.x & 7, q = items >> 3, in_x = blockIdx.x >> 3;
  if (in_x >= q + (x < (items & 7))) return;
  const uint32_t it = x * q + min(x, items & 7) + in_x;
  const Fp8Found f = fp8_find<G::BM>(p, per, c, (int)(it / (uint32_t)cut.tiles_n));
  const int tiles = fp8_tiles_of<G::BM>({f.first, f.end});
  const uint32_t in = it - (uint32_t)f.before * (uint32_t)cut.tiles_n;
  if (in >= (uint64_t)tiles * (uint32_t)cut.tiles_n) return;
  const int tn = (int)(in / (uint32_t)tiles);
  const int64_t m0 = f.first + (int64_t)((int)in - tn * tiles) * G::BM;
  fp8_tile_body<WM, WN, MI, NI, NBUF, true>(
      p, cut,
      Fp8Tile{m0, min((int64_t)f.end, m0 + G::BM), tn * G::BN, 0,
              (p.K + kScaleBlock - 1) / kScaleBlock, 0, f.e},
      lds);
}

// The splits' partial sums, added in split order.
static __global__ __launch_bounds__(256) void fp8_join_kernel(Fp8Params p, int splits) {
  const int per_row = (p.N + 3) / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t total = (int64_t)p.M * per_row;
  if (at >= total) return;
  const int64_t m = at / per_row;
  const v4f* part = static_cast<const v4f*>(p.partial) + at;
  v4f s = part[0];
#pragma unroll 4
  for (int z = 1; z < splits; ++z) s += part[z * total];
  fp8_store(p, s, m, 4 * (int)(at - m * per_row));
}

template <int WM, int WN, int MI, int NI, int NBUF>
hipError_t fp8_tile_launch(const Fp8Params& p, int splits, hipStream_t stream) {
  using G = Fp8Geom<WM, WN, MI, NI, NBUF>;
  Fp8Cut cut;
  cut.tiles_m = (p.M + G::BM - 1) / G::BM;
  cut.tiles_n = (p.N + G::BN - 1) / G::BN;
  const int KB = (p.K + kScaleBlock - 1) / kScaleBlock;
  cut.stages_per_split = (KB + splits - 1) / splits;
  cut.splits = (KB + cut.stages_per_split - 1) / cut.stages_per_split;
  const int64_t grid = (int64_t)cut.tiles_m * cut.tiles_n * cut.splits;
  if (grid > most_blocks(64 * WM * WN)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, MI, NI, NBUF>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, stream, p, cut);
  if (cut.splits > 1) {
    const int64_t pieces = (int64_t)p.M * ((p.N + 3) / 4);
    hipLaunchKernelGGL(fp8_join_kernel, dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0,
                       stream, p, cut.splits);
  }
  return hipGetLastError();
}

template <int WM, int WN, int MI, int NI, int NBUF>
hipError_t fp8_grouped_launch(const Fp8Params& p, hipStream_t stream) {
  using G = Fp8Geom<WM, WN, MI, NI, NBUF>;
  Fp8Cut cut;
  cut.tiles_n = (p.N + G::BN - 1) / G::BN;
  cut.tiles_m = 0;
  cut.splits = 1;
  cut.stages_per_split = (p.K + kScaleBlock - 1) / kScaleBlock;
  const int64_t grid = fp8_grouped_blocks(G::BM, G::BN, p.M, p.E, p.N);
  if (grid > most_blocks(64 * WM * WN)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((fp8_grouped_kernel<WM, WN, MI, NI, NBUF>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, stream, p, cut);
  return hipGetLastError();
}

}  // namespace mi355moe
