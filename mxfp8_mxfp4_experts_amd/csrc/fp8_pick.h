// Which kernel, variant and split of K a block-scaled FP8 product takes: host code, from the sizes
// alone (fp8.hip launches what is picked here).
#pragma once

#include "dense_pick.h"   // kCus, kMaxSplits, most_partials
#include "grid.h"

namespace mi355moe {

constexpr int kFp8Waves = 16;        // wavefronts of the direct kernels' workgroups
constexpr int kRawPieces = 4;        // pieces of 8 elements that a thread quantises there
constexpr int kFp8DirectMost = 512;  // tokens up to which the direct kernel is considered
constexpr int kFp8DirectRows = 8;    // and up to which it is always taken

// The estimates below, in ns, are fitted to every variant and split of 900 products (M 1 .. 8192,
// N 64 .. 3584, K 128 .. 7168, log-uniform): what is picked is 2.2% slower than the best of them
// in the mean, 43% at worst.
//
// Direct kernel: a workgroup reads its columns' and tokens' codes at the rate of a CU (with Q = 1
// half of what it takes with 2: fewer loads are in flight) and takes a fixed time, more where K is
// longer than its wavefronts take at once; the chip reads weights at about 5600 bytes/ns.  (1 x
// 3584 x 7168: 7.6 us with Q = 1, 8.4 with 2, 10.4 with 4; 8 x 500 x 2992: 4.3, 3.5, 3.8.)
struct DirectCost {
  float rate, fixed, more;
};
constexpr DirectCost kFp8Direct[3] = {{61, 1160, 720}, {130, 1020, 680}, {46, 910, 300}};
constexpr DirectCost kFp8Raw[3] = {{72, 1540, 520}, {106, 1410, 650}, {77, 1390, 300}};
inline float fp8_chip_ns(const DirectCost& c, int q, int M, int N, int K, float bytes, float more) {
  const int cols = 16 / q;
  const int64_t wgs = (int64_t)((N + cols - 1) / cols) * ((M + cols - 1) / cols);
  const float one = bytes / c.rate + c.fixed + (K > 128 * q * kFp8Waves ? c.more : 0.0f) + more;
  const float cu = (float)((wgs + kCus - 1) / kCus) * one, chip = (float)N * K / 5600.0f;
  return 1900.0f + (cu > chip ? cu : chip);
}
inline float fp8_direct_ns(int i, int M, int N, int K) {
  const int q = 1 << i, c = 16 / q;
  return fp8_chip_ns(kFp8Direct[i], q, M, N, K, (float)(c + (M < c ? M : c)) * K, 0.0f);
}
inline int fp8_direct_q(int M, int N, int K) {
  int best = 0;
  for (int i = 1; i < 3; ++i)
    if (fp8_direct_ns(i, M, N, K) < fp8_direct_ns(best, M, N, K)) best = i;
  return 1 << best;
}

// The tiled kernel's variants: one stage's time in launches of up to half the workgroups that run
// at once and in fuller ones (one and two per CU; of 256 x 256 tiles half a workgroup and one), and
// what a workgroup takes besides (first loads, epilogue); a split's join and each partial sum.
struct Fp8Variant {
  int bm, bn, per_cu, threads;
  float one, one_fixed, two, two_fixed, join, part;
};
constexpr Fp8Variant kFp8Variants[] = {
    {256, 256, 1, 512, 1136, 5840, 1451, 10090, 0, 0},
    {128, 128, 2, 256, 547, 2627, 1060, 4957, 1129, 0.0029f},
    {64, 128, 2, 256, 338, 1936, 704, 3020, 1744, 0.0023f},
    {64, 64, 2, 256, 232, 1467, 463, 2103, 1993, 0.0021f},
    {32, 64, 2, 256, 194, 1100, 321, 1614, 2128, 0.0019f},
};
constexpr int kFp8NumVariants = sizeof(kFp8Variants) / sizeof(kFp8Variants[0]);

inline float fp8_tiled_ns(const Fp8Variant& v, int64_t wgs, int stages) {
  const int at_once = kCus * v.per_cu, rest = (int)(wgs % at_once);
  const float one = stages * v.one + v.one_fixed, two = stages * v.two + v.two_fixed;
  return 2000.0f + (float)(wgs / at_once) * two +
         (rest == 0 ? 0.0f : rest <= at_once / 2 && rest <= kCus ? one : two);
}

struct Fp8Pick {
  int variant;   // -1: the direct kernel
  int splits;
  float ns;      // estimated
};

// Splits are for launches that leave CUs idle; each has three stages at least.
inline int fp8_most_splits(int K) {
  const int stages = (K + 127) / 128;
  return kMaxSplits < stages / 3 ? kMaxSplits : stages / 3;
}
inline bool fp8_may_split(int M, int K) { return M > kFp8DirectRows && fp8_most_splits(K) > 1; }

inline Fp8Pick fp8_pick(int M, int N, int K) {
  Fp8Pick best{-1, 1, 3.4e38f};
  if (M <= kFp8DirectMost) {
    const int q = fp8_direct_q(M, N, K);
    best.ns = fp8_direct_ns(q == 1 ? 0 : q == 2 ? 1 : 2, M, N, K);
  }
  if (M <= kFp8DirectRows) return best;
  const int stages = (K + 127) / 128;
  const int64_t sums = (int64_t)M * ((N + 3) / 4 * 4);
  int most = fp8_most_splits(K);
  while (most > 1 && most * sums > most_partials(M, N)) --most;
  for (int i = 0; i < kFp8NumVariants; ++i) {
    const Fp8Variant& v = kFp8Variants[i];
    const int64_t tiles = (int64_t)((M + v.bm - 1) / v.bm) * ((N + v.bn - 1) / v.bn);
    for (int s = 1; s == 1 || (v.per_cu == 2 && s <= most && tiles * s <= 3 * kCus); ++s) {
      float t = fp8_tiled_ns(v, tiles * s, (stages + s - 1) / s);
      if (s > 1) t += v.join + v.part * (float)M * N * s;
      if (t < best.ns) best = {i, s, t};
    }
  }
  return best;
}

// One launch that quantises every workgroup's tokens anew (its Q), or two (0)?  The estimate of the
// one, against the other's with 2.7 us for the quantisation, and half a microsecond because a
// second launch costs the host 3.5 us.  (1 x 3584 x 7168: 8.0 us against 9.9; 64 x 512 x 512 3.9
// against 6.0; 32 x 3000 x 1024 8.3 against 7.2.)
inline int fp8_raw(int M, int N, int K) {
  const int KB = (K + 127) / 128;
  int best = 0;
  float least = 0.0f;
  for (int i = 0; i < 3; ++i) {
    const int q = 1 << i, c = 16 / q, t = M < c ? M : c;
    if (t * KB > kRawPieces * 4 * kFp8Waves || M > kFp8DirectMost) continue;
    const float ns = fp8_chip_ns(kFp8Raw[i], q, M, N, K, (float)(c + 2 * t) * K,
                                 t * KB > 4 * kFp8Waves ? 1280.0f : 0.0f);
    if (!best || ns < least) {
      best = q;
      least = ns;
    }
  }
  return best && least <= fp8_pick(M, N, K).ns + 3200.0f ? best : 0;
}

// A grouped launch: a workgroup for every tile that there can be, in eights.
inline int64_t fp8_grouped_blocks(int bm, int bn, int R, int E, int N) {
  const int64_t tiles = ((int64_t)R / bm + (E < R ? E : R)) * ((N + bn - 1) / bn);
  return (tiles + 7) / 8 * 8;
}

// Grouped: the rows of each expert are known on the GPU only, so as if the R routes were spread
// evenly over the experts, with half a tile to spare for each: routes that are dropped count too.
// (28 experts, 3584 x 3584, 4096 routes of which 1020 are kept: 88.6 us in the 256 x 256 tiles taken,
// 78.9 in 64 x 128; 8192 of which 2087: 95.0, and 94.2 in 128 x 128; the weights alone take 72.)  (Rows by the thousand million are
// too many for a launch of small tiles.)
inline int fp8_pick_grouped(int R, int E, int N, int K) {
  const int stages = (K + 127) / 128, used = E < R ? E : R;
  int best = 0;
  float least = 3.4e38f;
  for (int i = 0; i < kFp8NumVariants; ++i) {
    const Fp8Variant& v = kFp8Variants[i];
    if (i > 0 && fp8_grouped_blocks(v.bm, v.bn, R, E, N) > most_blocks(v.threads)) continue;
    const int64_t tiles = (int64_t)R / v.bm + (used + 1) / 2;
    const float t = fp8_tiled_ns(v, (tiles > used ? tiles : used) * ((N + v.bn - 1) / v.bn), stages);
    if (t < least) {
      least = t;
      best = i;
    }
  }
  return best;
}

}  // namespace mi355moe
