// Which kernel, variant and split of K a dense product takes: host code, from
// the sizes alone (dense.hip launches what is picked here; K in bytes).
#pragma once

#include <stdint.h>

namespace mi355moe {

constexpr int kStageK = 128;           // bytes of K per stage of the tiled kernel
constexpr int kDirectWaves = 16;       // wavefronts of the direct kernel's workgroups
constexpr int kFusedUnits = 4;         // units of 512 elements a wavefront quantises

// Estimated time of the direct kernel past its launch, in ns.  A workgroup reads
// its columns and its tokens, a CU about 90 bytes/ns where a load instruction
// takes whole 128-byte lines (Q of 2 or 4) and 51 where it takes half lines; first
// loads and the join take half a microsecond, longer with more sums per output;
// the chip reads its weights at about 5600 bytes/ns.  (Router product of 32
// tokens, 896 x 7168: 14.9 us with Q = 1, 9.5 with 2; INT8 16 x 3584 x 7168: 8.7 us
// with 1, 11.2 with 2.)
constexpr int kCus = 256;
inline float direct_ns(int q, int M, int N, int64_t Kb) {
  const int c = 16 / q;
  const int64_t wgs = (int64_t)((N + c - 1) / c) * ((M + c - 1) / c);
  const float bytes = (float)(c + (M < c ? M : c)) * Kb;
  const float one = q == 1 ? bytes / 51.0f + 530.0f : bytes / 90.0f + (q == 2 ? 490.0f : 850.0f);
  const float per_cu = (float)((wgs + kCus - 1) / kCus) * one;
  const float chip = (float)N * Kb / 5600.0f;
  return per_cu > chip ? per_cu : chip;
}
// The Q of least estimated time.
inline int direct_q(int M, int N, int64_t Kb) {
  int best = 1;
  for (int q = 2; q <= 4; q *= 2)
    if (direct_ns(q, M, N, Kb) < direct_ns(best, M, N, Kb)) best = q;
  return best;
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
inline int64_t most_partials(int M, int N) {
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
inline Pick pick(int M, int N, int64_t Kb) {
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

// One launch that quantises every workgroup's tokens anew, or two?  The estimate
// of the one (fitted as those above, to 258 products of 1 .. 1024 tokens, 160 of
// them faster in one launch: 64 x 512 x 512 4.2 against 6.0 us, 256 x 240 x 736 5.2
// against 5.6, 28 x 2889 x 1104 8.2 against 6.6) against the other's with 2.7 us
// for the quantisation, and half a microsecond because a second launch costs the
// host 3.5 us.  On 128 other products the choice is 1.3% slower than the better.
inline int fused_q(int M, int N, int K) {
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

}  // namespace mi355moe
