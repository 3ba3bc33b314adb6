// Group-limited top-k routing: sigmoid or softmax scores, a correction bias
// that only takes part in the choice, the best groups of experts, then the
// best experts in them, weights renormalised or not.
//
//   s_e   = sigmoid(l_e), or exp(l_e - max) / sum (over the experts that their
//           logits do not mask, whatever their biases), evaluated in double and
//           rounded once to float
//   key_e = s_e + bias_e (float); an expert is masked when l_e is -inf or the
//           lowest finite float, or its key is -inf
//   worth of a group: its best key, or the float sum of its best two
//   the topk_group groups of most worth; in them the K largest keys; equal
//   keys (worths) rank the lower expert (group) first; NaN ranks below every
//   number, a masked expert is never taken: slots left over hold id -1 and
//   weight 0
//   w_k   = s_k [/ sum_j s_j in double; 0 where that sum is 0] * scaling
//
// One wavefront per token, no barriers.  Doubles for every expert would bound
// the kernel, so the choice is narrowed in float first, with a margin that
// covers the float evaluation's error, and only the candidates (usually 16 to
// 40 of hundreds) get their exact scores:
//   * float scores differ from the exact ones by less than kScoreErr = 2^-21.
//     Sigmoid: the exponent's argument rounds by |l| 2^-24 relative, which is
//     s(1-s)|l| 2^-24 < 2^-26 of the score, v_exp_f32's ulp s(1-s) 2^-23 <=
//     2^-25, the sum and the rounding of the exact score 2^-24 and 2^-25,
//     v_rcp_f32's ulp 2^-23: 17/16 of 2^-22 together.  Softmax: two roundings of the
//     argument x, p|x| 2^-23 < 2^-24, exponential, scale and product 2^-23 +
//     2^-24 + 2^-24, the exact score's 2^-25: below 2^-21.5;
//   * a key adds bias in float, rounding by at most 2^-24 |key| on each side
//     (kKeyRel = 2^-23 for both), and so does the sum of two keys;
//   * an expert among the K largest exact keys then has a float key above the
//     K-th largest float key less twice that error; the K-th largest of the
//     lanes' largest keys is a lower bound of that, found by bisection with
//     ballots.
// Where the worths of the last group inside and the first one outside are
// within their errors (about one token in 3000 at 896 experts in 8 groups), the
// groups' worths are taken exactly, again from candidates only.  With more than
// 64 candidates, or NaN or huge keys, the wavefront evaluates everything
// exactly; likewise where a lane has more than 16 experts, whose keys would not
// stay in registers (one group: 8192 x 1024 14.5 us, 8192 x 1056 66, 8192 x 2048
// 123, 8192 x 4096 439; 9 groups of 99, 25 experts a lane, 37).
//
// The exact path's sum of exponentials runs in another order than the narrowed
// one's, both in double: a softmax score next to a rounding boundary of float may
// so differ by its last bit between the two; sigmoid scores are the same.
//
// Vector instructions bound it at many tokens, about 790 a token and wavefront
// (8192 x 896, 8 groups of which 4, top 16: 52.9 us with every score exact, 16.3
// narrowed; 30 MB, 1.9 TB/s), and one wavefront's chain at few (8 tokens: 6.1 us).
#include "common.h"
#include "launch.h"
#include "route_dev.h"

namespace mi355moe {

namespace {

constexpr float kLowest = -3.402823466e38f;
constexpr float kInf = __builtin_inff();
constexpr float kScoreErr = 4.76837158203125e-07f;     // 2^-21
constexpr float kKeyRel = 1.1920928955078125e-07f;     // 2^-23
constexpr int kWaves = 4;

// The float that ordered_key mapped to k.
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 1u ? __uint_as_float(0x7FC00000u)
                 : __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// 0 for an expert that may not be taken, else the ordered key.
__device__ __forceinline__ uint32_t route_key(float logit, float score, float bias) {
  const float key = score + bias;
  return (logit <= kLowest || key == -kInf) ? 0u : ordered_key(key);
}

// Largest float of the wavefront; no NaN among them.
__device__ __forceinline__ float wave_fmax(float v) {
  return key_value(wave_max_u32(ordered_key(v)));
}

// The best two keys of two disjoint sets, (k0, k1) and another lane's.
template <int CTRL>
__device__ __forceinline__ void top2_dpp(uint32_t& k0, uint32_t& k1) {
  const uint32_t o0 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)k0, CTRL, 0xf, 0xf, false);
  const uint32_t o1 = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)k1, CTRL, 0xf, 0xf, false);
  k1 = umax32(umin32(k0, o0), umax32(k1, o1));
  k0 = umax32(k0, o0);
}
__device__ __forceinline__ void top2_xor(uint32_t& k0, uint32_t& k1, int off) {
  const uint32_t o0 = (uint32_t)__shfl_xor((int)k0, off);
  const uint32_t o1 = (uint32_t)__shfl_xor((int)k1, off);
  k1 = umax32(umin32(k0, o0), umax32(k1, o1));
  k0 = umax32(k0, o0);
}
// Over each run of 1 << log2l lanes, the same result in all of them: pairs by
// quad permutation, quads and halves of a row by mirroring (lanes already hold
// their quad's result, so any lane of the other quad will do), rows by shuffles.
__device__ __forceinline__ void top2_lanes(uint32_t& k0, uint32_t& k1, int log2l) {
  if (log2l > 0) top2_dpp<0xB1>(k0, k1);    // quad_perm [1, 0, 3, 2]
  if (log2l > 1) top2_dpp<0x4E>(k0, k1);    // quad_perm [2, 3, 0, 1]
  if (log2l > 2) top2_dpp<0x141>(k0, k1);   // row_half_mirror
  if (log2l > 3) top2_dpp<0x140>(k0, k1);   // row_mirror
  if (log2l > 4) top2_xor(k0, k1, 16);
  if (log2l > 5) top2_xor(k0, k1, 32);
}
// Wavefront sum of doubles, uniform result (the steps of wave_max_u32).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dadd_dpp(double v) {
  const long long b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xf, false);
  return v + __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double wave_dsum(double v) {
  v = dadd_dpp<0x111, 0xf>(v);
  v = dadd_dpp<0x112, 0xf>(v);
  v = dadd_dpp<0x114, 0xf>(v);
  v = dadd_dpp<0x118, 0xf>(v);
  v = dadd_dpp<0x142, 0xa>(v);
  v = dadd_dpp<0x143, 0xc>(v);
  const long long b = __double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// A token's softmax normaliser: the largest unmasked logit and the sum.
struct Softmax {
  float top;
  double total;
};

template <bool SOFTMAX>
__device__ __forceinline__ float exact_score(float l, const Softmax& sm) {
  if constexpr (SOFTMAX)
    return l <= kLowest ? 0.0f : (float)(exp((double)l - (double)sm.top) / sm.total);
  return sigmoid_score(l);
}

// This wavefront's LDS writes before its reads of other lanes' entries.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Set bits of mask below this lane's.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

struct WaveLds {
  uint32_t* keys;      // [E]: candidates' experts, or the exact path's keys
  uint64_t* cand;      // [64]
  float* score;        // [64]: candidates' scores, then the slots'
  int* id;             // [64]
  uint32_t* worth;     // [kMaxGroups], the exact path's
};

// Lane k's expert by the exact scores of all experts (-1: none).
template <bool SOFTMAX>
__device__ int exact_choice(const RouteGroupsParams& p, const float* row, const Softmax& sm,
                            const WaveLds& s, int lane) {
  const int E = p.E, K = p.K, G = p.n_group, per = E / G;
#pragma unroll 4
  for (int e = lane; e < E; e += 64) {
    const float l = row[e];
    s.keys[e] = route_key(l, exact_score<SOFTMAX>(l, sm), p.bias ? p.bias[e] : 0.0f);
  }
  wave_lds_fence();
  if (G > 1) {
    for (int g = 0; g < G; ++g) {
      uint32_t k0 = 0, k1 = 0;   // the group's best two keys
      for (int i = lane; i < per; i += 64) {
        const uint32_t k = s.keys[g * per + i];
        k1 = umax32(k1, umin32(k0, k));
        k0 = umax32(k0, k);
      }
      top2_lanes(k0, k1, 6);
      uint32_t w = k0;           // 0: every expert of the group is masked
      if (p.group_score == MOE_GROUP_TOP2 && k1 != 0u)
        w = ordered_key(key_value(k0) + key_value(k1));
      if (lane == 0) s.worth[g] = w;
    }
    wave_lds_fence();
    const uint32_t mine = lane < G ? s.worth[lane] : 0u;
    int before = 0;
    for (int j = 0; j < G; ++j) {
      const uint32_t o = s.worth[j];
      before += (o > mine || (o == mine && j < lane)) ? 1 : 0;
    }
    const uint64_t keep = __ballot(lane < G && before < p.topk_group);
    for (int e = lane; e < E; e += 64)
      if (!((keep >> (e / per)) & 1ull)) s.keys[e] = 0u;
    wave_lds_fence();
  }
  int id = -1;
  if (E <= 64 * kRegExpertsPerLane) {
    if (!select_topk_threshold(s.keys, E, K, lane, s.cand, id))
      id = select_topk_rounds(s.keys, E, K, lane);
  } else {
    uint64_t last = ~0ull;
    for (int k = 0; k < K; ++k) {
      uint64_t best = 0;
      for (int e = lane; e < E; e += 64) {
        const uint64_t c = ((uint64_t)s.keys[e] << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)e);
        best = (c < last && c > best) ? c : best;
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const uint64_t o = __shfl_xor(best, off);
        best = o > best ? o : best;
      }
      last = best;
      if (lane == k) id = (int)(0xFFFFFFFFu - (uint32_t)best);
    }
  }
  return (lane >= K || id < 0 || id >= E || s.keys[id] == 0u) ? -1 : id;
}

// Lane k writes slot k: expert id (-1: none) of score sc.
__device__ __forceinline__ void write_slots(const RouteGroupsParams& p, int64_t t, int id, float sc,
                                            const WaveLds& s, int lane) {
  double w = (double)sc;
  if (p.renormalise) {
    double* d = reinterpret_cast<double*>(s.cand);
    wave_lds_fence();
    d[lane] = w;
    wave_lds_fence();
    double sum = 0.0;
#pragma unroll 8
    for (int k = 0; k < p.K; ++k) sum += d[k];   // left to right
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (lane < p.K) {
    p.topk_idx[t * p.K + lane] = id;
    p.topk_w[t * p.K + lane] = id >= 0 ? (float)(w * (double)p.scaling) : 0.0f;
  }
}

// Float keys of the narrowed choice as unsigned numbers in the same order: the
// ordered key less that of -inf, so 0 is "may not be taken" and a negative NaN,
// wrapping around, is the largest of all.
constexpr uint32_t kKeyBase = 0x007FFFFFu;
__device__ __forceinline__ uint32_t near_key(float f) {
  const uint32_t b = __float_as_uint(f);
  return (b ^ ((uint32_t)((int)b >> 31) | 0x80000000u)) - kKeyBase;
}
__device__ __forceinline__ float near_value(uint32_t k) { return key_value(k + kKeyBase); }
// Keys of 2^120 and above, NaN among them; keys of -2^120 and below are the
// numbers 1 .. kLowOdd.  Sums of two keys between those stay finite.
constexpr uint32_t kHighOdd = 0xFB800000u - kKeyBase, kLowOdd = 0x047FFFFFu - kKeyBase;

// The narrowed choice.  The wavefront's 64 lanes are split evenly over the
// groups (L lanes each, L = 64 over n_group rounded up to a power of two);
// lane i of group g holds experts i, i + L, ... of it, at most S.  Returns
// false, having written nothing, where float cannot tell.
template <bool SOFTMAX, int S>
__device__ __forceinline__ bool narrowed_choice(const RouteGroupsParams& p, const float* row,
                                                int64_t t, int log2l, Softmax& sm,
                                                const WaveLds& s, int lane) {
  const int E = p.E, K = p.K, G = p.n_group, per = E / G;
  const int L = 1 << log2l, g = lane >> log2l, i0 = lane & (L - 1);
  const int slots = (per + L - 1) >> log2l;          // uniform, <= S
  const int left = g < G ? per - i0 : 0;             // this lane's experts: L j < left
  const int e0 = (g < G ? g : G - 1) * per + i0;     // its first expert
  // Through buffers of the row's (the bias's) size: 32-bit offsets, zeros past the
  // end and for no bias at all.
  const __amdgpu_buffer_rsrc_t lr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(row), 0, (uint32_t)(4 * E), 0x00020000);
  const __amdgpu_buffer_rsrc_t br = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float*>(p.bias), 0, p.bias ? (uint32_t)(4 * E) : 0u, 0x00020000);
  float l[S], b[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int at = 4 * (e0 + L * j);   // past the row for slots that do not exist
    l[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(lr, at, 0, 0));
    b[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(br, at, 0, 0));
  }
  if (per != L * slots || (G << log2l) != 64) {        // some lanes have fewer
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (L * j >= left) l[j] = -kInf;
  }
  float scale = 1.0f, top = 0.0f;
  if constexpr (SOFTMAX) {
    top = -kInf;
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (j < slots && l[j] > kLowest) top = fmaxf(top, l[j]);
    top = wave_fmax(top);
    double part = 0.0;
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (j < slots) part += l[j] <= kLowest ? 0.0 : exp((double)l[j] - (double)top);
    sm.top = top;
    sm.total = wave_dsum(part);
    scale = (float)(1.0 / sm.total);
  }
  uint32_t key[S], best = 0, second = 0, low = ~0u;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    key[j] = 0;
    if (j >= slots) continue;
    float a;
    if constexpr (SOFTMAX)
      a = __builtin_amdgcn_exp2f((l[j] - top) * 1.44269504f) * scale;
    else
      a = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[j] * -1.44269504f));
    key[j] = near_key(l[j] <= kLowest ? -kInf : a + b[j]);
    low = umin32(low, key[j] - 1u);
    second = umax32(second, umin32(best, key[j]));
    best = umax32(best, key[j]);
  }
  if (__ballot(best >= kHighOdd || low < kLowOdd)) return false;

  bool in = g < G;                   // whether this lane's group stays
  if (G > 1) {
    uint32_t k0 = best, k1 = second;
    top2_lanes(k0, k1, log2l);
    // Every lane of a group now has its best two keys.
    float w = k0 ? near_value(k0) : -kInf;
    float err = kScoreErr + kKeyRel * fabsf(k0 ? w : 0.0f);
    if (p.group_score == MOE_GROUP_TOP2 && k1) {
      const float v = near_value(k1);
      err += kScoreErr + kKeyRel * fabsf(v);
      w += v;
      err += kKeyRel * fabsf(w);
    }
    int before = 0;
    for (int j = 0; j < G; ++j) {
      const float o =
          __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), j << log2l));
      before += (o > w || (o == w && j < g)) ? 1 : 0;
    }
    in = g < G && before < p.topk_group;
    // Certain if every group inside stands above every one outside by their errors.
    const float lo = -wave_fmax(in && k0 ? err - w : -kInf);
    const float out_top = wave_fmax(g < G && !in && k0 ? w + err : -kInf);
    if (!(lo > out_top)) {
      // Else the groups' exact worths, from the few experts that can be among
      // their group's best.
      uint32_t from = 1u;
      const uint32_t kth = p.group_score == MOE_GROUP_TOP2 && k1 ? k1 : k0;
      if (kth) {
        const float v = near_value(kth);
        from = umax32(1u, near_key(v - 4.0f * (kScoreErr + kKeyRel * fabsf(v))));
      }
      int n = 0;
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const bool c = key[j] >= from;
        const uint64_t mask = __ballot(c);
        const int at = n + lanes_below(mask);
        n += __popcll(mask);
        if (c) s.keys[at] = (uint32_t)(e0 + L * j);
      }
      if (n > 64) return false;
      wave_lds_fence();
      uint64_t mine = 0;             // the exact key, and its group's number plus one
      if (lane < n) {
        const int id = (int)s.keys[lane];
        const float cl = row[id];
        mine = ((uint64_t)route_key(cl, exact_score<SOFTMAX>(cl, sm), p.bias ? p.bias[id] : 0.0f)
                << 32) | (uint64_t)(id / per + 1);
      }
      s.cand[lane] = mine;
      wave_lds_fence();
      uint32_t x0 = 0, x1 = 0;       // lane j < G: group j's best two exact keys
      for (int j = 0; j < n; j += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t c = s.cand[j + i];
          const uint32_t k = (uint32_t)c == (uint32_t)lane + 1u ? (uint32_t)(c >> 32) : 0u;
          x1 = umax32(x1, umin32(x0, k));
          x0 = umax32(x0, k);
        }
      }
      uint32_t xw = x0;
      if (p.group_score == MOE_GROUP_TOP2 && x1) xw = ordered_key(key_value(x0) + key_value(x1));
      before = 0;
      for (int j = 0; j < G; ++j) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)xw, j);
        before += (o > xw || (o == xw && j < lane)) ? 1 : 0;
      }
      const uint64_t keep = __ballot(lane < G && before < p.topk_group);
      in = g < G && ((keep >> g) & 1ull);
      wave_lds_fence();
    }
    if (!in) best = 0u;
  }
  const uint64_t in_mask = __ballot(in);

  // A lower bound of the K-th largest key, to its upper 16 bits (two bits a
  // step): by the lanes' largest keys where at least K lanes hold one, else by
  // all keys.
  const bool by_lane = __popcll(__ballot(best != 0u)) >= K;
  auto enough = [&](uint32_t c) __attribute__((always_inline)) {
    if (by_lane) return __popcll(__ballot(best >= c)) >= K;
    int n = 0;
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (j < slots) n += __popcll(__ballot(key[j] >= c) & in_mask);
    return n >= K;
  };
  uint32_t bound = 0;
#pragma unroll 1
  for (int bit = 30; bit >= 16; bit -= 2) {
    const uint32_t c1 = bound | (1u << bit), c2 = bound | (2u << bit), c3 = bound | (3u << bit);
    const bool e1 = enough(c1), e2 = enough(c2), e3 = enough(c3);
    bound = e3 ? c3 : e2 ? c2 : e1 ? c1 : bound;
  }
  uint32_t least = 1u;
  if (bound) {     // 0: fewer than K keys, all are candidates
    const float v = near_value(bound);
    least = umax32(1u, near_key(v - 4.0f * (kScoreErr + kKeyRel * fabsf(v))));
  }
  if (!in) least = ~0u;              // above every key here
  int n = 0;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    if (j >= slots) continue;
    const bool c = key[j] >= least;
    const uint64_t mask = __ballot(c);
    const int at = n + lanes_below(mask);
    n += __popcll(mask);
    if (c) s.keys[at] = (uint32_t)(e0 + L * j);
  }
  if (n > 64) return false;
  wave_lds_fence();
  // Exact keys of the candidates, and each one's rank among them.
  uint64_t mine = 0;
  float sc = 0.0f;
  int id = -1;
  if (lane < n) {
    id = (int)s.keys[lane];
    const float cl = row[id];
    sc = exact_score<SOFTMAX>(cl, sm);
    const uint32_t k = route_key(cl, sc, p.bias ? p.bias[id] : 0.0f);
    if (k) mine = ((uint64_t)k << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)id);
  }
  s.cand[lane] = mine;
  wave_lds_fence();
  int rank = 0;
  for (int j = 0; j < n; j += 8) {         // past the last: 0, above nothing
#pragma unroll
    for (int i = 0; i < 8; ++i) rank += s.cand[j + i] > mine ? 1 : 0;
  }
  // Slot k takes the candidate of rank k.
  s.id[lane] = -1;
  s.score[lane] = 0.0f;
  wave_lds_fence();
  if (mine) {
    s.id[rank] = id;
    s.score[rank] = sc;
  }
  wave_lds_fence();
  const int slot_id = s.id[lane];
  const float slot_sc = s.score[lane];
  write_slots(p, t, slot_id, slot_sc, s, lane);
  return true;
}

template <bool SOFTMAX>
__device__ void exact_token(const RouteGroupsParams& p, const float* row, int64_t t,
                            const WaveLds& s, int lane) {
  Softmax sm{0.0f, 1.0};
  if constexpr (SOFTMAX) {
    float top = -kInf;
    for (int e = lane; e < p.E; e += 64) {
      const float l = row[e];
      if (l > kLowest) top = fmaxf(top, l);
    }
    sm.top = wave_fmax(top);
    double part = 0.0;
    for (int e = lane; e < p.E; e += 64) {
      const float l = row[e];
      if (!(l <= kLowest)) part += exp((double)l - (double)sm.top);
    }
    sm.total = wave_dsum(part);
  }
  const int id = exact_choice<SOFTMAX>(p, row, sm, s, lane);
  const float sc = id >= 0 ? exact_score<SOFTMAX>(row[id], sm) : 0.0f;
  write_slots(p, t, id, sc, s, lane);
}

// S = 0: every token exactly.
template <bool SOFTMAX, int S>
__global__ __launch_bounds__(64 * kWaves) void route_groups_kernel(RouteGroupsParams p, int log2l) {
  extern __shared__ uint32_t keys_s[];   // [wavefronts][E]
  __shared__ uint64_t cand_s[kWaves][64];
  __shared__ float score_s[kWaves][64];
  __shared__ int id_s[kWaves][64];
  __shared__ uint32_t worth_s[kWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) + wave;
  if (t >= p.T) return;
  const float* row = p.logits + t * p.ld;
  const WaveLds s{keys_s + (size_t)wave * p.E, cand_s[wave], score_s[wave], id_s[wave],
                  worth_s[wave]};
  if constexpr (S > 0) {
    Softmax sm{0.0f, 1.0};
    if (narrowed_choice<SOFTMAX, S>(p, row, t, log2l, sm, s, lane)) return;
  }
  exact_token<SOFTMAX>(p, row, t, s, lane);
}

template <bool SOFTMAX>
hipError_t launch(const RouteGroupsParams& p, hipStream_t stream) {
  int log2l = 6;
  while ((64 >> log2l) < p.n_group) --log2l;
  const int per = p.E / p.n_group, slots = (per + (1 << log2l) - 1) >> log2l;
  const int waves = p.E <= 2048 ? kWaves : 2;    // their exact paths' keys in 32 KB of LDS
  const dim3 grid((p.T + waves - 1) / waves), block(64 * waves);
  const size_t lds = sizeof(uint32_t) * (size_t)p.E * waves;
  if (slots <= 2)
    hipLaunchKernelGGL((route_groups_kernel<SOFTMAX, 2>), grid, block, lds, stream, p, log2l);
  else if (slots <= 4)
    hipLaunchKernelGGL((route_groups_kernel<SOFTMAX, 4>), grid, block, lds, stream, p, log2l);
  else if (slots <= 8)
    hipLaunchKernelGGL((route_groups_kernel<SOFTMAX, 8>), grid, block, lds, stream, p, log2l);
  else if (slots <= 16)
    hipLaunchKernelGGL((route_groups_kernel<SOFTMAX, 16>), grid, block, lds, stream, p, log2l);
  else
    hipLaunchKernelGGL((route_groups_kernel<SOFTMAX, 0>), grid, block, lds, stream, p, log2l);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_groups(const RouteGroupsParams& p, hipStream_t stream) {
  return p.score == MOE_SCORE_SOFTMAX ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace mi355moe
