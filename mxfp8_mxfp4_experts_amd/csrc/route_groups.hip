// Group-limited top-k routing: sigmoid or softmax scores, a correction bias
// that only takes part in the choice, the best groups of experts, then the
// best experts in them, weights renormalised or not.
//
//   s_e   = sigmoid(l_e), or exp(l_e - max) / sum (over the unmasked experts),
//           evaluated in double and rounded once to float
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
//   * float scores differ from the exact ones by less than kScoreErr = 2^-20:
//     the exponent's argument carries |l| 2^-24 relative, which the sigmoid
//     damps to s(1-s)|l| 2^-24 < 2^-26; v_exp_f32 and v_rcp_f32 are within an
//     ulp (2^-23), the sum and the product round once each;
//   * a key adds bias in float, rounding by at most 2^-24 |key| on each side;
//   * an expert among the K largest exact keys then has a float key above the
//     K-th largest float key less twice that error; the K-th largest of the
//     lanes' largest keys is a lower bound of that, found by bisection with
//     ballots.
// Where float cannot tell (worths of the last group in and the first one out
// within their error, more than 64 candidates, NaN or huge keys), the
// wavefront evaluates everything exactly instead.
#include "common.h"
#include "launch.h"
#include "route_dev.h"

namespace mi355moe {

namespace {

constexpr float kLowest = -3.402823466e38f;
constexpr float kInf = __builtin_inff();
constexpr float kScoreErr = 9.5367431640625e-07f;     // 2^-20
constexpr float kKeyRel = 2.384185791015625e-07f;     // 2^-22
constexpr uint32_t kHuge = 0xFB800000u;   // the ordered key of 2^120: sums of two stay finite
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

__device__ __forceinline__ float wave_fmax(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ double wave_dsum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
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

struct WaveLds {
  uint32_t* keys;      // [E]: the exact path's keys
  uint64_t* cand;      // [64]
  float* score;        // [64]: candidates' scores, then the slots'
  int* id;             // [64]
  uint32_t* worth;     // [kMaxGroups]
};

// Lane k's expert by the exact scores of all experts (-1: none).
template <bool SOFTMAX>
__device__ int exact_choice(const RouteGroupsParams& p, const float* row, const Softmax& sm,
                            const WaveLds& s, int lane) {
  const int E = p.E, K = p.K, G = p.n_group, per = E / G;
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
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const uint32_t o0 = (uint32_t)__shfl_xor((int)k0, off);
        const uint32_t o1 = (uint32_t)__shfl_xor((int)k1, off);
        k1 = umax32(umin32(k0, o0), umax32(k1, o1));
        k0 = umax32(k0, o0);
      }
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
    wave_lds_fence();
    s.score[lane] = sc;
    wave_lds_fence();
    double sum = 0.0;
    for (int k = 0; k < p.K; ++k) sum += (double)s.score[k];   // left to right
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (lane < p.K) {
    p.topk_idx[t * p.K + lane] = id;
    p.topk_w[t * p.K + lane] = id >= 0 ? (float)(w * (double)p.scaling) : 0.0f;
  }
}

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
  float l[S], b[S];
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const int i = i0 + L * j;
    const bool in = g < G && i < per;
    l[j] = in ? row[g * per + i] : -kInf;
    b[j] = in && p.bias ? p.bias[g * per + i] : 0.0f;
  }
  float scale = 1.0f, top = 0.0f;
  if constexpr (SOFTMAX) {
    top = -kInf;
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (l[j] > kLowest) top = fmaxf(top, l[j]);
    top = wave_fmax(top);
    double part = 0.0;
#pragma unroll
    for (int j = 0; j < S; ++j)
      if (!(l[j] <= kLowest)) part += exp((double)l[j] - (double)top);
    sm.top = top;
    sm.total = wave_dsum(part);
    scale = (float)(1.0 / sm.total);
  }
  uint32_t key[S], best = 0, second = 0;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    float a;
    if constexpr (SOFTMAX)
      a = __builtin_amdgcn_exp2f((l[j] - top) * 1.44269504f) * scale;
    else
      a = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[j] * -1.44269504f));
    key[j] = route_key(l[j], a, b[j]);
    odd |= key[j] >= kHuge || (key[j] != 0u && key[j] <= ~kHuge);
    second = umax32(second, umin32(best, key[j]));
    best = umax32(best, key[j]);
  }
  if (__ballot(odd)) return false;

  if (G > 1) {
    uint32_t k0 = best, k1 = second;
    for (int off = L >> 1; off > 0; off >>= 1) {
      const uint32_t o0 = (uint32_t)__shfl_xor((int)k0, off);
      const uint32_t o1 = (uint32_t)__shfl_xor((int)k1, off);
      k1 = umax32(umin32(k0, o0), umax32(k1, o1));
      k0 = umax32(k0, o0);
    }
    // Every lane of a group now has its best two keys.
    float w = k0 ? key_value(k0) : -kInf;
    float err = kScoreErr + kKeyRel * fabsf(k0 ? w : 0.0f);
    if (p.group_score == MOE_GROUP_TOP2 && k1) {
      const float v = key_value(k1);
      err += kScoreErr + kKeyRel * fabsf(v);
      w += v;
      err += kKeyRel * fabsf(w);
    }
    int before = 0;
    float out_top = -kInf;       // the best worth below this group's rank, with its error
    for (int j = 0; j < G; ++j) {
      const float o = __shfl(w, j << log2l);
      before += (o > w || (o == w && j < g)) ? 1 : 0;
    }
    const bool in = g < G && before < p.topk_group;
    // Certain if every group inside stands above every one outside by their errors.
    float lo = in && k0 ? w - err : kInf;
    if (g < G && !in && k0) out_top = w + err;
    lo = -wave_fmax(-lo);
    out_top = wave_fmax(out_top);
    if (!(lo > out_top)) return false;
    if (!in) {
#pragma unroll
      for (int j = 0; j < S; ++j) key[j] = 0u;
      best = 0u;
    }
  }

  // A lower bound of the K-th largest key, to 20 of its bits: by the lanes'
  // largest keys where at least K lanes hold one, else by all keys.
  uint32_t bound = 0;
  if (__popcll(__ballot(best != 0u)) >= K) {
#pragma unroll 4
    for (int bit = 31; bit >= 12; --bit) {
      const uint32_t c = bound | (1u << bit);
      if (__popcll(__ballot(best >= c)) >= K) bound = c;
    }
  } else {
    for (int bit = 31; bit >= 12; --bit) {
      const uint32_t c = bound | (1u << bit);
      int n = 0;
#pragma unroll
      for (int j = 0; j < S; ++j) n += __popcll(__ballot(key[j] >= c));
      if (n >= K) bound = c;
    }
  }
  uint32_t least = 1u;
  if (bound > 0x00800000u) {     // below: fewer than K keys, all are candidates
    const float v = key_value(bound);
    least = umax32(1u, ordered_key(v - 4.0f * (kScoreErr + kKeyRel * fabsf(v))));
  }
  int n = 0;
  const uint64_t below = (1ull << lane) - 1;
#pragma unroll
  for (int j = 0; j < S; ++j) {
    const bool c = key[j] >= least;
    const uint64_t mask = __ballot(c);
    const int at = n + __popcll(mask & below);
    n += __popcll(mask);
    if (c && at < 64) {
      s.id[at] = g * per + i0 + L * j;
      s.score[at] = l[j];
      s.worth[at] = __float_as_uint(b[j]);
    }
  }
  if (n > 64) return false;
  wave_lds_fence();
  // Exact keys of the candidates, and each one's rank among them.
  uint64_t mine = 0;
  float sc = 0.0f;
  int id = -1;
  if (lane < n) {
    id = s.id[lane];
    const float cl = s.score[lane];
    sc = exact_score<SOFTMAX>(cl, sm);
    const uint32_t k = route_key(cl, sc, __uint_as_float(s.worth[lane]));
    if (k) mine = ((uint64_t)k << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)id);
  }
  s.cand[lane] = mine;
  wave_lds_fence();
  int rank = 0;
  for (int j = 0; j < n; ++j) rank += s.cand[j] > mine ? 1 : 0;
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
