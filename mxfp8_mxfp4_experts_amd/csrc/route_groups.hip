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
// One workgroup per token: its four wavefronts evaluate the scores (a double
// exp each, which is what bounds the kernel) and the groups' worths; the
// first one selects.
#include "common.h"
#include "launch.h"
#include "route_dev.h"

namespace mi355moe {

namespace {

constexpr float kLowest = -3.402823466e38f;
constexpr int kThreads = 256;
constexpr int kPerThread = kMaxExperts / kThreads;

__device__ __forceinline__ double block_reduce_sum(double v, double* s) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
}
__device__ __forceinline__ float block_reduce_max(float v, float* s) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
}

// The float that ordered_key mapped to k (k >= 2).
__device__ __forceinline__ float key_value(uint32_t k) {
  return k == 1u ? __uint_as_float(0x7FC00000u)
                 : __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// 0 for an expert that may not be taken, else the ordered key.
__device__ __forceinline__ uint32_t route_key(float logit, float score, float bias) {
  const float key = score + bias;
  return (logit <= kLowest || key == -__builtin_inff()) ? 0u : ordered_key(key);
}

__global__ __launch_bounds__(kThreads) void route_groups_kernel(RouteGroupsParams p) {
  extern __shared__ uint32_t keys_s[];   // [E]
  __shared__ uint64_t cand_s[64];
  __shared__ uint32_t worth_s[kMaxGroups];
  __shared__ double dsum_s[4];
  __shared__ float fmax_s[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = p.E, K = p.K, G = p.n_group, per = E / G;
  const int64_t t = blockIdx.x;
  const float* row = p.logits + t * p.ld;

  float top = -__builtin_inff();
  double total = 1.0;
  if (p.score == MOE_SCORE_SOFTMAX) {
    for (int e = tid; e < E; e += kThreads) {
      const float l = row[e];
      if (l > kLowest) top = fmaxf(top, l);
    }
    top = block_reduce_max(top, fmax_s);
    double part = 0.0;
    for (int e = tid; e < E; e += kThreads) {
      const float l = row[e];
      if (!(l <= kLowest)) part += exp((double)l - (double)top);
    }
    total = block_reduce_sum(part, dsum_s);
  }
  auto score_of = [&](float l) -> float {
    if (p.score == MOE_SCORE_SOFTMAX)
      return l <= kLowest ? 0.0f : (float)(exp((double)l - (double)top) / total);
    return sigmoid_score(l);
  };
  for (int e = tid; e < E; e += kThreads) {
    const float l = row[e];
    keys_s[e] = route_key(l, score_of(l), p.bias ? p.bias[e] : 0.0f);
  }
  __syncthreads();

  if (G > 1) {
    for (int g = wave; g < G; g += 4) {
      uint32_t k0 = 0, k1 = 0;   // the group's best two keys
      for (int i = lane; i < per; i += 64) {
        const uint32_t k = keys_s[g * per + i];
        k1 = k > k0 ? k0 : (k > k1 ? k : k1);
        k0 = k > k0 ? k : k0;
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const uint32_t o0 = (uint32_t)__shfl_xor((int)k0, off);
        const uint32_t o1 = (uint32_t)__shfl_xor((int)k1, off);
        k1 = umax32(umin32(k0, o0), umax32(k1, o1));
        k0 = umax32(k0, o0);
      }
      if (lane == 0) {
        uint32_t w = k0;
        if (p.group_score == MOE_GROUP_TOP2 && k1 != 0u)
          w = ordered_key(key_value(k0) + key_value(k1));
        worth_s[g] = w;   // 0: every expert of the group is masked
      }
    }
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
      const int g = e / per;
      const uint32_t mine = worth_s[g];
      int before = 0;
      for (int j = 0; j < G; ++j) {
        const uint32_t o = worth_s[j];
        before += (o > mine || (o == mine && j < g)) ? 1 : 0;
      }
      if (before >= p.topk_group) keys_s[e] = 0u;
    }
    __syncthreads();
  }
  if (wave != 0) return;

  int id = -1;
  if (E <= 64 * kRegExpertsPerLane) {
    if (!select_topk_threshold(keys_s, E, K, lane, cand_s, id))
      id = select_topk_rounds(keys_s, E, K, lane);
  } else {
    uint64_t last = ~0ull;
    for (int k = 0; k < K; ++k) {
      uint64_t best = 0;
      for (int e = lane; e < E; e += 64) {
        const uint64_t c = ((uint64_t)keys_s[e] << 32) | (uint64_t)(0xFFFFFFFFu - (uint32_t)e);
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
  if (lane >= K || id < 0 || id >= E || keys_s[id] == 0u) id = -1;
  const float s = id >= 0 ? score_of(row[id]) : 0.0f;
  double w = (double)s;
  if (p.renormalise) {
    double sum = 0.0;
    for (int k = 0; k < K; ++k) sum += (double)__shfl(s, k);   // left to right
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (lane < K) {
    p.topk_idx[t * K + lane] = id;
    p.topk_w[t * K + lane] = id >= 0 ? (float)(w * (double)p.scaling) : 0.0f;
  }
}

}  // namespace

hipError_t launch_route_groups(const RouteGroupsParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(route_groups_kernel, dim3(p.T), dim3(kThreads), sizeof(uint32_t) * p.E,
                     stream, p);
  return hipGetLastError();
}

}  // namespace mi355moe
