// Tokens into expert order and back, and the gradients of both ways.
//
//   sort     rows[route_row[t, k]] = x[t]
//   unsort   out[t] = sum over kept k of w[t, k] rows[route_row[t, k]] (or without w, which is
//            also the sort's gradient), in k order, float sums, one rounding
//   grad     of the weighted unsort: drows[route_row[t, k]] = w[t, k] dout[t] and
//            dw[t, k] = <dout[t], rows[route_row[t, k]]> (float)
//
// All three run token by token, so that what a token's routes share (x[t], out[t], dout[t]) is
// read or written once and what they differ in moves as whole rows; nothing is added with
// atomics, and equal calls give equal bits.
//
// Memory bounds them at many tokens: 4096 tokens x 8 routes x 3584 in bf16, sort 264 MB in 45 us,
// 5.9 TB/s; unsort 50 us, 5.3; gradients 499 MB in 90 us, 5.5 (a copy of 2 GiB reaches 5.0).  That
// takes loads and stores that leave the caches alone (NT): with plain ones 51, 56 and 99 us.  Rows that
// the caches hold for what comes next, or from what came before, are left in them: 256 tokens x 8
// (15 MB) unsort 5.9 us plain and 7.2 past the caches.  At few tokens the chain of place, load and
// store bounds them: 8 x 16 x 7168 sort 3.6 us, unsort 5.0.
//
// A row is cut into pieces of 16 bytes.  Rows may start at any element and have any length: the
// pieces are accessed at element alignment (gfx950 takes that), and a row's last piece is moved
// back to end with the row, where it repeats elements of the piece before it (the same values
// stored twice; a sum counts them once).  Rows shorter than a piece go element by element.
#include "common.h"
#include "grid.h"
#include "launch.h"
#include "q8_dev.h"

namespace mi355moe {

namespace {

// V elements of type T as floats, and the raw piece they are loaded as.
template <class T, int V>
struct Piece;
template <>
struct Piece<uint16_t, 8> {
  typedef uint32_t Raw __attribute__((ext_vector_type(4), aligned(2)));
  static __device__ __forceinline__ void floats(Raw v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
      f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
    }
  }
  static __device__ __forceinline__ Raw raw(const float (&f)[8]) {
    return Raw{f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]),
               f32x2_to_bf16x2(f[4], f[5]), f32x2_to_bf16x2(f[6], f[7])};
  }
};
template <>
struct Piece<uint16_t, 1> {
  typedef uint16_t Raw;
  static __device__ __forceinline__ void floats(Raw v, float (&f)[1]) { f[0] = bf16_to_f32(v); }
  static __device__ __forceinline__ Raw raw(const float (&f)[1]) {
    return (Raw)f32x2_to_bf16x2(f[0], 0.0f);
  }
};
template <>
struct Piece<float, 4> {
  typedef float Raw __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ void floats(Raw v, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  }
  static __device__ __forceinline__ Raw raw(const float (&f)[4]) {
    return Raw{f[0], f[1], f[2], f[3]};
  }
};
template <>
struct Piece<float, 1> {
  typedef float Raw;
  static __device__ __forceinline__ void floats(Raw v, float (&f)[1]) { f[0] = v; }
  static __device__ __forceinline__ Raw raw(const float (&f)[1]) { return f[0]; }
};

template <class T, int V, bool NT = false>
__device__ __forceinline__ typename Piece<T, V>::Raw load(const void* base, int64_t at) {
  const auto* q =
      reinterpret_cast<const typename Piece<T, V>::Raw*>(static_cast<const T*>(base) + at);
  if constexpr (NT) return __builtin_nontemporal_load(q);
  return *q;
}
template <class T, int V, bool NT = false>
__device__ __forceinline__ void store(void* base, int64_t at, typename Piece<T, V>::Raw v) {
  auto* q = reinterpret_cast<typename Piece<T, V>::Raw*>(static_cast<T*>(base) + at);
  if constexpr (NT)
    __builtin_nontemporal_store(v, q);
  else
    *q = v;
}

// The row of route r of token t, or -1 (dropped, or past the buffer).
__device__ __forceinline__ int kept_row(const SortParams& p, int64_t t, int k) {
  const int row = p.route_row[t * p.top_k + k];
  return (uint32_t)row < (uint32_t)p.n_rows ? row : -1;
}

constexpr int kWaves = 4;      // wavefronts per workgroup, each with a run of pieces of its own

// Wavefront u takes pieces [64 c, 64 (c + 1)) of token t, u = t * runs + c.
struct Place {
  int64_t t;
  int c;
};
__device__ __forceinline__ bool place(const SortParams& p, int pieces, Place& at) {
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int runs = (pieces + 63) / 64;
  const int64_t u = (int64_t)blockIdx.x * kWaves + wave;
  at.t = u / runs;
  at.c = (int)(u - at.t * runs);
  return at.t < p.T;
}

// The places of G slots from k0 on are known before the first is used.
template <class T, int V, bool NT>
__global__ __launch_bounds__(64 * kWaves) void sort_kernel(SortParams p) {
  using R = typename Piece<T, V>::Raw;
  constexpr int G = 8;
  const int pieces = (p.H + V - 1) / V;
  Place at;
  if (!place(p, pieces, at)) return;
  const int piece = 64 * at.c + ((int)threadIdx.x & 63);
  if (piece >= pieces) return;
  const int col = min(piece * V, p.H - V);
  const R v = load<T, V>(p.x, at.t * p.ld_x + col);
  for (int k0 = 0; k0 < p.top_k; k0 += G) {
    int row[G];
#pragma unroll
    for (int j = 0; j < G; ++j) row[j] = k0 + j < p.top_k ? kept_row(p, at.t, k0 + j) : -1;
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (row[j] >= 0) store<T, V, NT>(p.rows, row[j] * p.ld_rows + col, v);
  }
}

// Slots in groups of G: their rows' loads are all on their way before the first is used.
template <class T, int V, bool WEIGHTED, bool NT>
__global__ __launch_bounds__(64 * kWaves) void unsort_kernel(SortParams p) {
  using R = typename Piece<T, V>::Raw;
  constexpr int G = 8;
  const int pieces = (p.H + V - 1) / V;
  Place at;
  if (!place(p, pieces, at)) return;
  const int piece = 64 * at.c + ((int)threadIdx.x & 63);
  if (piece >= pieces) return;
  const int col = min(piece * V, p.H - V);
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.0f;
  for (int k0 = 0; k0 < p.top_k; k0 += G) {
    int row[G];
    float w[G];
    R v[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      row[j] = k0 + j < p.top_k ? kept_row(p, at.t, k0 + j) : -1;
      w[j] = 1.0f;
      if (WEIGHTED && k0 + j < p.top_k) w[j] = p.w[at.t * p.top_k + k0 + j];
    }
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (row[j] >= 0) v[j] = load<T, V, NT>(p.rows, row[j] * p.ld_rows + col);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (row[j] < 0) continue;
      float f[V];
      Piece<T, V>::floats(v[j], f);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = WEIGHTED ? fmaf(w[j], f[i], acc[i]) : acc[i] + f[i];
    }
  }
  store<T, V>(p.x, at.t * p.ld_x + col, Piece<T, V>::raw(acc));
}

// Unit (token, group of G slots): drows and the dot products of those slots, by a workgroup (WAVE
// false) or, for rows of few pieces, by a wavefront.
template <class T, int V, int G, bool WAVE, bool NT>
__global__ __launch_bounds__(64 * kWaves) void unsort_grad_kernel(SortParams p) {
  using R = typename Piece<T, V>::Raw;
  __shared__ float sum_s[kWaves][G];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int groups = (p.top_k + G - 1) / G;
  const int64_t unit = WAVE ? (int64_t)blockIdx.x * kWaves + wave : (int64_t)blockIdx.x;
  const int64_t t = unit / groups;
  if (t >= p.T) return;
  const int k0 = (int)(unit - t * groups) * G;
  const int pieces = (p.H + V - 1) / V;
  int row[G];
  float w[G], dot[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    row[j] = k0 + j < p.top_k ? kept_row(p, t, k0 + j) : -1;
    w[j] = k0 + j < p.top_k ? p.w[t * p.top_k + k0 + j] : 0.0f;
    dot[j] = 0.0f;
  }
  for (int piece = WAVE ? lane : tid; piece < pieces; piece += WAVE ? 64 : 64 * kWaves) {
    const int col = min(piece * V, p.H - V), again = piece * V - col;   // elements counted before
    const R d = load<T, V>(p.dout, t * p.ld_dout + col);
    R v[G];
    if (p.dw) {
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (row[j] >= 0) v[j] = load<T, V, NT>(p.rows, row[j] * p.ld_rows + col);
    }
    float g[V];
    Piece<T, V>::floats(d, g);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (row[j] < 0) continue;
      if (p.drows) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = w[j] * g[i];
        store<T, V, NT>(p.drows, row[j] * p.ld_drows + col, Piece<T, V>::raw(o));
      }
      if (p.dw) {
        float f[V];
        Piece<T, V>::floats(v[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (V == 1 || i >= again) dot[j] = fmaf(g[i], f[i], dot[j]);
      }
    }
  }
  if (!p.dw) return;
  float mine = 0.0f;                        // lane j: slot j's
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const float s = wave_sum(dot[j]);
    if (lane == j) mine = s;
  }
  if constexpr (!WAVE) {
    if (lane < G) sum_s[wave][lane] = mine;
    __syncthreads();
    if (tid < G) {
      mine = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) mine += sum_s[i][tid];
    }
  }
  if ((WAVE ? lane : tid) < G && k0 + lane < p.top_k) p.dw[t * p.top_k + k0 + lane] = mine;
}

// Rows of more bytes than this go past the caches.  (Gradients of 1024 tokens x 8 x 3584 in bf16, 59
// MB: 25.9 us with plain loads and stores, 24.4 past the caches; unsort 12.7 and 12.7; of 2048, 117
// MB: 51.7 and 47.0; 30.2 and 25.6.)
constexpr int64_t kCached = 64 << 20;
// Sorted rows that begin or end within 64 bytes go through the caches all the same: 4096 x 8 x 3592
// in bf16 take 43 us so and 67 past them where the memory-side cache still holds the rows, 65 and
// 69 where not (3616 columns 44 .. 49 and 52, 58 and 52).
constexpr int kHalfLine = 64;
// Slots of a token that one unit of the gradients takes: with 8 instead of 4, 8 tokens x 16 slots
// take 8.5 us instead of 5.9 and 4096 x 8 93 instead of 90.
constexpr int kGradSlots = 4;

// The tokens from t on.
template <class T>
void advance(SortParams& p, int64_t t) {
  if (p.x) p.x = static_cast<T*>(p.x) + t * p.ld_x;
  if (p.dout) p.dout = static_cast<const T*>(p.dout) + t * p.ld_dout;
  p.route_row += t * p.top_k;
  if (p.w) p.w += t * p.top_k;
  if (p.dw) p.dw += t * p.top_k;
}

// More tokens than a launch takes go in several, one after another (2^26 of up to 512 elements in
// bf16, fewer of longer ones).
template <class T, int V, bool NT>
hipError_t sort_launch(SortParams p, SortOp op, hipStream_t stream) {
  constexpr int G = kGradSlots, kThreads = 64 * kWaves;
  const int64_t pieces = (p.H + V - 1) / V;
  const bool grad = op == SortOp::kGrad;
  const bool wave = pieces <= 64;   // 8192 x 2 x 512 in bf16: 9.9 us by workgroups, 5.4 so
  const int64_t units = grad ? (p.top_k + G - 1) / G : (pieces + 63) / 64;
  const int per_block = grad && !wave ? 1 : kWaves;
  const int64_t most = most_items(kThreads, per_block, units);
  for (int64_t left = p.T; left > 0; left -= p.T) {
    p.T = (int)(left < most ? left : most);
    const dim3 grid((unsigned)((p.T * units + per_block - 1) / per_block)), block(kThreads);
    if (op == SortOp::kSort)
      hipLaunchKernelGGL((sort_kernel<T, V, NT>), grid, block, 0, stream, p);
    else if (grad && wave)
      hipLaunchKernelGGL((unsort_grad_kernel<T, V, G, true, NT>), grid, block, 0, stream, p);
    else if (grad)
      hipLaunchKernelGGL((unsort_grad_kernel<T, V, G, false, NT>), grid, block, 0, stream, p);
    else if (p.w)
      hipLaunchKernelGGL((unsort_kernel<T, V, true, NT>), grid, block, 0, stream, p);
    else
      hipLaunchKernelGGL((unsort_kernel<T, V, false, NT>), grid, block, 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    advance<T>(p, p.T);
  }
  return hipSuccess;
}
template <class T, int V>
hipError_t sort_launch(const SortParams& p, SortOp op, hipStream_t stream) {
  const int64_t rows = (int64_t)p.T * p.top_k < p.n_rows ? (int64_t)p.T * p.top_k : p.n_rows;
  const uint64_t bytes = (uint64_t)(p.ld_rows | p.H) * sizeof(T);
  const bool odd = op == SortOp::kSort &&
                   (bytes | reinterpret_cast<uintptr_t>(p.rows)) % kHalfLine != 0;
  return rows * p.H * (int64_t)sizeof(T) > kCached && !odd ? sort_launch<T, V, true>(p, op, stream)
                                                           : sort_launch<T, V, false>(p, op, stream);
}

}  // namespace

hipError_t launch_sort(const SortParams& p, SortOp op, bool f32, hipStream_t stream) {
  if (f32)
    return p.H >= 4 ? sort_launch<float, 4>(p, op, stream) : sort_launch<float, 1>(p, op, stream);
  return p.H >= 8 ? sort_launch<uint16_t, 8>(p, op, stream)
                  : sort_launch<uint16_t, 1>(p, op, stream);
}

}  // namespace mi355moe
