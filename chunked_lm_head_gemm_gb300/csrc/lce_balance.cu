// The routing's balance loss with per-expert counts (lce_balance_forward /
// lce_balance_backward, lce_expert_counts).
//
// With p_t the normalised scores of token t, counts_e the slots of expert e, N
// the tokens that take part and f_e = E counts_e / (N K): loss = coef sum_e f_e
// mean_t p_te. Its gradient, the counts being constant, is dz_tj = coef / N
// p_tj slope_tj (f_j - sum_e f_e p_te), slope 1 for the softmax and 1 - s_tj
// for sigmoid scores. As the p of a row add up to 1, f may be shifted: f - 1
// is used, formed in fp64 from the counts, so that an even load, where the
// differences are small, loses nothing to rounding.
//
// Bound: the bytes of the logits (read in each direction) and dlogits.
#include <math.h>

#include "lce_host.h"
#include "lce_vec.cuh"

namespace lce {
namespace {

constexpr int MAX_E = 1024;
constexpr int WARPS = 8;
constexpr int64_t MAX_BLOCKS = 304;

struct BalanceArgs {
  const void* logits;
  const int32_t* experts;
  const uint8_t* mask;
  int64_t L;
  int E, K;
  int scoring;
  float coef;
  float* loss;
  int32_t* counts;
  float* slopes;
  const float* dloss;
  void* dlogits;
  float* part_p;    // [blocks][E] sums of p
  int* part_n;      // [blocks][E + 1] slots of each expert, tokens
  int blocks;
  unsigned* err;
};

__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = fmaxf(v, __shfl_xor_sync(ALL_LANES, v, o));
  return v;
}

// A row's normalised scores in place of its logits (0 where all are -inf),
// and with SLOPE the factor of the score's derivative. Element lane + 32 i.
// Sigmoid scores are taken relative to the row's largest, e^{min(z, 0) - m} /
// (1 + e^{-|z|}), so that a row of very negative logits keeps its ratios.
template <int PER, bool SLOPE>
__device__ __forceinline__ void probabilities(float (&z)[PER],
                                              float (&slope)[PER], int scoring) {
  float m = -INFINITY;
  const bool sig = scoring == LCE_SIGMOID;
#pragma unroll
  for (int i = 0; i < PER; ++i) m = fmaxf(m, sig ? fminf(z[i], 0.f) : z[i]);
  m = lanes_max(m);
  if (m == -INFINITY) m = 0.f;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (sig) {
      const float q = expf(-fabsf(z[i])), d = 1.f / (1.f + q);
      const float e = z[i] < 0.f ? (m == 0.f ? q : expf(z[i] - m)) : 1.f;
      if (SLOPE) slope[i] = z[i] < 0.f ? d : q * d;
      z[i] = e * d;
    } else {
      z[i] = expf(z[i] - m);
    }
    t += z[i];
  }
  t = lanes_sum(t);
  const float inv = t == 0.f ? 0.f : 1.f / t;
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] *= inv;
}

template <typename T, int PER>
__device__ __forceinline__ void load_row(const T* row, int E, int lane,
                                         float (&z)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + 32 * i;
    z[i] = j < E ? to_float(row[j]) : -INFINITY;
  }
}

__device__ __forceinline__ void count_slots(const int32_t* experts,
                                            const uint8_t* mask, int64_t t0,
                                            int64_t t1, int K, int E, int* hist,
                                            unsigned* err) {
  for (int64_t i = t0 * K + threadIdx.x; i < t1 * K; i += blockDim.x) {
    if (mask && !mask[i / K]) continue;
    const int e = experts[i];
    if (e >= 0 && e < E)
      atomicAdd(&hist[e], 1);
    else if (e != -1)
      atomicOr(err, ERRBIT_EXPERT_RANGE);
  }
}

// Block b takes rows [b, b + 1) L / blocks.
template <typename T, int PER>
__global__ void __launch_bounds__(WARPS * 32) k_balance(const BalanceArgs a) {
  extern __shared__ float smem[];
  float* sums = smem;                                   // [WARPS][E]
  int* hist = reinterpret_cast<int*>(smem + WARPS * a.E);  // [E + 1]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t t0 = a.L * blockIdx.x / a.blocks;
  const int64_t t1 = a.L * (blockIdx.x + 1) / a.blocks;
  count_slots(a.experts, a.mask, t0, t1, a.K, a.E, hist, a.err);
  float acc[PER] = {}, z[PER], unused[PER];
  int tokens = 0;
  for (int64_t t = t0 + warp; t < t1; t += WARPS) {
    if (a.mask && !a.mask[t]) continue;
    ++tokens;
    load_row(static_cast<const T*>(a.logits) + t * a.E, a.E, lane, z);
    probabilities<PER, false>(z, unused, a.scoring);
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] += z[i];
  }
  if (lane == 0) atomicAdd(&hist[a.E], tokens);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + 32 * i;
    if (j < a.E) sums[warp * a.E + j] = acc[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) {
    a.part_n[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + e] = hist[e];
    if (e == a.E) continue;
    float s = 0.f;
    for (int w = 0; w < WARPS; ++w) s += sums[w * a.E + e];
    a.part_p[static_cast<int64_t>(blockIdx.x) * a.E + e] = s;
  }
}

__global__ void __launch_bounds__(1024) k_balance_join(const BalanceArgs a) {
  __shared__ int tokens_of[32];
  __shared__ double part[32];
  int n = 0;
  for (int b = threadIdx.x; b < a.blocks; b += blockDim.x)
    n += a.part_n[static_cast<int64_t>(b) * (a.E + 1) + a.E];
  n = block_sum(n, tokens_of);
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double term = 0.0;
  const int e = threadIdx.x;
  if (e < a.E) {
    int c = 0;
    double p = 0.0;
    for (int b = 0; b < a.blocks; ++b) {
      c += a.part_n[static_cast<int64_t>(b) * (a.E + 1) + e];
      p += a.part_p[static_cast<int64_t>(b) * a.E + e];
    }
    const double f = c * inv * a.E / a.K;
    term = f * (p * inv);
    a.counts[e] = c;
    a.slopes[e] = static_cast<float>(a.coef * inv * (f - 1.0));
  }
  const double loss = block_sum(term, part) * a.coef;
  if (threadIdx.x == 0) *a.loss = static_cast<float>(loss);
}

template <typename T, int PER>
__global__ void __launch_bounds__(WARPS * 32)
    k_balance_bwd(const BalanceArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float d = *a.dloss;
  float f[PER], z[PER], slope[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = lane + 32 * i;
    f[i] = j < a.E ? a.slopes[j] * d : 0.f;
  }
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * WARPS + warp; t < a.L;
       t += static_cast<int64_t>(gridDim.x) * WARPS) {
    T* out = static_cast<T*>(a.dlogits) + t * a.E;
    const bool on = !a.mask || a.mask[t];
    float dot = 0.f;
    if (on) {
      load_row(static_cast<const T*>(a.logits) + t * a.E, a.E, lane, z);
      probabilities<PER, true>(z, slope, a.scoring);
#pragma unroll
      for (int i = 0; i < PER; ++i) dot = fmaf(f[i], z[i], dot);
      dot = lanes_sum(dot);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = lane + 32 * i;
      if (j >= a.E) continue;
      float v = 0.f;
      if (on) v = z[i] * (f[i] - dot);
      if (on && a.scoring == LCE_SIGMOID) v *= slope[i];
      out[j] = from_float<T>(v);
    }
  }
}

constexpr int COUNT_THREADS = 256;

__global__ void __launch_bounds__(COUNT_THREADS)
    k_expert_counts(const int32_t* experts, const uint8_t* mask, int64_t L,
                    int K, int E, int32_t* counts, unsigned* err) {
  __shared__ int hist[MAX_E];
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  count_slots(experts, mask, L * blockIdx.x / gridDim.x,
              L * (blockIdx.x + 1) / gridDim.x, K, E, hist, err);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    if (gridDim.x == 1)
      counts[e] = hist[e];
    else if (hist[e])
      atomicAdd(&counts[e], hist[e]);  // integers: the order is of no account
  }
}

// Blocks of a forward pass: a warp has a row at least.
int blocks_of(int64_t L) {
  const int64_t n = ceil_div(L, WARPS);
  return static_cast<int>(n < 1 ? 1 : n < MAX_BLOCKS ? n : MAX_BLOCKS);
}

bool sizes_ok(int64_t L, int64_t E) {
  return L >= 0 && L <= (1ll << 30) && E >= 1 && E <= MAX_E;
}
bool slots_ok(int64_t L, int64_t K) {
  return K >= 1 && K <= 32 && L * K <= (1ll << 30);
}

template <typename T>
cudaError_t launch_forward(const BalanceArgs& a, cudaStream_t s) {
  const size_t smem = (WARPS * a.E + a.E + 1) * sizeof(float);
  auto kern = a.E <= 128   ? k_balance<T, 4>
              : a.E <= 256 ? k_balance<T, 8>
              : a.E <= 512 ? k_balance<T, 16>
                           : k_balance<T, 32>;
  kern<<<a.blocks, WARPS * 32, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_backward(const BalanceArgs& a, int grid, cudaStream_t s) {
  auto kern = a.E <= 128   ? k_balance_bwd<T, 4>
              : a.E <= 256 ? k_balance_bwd<T, 8>
              : a.E <= 512 ? k_balance_bwd<T, 16>
                           : k_balance_bwd<T, 32>;
  kern<<<grid, WARPS * 32, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_balance_workspace_size(int64_t L, int64_t E) {
  if (!sizes_ok(L, E)) return 0;
  return static_cast<size_t>(blocks_of(L)) * (2 * E + 1) * 4;
}

lce_status lce_balance_forward(const void* logits, lce_dtype dt,
                               const int32_t* experts, const uint8_t* mask,
                               int64_t L, int64_t E, int64_t top_k,
                               lce_scoring scoring, float coef, float* loss,
                               int32_t* counts, float* slopes, void* ws,
                               size_t ws_bytes, void* stream) {
  if (!sizes_ok(L, E) || !slots_ok(L, top_k)) return LCE_ERR_INVALID_ARG;
  if (dt != LCE_BF16 && dt != LCE_F32) return LCE_ERR_UNSUPPORTED;
  if ((scoring != LCE_SOFTMAX && scoring != LCE_SIGMOID) || !isfinite(coef))
    return LCE_ERR_INVALID_ARG;
  if (!loss || !counts || !slopes || !ws || !aligned_to(loss, 4) ||
      !aligned_to(counts, 4) || !aligned_to(slopes, 4) || !aligned_to(ws, 16))
    return LCE_ERR_INVALID_ARG;
  if (L > 0 && (!logits || !experts || !aligned_to(experts, 4) ||
                !aligned_to(logits, dt == LCE_F32 ? 4 : 2)))
    return LCE_ERR_INVALID_ARG;
  if (ws_bytes < lce_balance_workspace_size(L, E)) return LCE_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BalanceArgs a{};
  a.logits = logits;
  a.experts = experts;
  a.mask = mask;
  a.L = L;
  a.E = static_cast<int>(E);
  a.K = static_cast<int>(top_k);
  a.scoring = scoring;
  a.coef = coef;
  a.loss = loss;
  a.counts = counts;
  a.slopes = slopes;
  a.blocks = blocks_of(L);
  a.part_p = static_cast<float*>(ws);
  a.part_n = reinterpret_cast<int*>(a.part_p + a.blocks * E);
  a.err = dev->err;
  ProfScope ps(LCE_K_BALANCE, s);
  cudaError_t e = dt == LCE_F32 ? launch_forward<float>(a, s)
                                : launch_forward<__nv_bfloat16>(a, s);
  if (e == cudaSuccess) {
    k_balance_join<<<1, 1024, 0, s>>>(a);
    e = cudaGetLastError();
  }
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "balance");
}

lce_status lce_balance_backward(const void* logits, lce_dtype dt,
                                const uint8_t* mask, int64_t L, int64_t E,
                                lce_scoring scoring, const float* slopes,
                                const float* dloss, void* dlogits,
                                void* stream) {
  if (!sizes_ok(L, E)) return LCE_ERR_INVALID_ARG;
  if (dt != LCE_BF16 && dt != LCE_F32) return LCE_ERR_UNSUPPORTED;
  if (scoring != LCE_SOFTMAX && scoring != LCE_SIGMOID)
    return LCE_ERR_INVALID_ARG;
  const uintptr_t elt = dt == LCE_F32 ? 4 : 2;
  if (L == 0) return LCE_OK;
  if (!logits || !slopes || !dloss || !dlogits || !aligned_to(logits, elt) ||
      !aligned_to(dlogits, elt) || !aligned_to(slopes, 4) ||
      !aligned_to(dloss, 4))
    return LCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  BalanceArgs a{};
  a.logits = logits;
  a.mask = mask;
  a.L = L;
  a.E = static_cast<int>(E);
  a.scoring = scoring;
  a.slopes = const_cast<float*>(slopes);
  a.dloss = dloss;
  a.dlogits = dlogits;
  const int64_t need = ceil_div(L, WARPS), most = dev->num_sms * 8;
  const int grid = static_cast<int>(need < most ? need : most);
  ProfScope ps(LCE_K_BALANCE_BWD, s);
  const cudaError_t e = dt == LCE_F32
                            ? launch_backward<float>(a, grid, s)
                            : launch_backward<__nv_bfloat16>(a, grid, s);
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "balance_bwd");
}

lce_status lce_expert_counts(const int32_t* experts, const uint8_t* mask,
                             int64_t L, int64_t E, int64_t top_k,
                             int32_t* counts, void* stream) {
  if (!sizes_ok(L, E) || !slots_ok(L, top_k)) return LCE_ERR_INVALID_ARG;
  if (!counts || !aligned_to(counts, 4) ||
      (L > 0 && (!experts || !aligned_to(experts, 4))))
    return LCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t need = ceil_div(L * top_k, 16 * COUNT_THREADS);
  const int64_t most = dev->num_sms * 2;
  const int grid = static_cast<int>(need < 1 ? 1 : need < most ? need : most);
  cudaError_t e = cudaSuccess;
  ProfScope ps(LCE_K_EXPERT_COUNTS, s);
  if (grid > 1) e = cudaMemsetAsync(counts, 0, E * sizeof(int32_t), s);
  if (e == cudaSuccess) {
    k_expert_counts<<<grid, COUNT_THREADS, 0, s>>>(
        experts, mask, L, static_cast<int>(top_k), static_cast<int>(E), counts,
        dev->err);
    e = cudaGetLastError();
  }
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "expert_counts");
}

}  // extern "C"
