// Routing of tokens to experts (lce_route_forward / lce_route_backward): one
// warp per row of router logits. Scores, group ranks, the top_k selection
// and the weights stay in registers; a row is read once and only its top_k
// weights and indices are written.
//
// Bound: the logits' bytes forward (67 MB at L = 65536, E = 256 in fp32), the
// gradient's bytes backward. The selection's rounds are what a row costs in
// instructions, so each round is two warp-wide integer reductions (largest
// ordered key, then lowest index among the lanes that hold it) on keys kept
// as order-preserving integers.
#include <math.h>

#include <type_traits>

#include "lce_device.cuh"
#include "lce_host.h"

namespace lce {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int ROUTE_WARPS = 4;  // rows per block
constexpr int MAX_E = 1024;
constexpr int MAX_K = 32;
constexpr int MAX_GROUPS = 32;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t L;
  int E, K, groups, topk_group, group_top;
  int scoring, renorm;
  float scale;
  int buf;  // shared-memory elements of one warp (group ranks), or 0
  void* weights;
  int32_t* experts;
};

// fp32 as an unsigned integer of the same order (-0 as +0); every number,
// the infinities included, lies above 0, which marks "out of the running".
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  return static_cast<float>(*p);
}
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
  v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// Element of slot i of a lane: runs of V contiguous elements per lane, so
// that loads are wide and a lane's slots rise with the element index.
template <int V>
__device__ __forceinline__ int element(int i, int lane) {
  return (i / V) * (32 * V) + lane * V + (i % V);
}

// The row's logits, -inf beyond E.
template <typename T, int PER, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int lane,
                                         float (&z)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; i += V) {
    const int j = element<V>(i, lane);
    if (V == 4) {
      float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (j < E) load4(row + j, q);  // E % 4 == 0
#pragma unroll
      for (int k = 0; k < 4; ++k) z[i + k] = q[k];
    } else {
      z[i] = j < E ? load1(row + j) : -INFINITY;
    }
  }
}

// Scores of the row in place of its logits. Softmax: exp(z - max) / sum, 0
// everywhere when no logit is above -inf; NaN logits reach the sum and with
// it every score. Error of a score, relative: below 2^-19 (expf 2 ulp twice,
// the rounding of z - max times at most ln of the score's reciprocal, a sum
// of at most 1024 terms, one division).
template <int PER>
__device__ __forceinline__ void scores(float (&z)[PER], int scoring) {
  if (scoring == LCE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < PER; ++i) z[i] = 1.f / (1.f + expf(-z[i]));
    return;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) m = fmaxf(m, z[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.f;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    z[i] = expf(z[i] - m);
    t += z[i];
  }
  t = warp_sum(t);
  if (t == 0.f) t = 1.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] /= t;
}

// Sigmoid scores of chosen logits so low that their fp32 sum loses its
// digits or vanishes (below 2^-90, logits under about -60), in fp64: this
// lane's score and the warp's sum. Lanes without a logit pass -inf.
constexpr float TINY_SUM = 0x1p-90f;
__device__ __noinline__ double sigmoid64(float z, double* sum) {
  const double p = 1.0 / (1.0 + exp(-static_cast<double>(z)));
  *sum = warp_sum(p);
  return p;
}

// Bound of the error of an fp32 key against exact arithmetic: the score's
// (scores are at most 1) and the bias addition's rounding.
__device__ __forceinline__ float key_error(float v) {
  return 0x1p-19f + 0x1p-23f * fabsf(v);
}

// Group ranks from per-element values: the values go through shared memory
// (stride chosen so that the lanes of different groups hit different banks),
// lpg lanes scan a group for its two largest values. Lane g < groups returns
// the rank of group g, -inf where the sum is not a number (inf - inf).
struct GroupGeom {
  int per, lpg, stride;
  __host__ __device__ __forceinline__ GroupGeom(int E, int groups) {
    per = E / groups;
    int p = 1;
    while (p < groups) p *= 2;
    lpg = 32 / p;
    stride = per + (lpg - per % 32 + 32) % 32;
  }
};

template <typename F, int PER, int V>
__device__ __forceinline__ F group_rank(const F (&v)[PER], F* buf, int E,
                                        int groups, int top, int lane) {
  const GroupGeom gg(E, groups);
  const F lowest = static_cast<F>(-INFINITY);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = element<V>(i, lane);
    if (j < E) buf[(j / gg.per) * gg.stride + j % gg.per] = v[i];
  }
  __syncwarp();
  const int g = lane / gg.lpg, sub = lane % gg.lpg;
  F a = lowest, b = lowest;
  if (g < groups)
    for (int r = sub; r < gg.per; r += gg.lpg) {
      const F x = buf[g * gg.stride + r];
      if (x > a) {
        b = a;
        a = x;
      } else if (x > b) {
        b = x;
      }
    }
  for (int o = gg.lpg >> 1; o > 0; o >>= 1) {
    const F xa = __shfl_xor_sync(FULL, a, o), xb = __shfl_xor_sync(FULL, b, o);
    const F lo = a < xa ? a : xa, hi = a < xa ? xa : a;
    const F nb = b < xb ? xb : b;
    a = hi;
    b = lo < nb ? nb : lo;
  }
  F rank = top == 2 ? a + b : a;
  if (isnan(rank)) rank = lowest;
  __syncwarp();
  // lane g holds group g
  return __shfl_sync(FULL, rank, (lane * gg.lpg) & 31);
}

// Bit g set: group g is kept, the `take` largest ranks with ties to the
// lowest index. Every lane returns the whole mask.
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(F rank, int groups, int take,
                                                int lane) {
  int above = 0;
  for (int g = 0; g < groups; ++g) {
    const F r = __shfl_sync(FULL, rank, g);
    if (r > rank || (r == rank && g < lane)) ++above;
  }
  return __ballot_sync(FULL, lane < groups && above < take);
}

// ---------------------------------------------------------------------------
// the row in 64 bits: taken when two fp32 keys that decide something lie
// within their error bounds
// ---------------------------------------------------------------------------
template <typename T, int PER, int V>
__device__ __noinline__ int select_exact(const RouteArgs& a, const T* row,
                                         double* buf, int lane) {
  const float* bias = a.bias;
  const bool key_is_logit = bias == nullptr;
  float z32[PER];
  load_row<T, PER, V>(row, a.E, lane, z32);
  double v[PER];
  if (a.scoring == LCE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[i] = 1.0 / (1.0 + exp(-static_cast<double>(z32[i])));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, z32[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = exp(static_cast<double>(z32[i]) - static_cast<double>(m));
      t += v[i];
    }
    t = warp_sum(t);
    if (t == 0.0) t = 1.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) v[i] /= t;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = element<V>(i, lane);
    if (bias != nullptr && j < a.E) v[i] += static_cast<double>(bias[j]);
    if (j >= a.E || !(z32[i] > -INFINITY) || isnan(v[i])) v[i] = -INFINITY;
  }
  uint32_t kept = FULL;
  const int per = a.E / a.groups;
  if (a.groups > 1) {
    const double rank =
        group_rank<double, PER, V>(v, buf, a.E, a.groups, a.group_top, lane);
    kept = keep_groups(rank, a.groups, a.topk_group, lane);
  }
  if (key_is_logit)
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[i] = z32[i] > -INFINITY ? static_cast<double>(z32[i]) : -INFINITY;
  uint32_t open = 0;  // slots still in the running
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = element<V>(i, lane);
    if (j < a.E && (a.groups == 1 || (kept >> (j / per) & 1u))) open |= 1u << i;
  }
  int mine = 0;
  for (int k = 0; k < a.K; ++k) {
    double best = 0.0;
    int at = MAX_E * 2;  // none
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if ((open >> i & 1u) && (at == MAX_E * 2 || v[i] > best)) {
        best = v[i];
        at = element<V>(i, lane);
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(FULL, best, o);
      const int oa = __shfl_xor_sync(FULL, at, o);
      const bool theirs =
          oa != MAX_E * 2 &&
          (at == MAX_E * 2 || ob > best || (ob == best && oa < at));
      if (theirs) {
        best = ob;
        at = oa;
      }
    }
    if (lane == k) mine = at;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (element<V>(i, lane) == at) open &= ~(1u << i);
  }
  return mine;
}

// The value at element j of the row (j the same in every lane).
template <int PER, int V>
__device__ __forceinline__ float gather_slot(const float (&v)[PER], int j) {
  const int slot = (j / (32 * V)) * V + j % V;
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i == slot) r = v[i];
  return __shfl_sync(FULL, r, (j / V) % 32);
}

template <typename T, int PER, int V>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
    k_route(const RouteArgs a) {
  extern __shared__ double route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x * static_cast<int64_t>(ROUTE_WARPS) + warp;
  if (row >= a.L) return;
  double* buf = route_smem + warp * a.buf;
  const T* zr = static_cast<const T*>(a.logits) + row * a.E;
  float z[PER];
  load_row<T, PER, V>(zr, a.E, lane, z);
  float s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) s[i] = z[i];
  scores<PER>(s, a.scoring);

  const bool key_is_logit = a.bias == nullptr;
  const int per = a.E / a.groups;
  float v[PER];  // keys
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = element<V>(i, lane);
    const bool live = j < a.E && z[i] > -INFINITY;
    v[i] = -INFINITY;
    if (live) {
      const float t = key_is_logit ? z[i] : s[i] + a.bias[j];
      if (!isnan(t)) v[i] = t;
    }
  }
  bool unsure = false;
  uint32_t kept = FULL;
  if (a.groups > 1) {
    float rank;
    const bool exact = key_is_logit && a.group_top == 1;
    if (key_is_logit && a.group_top == 2) {
      float u[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) u[i] = z[i] > -INFINITY ? s[i] : -INFINITY;
      rank = group_rank<float, PER, V>(u, reinterpret_cast<float*>(buf), a.E,
                                       a.groups, 2, lane);
    } else {
      rank = group_rank<float, PER, V>(v, reinterpret_cast<float*>(buf), a.E,
                                       a.groups, a.group_top, lane);
    }
    kept = keep_groups(rank, a.groups, a.topk_group, lane);
    if (!exact && a.topk_group < a.groups) {
      const bool in = kept >> lane & 1u;
      // the lowest kept rank against the highest one left out
      const float lo = -warp_max(lane < a.groups && in ? -rank : -INFINITY);
      const float hi = warp_max(lane < a.groups && !in ? rank : -INFINITY);
      if (hi > -INFINITY)
        unsure = !(lo - hi > 2.f * (key_error(lo) + key_error(hi)));
    }
  }
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = element<V>(i, lane);
    const bool in = j < a.E && (a.groups == 1 || (kept >> (j / per) & 1u));
    key[i] = in ? ordered(v[i]) : 0u;
  }

  int mine = 0;          // lane k: the k-th expert
  uint32_t last = 0;     // the previous round's key, its logit and its bias
  float last_z = 0.f, last_b = 0.f;
  const int open = a.groups == 1 ? a.E : a.topk_group * per;
  // With a bias the rounds go on past top_k until a key clearly below the
  // last one shows that nothing left out could belong in.
  for (int k = 0; k < open && !unsure; ++k) {
    if (k >= a.K && key_is_logit) break;
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(FULL, best);
    const int j = static_cast<int>(__reduce_min_sync(
        FULL, best == top ? static_cast<unsigned>(element<V>(at, lane))
                          : FULL));
    if (!key_is_logit) {
      const float jz = gather_slot<PER, V>(z, j), jb = a.bias[j];
      if (k > 0) {
        const float hi = from_ordered(last), lo = from_ordered(top);
        const bool apart =
            lo == -INFINITY || hi - lo > key_error(hi) + key_error(lo);
        if (apart && k >= a.K) break;
        // equal inputs have equal keys, whatever the rounding
        if (!apart && !(jz == last_z && jb == last_b)) unsure = true;
      }
      last = top;
      last_z = jz;
      last_b = jb;
    }
    if (lane == k) mine = j;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (element<V>(i, lane) == j) key[i] = 0u;
  }
  if (unsure)  // the same for the whole warp
    mine = select_exact<T, PER, V>(a, zr, buf, lane);

  float w = 0.f;
  for (int k = 0; k < a.K; ++k) {
    const int j = __shfl_sync(FULL, mine, k);
    const float x = gather_slot<PER, V>(s, j);
    if (lane == k) w = x;
  }
  const bool out = lane < a.K;
  if (a.renorm) {
    const float t = warp_sum(out ? w : 0.f);
    if (t < TINY_SUM && a.scoring == LCE_SIGMOID) {  // the same for the warp
      float zk = -INFINITY;
      for (int k = 0; k < a.K; ++k) {
        const float x = gather_slot<PER, V>(z, __shfl_sync(FULL, mine, k));
        if (lane == k) zk = x;
      }
      double t64;
      const double p = sigmoid64(zk, &t64);
      w = t64 == 0.0 ? 0.f : static_cast<float>(p / t64);
    } else {
      w = t == 0.f ? 0.f : w / t;
    }
  }
  w *= a.scale;
  if (out) {
    store1(static_cast<T*>(a.weights) + row * a.K + lane, w);
    a.experts[row * a.K + lane] = mine;
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct RouteBwdArgs {
  const void* logits;
  const int32_t* experts;
  const void* dweights;
  int64_t L;
  int E, K, scoring, renorm;
  float scale;
  void* dlogits;
  unsigned* err;
};

// One warp per row. Only the plain softmax needs the whole row again (its
// gradient is nonzero everywhere); the other forms read the chosen logits
// alone and write zeros elsewhere. The row is written first, the chosen
// elements after it by the same warp.
template <typename T, int PER, int V, bool WHOLE>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
    k_route_bwd(const RouteBwdArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x * static_cast<int64_t>(ROUTE_WARPS) + warp;
  if (row >= a.L) return;
  const T* zr = static_cast<const T*>(a.logits) + row * a.E;
  T* dr = static_cast<T*>(a.dlogits) + row * a.E;

  int j = -1;
  float u = 0.f;
  if (lane < a.K) {
    j = a.experts[row * a.K + lane];
    if (j < 0 || j >= a.E) {
      atomicOr(a.err, ERRBIT_EXPERT_RANGE);
      j = -1;
    } else {
      u = a.scale *
          load1(static_cast<const T*>(a.dweights) + row * a.K + lane);
    }
  }
  float p = 0.f, d = 0.f;
  float fill[PER];
  if (WHOLE) {
    load_row<T, PER, V>(zr, a.E, lane, fill);
    scores<PER>(fill, LCE_SOFTMAX);
    for (int k = 0; k < a.K; ++k) {
      const int jk = __shfl_sync(FULL, j, k);
      const float x = gather_slot<PER, V>(fill, jk < 0 ? 0 : jk);
      if (lane == k && j >= 0) p = x;
    }
    const float dot = warp_sum(u * p);
    d = p * u;  // the element's own share; -p dot once per element, below
#pragma unroll
    for (int i = 0; i < PER; ++i) fill[i] *= -dot;
  } else {
    const float z = j >= 0 ? load1(zr + j) : -INFINITY;
    if (a.scoring == LCE_SOFTMAX) {  // renormalised: a softmax of the chosen
      float m = warp_max(z);
      if (m == -INFINITY) m = 0.f;
      p = j >= 0 ? expf(z - m) : 0.f;
      float t = warp_sum(p);
      if (t == 0.f) t = 1.f;
      const float q = p / t;
      const float dot = warp_sum(u * q);
      d = q * (u - dot);
    } else {
      p = j >= 0 ? 1.f / (1.f + expf(-z)) : 0.f;
      const float slope = j >= 0 ? p / (1.f + expf(z)) : 0.f;  // p (1 - p)
      if (a.renorm) {
        const float t = warp_sum(p);
        float q = t == 0.f ? 0.f : p / t;
        float gain = t == 0.f ? 0.f : slope / t;
        if (t < TINY_SUM) {
          double t64;
          const double p64 = sigmoid64(z, &t64);
          q = t64 == 0.0 ? 0.f : static_cast<float>(p64 / t64);
          gain = q;  // p (1 - p) / t with 1 - p = 1
        }
        const float dot = warp_sum(u * q);
        d = gain * (u - dot);
      } else {
        d = slope * u;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PER; i += V) {
    const int e = element<V>(i, lane);
    if (e >= a.E) continue;
    if (V == 4) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = WHOLE ? fill[i + k] : 0.f;
      store4(dr + e, q);
    } else {
      store1(dr + e, WHOLE ? fill[i] : 0.f);
    }
  }
  // shares of an index given more than once add up in the first lane of it
  float sum = 0.f;
  bool first = j >= 0;
  for (int k = 0; k < a.K; ++k) {
    const int jk = __shfl_sync(FULL, j, k);
    const float dk = __shfl_sync(FULL, d, k);
    if (jk == j) {
      sum += dk;
      if (k < lane) first = false;
    }
  }
  if (WHOLE) {
    const float dot = warp_sum(u * p);
    sum -= p * dot;
  }
  __syncwarp();  // the row's stores come before the chosen elements'
  if (first) store1(dr + j, sum);
}

template <typename T, int PER, int V>
cudaError_t launch_route_t(const RouteArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(double) * ROUTE_WARPS * a.buf;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(
        k_route<T, PER, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = static_cast<unsigned>(ceil_div(a.L, ROUTE_WARPS));
  k_route<T, PER, V><<<grid, ROUTE_WARPS * 32, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int PER, int V>
cudaError_t launch_route_bwd_t(const RouteBwdArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(ceil_div(a.L, ROUTE_WARPS));
  if (a.scoring == LCE_SOFTMAX && !a.renorm)
    k_route_bwd<T, PER, V, true><<<grid, ROUTE_WARPS * 32, 0, s>>>(a);
  else
    k_route_bwd<T, PER, V, false><<<grid, ROUTE_WARPS * 32, 0, s>>>(a);
  return cudaGetLastError();
}

// Slots per lane by E; wide loads when every row starts on 4 elements.
template <typename T, int V, class Args>
cudaError_t by_width(const Args& a, cudaStream_t s) {
  constexpr bool FWD = std::is_same<Args, RouteArgs>::value;
  const int per = a.E <= 128 ? 4 : a.E <= 256 ? 8 : a.E <= 512 ? 16 : 32;
  if constexpr (FWD) {
    switch (per) {
      case 4: return launch_route_t<T, 4, V>(a, s);
      case 8: return launch_route_t<T, 8, V>(a, s);
      case 16: return launch_route_t<T, 16, V>(a, s);
      default: return launch_route_t<T, 32, V>(a, s);
    }
  } else {
    switch (per) {
      case 4: return launch_route_bwd_t<T, 4, V>(a, s);
      case 8: return launch_route_bwd_t<T, 8, V>(a, s);
      case 16: return launch_route_bwd_t<T, 16, V>(a, s);
      default: return launch_route_bwd_t<T, 32, V>(a, s);
    }
  }
}

template <class Args>
cudaError_t dispatch(const Args& a, lce_dtype dt, bool wide, cudaStream_t s) {
  if (dt == LCE_F32)
    return wide ? by_width<float, 4>(a, s) : by_width<float, 1>(a, s);
  return wide ? by_width<__nv_bfloat16, 4>(a, s)
              : by_width<__nv_bfloat16, 1>(a, s);
}

// What both calls check of their sizes and options.
lce_status check(int64_t L, int64_t E, lce_dtype dt, const lce_route_opts* o) {
  if (!o || L < 0 || E < 1) return LCE_ERR_INVALID_ARG;
  if (dt != LCE_BF16 && dt != LCE_F32) return LCE_ERR_UNSUPPORTED;
  if (E > MAX_E || L > (1ll << 31)) return LCE_ERR_INVALID_ARG;
  if (o->scoring != LCE_SOFTMAX && o->scoring != LCE_SIGMOID)
    return LCE_ERR_INVALID_ARG;
  if (o->top_k < 1 || o->top_k > MAX_K || o->top_k > E ||
      (o->renormalize != 0 && o->renormalize != 1) || !isfinite(o->scale))
    return LCE_ERR_INVALID_ARG;
  return LCE_OK;
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

lce_status lce_route_forward(const void* logits, lce_dtype dt,
                             const float* bias, int64_t L, int64_t E,
                             const lce_route_opts* opts, void* weights,
                             int32_t* experts, void* stream) {
  lce_status st = check(L, E, dt, opts);
  if (st != LCE_OK) return st;
  const lce_route_opts& o = *opts;
  if (o.n_group < 1 || o.n_group > MAX_GROUPS || E % o.n_group ||
      o.topk_group < 1 || o.topk_group > o.n_group ||
      o.top_k > o.topk_group * (E / o.n_group))
    return LCE_ERR_INVALID_ARG;
  if (o.n_group > 1 && (o.group_top < 1 || o.group_top > 2 ||
                        o.group_top > E / o.n_group))
    return LCE_ERR_INVALID_ARG;
  const uintptr_t elt = dt == LCE_F32 ? 4 : 2;
  if (!aligned_to(bias, 4)) return LCE_ERR_INVALID_ARG;
  if (L == 0) return LCE_OK;
  if (!logits || !weights || !experts || !aligned_to(logits, elt) ||
      !aligned_to(weights, elt) || !aligned_to(experts, 4))
    return LCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != LCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.L = L;
  a.E = static_cast<int>(E);
  a.K = o.top_k;
  a.groups = o.topk_group == o.n_group ? 1 : o.n_group;  // all kept: no groups
  a.topk_group = o.topk_group;
  a.group_top = o.group_top;
  a.scoring = o.scoring;
  a.renorm = o.renormalize;
  a.scale = o.scale;
  if (a.groups > 1) a.buf = a.groups * GroupGeom(a.E, a.groups).stride;
  a.weights = weights;
  a.experts = experts;
  ProfScope ps(LCE_K_ROUTE, s);
  const cudaError_t e =
      dispatch(a, dt, E % 4 == 0 && aligned_to(logits, 4 * elt), s);
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "route");
}

lce_status lce_route_backward(const void* logits, lce_dtype dt,
                              const int32_t* experts, const void* dweights,
                              int64_t L, int64_t E,
                              const lce_route_opts* opts, void* dlogits,
                              void* stream) {
  lce_status st = check(L, E, dt, opts);
  if (st != LCE_OK) return st;
  if (L == 0) return LCE_OK;
  const uintptr_t elt = dt == LCE_F32 ? 4 : 2;
  if (!logits || !experts || !dweights || !dlogits ||
      !aligned_to(logits, elt) || !aligned_to(dweights, elt) ||
      !aligned_to(dlogits, elt) || !aligned_to(experts, 4))
    return LCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  if ((st = device_info(&dev)) != LCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouteBwdArgs a{};
  a.logits = logits;
  a.experts = experts;
  a.dweights = dweights;
  a.L = L;
  a.E = static_cast<int>(E);
  a.K = opts->top_k;
  a.scoring = opts->scoring;
  a.renorm = opts->renormalize;
  a.scale = opts->scale;
  a.dlogits = dlogits;
  a.err = dev->err;
  ProfScope ps(LCE_K_ROUTE_BWD, s);
  const cudaError_t e = dispatch(a, dt,
                                 E % 4 == 0 && aligned_to(logits, 4 * elt) &&
                                     aligned_to(dlogits, 4 * elt),
                                 s);
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "route_bwd");
}

}  // extern "C"
