// Routing of tokens to experts (lce_route_forward / lce_route_backward): a
// warp to a row of router logits (k_route), or four rows to a warp where there
// are many (k_route_many). A row is read once, its scores, group ranks and
// top_k selection stay on the SM (in registers; k_route_many's keys in shared
// memory), and only its top_k weights and indices are written.
//
// Bound: the logits' bytes (67 MB at L = 65536, E = 256 in fp32), but the
// instructions of the selection come first. So the selection does not search
// the row top_k times: the n-th largest of the 32 lanes' maxima is a lower
// bound of the row's n-th largest key, and the few keys that reach it (about
// n + 2 of 256) are packed one to a lane and ranked against each other at
// once. Scores of a whole row are computed only where its keys or its sum
// need them, with the fast exponential; the chosen ones again, exactly.
// Against top_k rounds of two warp-wide reductions over the whole row, both a
// warp to a row: L = 32768, E = 128, top 8 of bf16 39 -> 31 us; L = 65536, E =
// 256 in 8 groups with a bias 223 -> 121 us, which k_route_many does in 61.
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

// The row's maximum for the softmax (0 for a row without a finite logit).
template <int PER>
__device__ __forceinline__ float row_max(const float (&z)[PER]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) m = fmaxf(m, z[i]);
  m = warp_max(m);
  return m == -INFINITY ? 0.f : m;
}

// Scores of the row in place of its logits, by ex2.approx. Softmax: exp(z -
// max) / sum, 0 everywhere when no logit is above -inf; NaN logits reach the
// sum and with it every score. Returns the sum (1 for an empty row; sigmoid:
// 1). With e the error of ex2.approx, 2^-22, and that of its argument,
// 1.5 * 2^-24 of it: a sigmoid score is off by at most s (1 - s) (e + 1.5 *
// 2^-24 |z|) + 2^-22 + 2^-24 < 2^-21; a softmax score, whose terms lose 2.5 *
// 2^-24 d to an argument -d and whose sum of at most 1024 adds 36 * 2^-24, by
// at most 2^-17 of itself (d < 17) or 2^-24 (beyond, where it is tiny).
template <int PER>
__device__ __forceinline__ float scores(float (&z)[PER], int scoring,
                                        float m) {
  if (scoring == LCE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      z[i] = __fdividef(1.f, 1.f + ex2(-z[i] * LOG2E));
    return 1.f;
  }
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    z[i] = ex2((z[i] - m) * LOG2E);
    t += z[i];
  }
  t = warp_sum(t);
  if (t == 0.f) t = 1.f;
  const float r = 1.f / t;
#pragma unroll
  for (int i = 0; i < PER; ++i) z[i] *= r;
  return t;
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

// Bound of the error of an fp32 key v with bias b: the score's (scores())
// and the rounding of the addition.
__device__ __forceinline__ float key_error(float v, float b, int scoring) {
  const float s = scoring == LCE_SIGMOID
                      ? 0x1p-21f
                      : 0x1p-17f * fabsf(v - b) + 0x1p-24f;
  return s + 0x1p-23f * fabsf(v);
}

// Group ranks from per-element values: the values go through shared memory
// (stride chosen so that the lanes of different groups hit different banks),
// lpg lanes scan a group for its two largest values. Lane g < groups returns
// the rank of group g, -inf where the sum is not a number (inf - inf).
struct GroupGeom {
  int per, lpg, stride;
  unsigned recip;  // ceil(2^20 / per): j / per = j recip >> 20 for j < 1024
  GroupGeom() = default;
  GroupGeom(int E, int groups) {
    per = E / groups;
    recip = ((1u << 20) + per - 1) / per;
    int p = 1;
    while (p < groups) p *= 2;
    lpg = 32 / p;
    stride = per + (lpg - per % 32 + 32) % 32;
  }
  __device__ __forceinline__ int group(int j) const {
    return static_cast<int>(static_cast<unsigned>(j) * recip >> 20);
  }
};

struct RouteArgs {
  const void* logits;
  const float* bias;
  int64_t L;
  int E, K, groups, topk_group, group_top;
  int scoring, renorm;
  float scale;
  GroupGeom gg;
  int warp_smem;  // shared memory of one warp, in doubles
  void* weights;
  int32_t* experts;
};

template <typename F, int PER, int V>
__device__ __forceinline__ F group_rank(const F (&v)[PER], F* buf,
                                        const RouteArgs& a_, int top,
                                        int lane) {
  const GroupGeom& gg = a_.gg;
  const int E = a_.E, groups = a_.groups;
  const F lowest = static_cast<F>(-INFINITY);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = element<V>(i, lane);
    if (j < E) buf[j + gg.group(j) * (gg.stride - gg.per)] = v[i];
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
// the whole row in 64 bits: taken when two group ranks lie within their error
// bounds, or when more than 32 keys with a bias reach the threshold
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
  if (a.groups > 1) {
    const double rank = group_rank<double, PER, V>(v, buf, a, a.group_top, lane);
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
    if (j < a.E && (a.groups == 1 || (kept >> a.gg.group(j) & 1u)))
      open |= 1u << i;
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

// The candidates' order in 64 bits, where neighbours lie within their fp32
// errors: one exact key a lane, compared as ordered integers (the fp64 pipe
// is 64 times slower than fp32's, so it sees one exponential and one division
// a lane, not the whole row; a softmax needs the row's sum in fp64 too).
// Returns lane k's k-th candidate.
template <typename T, int PER, int V>
__device__ __noinline__ int rank_exact(const RouteArgs& a, const T* row,
                                       bool live, int j, float z, float b,
                                       int lane, uint2* list) {
  double p;
  if (a.scoring == LCE_SIGMOID) {
    p = 1.0 / (1.0 + exp(-static_cast<double>(z)));
  } else {
    float zs[PER];
    load_row<T, PER, V>(row, a.E, lane, zs);
    const float m = row_max<PER>(zs);
    double t = 0.0;
#pragma unroll 1
    for (int i = 0; i < PER; ++i)
      t += exp(static_cast<double>(zs[i]) - static_cast<double>(m));
    t = warp_sum(t);
    p = exp(static_cast<double>(z) - static_cast<double>(m)) / t;
  }
  double v = p + static_cast<double>(b);
  if (!(z > -INFINITY) || isnan(v)) v = -INFINITY;
  const long long bits = __double_as_longlong(v + 0.0);
  const unsigned long long key =
      live ? (bits < 0 ? ~static_cast<unsigned long long>(bits)
                       : static_cast<unsigned long long>(bits) | 1ull << 63)
           : 0ull;
  __syncwarp();
  list[lane] = make_uint2(static_cast<unsigned>(key >> 32),
                          static_cast<unsigned>(key));
  list[32 + lane] = make_uint2(static_cast<unsigned>(j), 0u);
  __syncwarp();
  int rank = 0;
  for (int q = 0; q < 32; ++q) {
    const uint2 o = list[q];
    const unsigned long long ok =
        static_cast<unsigned long long>(o.x) << 32 | o.y;
    const int oj = static_cast<int>(list[32 + q].x);
    if (ok > key || (ok == key && oj < j && ok != 0ull)) ++rank;
  }
  __syncwarp();
  if (live) list[rank] = make_uint2(static_cast<unsigned>(j), 0u);
  __syncwarp();
  return static_cast<int>(list[lane].x);
}

// top_k rounds over the whole row, each the largest key and the lowest index
// that has it: for exact keys of which more than 32 reach the threshold.
template <int PER, int V>
__device__ __forceinline__ int select_rounds(const uint32_t (&keys)[PER], int K,
                                          int lane) {
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = keys[i];
  int mine = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    const uint32_t top = __reduce_max_sync(FULL, best);
    unsigned j = FULL;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == top) j = static_cast<unsigned>(element<V>(i, lane));
    j = __reduce_min_sync(FULL, j);
    if (lane == k) mine = static_cast<int>(j);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (static_cast<unsigned>(element<V>(i, lane)) == j) key[i] = 0u;
  }
  return mine;
}

// The chosen score of one lane from its logit, to fp32 accuracy.
__device__ __forceinline__ float one_score(float z, int scoring, float m,
                                           float t) {
  return scoring == LCE_SIGMOID ? 1.f / (1.f + expf(-z)) : expf(z - m) / t;
}

// smem of a warp: two lists of 32 (key, element), then the group ranks.
constexpr int LIST_BYTES = 2 * 32 * 8;

// One row by a whole warp.
template <typename T, int PER, int V>
__device__ __forceinline__ void route_row(const RouteArgs& a, int64_t row,
                                          int lane, double* smem) {
  uint2* list = reinterpret_cast<uint2*>(smem);
  double* buf = smem + LIST_BYTES / 8;
  const T* zr = static_cast<const T*>(a.logits) + row * a.E;
  float z[PER];
  load_row<T, PER, V>(zr, a.E, lane, z);

  const bool biased = a.bias != nullptr;
  const bool rank_scores = a.groups > 1 && a.group_top == 2;
  const bool softmax = a.scoring == LCE_SOFTMAX;
  // a softmax renormalised over the chosen needs neither maximum nor sum
  const bool whole = biased || rank_scores || (softmax && !a.renorm);
  float m = 0.f, t = 1.f;
  float v[PER];  // keys
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = z[i];
  if (whole) {
    if (softmax) m = row_max<PER>(z);
    t = scores<PER>(v, a.scoring, m);
  }
  if (biased) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = element<V>(i, lane);
      if (j < a.E) v[i] += a.bias[j];
    }
  }
  bool unsure = false;
  uint32_t kept = FULL;
  if (a.groups > 1) {
    // masked experts, and keys that are no numbers, rank lowest
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!(z[i] > -INFINITY) || isnan(v[i])) v[i] = -INFINITY;
    const bool exact = !biased && !rank_scores;
    if (exact) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        v[i] = z[i] > -INFINITY ? z[i] : -INFINITY;
    }
    const float rank = group_rank<float, PER, V>(
        v, reinterpret_cast<float*>(buf), a, a.group_top, lane);
    kept = keep_groups(rank, a.groups, a.topk_group, lane);
    if (!exact) {
      const bool in = kept >> lane & 1u;
      // the lowest kept rank against the highest one left out; of the
      // softmax scores in a rank none is above the row's largest, 1 / t
      const float lo = -warp_max(lane < a.groups && in ? -rank : -INFINITY);
      const float hi = warp_max(lane < a.groups && !in ? rank : -INFINITY);
      const float top = softmax ? 1.f / t : 0.f;
      float big = 0.f;  // the largest key's size: what additions round by
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (v[i] > -INFINITY) big = fmaxf(big, fabsf(v[i]));
      big = warp_max(big);
      const float err = key_error(top, 0.f, a.scoring) + 0x1p-22f * big;
      if (hi > -INFINITY) unsure = !(lo - hi > 4.f * err);
    }
  }
  uint32_t key[PER], largest = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int j = element<V>(i, lane);
    const bool in = j < a.E && (a.groups == 1 || (kept >> a.gg.group(j) & 1u));
    const float x = biased ? v[i] : z[i];
    const bool live = z[i] > -INFINITY && !isnan(x);
    key[i] = in ? ordered(live ? x : -INFINITY) : 0u;
    largest = max(largest, key[i]);
  }

  // threshold: the want-th largest of the lanes' maxima; every key if fewer
  // lanes than that are in the running
  const int open = a.groups == 1 ? a.E : a.topk_group * a.gg.per;
  const int want = min(open, a.K + (biased ? 1 : 0));
  uint32_t floor_key = 1u;
  {
    uint32_t cur = largest;
    for (int k = 0; k < want; ++k) {
      floor_key = __reduce_max_sync(FULL, cur);
      const unsigned who = __ballot_sync(FULL, cur == floor_key);
      if (lane == __ffs(who) - 1) cur = 0u;
    }
    if (biased && floor_key > 0u) {
      // down by what both sides of the border may be off, so that nothing
      // below it can belong to the chosen in exact arithmetic
      const float x = from_ordered(floor_key);
      const float s_max = softmax ? 1.f / t : 1.f;
      const float err = key_error(s_max, 0.f, a.scoring) +
                        0x1p-23f * (fabsf(x) + s_max);
      if (x > -INFINITY) floor_key = ordered(x - 4.f * err);
    }
    floor_key = max(floor_key, 1u);
  }
  int found = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool take = key[i] >= floor_key;
    const unsigned who = __ballot_sync(FULL, take);
    const int at = found + __popc(who & ((1u << lane) - 1u));
    if (take && at < 32)
      list[at] = make_uint2(key[i], static_cast<unsigned>(element<V>(i, lane)));
    found += __popc(who);
  }
  int mine = 0;  // lane k: the k-th expert
  if (found < want) unsure = true;  // an infinite bias has no finite border
  if (found > 32) {
    if (biased)
      unsure = true;
    else if (!unsure)
      mine = select_rounds<PER, V>(key, a.K, lane);
  } else if (!unsure) {
    __syncwarp();
    const uint2 own = lane < found ? list[lane] : make_uint2(0u, 0u);
    int rank = 0;
    for (int q = 0; q < found; ++q) {
      const uint2 o = list[q];
      if (o.x > own.x || (o.x == own.x && o.y < own.y)) ++rank;
    }
    if (lane < found) list[32 + rank] = own;
    __syncwarp();
    const uint2 at = list[32 + (lane < found ? lane : 0)];
    mine = static_cast<int>(at.y);
    if (biased) {
      // neighbours in the order: apart beyond their errors, or the same
      // inputs (equal keys, whatever the rounding)
      const float x = from_ordered(at.x), jz = load1(zr + mine),
                  jb = a.bias[mine];
      const float err = key_error(x, jb, a.scoring);
      const float nx = __shfl_down_sync(FULL, x, 1),
                  nz = __shfl_down_sync(FULL, jz, 1),
                  nb = __shfl_down_sync(FULL, jb, 1),
                  ne = __shfl_down_sync(FULL, err, 1);
      const bool pair = lane + 1 < found;
      const bool apart = pair && (nx == -INFINITY || x - nx > err + ne);
      const bool same = pair && nz == jz && nb == jb;
      const unsigned apart_of = __ballot_sync(FULL, apart);
      const unsigned fine = __ballot_sync(FULL, apart || same);
      // the first clear step at or past the last chosen key
      const unsigned past = apart_of >> (a.K - 1) << (a.K - 1);
      const int end = past ? __ffs(past) - 1 : found - 1;
      const unsigned before = end >= 31 ? 0x7fffffffu : (1u << end) - 1u;
      // a key further down with a larger score has a larger error, which may
      // reach over the step
      const float reach =
          warp_max(lane > end && lane < found ? x + err : -INFINITY);
      const bool clear = __shfl_sync(FULL, x - err, end) > reach ||
                         reach == -INFINITY;
      if ((fine & before) != before || !clear)  // the same for the whole warp
        mine = rank_exact<T, PER, V>(a, zr, lane < found, mine, jz, jb, lane,
                                     list);
    }
  }
  if (unsure)  // the same for the whole warp
    mine = select_exact<T, PER, V>(a, zr, buf, lane);

  const bool out = lane < a.K;
  const float zk = out ? load1(zr + mine) : -INFINITY;
  float w;
  if (a.renorm) {
    if (softmax) {
      m = warp_max(zk);
      if (m == -INFINITY) m = 0.f;
      w = out ? expf(zk - m) : 0.f;
      bool nan = false;  // a NaN anywhere in the row reaches every weight
#pragma unroll
      for (int i = 0; i < PER; ++i) nan |= isnan(z[i]);
      if (__any_sync(FULL, nan)) w = NAN;
    } else {
      w = out ? one_score(zk, LCE_SIGMOID, 0.f, 1.f) : 0.f;
    }
    const float sum = warp_sum(w);
    if (sum < TINY_SUM && !softmax) {  // the same for the warp
      double sum64;
      const double p = sigmoid64(zk, &sum64);
      w = sum64 == 0.0 ? 0.f : static_cast<float>(p / sum64);
    } else {
      w = sum == 0.f ? 0.f : w / sum;
    }
  } else {
    w = out ? one_score(zk, a.scoring, m, t) : 0.f;
  }
  w *= a.scale;
  if (out) {
    store1(static_cast<T*>(a.weights) + row * a.K + lane, w);
    a.experts[row * a.K + lane] = mine;
  }
}

template <typename T, int PER, int V>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
    k_route(const RouteArgs a) {
  extern __shared__ double route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x * static_cast<int64_t>(ROUTE_WARPS) + warp;
  if (row >= a.L) return;
  route_row<T, PER, V>(a, row, lane, route_smem + warp * a.warp_smem);
}

// ---------------------------------------------------------------------------
// many rows: four to a warp, eight lanes to a row. The steps are those of
// route_row, but the warp-wide reductions become three shuffles for four rows,
// and the kept groups alone are searched. The keys lie in shared memory
// (element j of a row belongs to lane j % 8; the row stride is 8 mod 32, so
// the 32 lanes hit 32 banks). Rows with a NaN, with more than 32
// candidates, or with softmax keys that fp32 does not settle go through
// route_row afterwards; sigmoid keys are settled in place in fp64, for a row
// that goes through route_row keeps its warp 20 us longer. Against a
// warp to a row: L = 32768, E = 128, top 8 of fp32 26 -> 14 us, E = 256 in 8
// groups with a bias 60 -> 31 us.
// ---------------------------------------------------------------------------
constexpr int MANY_LANES = 8;               // lanes of a row
constexpr int MANY_ROWS = 32 / MANY_LANES;  // rows of a warp
constexpr int MANY_MAXIMA = 32 / MANY_LANES;
constexpr int MANY_K = 8;
constexpr int MANY_LIST = 32;

// Shared memory of a warp: keys, candidates, sorted candidates, group ranks
// and kept groups.
__host__ __device__ __forceinline__ int many_stride(int E) {
  if (E < 2 * MANY_LIST) E = 2 * MANY_LIST;  // or the candidates' exact keys
  return E + (MANY_LANES - E % 32 + 32) % 32;
}
__host__ __device__ __forceinline__ int many_bytes(int E, int groups) {
  return MANY_ROWS *
         (many_stride(E) * 4 + MANY_LIST * 8 + (MANY_K + 2) * 8 + 2 * groups * 4);
}

// Reductions over a row's lanes, in each of them.
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = 1; o < MANY_LANES; o <<= 1)
    v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < MANY_LANES; o <<= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
__device__ __forceinline__ unsigned lanes_ballot(bool p, int lane) {
  return __ballot_sync(FULL, p) >> (lane & ~(MANY_LANES - 1)) &
         ((1u << MANY_LANES) - 1u);
}

template <typename T, int PER, int V>
__device__ __noinline__ void route_row_again(const RouteArgs& a, int64_t row,
                                             int lane, double* smem) {
  route_row<T, PER, V>(a, row, lane, smem);
}

template <typename T, int PER, int V>
__global__ void __launch_bounds__(ROUTE_WARPS * 32, PER <= 8 ? 8 : 4)
    k_route_many(const RouteArgs a) {
  extern __shared__ double route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 =
      (blockIdx.x * static_cast<int64_t>(ROUTE_WARPS) + warp) * MANY_ROWS;
  if (row0 >= a.L) return;
  double* smem = route_smem + warp * a.warp_smem;
  const int E = a.E, stride = many_stride(E);
  float* keys = reinterpret_cast<float*>(smem);
  uint2* lists = reinterpret_cast<uint2*>(keys + MANY_ROWS * stride);
  uint2* sorted = lists + MANY_ROWS * MANY_LIST;
  float* ranks = reinterpret_cast<float*>(sorted + MANY_ROWS * (MANY_K + 2));
  int* kept_list = reinterpret_cast<int*>(ranks + MANY_ROWS * a.groups);

  const bool biased = a.bias != nullptr;
  const bool softmax = a.scoring == LCE_SOFTMAX;
  const bool rank_scores = a.groups > 1 && a.group_top == 2;
  const bool whole = biased || rank_scores || (softmax && !a.renorm);

  // ---- the rows' logits, or their keys where those need no other element ----
  const int rows =
      a.L - row0 < MANY_ROWS ? static_cast<int>(a.L - row0) : MANY_ROWS;
  const T* base = static_cast<const T*>(a.logits) + row0 * E;
  const bool keys_now = biased && !softmax;
  float bias[PER];
  if (keys_now) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = element<V>(i, lane);
      bias[i] = j < E ? a.bias[j] : 0.f;
    }
  }
  unsigned nan_rows = 0;
  float big = 0.f;  // the largest key's size
#pragma unroll
  for (int r = 0; r < MANY_ROWS; ++r) {
    float z[PER];
    // rows past the last repeat it: they are computed and not written
    load_row<T, PER, V>(base + static_cast<int64_t>(min(r, rows - 1)) * E, E,
                        lane, z);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) nan |= isnan(z[i]);
    if (__any_sync(FULL, nan)) nan_rows |= 1u << r;
    if (keys_now) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float x =
            __fdividef(1.f, 1.f + ex2(-z[i] * LOG2E)) + bias[i];
        z[i] = z[i] > -INFINITY && !isnan(x) ? x : -INFINITY;
        if (z[i] > -INFINITY) big = fmaxf(big, fabsf(z[i]));
      }
    }
#pragma unroll
    for (int i = 0; i < PER; i += V) {
      const int j = element<V>(i, lane);
      if (j >= E) continue;
      if (V == 4)
        *reinterpret_cast<float4*>(keys + r * stride + j) =
            make_float4(z[i], z[i + (V > 1 ? 1 : 0)], z[i + (V > 2 ? 2 : 0)],
                        z[i + (V > 3 ? 3 : 0)]);
      else
        keys[r * stride + j] = z[i];
    }
  }
  if (keys_now) big = warp_max(big);
  __syncwarp();

  const int r = lane / MANY_LANES, s = lane % MANY_LANES;
  float* key = keys + r * stride;
  bool slow = nan_rows >> r & 1u;

  // ---- softmax maximum and sum -----------------------------------------------
  float m = 0.f, t = 1.f;
  if (softmax && whole) {
    m = -INFINITY;
    for (int j = s; j < E; j += MANY_LANES) m = fmaxf(m, key[j]);
    m = lanes_max(m);
    if (m == -INFINITY) m = 0.f;
    if (m == INFINITY) slow = true;
    t = 0.f;
    for (int j = s; j < E; j += MANY_LANES) t += ex2((key[j] - m) * LOG2E);
    t = lanes_sum(t);
    if (t == 0.f) t = 1.f;
  }
  const float rt = 1.f / t;
  auto score = [&](float z) {
    return softmax ? ex2((z - m) * LOG2E) * rt
                   : __fdividef(1.f, 1.f + ex2(-z * LOG2E));
  };
  if (biased && softmax) {
    for (int j = s; j < E; j += MANY_LANES) {
      const float k = key[j];
      float v = score(k) + a.bias[j];
      if (!(k > -INFINITY) || isnan(v)) v = -INFINITY;
      key[j] = v;
      if (v > -INFINITY) big = fmaxf(big, fabsf(v));
    }
    big = lanes_max(big);
  }

  // ---- groups ------------------------------------------------------------------
  const float s_max = softmax ? rt : 1.f;
  if (a.groups > 1) {
    const int per = a.gg.per;
    const bool by_score = rank_scores && !biased;
    for (int g = 0; g < a.groups; ++g) {
      float x = -INFINITY, y = -INFINITY;  // two largest
#pragma unroll 4
      for (int j = s; j < per; j += MANY_LANES) {
        float v = key[g * per + j];
        if (by_score && v > -INFINITY) v = score(v);
        y = fmaxf(y, fminf(x, v));
        x = fmaxf(x, v);
      }
#pragma unroll
      for (int o = 1; o < MANY_LANES; o <<= 1) {
        const float ox = __shfl_xor_sync(FULL, x, o),
                    oy = __shfl_xor_sync(FULL, y, o);
        y = fmaxf(fmaxf(y, oy), fminf(x, ox));
        x = fmaxf(x, ox);
      }
      float rank = a.group_top == 2 ? x + y : x;
      if (isnan(rank)) rank = -INFINITY;
      if (s == 0) ranks[r * a.groups + g] = rank;
    }
    __syncwarp();
    float lo = INFINITY, hi = -INFINITY;
    for (int g = s; g < a.groups; g += MANY_LANES) {
      const float mine = ranks[r * a.groups + g];
      int above = 0;
      for (int q = 0; q < a.groups; ++q) {
        const float o = ranks[r * a.groups + q];
        if (o > mine || (o == mine && q < g)) ++above;
      }
      if (above < a.topk_group) {
        kept_list[r * a.groups + above] = g;
        lo = fminf(lo, mine);
      } else {
        hi = fmaxf(hi, mine);
      }
    }
    lo = -lanes_max(-lo);
    hi = lanes_max(hi);
    if (biased || rank_scores) {
      const float size = biased ? big : s_max;
      const float err = key_error(s_max, 0.f, a.scoring) + 0x1p-22f * size;
      const bool close = hi > -INFINITY && !(lo - hi > 4.f * err);
      // an infinite key leaves no border to collect a group's largest by
      if (softmax || !(err < INFINITY)) {  // sigmoid: the same for the warp
        slow |= close;
      } else if (__any_sync(FULL, close)) {
        // ranks in 64 bits, a lane to a group: the exact values of the keys
        // that may be among its group_top largest
        double* exact = reinterpret_cast<double*>(lists + r * MANY_LIST);
        const T* zr = base + static_cast<int64_t>(min(r, rows - 1)) * E;
        for (int g0 = 0; g0 < a.groups; g0 += MANY_LANES) {
          const int g = g0 + s;
          float x = -INFINITY, y = -INFINITY;
          for (int j = 0; g < a.groups && j < per; ++j) {
            float v = key[g * per + j];
            if (by_score && v > -INFINITY) v = score(v);
            y = fmaxf(y, fminf(x, v));
            x = fmaxf(x, v);
          }
          const float from = (a.group_top == 2 ? y : x) - 4.f * err;
          int pick[4] = {0, 0, 0, 0}, n = 0;  // collected first: the lanes'
          for (int j = 0; g < a.groups && j < per; ++j) {  // exponentials run
            float v = key[g * per + j];                    // side by side
            if (!(v > -INFINITY)) continue;  // masked
            if (by_score) v = score(v);
            if (!(v >= from)) continue;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c == n) pick[c] = g * per + j;
            ++n;
          }
          if (n > 4) slow = true;
          double x64 = -INFINITY, y64 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (!__any_sync(FULL, c < n)) break;
            double e =
                1.0 / (1.0 + exp(-static_cast<double>(load1(zr + pick[c]))));
            if (biased) e += static_cast<double>(a.bias[pick[c]]);
            if (c < n) {
              y64 = fmax(y64, fmin(x64, e));
              x64 = fmax(x64, e);
            }
          }
          double rank = a.group_top == 2 ? x64 + y64 : x64;
          if (isnan(rank)) rank = -INFINITY;
          if (g < a.groups) exact[g] = rank;
        }
        __syncwarp();
        for (int g = s; g < a.groups; g += MANY_LANES) {
          const double mine = exact[g];
          int above = 0;
          for (int q = 0; q < a.groups; ++q) {
            const double o = exact[q];
            if (o > mine || (o == mine && q < g)) ++above;
          }
          if (above < a.topk_group) kept_list[r * a.groups + above] = g;
        }
      }
    }
    __syncwarp();
  }
  const int runs = a.groups > 1 ? a.topk_group : 1;
  const int per = a.groups > 1 ? a.gg.per : E;

  // ---- threshold: the want-th largest of 32 maxima of the row -----------------
  const int want = min(runs * per, a.K + (biased ? 1 : 0));
  float mx[MANY_MAXIMA];
#pragma unroll
  for (int q = 0; q < MANY_MAXIMA; ++q) mx[q] = -INFINITY;
  for (int x = 0; x < runs; ++x) {
    const float* run = key + (a.groups > 1 ? kept_list[r * a.groups + x] * per
                                           : 0);
    for (int i = s; i < per; i += 32) {
#pragma unroll
      for (int q = 0; q < MANY_MAXIMA; ++q)
        if (i + MANY_LANES * q < per)
          mx[q] = fmaxf(mx[q], run[i + MANY_LANES * q]);
    }
  }
  // each lane's maxima in falling order
  static_assert(MANY_MAXIMA == 4, "network of four");
  auto order = [&](int x, int y) {
    const float hi = fmaxf(mx[x], mx[y]), lo = fminf(mx[x], mx[y]);
    mx[x] = hi;
    mx[y] = lo;
  };
  order(0, 1), order(2, 3), order(0, 2), order(1, 3), order(1, 2);
  float floor_key = -INFINITY;  // -inf: every key is a candidate
  for (int k = 0; k < want; ++k) {
    floor_key = lanes_max(mx[0]);
    const unsigned who = lanes_ballot(mx[0] == floor_key, lane);
    if (s == __ffs(who) - 1) {
#pragma unroll
      for (int q = 0; q + 1 < MANY_MAXIMA; ++q) mx[q] = mx[q + 1];
      mx[MANY_MAXIMA - 1] = -INFINITY;
    }
  }
  if (biased && floor_key > -INFINITY) {
    const float err = key_error(s_max, 0.f, a.scoring) +
                      0x1p-23f * (fabsf(floor_key) + s_max);
    floor_key -= 4.f * err;
  }

  // ---- candidates, packed by row ------------------------------------------------
  uint2* list = lists + r * MANY_LIST;
  int found = 0;
  for (int x = 0; x < runs; ++x) {
    const int j0 = a.groups > 1 ? kept_list[r * a.groups + x] * per : 0;
#pragma unroll 4
    for (int i = 0; i < per; i += MANY_LANES) {
      const int j = i + s;
      const float k = j < per ? key[j0 + j] : 0.f;
      const bool take = j < per && k >= floor_key;
      const unsigned who = lanes_ballot(take, lane);
      const int at = found + __popc(who & ((1u << s) - 1u));
      if (take && at < MANY_LIST)
        list[at] =
            make_uint2(__float_as_uint(k), static_cast<unsigned>(j0 + j));
      found += __popc(who);
    }
  }
  if (found > MANY_LIST || found < want) slow = true;
  __syncwarp();
  // ---- their order ---------------------------------------------------------------
  uint2* fall = sorted + r * (MANY_K + 2);
  const int count = min(found, MANY_LIST);
  float reach = -INFINITY;  // how far up a key beyond the chosen may belong
  for (int c = s; c < count; c += MANY_LANES) {
    const uint2 own = list[c];
    const float v = __uint_as_float(own.x);
    int rank = 0;
#pragma unroll 4
    for (int q = 0; q < count; ++q) {
      const uint2 o = list[q];
      const float ov = __uint_as_float(o.x);
      if (ov > v || (ov == v && o.y < own.y)) ++rank;
    }
    if (rank <= MANY_K) fall[rank] = own;
    if (biased && softmax && rank >= a.K && v > -INFINITY)
      reach = fmaxf(reach, v + key_error(v, a.bias[own.y], a.scoring));
  }
  __syncwarp();
  const int64_t row = row0 + r;
  const bool in = r < rows;
  const T* zr = base + static_cast<int64_t>(in ? r : rows - 1) * E;
  if (biased) {
    // neighbours apart beyond their errors, or the same inputs; the last
    // chosen one apart from the next
    bool close = false;
    for (int k = s; k < a.K && k + 1 < count; k += MANY_LANES) {
      const uint2 p = fall[k], q = fall[k + 1];
      const float x = __uint_as_float(p.x), y = __uint_as_float(q.x);
      if (y == -INFINITY) continue;
      const float bx = a.bias[p.y], by = a.bias[q.y];
      const bool apart = x - y > key_error(x, bx, a.scoring) +
                                     key_error(y, by, a.scoring);
      if (!apart && (k + 1 == a.K || bx != by ||
                     load1(zr + p.y) != load1(zr + q.y)))
        close = true;
    }
    if (softmax) {
      // a larger score has a larger error: every key beyond the chosen is
      // held against the last of them, not the next one alone
      reach = lanes_max(reach);
      if (count > a.K && reach > -INFINITY) {
        const uint2 last = fall[a.K - 1];
        const float x = __uint_as_float(last.x);
        close |= !(x - key_error(x, a.bias[last.y], a.scoring) > reach);
      }
      slow |= close;  // the exact scores need the row's sum
    } else if (__any_sync(FULL, close)) {
      // the order in 64 bits: exact keys of the candidates as ordered
      // integers, in the place of the row's fp32 keys
      unsigned long long* exact = reinterpret_cast<unsigned long long*>(key);
      for (int c = s; c < count; c += MANY_LANES) {
        const unsigned j = list[c].y;
        const float z = load1(zr + j);
        double v = 1.0 / (1.0 + exp(-static_cast<double>(z))) +
                   static_cast<double>(a.bias[j]);
        if (!(z > -INFINITY) || isnan(v)) v = -INFINITY;
        const long long bits = __double_as_longlong(v + 0.0);
        exact[c] = static_cast<unsigned long long>(bits) ^
                   (static_cast<unsigned long long>(bits >> 63) | 1ull << 63);
      }
      __syncwarp();
      for (int c = s; c < count; c += MANY_LANES) {
        const unsigned long long own = exact[c];
        const unsigned j = list[c].y;
        int rank = 0;
#pragma unroll 4
        for (int q = 0; q < count; ++q) {
          const unsigned long long o = exact[q];
          if (o > own || (o == own && list[q].y < j)) ++rank;
        }
        if (rank <= MANY_K) fall[rank] = list[c];
      }
      __syncwarp();
    }
  }
  slow = lanes_ballot(slow, lane) != 0u;

  // ---- weights: lane s has choice s ----------------------------------------------
  static_assert(MANY_K <= MANY_LANES, "a lane to a choice");
  const bool out = s < a.K && !slow;
  const int chosen = out ? static_cast<int>(fall[s].y) : 0;
  const float zk = out ? load1(zr + chosen) : -INFINITY;
  if (a.renorm && softmax) {
    m = lanes_max(zk);
    if (m == -INFINITY) m = 0.f;
    t = 1.f;
  }
  float w = s < a.K ? one_score(zk, a.scoring, m, t) : 0.f;
  if (a.renorm) {
    const float sum = lanes_sum(w);
    if (!softmax && sum < TINY_SUM) slow = true;  // the same for the row
    w = sum == 0.f ? 0.f : w / sum;
  }
  if (in && !slow && s < a.K) {
    store1(static_cast<T*>(a.weights) + row * a.K + s, w * a.scale);
    a.experts[row * a.K + s] = chosen;
  }
  unsigned again = __ballot_sync(FULL, slow && in && s == 0);
  __syncwarp();
  while (again) {
    const int q = (__ffs(again) - 1) / MANY_LANES;
    again &= again - 1u;
    route_row_again<T, PER, V>(a, row0 + q, lane, smem);
    __syncwarp();
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

// Sums over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float row_top(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

// The choices of a row sit in LANES lanes (8 when top_k <= 8: four rows to a
// warp). Only the plain softmax needs the whole row again (its gradient is
// nonzero everywhere; one row to a warp); the other forms read the chosen
// logits alone and write zeros elsewhere, so they are bound by dlogits'
// bytes. The rows are written first, the chosen elements after them by the
// same warp. Four rows to a warp against one: L = 32768, E = 128, top 8 of
// bf16 26.6 -> 7.9 us, L = 65536, E = 256, fp32 27.4 -> 16.7 us.
template <typename T, int PER, int V, int LANES, bool WHOLE>
__global__ void __launch_bounds__(ROUTE_WARPS * 32)
    k_route_bwd(const RouteBwdArgs a) {
  constexpr int ROWS = 32 / LANES;
  static_assert(!WHOLE || ROWS == 1, "one row to a warp");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 =
      (blockIdx.x * static_cast<int64_t>(ROUTE_WARPS) + warp) * ROWS;
  if (row0 >= a.L) return;
  const int64_t row = row0 + lane / LANES;
  const int k = lane % LANES;
  const T* zr = static_cast<const T*>(a.logits) + row * a.E;
  T* dr = static_cast<T*>(a.dlogits) + row * a.E;

  int j = -1;
  float u = 0.f;
  if (k < a.K && row < a.L) {
    j = a.experts[row * a.K + k];
    if (j < 0 || j >= a.E) {
      atomicOr(a.err, ERRBIT_EXPERT_RANGE);
      j = -1;
    } else {
      u = a.scale * load1(static_cast<const T*>(a.dweights) + row * a.K + k);
    }
  }
  const float z = j >= 0 ? load1(zr + j) : -INFINITY;
  float p = 0.f, d = 0.f, dot = 0.f;
  if (WHOLE) {
    float fill[PER];
    load_row<T, PER, V>(zr, a.E, lane, fill);
    const float m = row_max<PER>(fill);
    const float t = scores<PER>(fill, LCE_SOFTMAX, m);
    if (j >= 0) p = one_score(z, LCE_SOFTMAX, m, t);
    dot = row_sum<LANES>(u * p);
    d = p * u;  // an element's own shares; -p dot once per element
#pragma unroll
    for (int i = 0; i < PER; i += V) {
      const int e = element<V>(i, lane);
      if (e >= a.E) continue;
      if (V == 4) {
        float q[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) q[x] = -fill[i + x] * dot;
        store4(dr + e, q);
      } else {
        store1(dr + e, -fill[i] * dot);
      }
    }
  } else {
    // the warp's rows are contiguous: zeros, 16 bytes a lane where aligned
    const int64_t left = a.L - row0;
    const int n = static_cast<int>(left < ROWS ? left : ROWS) * a.E;
    T* d0 = static_cast<T*>(a.dlogits) + row0 * a.E;
    constexpr int W = V == 4 ? 16 / sizeof(T) : 1;
    if (V == 4 && n % W == 0 && (reinterpret_cast<uintptr_t>(d0) & 15u) == 0) {
      for (int e = lane; e < n / W; e += 32)
        reinterpret_cast<uint4*>(d0)[e] = make_uint4(0, 0, 0, 0);
    } else {
      for (int e = lane; e < n; e += 32) store1(d0 + e, 0.f);
    }
    if (a.scoring == LCE_SOFTMAX) {  // renormalised: a softmax of the chosen
      float m = row_top<LANES>(z);
      if (m == -INFINITY) m = 0.f;
      p = j >= 0 ? expf(z - m) : 0.f;
      float t = row_sum<LANES>(p);
      if (t == 0.f) t = 1.f;
      const float q = p / t;
      const float all = row_sum<LANES>(u * q);
      d = q * (u - all);
    } else {
      p = j >= 0 ? 1.f / (1.f + expf(-z)) : 0.f;
      const float slope = j >= 0 ? p / (1.f + expf(z)) : 0.f;  // p (1 - p)
      if (a.renorm) {
        const float t = row_sum<LANES>(p);
        float q = t == 0.f ? 0.f : p / t;
        float gain = t == 0.f ? 0.f : slope / t;
        if (__any_sync(FULL, t < TINY_SUM)) {
          const double p64 = 1.0 / (1.0 + exp(-static_cast<double>(z)));
          double t64 = p64;
#pragma unroll
          for (int o = LANES / 2; o > 0; o >>= 1)
            t64 += __shfl_xor_sync(FULL, t64, o);
          if (t < TINY_SUM) {
            q = t64 == 0.0 ? 0.f : static_cast<float>(p64 / t64);
            gain = q;  // p (1 - p) / t with 1 - p = 1
          }
        }
        const float all = row_sum<LANES>(u * q);
        d = gain * (u - all);
      } else {
        d = slope * u;
      }
    }
  }
  // shares of an index given more than once in a row add up in the first
  // lane that has it, in the order of the choices
  const unsigned mates =
      (LANES == 32 ? FULL : ((1u << LANES) - 1u) << (lane & ~(LANES - 1)));
  const unsigned same = __match_any_sync(FULL, j) & mates;
  const bool first = j >= 0 && (same & ((1u << lane) - 1u)) == 0u;
  float sum = d;
  if (__any_sync(FULL, j >= 0 && (same & (same - 1u)) != 0u)) {
    sum = 0.f;
    for (int q = 0; q < LANES; ++q) {
      const int from = (lane & ~(LANES - 1)) + q;
      const float dq = __shfl_sync(FULL, d, from);
      if (same >> from & 1u) sum += dq;
    }
  }
  if (WHOLE) sum -= p * dot;
  __syncwarp();  // the rows' stores come before the chosen elements'
  if (first) store1(dr + j, sum);
}

// Four rows to a warp from MANY_MIN rows on: at E = 128 (fp32, top 8) L = 2048
// takes 4.7 us a warp to a row and 5.1 us four to a warp, L = 4096 5.8 and 5.1.
constexpr int64_t MANY_MIN = 3000;
constexpr int MANY_MAX_E = 512;  // shared memory of the keys

// The largest size of any call: a group's stride is below its experts + 32,
// and what a warp of k_route_many adds to that is less.
constexpr int MAX_WARP_BYTES = LIST_BYTES + 8 * (MAX_E + 31 * MAX_GROUPS);
constexpr int MAX_ROUTE_SMEM = ROUTE_WARPS * MAX_WARP_BYTES;
static_assert(MAX_WARP_BYTES % 16 == 0, "rows of doubles");
static_assert(MANY_ROWS * ((MANY_MAX_E + 31) * 4 + MANY_LIST * 8 +
                           (MANY_K + 2) * 8 + 2 * MAX_GROUPS * 4) <=
                  MAX_WARP_BYTES,
              "k_route_many's part");

template <typename T, int PER, int V>
cudaError_t launch_route_t(const RouteArgs& args, cudaStream_t s) {
  RouteArgs a = args;
  constexpr bool FITS = 32 * PER <= MANY_MAX_E;  // by_width: E <= 32 PER
  const bool many = FITS && a.L >= MANY_MIN && a.K <= MANY_K;
  int bytes = LIST_BYTES + (a.groups > 1 ? 8 * a.groups * a.gg.stride : 0);
  if (many && many_bytes(a.E, a.groups) > bytes)
    bytes = many_bytes(a.E, a.groups);
  a.warp_smem = (bytes + 15) / 16 * 2;
  const size_t smem = sizeof(double) * ROUTE_WARPS * a.warp_smem;
  auto kern = k_route<T, PER, V>;
  if constexpr (FITS) {
    if (many) kern = k_route_many<T, PER, V>;
  }
  if (smem > 48 * 1024) {
    // one value for every call: the limit is the process's, and another
    // thread may launch between this and the launch below
    cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_ROUTE_SMEM);
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = static_cast<unsigned>(
      ceil_div(a.L, ROUTE_WARPS * (many ? MANY_ROWS : 1)));
  kern<<<grid, ROUTE_WARPS * 32, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int PER, int V>
cudaError_t launch_route_bwd_t(const RouteBwdArgs& a, cudaStream_t s) {
  const bool whole = a.scoring == LCE_SOFTMAX && !a.renorm;
  const bool four = !whole && a.K <= 8;
  auto kern = whole  ? k_route_bwd<T, PER, V, 32, true>
              : four ? k_route_bwd<T, PER, V, 8, false>
                     : k_route_bwd<T, PER, V, 32, false>;
  const unsigned grid = static_cast<unsigned>(
      ceil_div(a.L, ROUTE_WARPS * (four ? 4 : 1)));
  kern<<<grid, ROUTE_WARPS * 32, 0, s>>>(a);
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
  a.gg = GroupGeom(a.E, a.groups);
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
