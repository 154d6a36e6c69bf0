// Device helpers of the row-wise operators (norms, balance loss, gradient
// clipping): typed loads and stores, warp and block reductions.
#pragma once
#include "lce_device.cuh"

namespace lce {

constexpr unsigned ALL_LANES = 0xffffffffu;

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Element i of an array of either type.
__device__ __forceinline__ float load_as_float(const void* p, bool f32,
                                               int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : to_float(static_cast<const __nv_bfloat16*>(p)[i]);
}
// Elements i to i + 3, which begin on four elements.
__device__ __forceinline__ void load4(const void* p, bool f32, int64_t i,
                                      float (&v)[4]) {
  if (f32) {
    const float4 q =
        *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    const uint2 q = *reinterpret_cast<const uint2*>(
        static_cast<const __nv_bfloat16*>(p) + i);
    v[0] = __uint_as_float(q.x << 16);
    v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16);
    v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
}
__device__ __forceinline__ void store_from_float(void* p, bool f32, int64_t i,
                                                 float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

template <typename T, int V>
struct Chunk;  // V elements as they lie in memory
template <>
struct Chunk<float, 4> {
  uint4 q;
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w);
  }
  __device__ __forceinline__ void pack(const float* v) {
    q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                   __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Chunk<__nv_bfloat16, 8> {
  uint4 q;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? q.x : i < 4 ? q.y : i < 6 ? q.z : q.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ void pack(const float* v) {
    q = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Chunk<float, 2> {
  uint2 q;
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i ? q.y : q.x);
  }
  __device__ __forceinline__ void pack(const float* v) {
    q = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
  }
};
template <>
struct Chunk<__nv_bfloat16, 2> {
  uint32_t q;
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i ? q & 0xffff0000u : q << 16);
  }
  __device__ __forceinline__ void pack(const float* v) {
    q = pack_bf16x2(v[0], v[1]);
  }
};
template <typename T>
struct Chunk<T, 1> {
  T q;
  __device__ __forceinline__ float at(int) const { return to_float(q); }
  __device__ __forceinline__ void pack(const float* v) {
    q = from_float<T>(v[0]);
  }
};

template <typename T, int V>
__device__ __forceinline__ Chunk<T, V> load_chunk(const T* p) {
  Chunk<T, V> c;
  c.q = *reinterpret_cast<const decltype(c.q)*>(p);
  return c;
}
template <typename T, int V>
__device__ __forceinline__ void store_chunk(T* p, const float* v) {
  Chunk<T, V> c;
  c.pack(v);
  *reinterpret_cast<decltype(c.q)*>(p) = c.q;
}

// Elements 2 p and 2 p + 1 of a thread's chunks as a packed pair.
template <typename T, int V, int C>
__device__ __forceinline__ uint64_t pair_of(const Chunk<T, V> (&q)[C], int p) {
  if constexpr (V == 1)
    return f2pack(q[2 * p].at(0), q[2 * p + 1].at(0));
  else
    return f2pack(q[2 * p / V].at(2 * p % V), q[2 * p / V].at(2 * p % V + 1));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float sum_of_pair(uint64_t a) {
  float lo, hi;
  f2unpack(a, lo, hi);
  return lo + hi;
}
template <typename T, int V>
__device__ __forceinline__ Chunk<T, V> no_chunk() {
  Chunk<T, V> c;
  memset(&c, 0, sizeof c);
  return c;
}

template <typename V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(ALL_LANES, v, o);
  return v;
}

// Sums over the block, the same bits in every thread: warps by shuffles, then
// the warps' sums in warp order. `part` holds 32 values; the block must not
// use it again before its next barrier.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V* part) {
  v = lanes_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = 0;
  const int warps = (blockDim.x + 31) >> 5;
  for (int w = 0; w < warps; ++w) t += part[w];
  return t;
}

// A sum of fp32 values to about twice their precision: the rounding of every
// addition is kept (the two-sum of Knuth) and added at the end. fp64 additions
// are a sixty-fourth as fast on this chip, and its sums here are many.
struct LongSum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float s = hi + v, w = s - hi;
    lo += (hi - (s - w)) + (v - w);
    hi = s;
  }
  __device__ __forceinline__ void add(const LongSum& v) {
    add(v.hi);
    lo += v.lo;
  }
  // an infinite or NaN sum is hi's alone
  __device__ __forceinline__ double value() const {
    return isfinite(hi) ? static_cast<double>(hi) + static_cast<double>(lo)
                        : static_cast<double>(hi);
  }
  __device__ __forceinline__ float rounded() const {
    return isfinite(hi) ? hi + lo : hi;
  }
};

// The block's sum in thread 0, warps in order; 0 elsewhere.
__device__ __forceinline__ double block_total(double v, double* part) {
  v = lanes_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0) {
    const int warps = (blockDim.x + 31) >> 5;
    for (int w = 0; w < warps; ++w) t += part[w];
  }
  return t;
}

// A kernel launched with launch_early calls the first before it touches what
// earlier kernels read or write; the second lets the next kernel begin.
__device__ __forceinline__ void wait_for_earlier() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace lce
