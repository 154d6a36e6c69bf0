// The norm of many gradients together, and their clipping (lce_grad_norm /
// lce_clip_grads).
//
// norm = sqrt(sum of all g^2), out = min(1, max_norm / (norm + 1e-6)) g. A
// launch takes a table of tensors as its argument; their elements are cut into
// chunks, and a block takes every gridDim-th chunk.
//
// Squares of a group of a few elements are added in fp32, groups in fp64. A
// group whose sum leaves the range in which fp32 squares are exact to their
// rounding is added again in fp64 from the elements, so gradients far below
// 1e-19 or above 1e19 count in full.
//
// Bound: the bytes of the gradients, read for the norm, read and written for
// the clipping.
#include <math.h>

#include <algorithm>
#include <new>

#include "lce_host.h"
#include "lce_vec.cuh"

namespace lce {
namespace {

constexpr int TABLE = 96;        // tensors of a launch
constexpr int GRAD_BLOCKS = 608;
constexpr int GRAD_THREADS = 256;
constexpr int64_t CHUNK = 16384;  // elements

struct GradTable {
  const void* grad[TABLE];
  void* out[TABLE];
  int64_t size[TABLE];
  int64_t first[TABLE + 1];  // chunks before a tensor's own
  uint8_t f32[TABLE];
  int count;
};

__device__ __forceinline__ int tensor_of(const GradTable& t, int64_t chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <int N>
__device__ __forceinline__ void add_squares(const float (&v)[N], double& sum) {
  float s = 0.f;
  bool any = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s = fmaf(v[i], v[i], s);
    any |= v[i] != 0.f;
  }
  if (s >= 1e-28f && s <= 1e37f) {
    sum += static_cast<double>(s);
  } else if (any) {
    for (int i = 0; i < N; ++i)
      sum += static_cast<double>(v[i]) * static_cast<double>(v[i]);
  }
}

__global__ void __launch_bounds__(GRAD_THREADS)
    k_grad_squares(const __grid_constant__ GradTable t, double* part) {
  __shared__ double warps[32];
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = tensor_of(t, c);
    const int64_t i0 = (c - t.first[k]) * CHUNK;
    const int64_t i1 = min(i0 + CHUNK, t.size[k]);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += GRAD_THREADS) {
      const float v[1] = {load_as_float(t.grad[k], t.f32[k], i)};
      add_squares(v, sum);
    }
  }
  sum = block_sum(sum, warps);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(1024)
    k_grad_norm(const double* part, int64_t n, float* norm) {
  __shared__ double warps[32];
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) sum += part[i];
  sum = block_sum(sum, warps);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

__global__ void __launch_bounds__(GRAD_THREADS)
    k_clip(const __grid_constant__ GradTable t, const float* norm,
           float max_norm) {
  const double r =
      static_cast<double>(max_norm) / (static_cast<double>(*norm) + 1e-6);
  // a norm that is NaN makes every gradient NaN
  const float scale = isinf(max_norm) || r >= 1.0 ? 1.f : static_cast<float>(r);
  for (int64_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int k = tensor_of(t, c);
    if (scale == 1.f && t.out[k] == t.grad[k]) continue;
    const int64_t i0 = (c - t.first[k]) * CHUNK;
    const int64_t i1 = min(i0 + CHUNK, t.size[k]);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += GRAD_THREADS)
      store_from_float(t.out[k], t.f32[k], i,
                       load_as_float(t.grad[k], t.f32[k], i) * scale);
  }
}

int64_t bytes_of(lce_dtype dt, int64_t n) { return n * (dt == LCE_F32 ? 4 : 2); }

lce_status check(const void* const* grads, const lce_dtype* dts,
                 const int64_t* sizes, int64_t n) {
  if (n < 0 || n > (1 << 20)) return LCE_ERR_INVALID_ARG;
  if (n > 0 && (!grads || !dts || !sizes)) return LCE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n; ++i) {
    if (dts[i] != LCE_BF16 && dts[i] != LCE_F32) return LCE_ERR_UNSUPPORTED;
    if (sizes[i] < 0 || sizes[i] > (1ll << 40)) return LCE_ERR_INVALID_ARG;
    if (sizes[i] > 0 &&
        (!grads[i] || !aligned_to(grads[i], dts[i] == LCE_F32 ? 4 : 2)))
      return LCE_ERR_INVALID_ARG;
  }
  return LCE_OK;
}

// What is written must not be read or written through another tensor: the
// outputs are disjoint, a gradient is its own output or apart from all, and the
// norm is apart from all.
lce_status check_disjoint(const void* const* grads, void* const* outs,
                          const lce_dtype* dts, const int64_t* sizes, int64_t n,
                          const float* norm) {
  struct Range {
    uintptr_t a, b;
  };
  Range* r = new (std::nothrow) Range[n];
  if (!r) return cuda_fail(cudaErrorMemoryAllocation, "clip_grads (host)");
  int64_t m = 0;
  for (int64_t i = 0; i < n; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(outs[i]);
    if (sizes[i] > 0) r[m++] = {a, a + bytes_of(dts[i], sizes[i])};
  }
  std::sort(r, r + m, [](const Range& x, const Range& y) { return x.a < y.a; });
  bool ok = true;
  for (int64_t i = 1; i < m; ++i) ok = ok && r[i - 1].b <= r[i].a;
  auto apart = [&](const void* from, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(from);
    // the last output that begins before the end
    const Range* p = std::lower_bound(
        r, r + m, a + bytes, [](const Range& x, uintptr_t v) { return x.a < v; });
    return p == r || p[-1].b <= a;
  };
  ok = ok && apart(norm, sizeof(float));
  for (int64_t i = 0; ok && i < n; ++i)
    if (sizes[i] > 0 && grads[i] != outs[i])
      ok = apart(grads[i], bytes_of(dts[i], sizes[i]));
  delete[] r;
  return ok ? LCE_OK : LCE_ERR_INVALID_ARG;
}

// Calls launch(table, index) for every table of up to TABLE tensors.
template <class F>
cudaError_t each_table(const void* const* grads, void* const* outs,
                       const lce_dtype* dts, const int64_t* sizes, int64_t n,
                       F&& launch) {
  GradTable t;
  int index = 0;
  t.count = 0;
  t.first[0] = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (sizes[i] > 0) {
      const int k = t.count++;
      t.grad[k] = grads[i];
      t.out[k] = outs ? outs[i] : nullptr;
      t.size[k] = sizes[i];
      t.f32[k] = dts[i] == LCE_F32;
      t.first[k + 1] = t.first[k] + ceil_div(sizes[i], CHUNK);
    }
    if (t.count == TABLE || (i == n - 1 && t.count > 0)) {
      const int64_t chunks = t.first[t.count];
      const int grid =
          static_cast<int>(chunks < GRAD_BLOCKS ? chunks : GRAD_BLOCKS);
      launch(t, grid, index++);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      t.count = 0;
    }
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_grad_norm_workspace_size(int64_t n) {
  if (n < 0 || n > (1 << 20)) return 0;
  return static_cast<size_t>(ceil_div(n < 1 ? 1 : n, TABLE)) * GRAD_BLOCKS *
         sizeof(double);
}

lce_status lce_grad_norm(const void* const* grads, const lce_dtype* dts,
                         const int64_t* sizes, int64_t n, float* norm, void* ws,
                         size_t ws_bytes, void* stream) {
  LCE_TRY(check(grads, dts, sizes, n));
  if (!norm || !aligned_to(norm, 4) || !ws || !aligned_to(ws, 16))
    return LCE_ERR_INVALID_ARG;
  if (ws_bytes < lce_grad_norm_workspace_size(n)) return LCE_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int64_t parts = 0;
  ProfScope ps(LCE_K_GRAD_NORM, s);
  cudaError_t e = each_table(
      grads, nullptr, dts, sizes, n, [&](const GradTable& t, int grid, int) {
        k_grad_squares<<<grid, GRAD_THREADS, 0, s>>>(t, part + parts);
        parts += grid;
      });
  if (e == cudaSuccess) {
    k_grad_norm<<<1, 1024, 0, s>>>(part, parts, norm);
    e = cudaGetLastError();
  }
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "grad_norm");
}

lce_status lce_clip_grads(const void* const* grads, void* const* outs,
                          const lce_dtype* dts, const int64_t* sizes, int64_t n,
                          const float* norm, float max_norm, void* stream) {
  LCE_TRY(check(grads, dts, sizes, n));
  if (n > 0 && !outs) return LCE_ERR_INVALID_ARG;
  if (!norm || !aligned_to(norm, 4) || !(max_norm >= 0.f))
    return LCE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n; ++i)
    if (sizes[i] > 0 &&
        (!outs[i] || !aligned_to(outs[i], dts[i] == LCE_F32 ? 4 : 2)))
      return LCE_ERR_INVALID_ARG;
  LCE_TRY(check_disjoint(grads, outs, dts, sizes, n, norm));
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(LCE_K_CLIP_GRADS, s);
  const cudaError_t e = each_table(
      grads, outs, dts, sizes, n, [&](const GradTable& t, int grid, int) {
        k_clip<<<grid, GRAD_THREADS, 0, s>>>(t, norm, max_norm);
      });
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "clip_grads");
}

}  // extern "C"
