// Layer norm and RMS norm of rows (lce_norm_forward / lce_norm_backward).
//
// Forward of a row x: mu its mean, v the mean of (x - mu)^2, r = 1 / sqrt(v +
// eps), n = (x - mu) r, y = n w + b (RMS norm: mu = 0, no b). Backward with g
// = dy w: dx = r (g - mean(g) - n mean(g n)) (RMS norm without mean(g)), dw =
// sum over rows of dy n, db = sum over rows of dy.
//
// Bound: the bytes of x and y, or of x, dy and dx.
#include <math.h>

#include "lce_host.h"
#include "lce_vec.cuh"

namespace lce {
namespace {

struct NormArgs {
  const void* x;
  const void* weight;
  const void* bias;
  const void* dy;
  void* y;   // y or dx
  float* mean;
  float* rstd;
  int64_t L;
  int H;
  float eps;
  int param_f32;
  float* part;  // [slabs][2][H] sums of dy n and dy
  int slabs;
};

// A block to a row.
template <typename T, bool LAYER>
__global__ void __launch_bounds__(256) k_norm_fwd(const NormArgs a) {
  __shared__ float part[2][32];
  const float inv = 1.f / a.H;
  for (int64_t row = blockIdx.x; row < a.L; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.H;
    T* y = static_cast<T*>(a.y) + row * a.H;
    float mu = 0.f;
    if (LAYER) {
      float t = 0.f;
      for (int j = threadIdx.x; j < a.H; j += blockDim.x) t += to_float(x[j]);
      mu = block_sum(t, part[0]) * inv;
    }
    float q = 0.f;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      const float d = to_float(x[j]) - mu;
      q = fmaf(d, d, q);
    }
    const float r = 1.f / sqrtf(block_sum(q, part[1]) * inv + a.eps);
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      float v = (to_float(x[j]) - mu) * r;
      if (a.weight) v *= load_as_float(a.weight, a.param_f32, j);
      if (a.bias) v += load_as_float(a.bias, a.param_f32, j);
      y[j] = from_float<T>(v);
    }
    if (threadIdx.x == 0) {
      if (LAYER && a.mean) a.mean[row] = mu;
      if (a.rstd) a.rstd[row] = r;
    }
    __syncthreads();
  }
}

template <typename T, bool LAYER>
__global__ void __launch_bounds__(256) k_norm_dx(const NormArgs a) {
  __shared__ float part[2][32];
  const float inv = 1.f / a.H;
  for (int64_t row = blockIdx.x; row < a.L; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.H;
    const T* dy = static_cast<const T*>(a.dy) + row * a.H;
    T* dx = static_cast<T*>(a.y) + row * a.H;
    const float mu = LAYER ? a.mean[row] : 0.f, r = a.rstd[row];
    float sg = 0.f, sgn = 0.f;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      float g = to_float(dy[j]);
      if (a.weight) g *= load_as_float(a.weight, a.param_f32, j);
      sg += g;
      sgn = fmaf(g, (to_float(x[j]) - mu) * r, sgn);
    }
    const float c1 = LAYER ? block_sum(sg, part[0]) * inv : 0.f;
    const float c2 = block_sum(sgn, part[1]) * inv;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      float g = to_float(dy[j]);
      if (a.weight) g *= load_as_float(a.weight, a.param_f32, j);
      const float n = (to_float(x[j]) - mu) * r;
      dx[j] = from_float<T>(r * (g - c1 - n * c2));
    }
    __syncthreads();
  }
}

// Sums over the rows of slab blockIdx.y, a thread to a column.
template <typename T, bool LAYER>
__global__ void __launch_bounds__(128) k_norm_dparams(const NormArgs a) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= a.H) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.L; row += a.slabs) {
    const float d = to_float(static_cast<const T*>(a.dy)[row * a.H + j]);
    const float v = to_float(static_cast<const T*>(a.x)[row * a.H + j]);
    const float mu = LAYER ? a.mean[row] : 0.f;
    dw = fmaf(d, (v - mu) * a.rstd[row], dw);
    db += d;
  }
  float* p = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.H;
  p[j] = dw;
  p[a.H + j] = db;
}

// The slabs' sums added in slab order.
__global__ void __launch_bounds__(128)
    k_norm_join(const float* __restrict__ part, int slabs, int H, void* dweight,
                void* dbias, int grad_f32) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= H) return;
  double dw = 0., db = 0.;
  for (int s = 0; s < slabs; ++s) {
    dw += part[(static_cast<int64_t>(s) * 2) * H + j];
    db += part[(static_cast<int64_t>(s) * 2 + 1) * H + j];
  }
  if (dweight) store_from_float(dweight, grad_f32, j, static_cast<float>(dw));
  if (dbias) store_from_float(dbias, grad_f32, j, static_cast<float>(db));
}

constexpr int64_t MAX_H = 1 << 20;
constexpr int64_t MAX_SLABS = 512;

int64_t slabs_of(int64_t L) { return L < MAX_SLABS ? (L > 0 ? L : 1) : MAX_SLABS; }

lce_status check(lce_norm_kind kind, lce_dtype dt, const void* x,
                 const void* weight, lce_dtype param_dt, int64_t L, int64_t H) {
  if (kind != LCE_LAYER_NORM && kind != LCE_RMS_NORM)
    return LCE_ERR_INVALID_ARG;
  if (L < 0 || L > (1ll << 31) || H < 1 || H > MAX_H)
    return LCE_ERR_INVALID_ARG;
  if ((dt != LCE_BF16 && dt != LCE_F32) ||
      (param_dt != LCE_BF16 && param_dt != LCE_F32))
    return LCE_ERR_UNSUPPORTED;
  if (!aligned_to(weight, param_dt == LCE_F32 ? 4 : 2) ||
      !aligned_to(x, dt == LCE_F32 ? 4 : 2) || (L > 0 && !x))
    return LCE_ERR_INVALID_ARG;
  return LCE_OK;
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_norm_workspace_size(int64_t L, int64_t H) {
  if (L < 0 || L > (1ll << 31) || H < 1 || H > MAX_H) return 0;
  return static_cast<size_t>(slabs_of(L)) * 2 * H * sizeof(float);
}

lce_status lce_norm_forward(lce_norm_kind kind, const void* x, lce_dtype dt,
                            const void* weight, const void* bias,
                            lce_dtype param_dt, int64_t L, int64_t H, float eps,
                            void* y, float* mean, float* rstd, void* stream) {
  LCE_TRY(check(kind, dt, x, weight, param_dt, L, H));
  if (!(eps >= 0.f) || isinf(eps) || (kind == LCE_RMS_NORM && (bias || mean)) ||
      !aligned_to(bias, param_dt == LCE_F32 ? 4 : 2) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return LCE_ERR_INVALID_ARG;
  if (L == 0) return LCE_OK;
  if (!y || !aligned_to(y, dt == LCE_F32 ? 4 : 2)) return LCE_ERR_INVALID_ARG;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.L = L;
  a.H = static_cast<int>(H);
  a.eps = eps;
  a.param_f32 = param_dt == LCE_F32;
  const unsigned grid =
      static_cast<unsigned>(L < dev->num_sms * 8 ? L : dev->num_sms * 8);
  const bool layer = kind == LCE_LAYER_NORM;
  auto kern = dt == LCE_F32
                  ? (layer ? k_norm_fwd<float, true> : k_norm_fwd<float, false>)
                  : (layer ? k_norm_fwd<__nv_bfloat16, true>
                           : k_norm_fwd<__nv_bfloat16, false>);
  ProfScope ps(LCE_K_NORM, s);
  kern<<<grid, 256, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "norm");
}

lce_status lce_norm_backward(lce_norm_kind kind, const void* x, lce_dtype dt,
                             const void* weight, lce_dtype param_dt,
                             const float* mean, const float* rstd,
                             const void* dy, int64_t L, int64_t H,
                             lce_dtype grad_dt, void* dx, void* dweight,
                             void* dbias, void* ws, size_t ws_bytes,
                             void* stream) {
  LCE_TRY(check(kind, dt, x, weight, param_dt, L, H));
  if (grad_dt != LCE_BF16 && grad_dt != LCE_F32) return LCE_ERR_UNSUPPORTED;
  const uintptr_t elt = dt == LCE_F32 ? 4 : 2, gelt = grad_dt == LCE_F32 ? 4 : 2;
  const bool layer = kind == LCE_LAYER_NORM, params = dweight || dbias;
  if ((!dx && !params) || (!layer && (mean || dbias)) || !aligned_to(dx, elt) ||
      !aligned_to(dy, elt) || !aligned_to(dweight, gelt) ||
      !aligned_to(dbias, gelt) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return LCE_ERR_INVALID_ARG;
  if (L > 0 && (!dy || !rstd || (layer && !mean))) return LCE_ERR_INVALID_ARG;
  if (params && (!ws || !aligned_to(ws, 16))) return LCE_ERR_INVALID_ARG;
  if (params && ws_bytes < lce_norm_workspace_size(L, H))
    return LCE_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormArgs a{};
  a.x = x;
  a.weight = weight;
  a.dy = dy;
  a.y = dx;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.L = L;
  a.H = static_cast<int>(H);
  a.param_f32 = param_dt == LCE_F32;
  a.part = static_cast<float*>(ws);
  a.slabs = static_cast<int>(slabs_of(L));
  const bool f32 = dt == LCE_F32;
  cudaError_t e = cudaSuccess;
  ProfScope ps(LCE_K_NORM_BWD, s);
  if (params) {
    const unsigned cols = static_cast<unsigned>(ceil_div(H, 128));
    auto kern =
        f32 ? (layer ? k_norm_dparams<float, true> : k_norm_dparams<float, false>)
            : (layer ? k_norm_dparams<__nv_bfloat16, true>
                     : k_norm_dparams<__nv_bfloat16, false>);
    kern<<<dim3(cols, static_cast<unsigned>(a.slabs)), 128, 0, s>>>(a);
    k_norm_join<<<cols, 128, 0, s>>>(a.part, a.slabs, a.H, dweight, dbias,
                                     grad_dt == LCE_F32);
    e = cudaGetLastError();
  }
  // last: dx may stand in x's or dy's place
  if (dx && L > 0 && e == cudaSuccess) {
    const unsigned grid =
        static_cast<unsigned>(L < dev->num_sms * 8 ? L : dev->num_sms * 8);
    auto kern = f32 ? (layer ? k_norm_dx<float, true> : k_norm_dx<float, false>)
                    : (layer ? k_norm_dx<__nv_bfloat16, true>
                             : k_norm_dx<__nv_bfloat16, false>);
    kern<<<grid, 256, 0, s>>>(a);
    e = cudaGetLastError();
  }
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "norm_bwd");
}

}  // extern "C"
