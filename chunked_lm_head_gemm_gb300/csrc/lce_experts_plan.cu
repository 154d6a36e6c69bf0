// The experts' gated MLP around its contractions: the plan that groups slots
// by expert (a stable counting sort), and the sums over a token's slots.
#include <cuda_fp16.h>

#include "lce_device.cuh"
#include "lce_experts.h"
#include "lce_host.h"

namespace lce {
namespace {

constexpr unsigned FULL = 0xffffffffu;

// The expert of a slot, or -1 (dropped). An index that is neither -1 nor in
// [0, E) raises the error bit and counts as dropped.
__device__ __forceinline__ int expert_of(const int32_t* experts, int64_t n,
                                         int64_t i, int E, unsigned* err) {
  if (i >= n) return -1;
  const int e = experts[i];
  if (e >= 0 && e < E) return e;
  if (e != -1 && err) atomicOr(err, ERRBIT_EXPERT_RANGE);
  return -1;
}

// One warp over the slots [i0, i1), 32 at a time: cnt[e] grows by the slots
// of e. With PLACE, cnt[e] holds the position of the warp's next slot of e
// in its segment, and every slot gets its row.
template <bool PLACE>
__device__ __forceinline__ void walk_slots(const int32_t* experts, int64_t n,
                                           int64_t i0, int64_t i1, int E,
                                           int K, int* cnt, const int* start,
                                           const Plan& p, unsigned* err) {
  const int lane = threadIdx.x & 31;
  for (int64_t i = i0 + lane; i - lane < i1; i += 32) {
    const int e = expert_of(experts, i < i1 ? n : 0, i, E, PLACE ? nullptr : err);
    const unsigned same = __match_any_sync(FULL, e);
    const int before = __popc(same & ((1u << lane) - 1u));
    if (e >= 0) {
      if (PLACE) {
        const int r = start[e] + cnt[e] + before;
        p.token[r] = static_cast<int>(i / K);
        p.slot[r] = static_cast<int>(i);
        p.row[i] = r;
      }
    } else if (PLACE && i < i1) {
      p.row[i] = -1;
    }
    __syncwarp();
    if (e >= 0 && before == 0) cnt[e] += __popc(same);
    __syncwarp();
  }
}

__device__ __forceinline__ int padded(int c) {
  return (c + SEG_ROWS - 1) / SEG_ROWS * SEG_ROWS;
}
__device__ __forceinline__ int tiles_of(int c) {
  return (padded(c) + BM - 1) / BM;
}

// One block of MAX_EXPERTS threads: segments, tiles and padding rows from
// the experts' counts. start[] (shared or global) gets each segment's row.
__device__ __forceinline__ void lay_out(int c, int E, const Plan& p,
                                        int* start) {
  __shared__ int warp_rows[32], warp_tiles[32];
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  if (e >= E) c = 0;
  const int rows = padded(c), tiles = tiles_of(c);
  int r = rows, t = tiles;  // inclusive scans over the experts
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(FULL, r, o), b = __shfl_up_sync(FULL, t, o);
    if (lane >= o) {
      r += a;
      t += b;
    }
  }
  if (lane == 31) {
    warp_rows[warp] = r;
    warp_tiles[warp] = t;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    r += warp_rows[w];
    t += warp_tiles[w];
  }
  if (e < E) {
    const int row0 = r - rows;
    int at = t - tiles;
    start[e] = row0;
    p.seg[e] = make_int2(row0, rows);
    p.count[e] = c;
    for (int q = 0; q < rows; q += BM)
      p.tile[at++] = RowTile{e, row0 + q, min(BM, rows - q), 0};
    for (int q = c; q < rows; ++q) {
      p.token[row0 + q] = -1;
      p.slot[row0 + q] = -1;
    }
    if (e == E - 1) *p.head = PlanHead{t, r};
  }
}

// Few slots: the whole plan in one block (a launch instead of four).
__global__ void __launch_bounds__(1024)
    k_plan_small(const int32_t* experts, int n, int K, int E, Plan p,
                 unsigned* err) {
  extern __shared__ int plan_smem[];
  int* cnt = plan_smem;          // [warps][E]
  const int warps = blockDim.x >> 5;
  int* start = cnt + warps * E;  // [E]
  const int warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int per = ((n + warps - 1) / warps + 31) / 32 * 32;
  const int i0 = min(n, warp * per), i1 = min(n, i0 + per);
  walk_slots<false>(experts, n, i0, i1, E, K, cnt + warp * E, nullptr, p, err);
  __syncthreads();
  int total = 0;
  if (threadIdx.x < E)
    for (int w = 0; w < warps; ++w) {
      const int c = cnt[w * E + threadIdx.x];
      cnt[w * E + threadIdx.x] = total;
      total += c;
    }
  lay_out(total, E, p, start);
  __syncthreads();
  walk_slots<true>(experts, n, i0, i1, E, K, cnt + warp * E, start, p, err);
}

constexpr int CHUNK_WARPS = 8;

// Many slots, step 1: each chunk's count of each expert.
__global__ void __launch_bounds__(CHUNK_WARPS * 32)
    k_plan_count(const int32_t* experts, int64_t n, int E, int chunks,
                 Plan p, unsigned* err) {
  extern __shared__ int plan_smem[];
  for (int e = threadIdx.x; e < E; e += blockDim.x) plan_smem[e] = 0;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * PLAN_CHUNK;
  for (int i = threadIdx.x; i < PLAN_CHUNK; i += blockDim.x) {
    const int e = expert_of(experts, n, i0 + i, E, err);
    if (e >= 0) atomicAdd(&plan_smem[e], 1);  // integers: order is no matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    p.hist[static_cast<int64_t>(e) * chunks + blockIdx.x] = plan_smem[e];
}

// Step 2: one warp per expert turns the chunk counts into the counts before.
__global__ void __launch_bounds__(256) k_plan_scan(int E, int chunks, Plan p) {
  const int e = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (e >= E) return;
  int* h = p.hist + static_cast<int64_t>(e) * chunks;
  int before = 0;
  for (int c0 = 0; c0 < chunks; c0 += 32) {
    const int c = c0 + lane < chunks ? h[c0 + lane] : 0;
    int r = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(FULL, r, o);
      if (lane >= o) r += a;
    }
    if (c0 + lane < chunks) h[c0 + lane] = before + r - c;
    before += __shfl_sync(FULL, r, 31);
  }
  if (lane == 0) p.count[e] = before;
}

// Step 3: segments and tiles.
__global__ void __launch_bounds__(1024) k_plan_layout(int E, Plan p) {
  __shared__ int start[MAX_EXPERTS];
  lay_out(threadIdx.x < E ? p.count[threadIdx.x] : 0, E, p, start);
}

// Step 4: every slot's row.
__global__ void __launch_bounds__(CHUNK_WARPS * 32)
    k_plan_place(const int32_t* experts, int64_t n, int K, int E, int chunks,
                 Plan p) {
  extern __shared__ int plan_smem[];
  int* cnt = plan_smem;                // [CHUNK_WARPS][E]
  int* start = cnt + CHUNK_WARPS * E;  // [E]
  const int warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < CHUNK_WARPS * E; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  constexpr int PER = PLAN_CHUNK / CHUNK_WARPS;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * PLAN_CHUNK;
  const int64_t i0 = min(n, c0 + warp * PER), i1 = min(n, i0 + PER);
  walk_slots<false>(experts, n, i0, i1, E, K, cnt + warp * E, nullptr, p,
                    nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int before = p.hist[static_cast<int64_t>(e) * chunks + blockIdx.x];
    for (int w = 0; w < CHUNK_WARPS; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = before;
      before += c;
    }
    start[e] = p.seg[e].x;
  }
  __syncthreads();
  walk_slots<true>(experts, n, i0, i1, E, K, cnt + warp * E, start, p,
                   nullptr);
}

// One warp per row, 16 bytes a lane, four loads in flight.
__global__ void __launch_bounds__(256)
    k_gather(const PlanHead* __restrict__ head, const int* __restrict__ token,
             int64_t H, const uint4* __restrict__ x, uint4* __restrict__ out,
             const uint4* __restrict__ y, uint4* __restrict__ out_y) {
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= head->rows) return;
  const int t = token[r];
  const int vecs = static_cast<int>(H / 8);
  const uint4* src = blockIdx.y ? y : x;
  uint4* dst = (blockIdx.y ? out_y : out) + static_cast<int64_t>(r) * vecs;
  src += static_cast<int64_t>(t < 0 ? 0 : t) * vecs;
  for (int i = threadIdx.x & 31; i < vecs; i += 128) {
    uint4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = t >= 0 && i + 32 * q < vecs ? __ldg(src + i + 32 * q)
                                         : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + 32 * q < vecs) dst[i + 32 * q] = v[q];
  }
}

template <typename T>
__device__ __forceinline__ float weight_at(const void* w, int64_t i) {
  return static_cast<float>(static_cast<const T*>(w)[i]);
}

// Eight columns of a token per thread; a token's rows are added in fp32 in
// the order of its slots, eight loads in flight. Bound by the rows' bytes.
template <typename T, bool WEIGHTED>
__global__ void __launch_bounds__(256)
    k_combine(const uint16_t* __restrict__ rows,
              const float* __restrict__ scale, const int* __restrict__ row,
              const void* __restrict__ w, int64_t L, int K, int64_t H,
              uint16_t* __restrict__ out) {
  const int64_t oct = H / 8, tiles = (H + 255) / 256;
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= L * oct) return;
  const int64_t t = i / oct, h = (i - t * oct) * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < K; k0 += 8) {
    uint4 v[8];
    float c[8];
    bool live[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t at = t * K + k0 + q;
      const int r = k0 + q < K ? row[at] : -1;
      live[q] = r >= 0;
      v[q] = make_uint4(0, 0, 0, 0);
      c[q] = 0.f;
      if (live[q]) {
        v[q] = __ldg(reinterpret_cast<const uint4*>(
            rows + static_cast<int64_t>(r) * H + h));
        c[q] = scale[r * tiles + (h >> 8)];
        if (WEIGHTED) c[q] *= weight_at<T>(w, at);
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (!live[q]) continue;
      const uint32_t x[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f =
            __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
        acc[2 * j] = fmaf(c[q], f.x, acc[2 * j]);
        acc[2 * j + 1] = fmaf(c[q], f.y, acc[2 * j + 1]);
      }
    }
  }
  *reinterpret_cast<uint4*>(out + t * H + h) =
      make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                 pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

template <typename T>
__global__ void __launch_bounds__(256)
    k_dweights(const float* __restrict__ part, int64_t stride, int tiles,
               const int* __restrict__ row, int64_t n, T* __restrict__ out) {
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= n) return;
  const int r = row[i];
  float sum = 0.f;
  if (r >= 0)
    for (int t = 0; t < tiles; ++t) sum += part[t * stride + r];
  out[i] = static_cast<T>(sum);
}

cudaError_t allow_smem(const void* kernel, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(kernel,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bytes));
}

}  // namespace

cudaError_t launch_plan(const int32_t* experts, int64_t n, int K, int E,
                        const Plan& p, unsigned* err, cudaStream_t s) {
  cudaError_t e;
  if (n <= PLAN_SMALL) {
    const size_t smem = sizeof(int) * 33 * static_cast<size_t>(E);
    if ((e = allow_smem(reinterpret_cast<const void*>(k_plan_small), smem)) !=
        cudaSuccess)
      return e;
    k_plan_small<<<1, 1024, smem, s>>>(experts, static_cast<int>(n), K, E,
                                       p, err);
    return cudaGetLastError();
  }
  const int chunks = static_cast<int>(ceil_div(n, PLAN_CHUNK));
  k_plan_count<<<chunks, CHUNK_WARPS * 32, sizeof(int) * E, s>>>(
      experts, n, E, chunks, p, err);
  k_plan_scan<<<(E + 7) / 8, 256, 0, s>>>(E, chunks, p);
  k_plan_layout<<<1, 1024, 0, s>>>(E, p);
  const size_t smem = sizeof(int) * (CHUNK_WARPS + 1) * static_cast<size_t>(E);
  if ((e = allow_smem(reinterpret_cast<const void*>(k_plan_place), smem)) !=
      cudaSuccess)
    return e;
  k_plan_place<<<chunks, CHUNK_WARPS * 32, smem, s>>>(experts, n, K, E, chunks,
                                                      p);
  return cudaGetLastError();
}

cudaError_t launch_gather(const Plan& p, int64_t max_rows, int64_t H,
                          const void* x, uint16_t* out, const void* y,
                          uint16_t* out_y, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(max_rows, 8)), y ? 2 : 1);
  k_gather<<<grid, 256, 0, s>>>(
      p.head, p.token, H, static_cast<const uint4*>(x),
      reinterpret_cast<uint4*>(out), static_cast<const uint4*>(y),
      reinterpret_cast<uint4*>(out_y));
  return cudaGetLastError();
}

cudaError_t launch_combine(const uint16_t* rows, const float* scale,
                           const int* row, const void* w, lce_dtype wdt,
                           int64_t L, int K, int64_t H, void* out,
                           cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(ceil_div(L * (H / 8), 256));
  uint16_t* o = static_cast<uint16_t*>(out);
  if (!w)
    k_combine<float, false>
        <<<grid, 256, 0, s>>>(rows, scale, row, w, L, K, H, o);
  else if (wdt == LCE_F32)
    k_combine<float, true>
        <<<grid, 256, 0, s>>>(rows, scale, row, w, L, K, H, o);
  else
    k_combine<__nv_bfloat16, true>
        <<<grid, 256, 0, s>>>(rows, scale, row, w, L, K, H, o);
  return cudaGetLastError();
}

cudaError_t launch_dweights(const float* part, int64_t stride, int tiles,
                            const int* row, int64_t n, lce_dtype wdt,
                            void* dweights, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(ceil_div(n, 256));
  if (wdt == LCE_F32)
    k_dweights<float><<<grid, 256, 0, s>>>(part, stride, tiles, row, n,
                                           static_cast<float*>(dweights));
  else
    k_dweights<__nv_bfloat16><<<grid, 256, 0, s>>>(
        part, stride, tiles, row, n, static_cast<__nv_bfloat16*>(dweights));
  return cudaGetLastError();
}

}  // namespace lce
