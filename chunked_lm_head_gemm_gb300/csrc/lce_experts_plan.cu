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

// A warp's slots, ITEMS to a lane: slot i0 + 32 q + lane in e[q], -1 where it
// is dropped or past the end. All loads are in flight at once.
template <int ITEMS>
__device__ __forceinline__ void load_slots(const int32_t* experts, int64_t n,
                                           int64_t i0, int E, int (&e)[ITEMS],
                                           unsigned* err) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < ITEMS; ++q)
    e[q] = expert_of(experts, n, i0 + 32 * q + lane, E, err);
}

// Counts a warp's slots into cnt[expert]; same[q] gets the lanes whose slot q
// goes to this lane's expert.
template <int ITEMS>
__device__ __forceinline__ void count_slots(const int (&e)[ITEMS],
                                            unsigned (&same)[ITEMS],
                                            int* cnt) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < ITEMS; ++q) same[q] = __match_any_sync(FULL, e[q]);
#pragma unroll
  for (int q = 0; q < ITEMS; ++q) {
    if (e[q] >= 0 && (same[q] & ((1u << lane) - 1u)) == 0u)
      cnt[e[q]] += __popc(same[q]);
    __syncwarp();
  }
}

// Gives a warp's slots their rows, in slot order; cnt[e] holds the position
// in its segment of the warp's next slot of e.
template <int ITEMS>
__device__ __forceinline__ void place_slots(const int (&e)[ITEMS],
                                            const unsigned (&same)[ITEMS],
                                            int64_t n, int64_t i0, int* cnt,
                                            const int* start, const Plan& p) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < ITEMS; ++q) {
    const int64_t i = i0 + 32 * q + lane;
    const int before = __popc(same[q] & ((1u << lane) - 1u));
    int at = 0;
    if (e[q] >= 0) at = cnt[e[q]];
    __syncwarp();
    if (e[q] >= 0) {
      const int r = start[e[q]] + at + before;
      p.slot[r] = static_cast<int>(i);
      p.row[i] = r;
      if (before == 0) cnt[e[q]] = at + __popc(same[q]);
    } else if (i < n) {
      p.row[i] = -1;
    }
    __syncwarp();
  }
}

__device__ __forceinline__ int padded(int c) {
  return (c + SEG_ROWS - 1) / SEG_ROWS * SEG_ROWS;
}
__device__ __forceinline__ int tiles_of(int c, int tile_m) {
  return (padded(c) + tile_m - 1) / tile_m;
}

// Static shared memory of lay_out, in 32-bit words.
constexpr int LAY_OUT_WORDS = 32 + 32 + MAX_EXPERTS;

// One block of 1024 threads: segments, tiles and padding rows from the
// experts' counts (c: thread e's expert). start[] (shared, E + 1 entries) gets
// each segment's row, cnt[] (shared) the counts.
__device__ __forceinline__ void lay_out(int c, int E, int tile_m,
                                        const Plan& p, int* start, int* cnt) {
  __shared__ int fixed[LAY_OUT_WORDS];
  int* warp_rows = fixed;
  int* warp_tiles = fixed + 32;
  int* first_tile = fixed + 64;
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  if (e >= E) c = 0;
  const int rows = padded(c), tiles = tiles_of(c, tile_m);
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
    start[e] = row0;
    cnt[e] = c;
    first_tile[e] = t - tiles;
    p.seg[e] = make_int2(row0, rows);
    if (e == E - 1) *p.head = PlanHead{t, r};
  }
  __syncthreads();
  // tiles and padding rows: a warp to an expert, its stores contiguous
  for (int x = warp; x < E; x += 32) {
    const int n = cnt[x], end = padded(n), first = first_tile[x];
    for (int q = lane; q < tiles_of(n, tile_m); q += 32)
      p.tile[first + q] = RowTile{x, first, start[x], end};
    for (int q = n + lane; q < end; q += 32) p.slot[start[x] + q] = -1;
  }
}

// Few slots: the whole plan in one block (a launch instead of three). Each of
// `workers` warps takes 32 ITEMS slots.
template <int ITEMS>
__global__ void __launch_bounds__(1024)
    k_plan_small(const int32_t* experts, int n, int E, int tile_m, Plan p,
                 unsigned* err) {
  extern __shared__ int plan_smem[];
  const int workers = (n + 32 * ITEMS - 1) / (32 * ITEMS);
  int* cnt = plan_smem;            // [workers][E]
  int* start = cnt + workers * E;  // [E]
  int* totals = start + E;         // [E]
  const int warp = threadIdx.x >> 5;
  const int i0 = warp * 32 * ITEMS;
  int e[ITEMS];
  unsigned same[ITEMS];
  if (warp < workers) load_slots<ITEMS>(experts, n, i0, E, e, err);
  for (int i = threadIdx.x; i < workers * E; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  if (warp < workers) count_slots<ITEMS>(e, same, cnt + warp * E);
  __syncthreads();
  int total = 0;
  if (threadIdx.x < E)
    for (int w = 0; w < workers; ++w) {
      const int c = cnt[w * E + threadIdx.x];
      cnt[w * E + threadIdx.x] = total;
      total += c;
    }
  lay_out(total, E, tile_m, p, start, totals);
  __syncthreads();
  if (warp < workers)
    place_slots<ITEMS>(e, same, n, i0, cnt + warp * E, start, p);
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

// Step 2, one block: the chunk counts become the counts before the chunk
// (a warp to an expert), then segments, tiles and padding.
__global__ void __launch_bounds__(1024) k_plan_layout(int E, int chunks,
                                                      int tile_m, Plan p) {
  __shared__ int start[MAX_EXPERTS], cnt[MAX_EXPERTS];
  begin_early();
  const int lane = threadIdx.x & 31;
  // four experts to a warp at a time, so that their loads overlap
  for (int e0 = (threadIdx.x >> 5) * 4; e0 < E; e0 += 128) {
    int before[4] = {0, 0, 0, 0};
    for (int c0 = 0; c0 < chunks; c0 += 32) {
      const int at = c0 + lane;
      int c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        c[q] = e0 + q < E && at < chunks
                   ? p.hist[static_cast<int64_t>(e0 + q) * chunks + at]
                   : 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        int r = c[q];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int a = __shfl_up_sync(FULL, r, o);
          if (lane >= o) r += a;
        }
        if (e0 + q < E && at < chunks)
          p.hist[static_cast<int64_t>(e0 + q) * chunks + at] =
              before[q] + r - c[q];
        before[q] += __shfl_sync(FULL, r, 31);
      }
    }
    if (lane == 0)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (e0 + q < E) cnt[e0 + q] = before[q];
  }
  __syncthreads();
  const int c = threadIdx.x < E ? cnt[threadIdx.x] : 0;
  lay_out(c, E, tile_m, p, start, cnt);
}

// Step 3: every slot's row.
__global__ void __launch_bounds__(CHUNK_WARPS * 32)
    k_plan_place(const int32_t* experts, int64_t n, int E, int chunks, Plan p) {
  extern __shared__ int plan_smem[];
  int* cnt = plan_smem;                // [CHUNK_WARPS][E]
  int* start = cnt + CHUNK_WARPS * E;  // [E]
  const int warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < CHUNK_WARPS * E; i += blockDim.x) cnt[i] = 0;
  constexpr int ITEMS = PLAN_CHUNK / CHUNK_WARPS / 32;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * PLAN_CHUNK +
                     warp * (32 * ITEMS);
  int mine[ITEMS];
  unsigned same[ITEMS];
  load_slots<ITEMS>(experts, n, i0, E, mine, nullptr);
  __syncthreads();
  begin_early();
  count_slots<ITEMS>(mine, same, cnt + warp * E);
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
  place_slots<ITEMS>(mine, same, n, i0, cnt + warp * E, start, p);
}

// Eight columns of a token per thread (threads x: columns, y: tokens): read
// once, written to each of the token's rows. The blocks past the tokens' zero
// an expert's padding rows each. Bound by the rows' bytes.
__global__ void __launch_bounds__(256)
    k_gather(Plan p, int64_t L, int K, int vecs, unsigned token_blocks,
             const uint4* __restrict__ x, uint4* __restrict__ out,
             const uint4* __restrict__ y, uint4* __restrict__ out_y) {
  begin_early();
  const uint4* src = blockIdx.z ? y : x;
  uint4* dst = blockIdx.z ? out_y : out;
  const int c = blockIdx.y * blockDim.x + threadIdx.x;
  if (c >= vecs) return;
  if (blockIdx.x >= token_blocks) {
    const int2 seg = p.seg[blockIdx.x - token_blocks];
    const int first = max(0, seg.y - SEG_ROWS);
    for (int q = first + threadIdx.y; q < seg.y; q += blockDim.y)
      if (p.slot[seg.x + q] < 0)
        dst[static_cast<int64_t>(seg.x + q) * vecs + c] =
            make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t t =
      blockIdx.x * static_cast<int64_t>(blockDim.y) + threadIdx.y;
  if (t >= L) return;
  const uint4 v = __ldg(src + t * vecs + c);
  const int* row = p.row + t * K;
  for (int k0 = 0; k0 < K; k0 += 8) {
    int r[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) r[q] = k0 + q < K ? row[k0 + q] : -1;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (r[q] >= 0) dst[static_cast<int64_t>(r[q]) * vecs + c] = v;
  }
}

template <typename T>
__device__ __forceinline__ float weight_at(const void* w, int64_t i) {
  return static_cast<float>(static_cast<const T*>(w)[i]);
}

// The routing weights' gradients: a slot's column pieces, in order.
struct DweightsArgs {
  const float* part;  // [pieces][stride]
  int64_t stride, n;
  int pieces;
  const int* row;
  void* out;          // NULL: none
  int f32;
};
__device__ __forceinline__ void sum_dweights(const DweightsArgs& d, int64_t i) {
  if (i >= d.n) return;
  const int r = d.row[i];
  float sum = 0.f;
  if (r >= 0)
    for (int t = 0; t < d.pieces; ++t) sum += d.part[t * d.stride + r];
  if (d.f32)
    static_cast<float*>(d.out)[i] = sum;
  else
    static_cast<__nv_bfloat16*>(d.out)[i] = __float2bfloat16_rn(sum);
}

__global__ void __launch_bounds__(256) k_dweights(const DweightsArgs d) {
  begin_early();
  sum_dweights(d, blockIdx.x * static_cast<int64_t>(256) + threadIdx.x);
}

// Eight columns of a token per thread (threads x: columns, y: tokens); a
// token's rows are added in fp32 in the order of its slots, KB loads in
// flight. Bound by the rows' bytes. Further blocks sum dweights, if wanted.
template <typename T, bool WEIGHTED, int KB>
__global__ void __launch_bounds__(256)
    k_combine(const uint16_t* rows, const float* scale, const int* row,
              const void* w, int64_t L, int K, int H, uint16_t* out,
              unsigned token_blocks, const DweightsArgs d) {
  begin_early();
  if (blockIdx.x >= token_blocks) {  // the blocks past the tokens'
    if (blockIdx.y == 0)
      sum_dweights(d, (blockIdx.x - token_blocks) * static_cast<int64_t>(256) +
                          threadIdx.y * blockDim.x + threadIdx.x);
    return;
  }
  const int64_t t =
      blockIdx.x * static_cast<int64_t>(blockDim.y) + threadIdx.y;
  const int h = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
  if (t >= L || h >= H) return;
  const int tiles = 2 * ((H + 255) / 256);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < K; k0 += KB) {
    int r[KB];
    uint4 v[KB];
    float c[KB];
#pragma unroll
    for (int q = 0; q < KB; ++q)
      r[q] = k0 + q < K ? row[t * K + k0 + q] : -1;
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      v[q] = make_uint4(0, 0, 0, 0);
      c[q] = 0.f;
      if (r[q] >= 0) {
        v[q] = *reinterpret_cast<const uint4*>(
            rows + static_cast<int64_t>(r[q]) * H + h);
        c[q] = scale[static_cast<int64_t>(r[q]) * tiles + (h >> 7)];
        if (WEIGHTED) c[q] *= weight_at<T>(w, t * K + k0 + q);
      }
    }
#pragma unroll
    for (int q = 0; q < KB; ++q) {
      if (r[q] < 0) continue;
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

// ---------------------------------------------------------------------------
// single tokens: few slots, no plan and no tensor cores. What bounds them is
// reading the chosen experts' weights once: 75 MB, 11 us, for one token at H
// = 2048, I = 768, top 8. So every warp of k_token_up is resident at once
// (40 registers, two 16-byte loads of each matrix in flight a lane; with four
// there are two waves of warps, 25 us against 22 for both kernels).
// k_token_down is launched early: its blocks (20 K registers) do not fit beside
// the ten of k_token_up on a full SM (51 K of 64 K), but take their places as
// they leave, and load their first weights before k_token_up as a whole has
// ended. Fetching the rows by bulk copies into shared memory took 26 us.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s = fmaf(__uint_as_float(x[j] << 16), __uint_as_float(y[j] << 16), s);
    s = fmaf(__uint_as_float(x[j] & 0xffff0000u),
             __uint_as_float(y[j] & 0xffff0000u), s);
  }
  return s;
}
__device__ __forceinline__ float dot8(uint4 a, float4 lo, float4 hi) {
  float s = __uint_as_float(a.x << 16) * lo.x;
  s = fmaf(__uint_as_float(a.x & 0xffff0000u), lo.y, s);
  s = fmaf(__uint_as_float(a.y << 16), lo.z, s);
  s = fmaf(__uint_as_float(a.y & 0xffff0000u), lo.w, s);
  s = fmaf(__uint_as_float(a.z << 16), hi.x, s);
  s = fmaf(__uint_as_float(a.z & 0xffff0000u), hi.y, s);
  s = fmaf(__uint_as_float(a.w << 16), hi.z, s);
  return fmaf(__uint_as_float(a.w & 0xffff0000u), hi.w, s);
}

__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

constexpr int TOKEN_WARPS = 4;

// a[slot][i] = silu(Wg_e[i] . x_t) (Wu_e[i] . x_t) in fp32, one warp per
// (slot, i). The call's first kernel: it begins when earlier work has ended,
// and lets k_token_down begin once each of its blocks runs.
__global__ void __launch_bounds__(TOKEN_WARPS * 32, 12)
    k_token_up(const uint4* __restrict__ x, const uint4* __restrict__ Wg,
               const uint4* __restrict__ Wu, const int32_t* __restrict__ experts,
               int n, int K, int H, int I, int E, float* __restrict__ a,
               unsigned* err) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * TOKEN_WARPS + (threadIdx.x >> 5);
  const int slot = blockIdx.y;
  const int e = expert_of(experts, n, slot, E,
                          blockIdx.x == 0 && threadIdx.x == 0 ? err : nullptr);
  if (e < 0 || i >= I) return;
  const int vecs = H / 8;
  const int64_t at = (static_cast<int64_t>(e) * I + i) * vecs;
  const uint4* xr = x + static_cast<int64_t>(slot / K) * vecs;
  float g = 0.f, u = 0.f;
  for (int c = lane; c < vecs; c += 64) {
    const bool two = c + 32 < vecs;
    const int d = two ? c + 32 : c;
    const uint4 g0 = load_stream(Wg + at + c), u0 = load_stream(Wu + at + c);
    const uint4 g1 = load_stream(Wg + at + d), u1 = load_stream(Wu + at + d);
    const uint4 x0 = __ldg(xr + c), x1 = __ldg(xr + d);
    g += dot8(g0, x0);
    u += dot8(u0, x0);
    if (two) {
      g += dot8(g1, x1);
      u += dot8(u1, x1);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    g += __shfl_xor_sync(FULL, g, o);
    u += __shfl_xor_sync(FULL, u, o);
  }
  if (lane == 0)
    a[static_cast<int64_t>(slot) * I + i] = g * sigmoid_fast(g) * u;
}

// y[t][h] = sum_k w_k Wd_e[h] . a[t, k]: TOKEN_SPLIT warps to an (t, h), each
// with every TOKEN_SPLIT-th slot, two at a time; a warp's first loads are on
// their way before it waits for k_token_up. The warps' sums are added in order.
constexpr int TOKEN_SPLIT = 4;
constexpr int TOKEN_HS = 2;  // (t, h) of a block

template <typename T>
__global__ void __launch_bounds__(TOKEN_SPLIT * TOKEN_HS * 32)
    k_token_down(const float* a, const uint4* __restrict__ Wd,
                 const int32_t* __restrict__ experts,
                 const void* __restrict__ weights, int n, int K, int H, int I,
                 int E, uint16_t* __restrict__ y) {
  __shared__ float part[TOKEN_HS][TOKEN_SPLIT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = warp % TOKEN_SPLIT;
  const int h = blockIdx.x * TOKEN_HS + warp / TOKEN_SPLIT;
  const int t = blockIdx.y;
  const int vecs = I / 8;
  const int cols = h < H ? vecs : 0;
  float acc = 0.f;
  bool waited = false;
  for (int k0 = sub; k0 < K; k0 += 2 * TOKEN_SPLIT) {
    int e[2];
    float w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int kk = k0 + k * TOKEN_SPLIT;
      e[k] = kk < K ? expert_of(experts, n, t * K + kk, E, nullptr) : -1;
      w[k] = e[k] >= 0 ? weight_at<T>(weights, t * K + kk) : 0.f;
    }
    for (int c0 = lane; c0 - lane < vecs; c0 += 128) {
      uint4 v[2][4];  // two slots by four columns
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4* wr =
            Wd + (static_cast<int64_t>(e[k] < 0 ? 0 : e[k]) * H + h) * vecs;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[k][q] = e[k] >= 0 && c0 + 32 * q < cols
                        ? load_stream(wr + c0 + 32 * q)
                        : make_uint4(0, 0, 0, 0);
      }
      if (!waited) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (e[k] < 0) continue;
        const float* ar =
            a + static_cast<int64_t>(t * K + k0 + k * TOKEN_SPLIT) * I;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (c0 + 32 * q >= cols) break;
          const float4* ap =
              reinterpret_cast<const float4*>(ar + (c0 + 32 * q) * 8);
          s += dot8(v[k][q], ap[0], ap[1]);
        }
        acc = fmaf(w[k], s, acc);
      }
    }
  }
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(FULL, acc, o);
  if (lane == 0) part[warp / TOKEN_SPLIT][sub] = acc;
  __syncthreads();
  if (threadIdx.x < TOKEN_HS) {
    const int out = blockIdx.x * TOKEN_HS + threadIdx.x;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < TOKEN_SPLIT; ++q) sum += part[threadIdx.x][q];
    if (out < H) y[static_cast<int64_t>(t) * H + out] = to_bf16_bits(sum);
  }
}

// Lets k_plan_small take its largest size where this call's, beside the
// static arrays, is above the default limit. The limit is one value for all
// threads of the process: set to a call's own size, another thread's smaller
// call would lower it before the launch.
cudaError_t allow_plan_small(const void* kernel, size_t bytes) {
  constexpr size_t STATIC = sizeof(int) * LAY_OUT_WORDS;
  if (bytes + STATIC <= 48 * 1024) return cudaSuccess;
  constexpr int LARGEST = sizeof(int) * (32 + 2) * MAX_EXPERTS;
  static_assert(LARGEST + STATIC <= 227 * 1024, "shared memory of a block");
  return cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LARGEST);
}

}  // namespace

cudaError_t launch_plan(const int32_t* experts, int64_t n, int E, int tile_m,
                        const Plan& p, unsigned* err, cudaStream_t s) {
  cudaError_t e;
  if (n <= PLAN_SMALL) {
    // slots of a lane: one while 32 warps suffice
    const int few = n <= 1024 ? 1 : PLAN_SMALL / 1024;
    const size_t smem =
        sizeof(int) * (ceil_div(n, 32 * few) + 2) * static_cast<size_t>(E);
    auto kern = few == 1 ? k_plan_small<1> : k_plan_small<PLAN_SMALL / 1024>;
    if ((e = allow_plan_small(reinterpret_cast<const void*>(kern), smem)) !=
        cudaSuccess)
      return e;
    kern<<<1, 1024, smem, s>>>(experts, static_cast<int>(n), E, tile_m, p,
                               err);
    return cudaGetLastError();
  }
  const int chunks = static_cast<int>(ceil_div(n, PLAN_CHUNK));
  k_plan_count<<<chunks, CHUNK_WARPS * 32, sizeof(int) * E, s>>>(
      experts, n, E, chunks, p, err);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_early(k_plan_layout, 1, 1024, 0, s, E, chunks, tile_m, p)) !=
      cudaSuccess)
    return e;
  static_assert(sizeof(int) * (CHUNK_WARPS + 1) * MAX_EXPERTS <= 48 * 1024,
                "default limit");
  const size_t smem = sizeof(int) * (CHUNK_WARPS + 1) * static_cast<size_t>(E);
  return launch_early(k_plan_place, chunks, CHUNK_WARPS * 32, smem, s, experts,
                      n, E, chunks, p);
}

namespace {
// Threads over the columns (x, in eights) and tokens (y) of a row kernel.
dim3 row_block(int64_t H) {
  unsigned bx = 32;
  while (bx < 256 && bx * 8 < H) bx *= 2;
  return dim3(bx, 256 / bx);
}
}  // namespace

cudaError_t launch_gather(const Plan& p, int64_t L, int K, int E, int64_t H,
                          const void* x, uint16_t* out, const void* y,
                          uint16_t* out_y, bool zero, cudaStream_t s) {
  const dim3 block = row_block(H);
  const unsigned tokens = static_cast<unsigned>(ceil_div(L, block.y));
  const dim3 grid(tokens + (zero ? E : 0),
                  static_cast<unsigned>(ceil_div(H, block.x * 8)), y ? 2 : 1);
  return launch_early(k_gather, grid, block, 0, s, p, L, K,
                      static_cast<int>(H / 8), tokens,
                      static_cast<const uint4*>(x),
                      reinterpret_cast<uint4*>(out),
                      static_cast<const uint4*>(y),
                      reinterpret_cast<uint4*>(out_y));
}

namespace {
template <typename T, bool WEIGHTED>
cudaError_t launch_combine_t(const uint16_t* rows, const float* scale,
                             const int* row, const void* w, int64_t L, int K,
                             int64_t H, uint16_t* out, const DweightsArgs& d,
                             cudaStream_t s) {
  const dim3 block = row_block(H);
  const unsigned tokens = static_cast<unsigned>(ceil_div(L, block.y));
  const unsigned more = d.out ? static_cast<unsigned>(ceil_div(d.n, 256)) : 0u;
  const dim3 grid(tokens + more,
                  static_cast<unsigned>(ceil_div(H, block.x * 8)));
  auto kern = K <= 2   ? k_combine<T, WEIGHTED, 2>
              : K <= 4 ? k_combine<T, WEIGHTED, 4>
                       : k_combine<T, WEIGHTED, 8>;
  return launch_early(kern, grid, block, 0, s, rows, scale, row, w, L, K,
                      static_cast<int>(H), out, tokens, d);
}
}  // namespace

cudaError_t launch_combine(const uint16_t* rows, const float* scale,
                           const int* row, const void* w, lce_dtype wdt,
                           int64_t L, int K, int64_t H, void* out,
                           cudaStream_t s) {
  uint16_t* o = static_cast<uint16_t*>(out);
  if (wdt == LCE_F32)
    return launch_combine_t<float, true>(rows, scale, row, w, L, K, H, o, {},
                                         s);
  return launch_combine_t<__nv_bfloat16, true>(rows, scale, row, w, L, K, H, o,
                                               {}, s);
}

cudaError_t launch_backward_sums(const uint16_t* rows, const float* scale,
                                 const int* row, int64_t L, int K, int64_t H,
                                 void* dx, const float* part, int64_t stride,
                                 int pieces, lce_dtype wdt, void* dweights,
                                 cudaStream_t s) {
  const DweightsArgs d{part, stride, L * K, pieces, row, dweights,
                       wdt == LCE_F32};
  if (dx)
    return launch_combine_t<float, false>(rows, scale, row, nullptr, L, K, H,
                                          static_cast<uint16_t*>(dx), d, s);
  if (!dweights) return cudaSuccess;
  return launch_early(k_dweights, static_cast<unsigned>(ceil_div(d.n, 256)),
                      256, 0, s, d);
}

cudaError_t launch_token(const void* x, const void* Wg, const void* Wu,
                         const void* Wd, const void* weights, lce_dtype wdt,
                         const int32_t* experts, int64_t L, int K, int64_t H,
                         int64_t I, int E, float* a, void* y, unsigned* err,
                         cudaStream_t s) {
  const int n = static_cast<int>(L) * K;
  const int h = static_cast<int>(H), i = static_cast<int>(I);
  k_token_up<<<dim3(static_cast<unsigned>(ceil_div(I, TOKEN_WARPS)), n),
               TOKEN_WARPS * 32, 0, s>>>(
      static_cast<const uint4*>(x), static_cast<const uint4*>(Wg),
      static_cast<const uint4*>(Wu), experts, n, K, h, i, E, a, err);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto kern = wdt == LCE_F32 ? k_token_down<float> : k_token_down<__nv_bfloat16>;
  return launch_early(
      kern,
      dim3(static_cast<unsigned>(ceil_div(H, TOKEN_HS)),
           static_cast<unsigned>(L)),
      TOKEN_SPLIT * TOKEN_HS * 32, 0, s, a, static_cast<const uint4*>(Wd),
      experts, weights, n, K, h, i, E, static_cast<uint16_t*>(y));
}

}  // namespace lce
