// Layer norm and RMS norm of rows (lce_norm_forward / lce_norm_backward).
//
// Forward of a row x: mu its mean, v the mean of (x - mu)^2, r = 1 / sqrt(v +
// eps), n = (x - mu) r, y = n w + b (RMS norm: mu = 0, no b). Backward with g
// = dy w: dx = r (g - mean(g) - n mean(g n)) (RMS norm without mean(g)), dw =
// sum over rows of dy n, db = sum over rows of dy.
//
// Bound: the bytes of x and y, or of x, dy and dx, each moved once. Up to
// MAX_FAST_H columns a row stays in the registers of its team, 16 elements to
// a thread: a team is a power of two of lanes for narrow rows (several rows to
// a warp), else the whole block. A thread has the same columns in every row,
// so it keeps its weights and its sums for dw and db in registers, and the
// backward needs no second pass over x and dy. Rows that start on 16 bytes
// come through a ring of shared memory by bulk copies, issued several rows
// ahead, so that enough bytes are under way without registers to hold them.
// Wider rows are read again where a pass over them needs it.
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
  void* y;  // y or dx
  float* mean;
  float* rstd;
  int64_t L;
  int H;
  float eps;
  int param_f32;
  int team;       // threads of a row; a block's for a whole block
  int tile_rows;  // rows that a group takes at a time
  int stages;     // tiles of a group in shared memory
  float* part;    // [slabs][2][H] sums of dy n and dy
  int slabs;
  int want_dx;
  uint64_t timeout_ns;
  unsigned* err;
};

constexpr int EPT = 16;           // elements of a row that a thread holds
constexpr int TEAM_WARPS = 8;     // warps of a block whose teams are lanes
constexpr int MAX_THREADS = 512;  // of a block that is a team
constexpr int MAX_FAST_H = EPT * MAX_THREADS;
constexpr int MAX_STAGES = 8;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Sums over a row's team: lanes by shuffles; a block also through shared
// memory, one barrier a call, with two areas in turn.
template <bool BLOCK, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int team,
                                         float (*area)[N][32], int& turn) {
  if (BLOCK) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum(v[i]);
    float(*p)[32] = area[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i][threadIdx.x >> 5] = v[i];
    }
    __syncthreads();
    const int warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = p[i][0];
      for (int w = 1; w < warps; ++w) t += p[i][w];
      v[i] = t;
    }
  } else {
    for (int o = team >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] += __shfl_xor_sync(ALL_LANES, v[i], o);
    }
  }
}

// A group (a warp of lane teams, or the block) and its ring of tiles. A tile
// is tile_rows rows, one after the other in memory; the group takes tiles
// first, first + step, ... Without RING the rows are read where they lie.
template <typename T, bool BLOCK, bool RING, int ARRAYS>
struct Tiles {
  const NormArgs& a;
  int64_t tiles, step, next;  // next: the tile to be fetched
  uint32_t ring, bars;
  uint32_t array_bytes;
  int fetch_stage, stage, phase;
  WaitCtx ctx;

  __device__ __forceinline__ Tiles(const NormArgs& args, unsigned char* smem,
                                   uint64_t* bar, uint32_t* abort_flag)
      : a(args) {
    const int groups = BLOCK ? 1 : TEAM_WARPS;
    const int group = BLOCK ? 0 : threadIdx.x >> 5;
    tiles = (a.L + a.tile_rows - 1) / a.tile_rows;
    step = static_cast<int64_t>(gridDim.x) * groups;
    next = static_cast<int64_t>(blockIdx.x) * groups + group;
    array_bytes = static_cast<uint32_t>(a.tile_rows) * a.H * sizeof(T);
    ring = smem_u32(smem) + group * a.stages * ARRAYS * array_bytes;
    bars = smem_u32(bar) + group * MAX_STAGES * 8;
    fetch_stage = stage = phase = 0;
    ctx = WaitCtx{abort_flag, a.err, a.timeout_ns};
    if (RING) {
      if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < groups * MAX_STAGES; ++i)
          mbar_init(smem_u32(bar) + 8 * i, 1);
        fence_mbar_init();
      }
      __syncthreads();
      for (int i = 0; i < a.stages; ++i) fetch();
    }
  }
  __device__ __forceinline__ bool leader() const {
    return BLOCK ? threadIdx.x == 0 : (threadIdx.x & 31) == 0;
  }
  // Fetches the group's next tile into the stage that was read last.
  __device__ __forceinline__ void fetch() {
    if (!RING) return;
    if (next < tiles && leader()) {
      const int64_t row = next * a.tile_rows;
      const int64_t left = a.L - row;
      const uint32_t bytes =
          left < a.tile_rows
              ? static_cast<uint32_t>(left) * a.H * sizeof(T)
              : array_bytes;
      const uint32_t bar = bars + 8 * fetch_stage;
      const uint32_t dst = ring + fetch_stage * ARRAYS * array_bytes;
      mbar_arrive_expect_tx(bar, ARRAYS * bytes);
      bulk_load(dst, static_cast<const T*>(a.x) + row * a.H, bytes, bar);
      if (ARRAYS == 2)
        bulk_load(dst + array_bytes, static_cast<const T*>(a.dy) + row * a.H,
                  bytes, bar);
    }
    next += step;
    fetch_stage = fetch_stage + 1 == a.stages ? 0 : fetch_stage + 1;
  }
  // Waits for the tile of the present stage. (Should the wait run out, which
  // raises the error, the rows are wrong but every barrier is still met.)
  __device__ __forceinline__ void wait() {
    if (RING) mbar_wait(bars + 8 * stage, phase, ctx, true);
  }
  __device__ __forceinline__ void advance() {
    stage = stage + 1 == a.stages ? 0 : stage + 1;
    if (stage == 0) phase ^= 1;
  }
  // Chunk k of row r of the tile (array 0: x, 1: dy).
  template <int V>
  __device__ __forceinline__ Chunk<T, V> chunk(int array, int64_t row, int r,
                                               int k) const {
    Chunk<T, V> c;
    if constexpr (RING) {
      const uint32_t at = ring + (stage * ARRAYS + array) * array_bytes +
                          (static_cast<uint32_t>(r) * a.H + k * V) * sizeof(T);
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(c.q.x), "=r"(c.q.y), "=r"(c.q.z), "=r"(c.q.w)
                   : "r"(at)
                   : "memory");
    } else {
      const T* p = static_cast<const T*>(array ? a.dy : a.x) + row * a.H;
      c.q = *reinterpret_cast<const decltype(c.q)*>(p + static_cast<int64_t>(k) * V);
    }
    return c;
  }
};

// A thread's columns of weight or bias, `absent` where there is none.
template <int V, int C>
__device__ __forceinline__ void load_params(const void* p, bool f32, int H,
                                            int id, int team, float absent,
                                            float (&w)[EPT]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = (id + team * c) * V + i;
      w[c * V + i] = j >= H ? 0.f : p ? load_as_float(p, f32, j) : absent;
    }
  }
}

template <typename T, int V, bool BLOCK, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) k_norm_fwd(const NormArgs a) {
  constexpr int C = EPT / V;
  constexpr bool RING = V > 1;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bar[TEAM_WARPS * MAX_STAGES];
  __shared__ uint32_t abort_flag;
  __shared__ float area[2][1][32];
  Tiles<T, BLOCK, RING, 1> tiles(a, smem, bar, &abort_flag);
  const int team = BLOCK ? blockDim.x : a.team;
  const int id = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  const int rows_at_once = BLOCK ? 1 : 32 / team;
  const int sub = BLOCK ? 0 : (threadIdx.x & 31) / team;
  const int chunks = a.H / V;
  const float inv = 1.f / a.H;
  int turn = 0;
  float w[EPT], b[EPT];
  load_params<V, C>(a.weight, a.param_f32, a.H, id, team, 1.f, w);
  if (LAYER) load_params<V, C>(a.bias, a.param_f32, a.H, id, team, 0.f, b);
  const int64_t first =
      BLOCK ? blockIdx.x
            : static_cast<int64_t>(blockIdx.x) * TEAM_WARPS + (threadIdx.x >> 5);
  for (int64_t t = first; t < tiles.tiles; t += tiles.step) {
    tiles.wait();
    for (int m = 0; m < a.tile_rows; m += rows_at_once) {
      const int r = m + sub;
      const int64_t row = t * a.tile_rows + r;
      const bool on = row < a.L;
      float v[EPT], s[1] = {0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int k = id + team * c;
        const bool has = on && k < chunks;
        Chunk<T, V> q;
        if (has) q = tiles.template chunk<V>(0, row, r, k);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          v[c * V + i] = has ? q.at(i) : 0.f;
          if (LAYER) s[0] += v[c * V + i];
        }
      }
      float mu = 0.f;
      if (LAYER) {
        team_sum<BLOCK, 1>(s, team, area, turn);
        mu = s[0] * inv;
        s[0] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool has = id + team * c < chunks;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = v[c * V + i] - mu;
          if (LAYER) v[c * V + i] = d;
          if (has) s[0] = fmaf(d, d, s[0]);
        }
      }
      team_sum<BLOCK, 1>(s, team, area, turn);
      if (BLOCK) tiles.fetch();  // every thread has its elements
      const float rs = 1.f / sqrtf(s[0] * inv + a.eps);
      if (on) {
        T* y = static_cast<T*>(a.y) + row * a.H;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int k = id + team * c;
          if (k >= chunks) continue;
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            o[i] = v[c * V + i] * rs * w[c * V + i];
            if (LAYER) o[i] += b[c * V + i];
          }
          Chunk<T, V> q;
          q.pack(o);
          *reinterpret_cast<decltype(q.q)*>(y + static_cast<int64_t>(k) * V) = q.q;
        }
        if (id == 0) {
          if (LAYER && a.mean) a.mean[row] = mu;
          if (a.rstd) a.rstd[row] = rs;
        }
      }
    }
    if (!BLOCK) {
      __syncwarp();
      tiles.fetch();
    }
    tiles.advance();
  }
}

// dx, and a slab's sums for dw and db: slab = block.
template <typename T, int V, bool BLOCK, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) k_norm_bwd(const NormArgs a) {
  constexpr int C = EPT / V;
  constexpr bool RING = V > 1;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bar[TEAM_WARPS * MAX_STAGES];
  __shared__ uint32_t abort_flag;
  __shared__ float area[2][2][32];
  __shared__ float sums[BLOCK ? 1 : 2 * 32 * EPT];
  Tiles<T, BLOCK, RING, 2> tiles(a, smem, bar, &abort_flag);
  const int team = BLOCK ? blockDim.x : a.team;
  const int id = BLOCK ? threadIdx.x : threadIdx.x & (team - 1);
  const int rows_at_once = BLOCK ? 1 : 32 / team;
  const int sub = BLOCK ? 0 : (threadIdx.x & 31) / team;
  const int chunks = a.H / V;
  const float inv = 1.f / a.H;
  int turn = 0;
  float w[EPT], dw[EPT], db[EPT];
  load_params<V, C>(a.weight, a.param_f32, a.H, id, team, 1.f, w);
#pragma unroll
  for (int i = 0; i < EPT; ++i) dw[i] = db[i] = 0.f;
  const int64_t first =
      BLOCK ? blockIdx.x
            : static_cast<int64_t>(blockIdx.x) * TEAM_WARPS + (threadIdx.x >> 5);
  for (int64_t t = first; t < tiles.tiles; t += tiles.step) {
    tiles.wait();
    for (int m = 0; m < a.tile_rows; m += rows_at_once) {
      const int r = m + sub;
      const int64_t row = t * a.tile_rows + r;
      const bool on = row < a.L;
      const float rs = on ? a.rstd[row] : 0.f;
      const float mu = LAYER && on ? a.mean[row] : 0.f;
      Chunk<T, V> x[C], dy[C];
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int k = id + team * c;
        if (!on || k >= chunks) continue;
        x[c] = tiles.template chunk<V>(0, row, r, k);
        dy[c] = tiles.template chunk<V>(1, row, r, k);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float d = dy[c].at(i), n = (x[c].at(i) - mu) * rs;
          const float g = d * w[c * V + i];
          dw[c * V + i] = fmaf(d, n, dw[c * V + i]);
          if (LAYER) {
            db[c * V + i] += d;
            s[0] += g;
          }
          s[1] = fmaf(g, n, s[1]);
        }
      }
      if (!a.want_dx) {
        if (BLOCK) __syncthreads();
        if (BLOCK) tiles.fetch();
        continue;
      }
      team_sum<BLOCK, 2>(s, team, area, turn);
      if (BLOCK) tiles.fetch();
      const float c1 = LAYER ? s[0] * inv : 0.f, c2 = s[1] * inv;
      if (on) {
        T* dx = static_cast<T*>(a.y) + row * a.H;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int k = id + team * c;
          if (k >= chunks) continue;
          float o[V];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float n = (x[c].at(i) - mu) * rs;
            const float g = dy[c].at(i) * w[c * V + i];
            o[i] = rs * (g - c1 - n * c2);
          }
          Chunk<T, V> q;
          q.pack(o);
          *reinterpret_cast<decltype(q.q)*>(dx + static_cast<int64_t>(k) * V) = q.q;
        }
      }
    }
    if (!BLOCK) {
      __syncwarp();
      tiles.fetch();
    }
    tiles.advance();
  }
  if (!a.part) return;
  float* p = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
  if (BLOCK) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = (id + team * c) * V + i;
        if (j >= a.H) continue;
        p[j] = dw[c * V + i];
        if (LAYER) p[a.H + j] = db[c * V + i];
      }
    }
    return;
  }
  // the warp's teams by shuffles, then the warps one after the other
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    for (int o = team; o < 32; o <<= 1) {
      dw[i] += __shfl_xor_sync(ALL_LANES, dw[i], o);
      if (LAYER) db[i] += __shfl_xor_sync(ALL_LANES, db[i], o);
    }
  }
  for (int turn_of = 0; turn_of < TEAM_WARPS; ++turn_of) {
    if ((threadIdx.x >> 5) == turn_of && sub == 0) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int j = (id + team * c) * V + i;
          if (j >= a.H) continue;
          sums[j] = turn_of ? sums[j] + dw[c * V + i] : dw[c * V + i];
          if (LAYER)
            sums[32 * EPT + j] =
                turn_of ? sums[32 * EPT + j] + db[c * V + i] : db[c * V + i];
        }
      }
    }
    __syncthreads();
  }
  for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
    p[j] = sums[j];
    if (LAYER) p[a.H + j] = sums[32 * EPT + j];
  }
}

// Rows of any width, a block to a row.
template <typename T, bool LAYER>
__global__ void __launch_bounds__(256) k_norm_fwd_wide(const NormArgs a) {
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
__global__ void __launch_bounds__(256) k_norm_dx_wide(const NormArgs a) {
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
__global__ void __launch_bounds__(128) k_norm_dparams_wide(const NormArgs a) {
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

// The slabs' sums added in fp64: a thread takes every JOIN_RUNS-th slab of a
// column, then the runs in order.
constexpr int JOIN_RUNS = 16;
__global__ void __launch_bounds__(32 * JOIN_RUNS)
    k_norm_join(const float* __restrict__ part, int slabs, int H, void* dweight,
                void* dbias, int grad_f32) {
  __shared__ double runs[JOIN_RUNS][32];
  const int col = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + col;
  void* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  double t = 0.0;
  if (j < H) {
#pragma unroll 4
    for (int s = run; s < slabs; s += JOIN_RUNS)
      t += part[(static_cast<int64_t>(s) * 2 + blockIdx.y) * H + j];
  }
  runs[run][col] = t;
  __syncthreads();
  if (run == 0 && j < H) {
    for (int q = 1; q < JOIN_RUNS; ++q) t += runs[q][col];
    store_from_float(out, grad_f32, j, static_cast<float>(t));
  }
}

constexpr int64_t MAX_H = 1 << 20;
constexpr int64_t MAX_SLABS = 1024;

int64_t slabs_of(int64_t L) {
  return L < MAX_SLABS ? (L > 0 ? L : 1) : MAX_SLABS;
}

// What is resident on an SM of a kernel with so many threads and bytes.
template <class K>
cudaError_t resident(K kern, int threads, size_t smem, int* n) {
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, threads, smem);
}

struct Geometry {
  bool block;
  int threads;
  size_t smem;
};

// Team, tile and ring of rows of H elements, `arrays` of them read, `v` to a
// chunk. Tiles of lane teams are about 2 KB, so that a copy is worth its
// issue.
Geometry geometry(NormArgs& a, int v, int size, int arrays) {
  const int per = EPT / v, chunks = static_cast<int>(ceil_div(a.H, v));
  Geometry g{};
  g.block = chunks > 32 * per;
  const int need = static_cast<int>(ceil_div(chunks, per));
  if (g.block) {
    g.threads = static_cast<int>(round_up(need, 32));
    a.team = g.threads;
    a.tile_rows = 1;
  } else {
    g.threads = TEAM_WARPS * 32;
    a.team = 1;
    while (a.team < need) a.team *= 2;
    const int at_once = 32 / a.team;
    a.tile_rows = at_once;
    if (v > 1)
      while (a.tile_rows * a.H * size < 2048 && a.tile_rows < 32)
        a.tile_rows += at_once;
  }
  a.stages = 1;
  if (v > 1) {
    const int groups = g.block ? 1 : TEAM_WARPS;
    const int64_t stage =
        static_cast<int64_t>(groups) * arrays * a.tile_rows * a.H * size;
    const int64_t goal = 48 * 1024;
    a.stages = static_cast<int>(goal / stage);
    a.stages = a.stages < 2 ? 2 : a.stages > MAX_STAGES ? MAX_STAGES : a.stages;
    g.smem = static_cast<size_t>(stage) * a.stages;
  }
  return g;
}

// The most shared memory that any geometry asks for: two stages of two rows
// of MAX_FAST_H fp32.
constexpr int MAX_NORM_SMEM = 2 * 2 * MAX_FAST_H * 4;

template <class K>
cudaError_t launch_rows(K kern, NormArgs& a, const Geometry& g, int num_sms,
                        cudaStream_t s, int* grid) {
  if (g.smem > 40 * 1024) {  // with the static part, up to 5 KB
    const cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_NORM_SMEM);
    if (e != cudaSuccess) return e;
  }
  const int64_t tiles = ceil_div(a.L, a.tile_rows);
  int64_t blocks = ceil_div(tiles, g.block ? 1 : TEAM_WARPS);
  if (blocks > num_sms) {
    int n = 0;
    const cudaError_t e = resident(kern, g.threads, g.smem, &n);
    if (e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(num_sms) * (n < 1 ? 1 : n);
    if (blocks > most) blocks = most;
  }
  if (a.part && blocks > MAX_SLABS) blocks = MAX_SLABS;
  *grid = static_cast<int>(blocks);
  kern<<<*grid, g.threads, g.smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int V, bool LAYER>
cudaError_t rows_fwd(NormArgs& a, int num_sms, cudaStream_t s) {
  const Geometry g = geometry(a, V, sizeof(T), 1);
  int grid;
  return g.block
             ? launch_rows(k_norm_fwd<T, V, true, LAYER>, a, g, num_sms, s, &grid)
             : launch_rows(k_norm_fwd<T, V, false, LAYER>, a, g, num_sms, s,
                           &grid);
}
template <typename T, int V, bool LAYER>
cudaError_t rows_bwd(NormArgs& a, int num_sms, cudaStream_t s) {
  const Geometry g = geometry(a, V, sizeof(T), 2);
  return g.block ? launch_rows(k_norm_bwd<T, V, true, LAYER>, a, g, num_sms, s,
                               &a.slabs)
                 : launch_rows(k_norm_bwd<T, V, false, LAYER>, a, g, num_sms, s,
                               &a.slabs);
}

template <typename T, bool LAYER>
cudaError_t forward(NormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool wide = a.H % V == 0 && aligned_to(a.x, 16) && aligned_to(a.y, 16);
  if (a.H <= MAX_FAST_H)
    return wide ? rows_fwd<T, V, LAYER>(a, num_sms, s)
                : rows_fwd<T, 1, LAYER>(a, num_sms, s);
  const int64_t most = num_sms * 8;
  k_norm_fwd_wide<T, LAYER>
      <<<static_cast<unsigned>(a.L < most ? a.L : most), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool LAYER>
cudaError_t backward(NormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const bool wide = a.H % V == 0 && aligned_to(a.x, 16) &&
                    aligned_to(a.dy, 16) && aligned_to(a.y, 16);
  if (a.H <= MAX_FAST_H)
    return wide ? rows_bwd<T, V, LAYER>(a, num_sms, s)
                : rows_bwd<T, 1, LAYER>(a, num_sms, s);
  if (a.part) {
    a.slabs = static_cast<int>(slabs_of(a.L));
    k_norm_dparams_wide<T, LAYER>
        <<<dim3(static_cast<unsigned>(ceil_div(a.H, 128)),
                static_cast<unsigned>(a.slabs)),
           128, 0, s>>>(a);
  }
  if (a.want_dx) {  // last: dx may stand in x's or dy's place
    const int64_t most = num_sms * 8;
    k_norm_dx_wide<T, LAYER>
        <<<static_cast<unsigned>(a.L < most ? a.L : most), 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

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
  a.timeout_ns = wait_timeout_ns();
  a.err = dev->err;
  const bool layer = kind == LCE_LAYER_NORM;
  auto run = dt == LCE_F32
                 ? (layer ? forward<float, true> : forward<float, false>)
                 : (layer ? forward<__nv_bfloat16, true>
                          : forward<__nv_bfloat16, false>);
  ProfScope ps(LCE_K_NORM, s);
  const cudaError_t e = run(a, dev->num_sms, s);
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
  a.want_dx = dx != nullptr;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.L = L;
  a.H = static_cast<int>(H);
  a.param_f32 = param_dt == LCE_F32;
  a.part = params ? static_cast<float*>(ws) : nullptr;
  a.slabs = 0;
  a.timeout_ns = wait_timeout_ns();
  a.err = dev->err;
  auto run = dt == LCE_F32
                 ? (layer ? backward<float, true> : backward<float, false>)
                 : (layer ? backward<__nv_bfloat16, true>
                          : backward<__nv_bfloat16, false>);
  cudaError_t e = cudaSuccess;
  ProfScope ps(LCE_K_NORM_BWD, s);
  if (L > 0) e = run(a, dev->num_sms, s);
  if (params && e == cudaSuccess) {
    k_norm_join<<<dim3(static_cast<unsigned>(ceil_div(H, 32)), dbias ? 2 : 1),
                  32 * JOIN_RUNS, 0, s>>>(a.part, a.slabs, a.H, dweight, dbias,
                                          grad_dt == LCE_F32);
    e = cudaGetLastError();
  }
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "norm_bwd");
}

}  // extern "C"
