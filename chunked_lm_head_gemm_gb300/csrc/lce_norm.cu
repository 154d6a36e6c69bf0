// Layer norm and RMS norm of rows (lce_norm_forward / lce_norm_backward).
//
// Forward of a row x: mu its mean, v the mean of (x - mu)^2, r = 1 / sqrt(v +
// eps), n = (x - mu) r, y = n w + b (RMS norm: mu = 0, no b). Backward with g
// = dy w: dx = r (g - mean(g) - n mean(g n)) (RMS norm without mean(g)), dw =
// sum over rows of dy n, db = sum over rows of dy.
//
// Bound: the bytes of x and y, or of x, dy and dx, each moved once. Up to 65536
// columns a row stays in the registers of its team, 16 elements to a thread: a
// power of two of lanes for narrow rows (several rows to a warp), a block up to
// 8192 columns, beyond that a larger block or a cluster, whose sums pass
// through distributed shared memory. A thread has the same columns in every
// row, so it keeps its weights and its sums for dw and db in registers, and the
// backward needs no second pass over x and dy. Rows come through a ring of
// shared memory by bulk copies, issued several rows ahead, so that enough bytes
// are under way without registers to hold them. Wider rows are read again where
// a pass over them needs it.
//
// Measured alone, 65536 x 4096 bf16 RMS norm: forward 170 us (6.3 TB/s),
// backward 224 us (7.2 TB/s) and 7 us for joining its blocks' sums; 1048576 x
// 128 bf16 89 and 127 us (6.0, 6.4 TB/s); 16384 x 2560 fp32 layer norm 54 and
// 70 us (6.3, 7.2 TB/s). Rows that are not on 16 bytes are bound by
// instructions: 65536 x 1001 bf16 RMS norm 53 and, with the join, 112 us (4.9,
// 3.5 TB/s).
#include <cooperative_groups.h>
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
  int team;       // threads of a row in a block; all for a whole block
  int cluster;    // blocks of a row
  int slice;      // columns of each of them (the last may have fewer)
  int tile_rows;  // rows that a group takes at a time
  int stages;     // tiles of a group in shared memory
  uint32_t array_bytes;  // of a tile's place there
  float* part;    // [slabs][2][H] sums of dy n and dy
  int slabs;
  int run;  // rows that a thread may add in registers, 48 at least
  int want_dx;
  int size;  // bytes of an element
  uint64_t timeout_ns;
  unsigned* err;
};

constexpr int EPT = 16;           // elements of a row that a thread holds
constexpr int PAIRS = EPT / 2;   // two elements of fp32 to an instruction
constexpr int TEAM_WARPS = 8;     // warps of a block whose teams are lanes
constexpr int MAX_THREADS = 512;  // of a block that is a team
constexpr int BLOCK_H = EPT * MAX_THREADS;  // the widest row of a block
constexpr int MAX_CLUSTER = 8;
constexpr int CLUSTER_H = BLOCK_H * MAX_CLUSTER;
// A row's team. BIG: a block of up to 1024 threads, whose barrier is a third of
// a cluster's, where that is faster at its 64 registers a thread: in the
// forward pass, and in the backward of an RMS norm of bf16, although it spills
// 168 to 180 bytes. 16384 rows of 16384 bf16: layer norm forward 222 us against
// 585, RMS norm backward 340 against 399.
enum Mode { LANES, BLOCK, CLUSTER, BIG };
constexpr int BIG_H = 2 * BLOCK_H;
constexpr int threads_of(Mode m) { return m == BIG ? 1024 : MAX_THREADS; }
constexpr int MAX_STAGES = 8;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src,
                                          uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Sums over a row's team: lanes by shuffles; a block's warps through shared
// memory, one barrier a call, with two areas in turn; a cluster's warps the
// same, each writing to every block.
template <Mode M>
constexpr int AREA = M == CLUSTER ? 16 * MAX_CLUSTER : M == BIG ? 32 : 16;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

template <Mode M, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], const NormArgs& a,
                                         int rank, float (*area)[N][AREA<M>],
                                         int& turn) {
  if constexpr (M == LANES) {
    for (int o = a.team >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] += __shfl_xor_sync(ALL_LANES, v[i], o);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum(v[i]);
    float(*p)[AREA<M>] = area[turn];
    turn ^= 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if constexpr (M != CLUSTER) {
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i][warp] = v[i];
      }
      __syncthreads();
    } else {
      if (lane < a.cluster) {  // lane l writes to block l
        auto cluster = cooperative_groups::this_cluster();
#pragma unroll
        for (int i = 0; i < N; ++i)
          *cluster.map_shared_rank(&p[i][16 * rank + warp], lane) = v[i];
      }
      cluster_sync();
    }
    // absent warps left zeros
    const int fours =
        M == CLUSTER ? 4 * a.cluster : (blockDim.x + 127) >> 7;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = 0.f;
      for (int w = 0; w < fours; ++w) {
        const float4 q = *reinterpret_cast<const float4*>(&p[i][4 * w]);
        t += (q.x + q.y) + (q.z + q.w);
      }
      v[i] = t;
    }
  }
}

// A thread's columns of a row's slice: n chunks of V, the first at column
// `first`, `stride` columns apart.
//
// Pairs (V = 2) of rows of odd width begin on a pair's address in every other
// row only. A team has rows of one parity, for which the pairs are shifted:
// where a row begins on an odd element, its first pair holds one element, else
// its last one does, and then the pairs are counted from the row's end. So the
// pair with one element is always the first chunk of thread 0.
struct Share {
  int first, stride, n;
  int outside;  // of the first chunk: 0 none, 1 the first element, 2 the second

  template <int V>
  static __device__ __forceinline__ Share of(int width, int id, int team,
                                             int odd_start) {
    Share p;
    if (V == 2 && (width & 1)) {
      const int pairs = (width + 1) >> 1;
      const int k = odd_start ? id : pairs - 1 - id;
      p.first = 2 * k - odd_start;
      p.stride = odd_start ? 2 * team : -2 * team;
      p.n = max(0, (pairs - id + team - 1) / team);
      p.outside = id ? 0 : odd_start ? 1 : 2;
    } else {
      p.first = id * V;
      p.stride = team * V;
      p.n = max(0, (width / V - id + team - 1) / team);
      p.outside = 0;
    }
    return p;
  }
  // Column of the thread's element i of EPT, -1 where it has none.
  template <int V>
  __device__ __forceinline__ int column(int i, int width) const {
    const int j = first + (i / V) * stride + i % V;
    return i / V < n && j < width ? j : -1;
  }
  __device__ __forceinline__ void mask(Chunk<__nv_bfloat16, 2>& c) const {
    c.q &= outside == 1 ? 0xffff0000u : outside == 2 ? 0xffffu : 0xffffffffu;
  }
  __device__ __forceinline__ void mask(Chunk<float, 2>& c) const {
    if (outside == 1) c.q.x = 0;
    if (outside == 2) c.q.y = 0;
  }
  template <typename T, int V>
  __device__ __forceinline__ void store(T* row, const float (&o)[EPT]) const {
#pragma unroll
    for (int c = 0; c < EPT / V; ++c) {
      if (c >= n) continue;
      T* at = row + first + c * stride;
      if (V == 2 && c == 0 && outside) {
        const int k = outside == 1;
        at[k] = from_float<T>(o[k]);
      } else {
        store_chunk<T, V>(at, &o[c * V]);
      }
    }
  }
};

// A group (a warp of lane teams, or the block) and its ring of tiles. A tile is
// tile_rows rows, one after the other in memory; the group takes tiles first,
// first + step, ... Of rows that are not on 16 bytes (chunks of less) the
// 16-byte units that cover the tile are copied; a tile whose units reach past
// the array's ends (the first and last, of arrays that do not begin or end on
// 16 bytes) is read where it lies.
template <typename T, int V, Mode M, int ARRAYS>
struct Tiles {
  static constexpr bool EXACT = V * sizeof(T) == 16;
  const NormArgs& a;
  int64_t tiles, step, tile, next;  // the present tile, the next to be fetched
  int rank, column, width;          // of the cluster's slice
  int last_rows;                    // of the last tile
  int64_t leap;                     // bytes from a tile of the group to the next
  const char* from[ARRAYS];         // of the tile to be fetched
  uint32_t ring, bars;
  int fetch_stage, stage, phase;
  uint32_t offset[ARRAYS];  // of the present tile in its stage
  bool copied[ARRAYS];
  bool gave_up;            // a wait ran out: nothing more is fetched
  int64_t lost, lost_end;  // its tile, and the one that would be fetched next
  int lost_stage, lost_phase;
  WaitCtx ctx;

  __device__ __forceinline__ Tiles(const NormArgs& args, unsigned char* smem,
                                   uint64_t* bar, uint32_t* abort_flag)
      : a(args) {
    const int groups = M == LANES ? TEAM_WARPS : 1;
    const int group = M == LANES ? threadIdx.x >> 5 : 0;
    const int block = M == CLUSTER ? blockIdx.x / a.cluster : blockIdx.x;
    rank = M == CLUSTER ? blockIdx.x % a.cluster : 0;
    column = M == CLUSTER ? rank * a.slice : 0;
    width = M == CLUSTER ? min(a.slice, a.H - column) : a.H;
    if (M == CLUSTER && V == 2 && (a.H & 1)) {
      // slices of whole pairs, in the order in which Share counts them
      const int odd =
          (reinterpret_cast<uintptr_t>(a.x) / sizeof(T) + block) & 1;
      const int pairs = (a.H + 1) / 2, first = rank * (a.slice / 2);
      const int last = min(first + a.slice / 2, pairs);
      column = max(0, odd ? 2 * first - 1 : 2 * (pairs - last));
      width = min(a.H, odd ? 2 * last - 1 : 2 * (pairs - first)) - column;
    }
    tiles = M == LANES ? (a.L + a.tile_rows - 1) / a.tile_rows : a.L;
    last_rows = static_cast<int>(a.L - (tiles - 1) * a.tile_rows);
    step = static_cast<int64_t>(M == CLUSTER ? gridDim.x / a.cluster
                                             : gridDim.x) * groups;
    tile = next = static_cast<int64_t>(block) * groups + group;
    leap = (M == LANES ? step * a.tile_rows : step) * a.H *
           static_cast<int64_t>(sizeof(T));
#pragma unroll
    for (int i = 0; i < ARRAYS; ++i)
      from[i] = array(i) + (first_row() * a.H + column) *
                               static_cast<int64_t>(sizeof(T));
    ring = smem_u32(smem) + group * a.stages * ARRAYS * a.array_bytes;
    bars = smem_u32(bar) + group * MAX_STAGES * 8;
    fetch_stage = stage = phase = 0;
    gave_up = false;
    ctx = WaitCtx{abort_flag, a.err, a.timeout_ns};
    if (threadIdx.x == 0) {
      *abort_flag = 0;
      for (int i = 0; i < groups * MAX_STAGES; ++i)
        mbar_init(smem_u32(bar) + 8 * i, 1);
      fence_mbar_init();
    }
    // also: every block of a cluster has begun before its sums are written
    if (M == CLUSTER)
      cluster_sync();
    else
      __syncthreads();
    for (int i = 0; i < a.stages; ++i) fetch();
  }
  __device__ __forceinline__ bool leader() const {
    return M == LANES ? (threadIdx.x & 31) == 0 : threadIdx.x == 0;
  }
  __device__ __forceinline__ const char* array(int i) const {
    return static_cast<const char*>(i ? a.dy : a.x);
  }
  __device__ __forceinline__ int64_t first_row() const {
    return M == LANES ? tile * a.tile_rows : tile;
  }
  __device__ __forceinline__ int rows_of(int64_t t) const {
    return M != LANES ? 1 : t == tiles - 1 ? last_rows : a.tile_rows;
  }
  // The units that cover the bytes of tile t of array i that begin at `begin`:
  // their own begin, and their bytes, 0 if they reach past the array.
  __device__ __forceinline__ uint32_t window(int i, int64_t t, uintptr_t begin,
                                             uintptr_t* at) const {
    const uint32_t bytes = ((rows_of(t) - 1) * a.H + width) * sizeof(T);
    *at = begin;
    if (EXACT) return bytes;
    *at = begin & ~static_cast<uintptr_t>(15);
    const uintptr_t to = (begin + bytes + 15) & ~static_cast<uintptr_t>(15);
    const uintptr_t base = reinterpret_cast<uintptr_t>(array(i));
    if (*at < base || to > base + a.L * a.H * sizeof(T)) return 0;
    return static_cast<uint32_t>(to - *at);
  }
  // Fetches the group's next tile into the stage that was read last.
  __device__ __forceinline__ void fetch() {
    if (next < tiles && leader() && !gave_up) {
      uintptr_t at[ARRAYS];
      uint32_t bytes[ARRAYS], all = 0;
#pragma unroll
      for (int i = 0; i < ARRAYS; ++i)
        all += bytes[i] = window(
            i, next, reinterpret_cast<uintptr_t>(from[i]), &at[i]);
      const uint32_t bar = bars + 8 * fetch_stage;
      mbar_arrive_expect_tx(bar, all);
#pragma unroll
      for (int i = 0; i < ARRAYS; ++i)
        if (EXACT || bytes[i])
          bulk_load(ring + (fetch_stage * ARRAYS + i) * a.array_bytes,
                    reinterpret_cast<const void*>(at[i]), bytes[i], bar);
    }
#pragma unroll
    for (int i = 0; i < ARRAYS; ++i) from[i] += leap;
    next += step;
    fetch_stage = fetch_stage + 1 == a.stages ? 0 : fetch_stage + 1;
  }
  // Waits for the present tile and returns its rows. Should the wait run out,
  // which raises the error, they are wrong, but every barrier is still met.
  __device__ __forceinline__ int wait() {
#pragma unroll
    for (int i = 0; i < ARRAYS; ++i) {
      offset[i] = ring + (stage * ARRAYS + i) * a.array_bytes;
      copied[i] = true;
      if (!EXACT) {
        const uintptr_t begin = reinterpret_cast<uintptr_t>(array(i)) +
                                (first_row() * a.H + column) * sizeof(T);
        uintptr_t at;
        copied[i] = window(i, tile, begin, &at) != 0;
        offset[i] += static_cast<uint32_t>(begin - at);
      }
    }
    if (!mbar_wait(bars + 8 * stage, phase, ctx, true) && !gave_up) {
      gave_up = true;
      lost = tile;
      lost_end = next < tiles ? next : tiles;
      lost_stage = stage;
      lost_phase = phase;
    }
    return M == LANES ? rows_of(tile) : 1;
  }
  __device__ __forceinline__ bool more() const { return tile < tiles; }
  // Whether the team's rows of odd width begin on an odd element: they are of
  // the parity of the team's place in its warp, or of the group's first tile,
  // its tiles being an even number of rows apart.
  __device__ __forceinline__ int odd_start(int rows_at_once, int sub) const {
    const int row = rows_at_once > 1 ? sub : static_cast<int>(tile & 1);
    return static_cast<int>(
        (reinterpret_cast<uintptr_t>(a.x) / sizeof(T) + row) & 1);
  }
  __device__ __forceinline__ void advance() {
    tile += step;
    stage = stage + 1 == a.stages ? 0 : stage + 1;
    if (stage == 0) phase ^= 1;
  }
  // After a wait that ran out: the copies still under way end, or are given
  // as long again, before the block does.
  __device__ __forceinline__ void drain() {
    if (!gave_up || !leader()) return;
    for (; lost < lost_end; lost += step) {
      mbar_wait(bars + 8 * lost_stage, lost_phase, ctx, false);
      lost_stage = lost_stage + 1 == a.stages ? 0 : lost_stage + 1;
      if (lost_stage == 0) lost_phase ^= 1;
    }
  }
  // The thread's chunks of row r of the present tile's slice (array 0: x, 1:
  // dy), zeros where it has none.
  __device__ __forceinline__ void row(int i, int r, const Share& p, bool on,
                                      Chunk<T, V> (&q)[EPT / V]) const {
    constexpr int C = EPT / V;
    const int n = on ? p.n : 0;
    if (EXACT || copied[i]) {
      const uint32_t at = offset[i] + (r * a.H + p.first) *
                                          static_cast<int>(sizeof(T));
#pragma unroll
      for (int c = 0; c < C; ++c) {
        q[c] = no_chunk<T, V>();
        if (c < n)
          load_shared(at + c * p.stride * static_cast<int>(sizeof(T)), q[c]);
      }
      if constexpr (V == 2) p.mask(q[0]);
    } else {
      const T* from = reinterpret_cast<const T*>(array(i)) +
                      (first_row() + r) * a.H + column;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int j = p.first + c * p.stride + k;
          v[k] = c < n && j >= 0 && j < width ? to_float(from[j]) : 0.f;
        }
        q[c].pack(v);
      }
    }
  }
  static __device__ __forceinline__ void load_shared(uint32_t at,
                                                     Chunk<T, V>& c) {
    if constexpr (EXACT) {
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(c.q.x), "=r"(c.q.y), "=r"(c.q.z), "=r"(c.q.w)
                   : "r"(at)
                   : "memory");
    } else if constexpr (V * sizeof(T) == 8) {
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                   : "=r"(c.q.x), "=r"(c.q.y)
                   : "r"(at)
                   : "memory");
    } else if constexpr (V == 2) {
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(c.q) : "r"(at) : "memory");
    } else if constexpr (sizeof(T) == 4) {
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(c.q) : "r"(at) : "memory");
    } else {
      unsigned short bits;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(at) : "memory");
      c.q = __ushort_as_bfloat16(bits);
    }
  }
};

// A thread's columns of weight or bias in pairs, `absent` where there is none.
template <int V>
__device__ __forceinline__ void load_params(const void* p, bool f32, int column,
                                            int width, const Share& share,
                                            float absent,
                                            uint64_t (&w)[PAIRS]) {
  auto at = [&](int i) {
    const int j = share.column<V>(i, width);
    return j < 0 ? 0.f : p ? load_as_float(p, f32, column + j) : absent;
  };
  // four at a time where a chunk has as many and they lie so
  if (V >= 4 && p &&
      (reinterpret_cast<uintptr_t>(p) & (f32 ? 15 : 7)) == 0) {
#pragma unroll
    for (int i = 0; i < PAIRS; i += 2) {
      const int j = share.column<V>(2 * i, width);
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (j >= 0) load4(p, f32, column + j, v);
      w[i] = f2pack(v[0], v[1]);
      w[i + 1] = f2pack(v[2], v[3]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) w[i] = f2pack(at(2 * i), at(2 * i + 1));
}

template <typename T, int V, Mode M, bool LAYER>
__global__ void __launch_bounds__(threads_of(M)) k_norm_fwd(const NormArgs a) {
  constexpr int C = EPT / V;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bar[TEAM_WARPS * MAX_STAGES];
  __shared__ uint32_t abort_flag;
  __shared__ __align__(16) float area[2][1][AREA<M>];
  for (int i = threadIdx.x; i < 2 * AREA<M>; i += blockDim.x)
    (&area[0][0][0])[i] = 0.f;
  __syncthreads();
  Tiles<T, V, M, 1> tiles(a, smem, bar, &abort_flag);
  const int team = M == LANES ? a.team : blockDim.x;
  const int id = M == LANES ? threadIdx.x & (team - 1) : threadIdx.x;
  const int rows_at_once = M == LANES ? 32 / team : 1;
  const int sub = M == LANES ? (threadIdx.x & 31) / team : 0;
  const Share share = Share::of<V>(tiles.width, id, team,
                                   tiles.odd_start(rows_at_once, sub));
  const float inv = 1.f / a.H;
  int turn = 0;
  uint64_t w[PAIRS], b[PAIRS];
  load_params<V>(a.weight, a.param_f32, tiles.column, tiles.width, share, 1.f,
                 w);
  if (LAYER)
    load_params<V>(a.bias, a.param_f32, tiles.column, tiles.width, share, 0.f,
                   b);
  for (; tiles.more(); tiles.advance()) {
    const int rows = tiles.wait();
    const int64_t row0 = tiles.first_row();
    T* out = static_cast<T*>(a.y) + row0 * a.H + tiles.column;
    for (int m = 0; m < rows; m += rows_at_once) {
      const int r = m + sub;
      const bool on = r < rows;
      Chunk<T, V> x[C];
      tiles.row(0, r, share, on, x);
      float mu = 0.f, s[1];
      uint64_t q = 0;  // a pair of zeros
      if (LAYER) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) q = add2(q, pair_of(x, i));
        s[0] = sum_of_pair(q);
        team_sum<M, 1>(s, a, tiles.rank, area, turn);
        mu = s[0] * inv;
        q = 0;
      }
      const uint64_t minus = f2pack(-mu, -mu);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        uint64_t d = pair_of(x, i);
        if (LAYER) {
          d = add2(d, minus);
          // elements outside the row
          if (V == 1 || (V == 2 && i == 0)) {
            float lo, hi;
            f2unpack(d, lo, hi);
            if (2 * i / V >= share.n || (V == 2 && share.outside == 1))
              lo = 0.f;
            if ((2 * i + 1) / V >= share.n || (V == 2 && share.outside == 2))
              hi = 0.f;
            d = f2pack(lo, hi);
          } else if (2 * i / V >= share.n) {
            d = 0;
          }
        }
        q = fma2(d, d, q);
      }
      s[0] = sum_of_pair(q);
      team_sum<M, 1>(s, a, tiles.rank, area, turn);
      if (M != LANES) tiles.fetch();  // every thread has its elements
      const float rs = rsqrtf(s[0] * inv + a.eps);
      const uint64_t rs2 = f2pack(rs, rs);
      if (on) {
        float o[EPT];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          uint64_t d = pair_of(x, i);
          if (LAYER) d = add2(d, minus);
          d = mul2(d, rs2);
          d = LAYER ? fma2(d, w[i], b[i]) : mul2(d, w[i]);
          f2unpack(d, o[2 * i], o[2 * i + 1]);
        }
        share.store<T, V>(out + r * a.H, o);
        if (id == 0 && tiles.rank == 0) {
          if (LAYER && a.mean) a.mean[row0 + r] = mu;
          if (a.rstd) a.rstd[row0 + r] = rs;
        }
      }
    }
    if (M == LANES) {
      __syncwarp();
      tiles.fetch();
    }
  }
  tiles.drain();
  if (M == CLUSTER) cluster_sync();  // no block ends before its sums are read
}

// The backward's blocks of 257 to 320 threads share an SM by two when they are
// built for it (at most 96 registers a thread): 32768 x 5120 bf16 RMS norm 165
// -> 143 us, layer norm 267 -> 212, although the layer norm spills (32 bytes
// there, to 96 in pairs; single elements spill 130 to 230 in either norm).
// Capped so for other sizes the kernels were up to 1.6 times as slow.
constexpr int PAIRED = 320;

// dx, and a slab's sums for dw and db: slab = block, or cluster.
template <typename T, int V, Mode M, bool LAYER, int BOUND = MAX_THREADS>
__global__ void __launch_bounds__(BOUND, BOUND == PAIRED ? 2 : 1)
    k_norm_bwd(const NormArgs a) {
  constexpr int C = EPT / V;
  constexpr int SUMS = LAYER ? 2 : 1;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t bar[TEAM_WARPS * MAX_STAGES];
  __shared__ uint32_t abort_flag;
  __shared__ __align__(16) float area[2][SUMS][AREA<M>];
  __shared__ float sums[M == LANES ? 2 * 32 * EPT : 1];
  for (int i = threadIdx.x; i < 2 * SUMS * AREA<M>; i += blockDim.x)
    (&area[0][0][0])[i] = 0.f;
  __syncthreads();
  Tiles<T, V, M, 2> tiles(a, smem, bar, &abort_flag);
  const int team = M == LANES ? a.team : blockDim.x;
  const int id = M == LANES ? threadIdx.x & (team - 1) : threadIdx.x;
  const int rows_at_once = M == LANES ? 32 / team : 1;
  const int sub = M == LANES ? (threadIdx.x & 31) / team : 0;
  const Share share = Share::of<V>(tiles.width, id, team,
                                   tiles.odd_start(rows_at_once, sub));
  const float inv = 1.f / a.H;
  int turn = 0;
  uint64_t w[PAIRS], dw[PAIRS], db[PAIRS];
  load_params<V>(a.weight, a.param_f32, tiles.column, tiles.width, share, 1.f,
                 w);
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) dw[i] = db[i] = 0;
  // the thread's sums into the slab: stored, or added to what is there
  auto slab = [&] {
    const int i = M == CLUSTER ? blockIdx.x / a.cluster : blockIdx.x;
    return a.part + static_cast<int64_t>(i) * 2 * a.H + tiles.column;
  };
  auto to_slab = [&](bool add) {
    float* p = slab();
    float aw[EPT], ab[EPT];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      f2unpack(dw[i], aw[2 * i], aw[2 * i + 1]);
      f2unpack(db[i], ab[2 * i], ab[2 * i + 1]);
    }
    if constexpr (V * sizeof(T) == 16) {  // H is a multiple of 4
      auto put = [&](float* to, const float* v) {
        float4 q = make_float4(v[0], v[1], v[2], v[3]);
        if (add) {
          const float4 o = *reinterpret_cast<const float4*>(to);
          q = make_float4(o.x + q.x, o.y + q.y, o.z + q.z, o.w + q.w);
        }
        *reinterpret_cast<float4*>(to) = q;
      };
#pragma unroll
      for (int i = 0; i < EPT; i += 4) {
        const int j = share.column<V>(i, tiles.width);
        if (j < 0) continue;
        put(p + j, &aw[i]);
        if (LAYER) put(p + a.H + j, &ab[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int j = share.column<V>(i, tiles.width);
        if (j < 0) continue;
        p[j] = add ? p[j] + aw[i] : aw[i];
        if (LAYER) p[a.H + j] = add ? p[a.H + j] + ab[i] : ab[i];
      }
    }
  };
  // the statistics of the next tile, a lane to a row, are under way while one
  // is computed
  const int lane = M == LANES ? threadIdx.x & 31 : 0;
  float rs_next = 0.f, mu_next = 0.f;
  auto look_ahead = [&](int64_t t) {
    const bool on = t < tiles.tiles && lane < tiles.rows_of(t);
    const int64_t row = (M == LANES ? t * a.tile_rows : t) + lane;
    rs_next = on ? a.rstd[row] : 0.f;
    if (LAYER) mu_next = on ? a.mean[row] : 0.f;
  };
  look_ahead(tiles.tile);
  constexpr bool RUNS = M == CLUSTER && V * sizeof(T) == 16;  // MAX_RUN
  bool again = false;
  for (int left = a.run; tiles.more(); tiles.advance()) {
    if (RUNS && left-- == 0) {
      if (a.part) to_slab(again);
      again = true;
      left = a.run - 1;
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) dw[i] = db[i] = 0;
    }
    const int rows = tiles.wait();
    const float rs_tile = rs_next, mu_tile = mu_next;
    look_ahead(tiles.tile + tiles.step);
    T* out = static_cast<T*>(a.y) + tiles.first_row() * a.H + tiles.column;
    for (int m = 0; m < rows; m += rows_at_once) {
      const int r = m + sub;
      const bool on = r < rows;
      float rs = rs_tile, mu = mu_tile;
      if (M == LANES) {
        rs = __shfl_sync(ALL_LANES, rs_tile, r);
        if (LAYER) mu = __shfl_sync(ALL_LANES, mu_tile, r);
      }
      const uint64_t rs2 = f2pack(rs, rs), minus = f2pack(-mu, -mu);
      Chunk<T, V> x[C], dy[C];
      tiles.row(0, r, share, on, x);
      tiles.row(1, r, share, on, dy);
      // d = x - mu, n = rs d: rs is applied to products and sums instead
      auto deviation = [&](int i) {
        const uint64_t d = pair_of(x, i);
        return LAYER ? add2(d, minus) : d;
      };
      uint64_t sg = 0, sgd = 0;
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const uint64_t u = pair_of(dy, i), ud = mul2(u, deviation(i));
        dw[i] = fma2(ud, rs2, dw[i]);
        sgd = fma2(ud, w[i], sgd);
        if (LAYER) {
          db[i] = add2(db[i], u);
          sg = fma2(u, w[i], sg);
        }
      }
      if (!a.want_dx) {
        if (M != LANES) {
          __syncthreads();
          tiles.fetch();
        }
        continue;
      }
      float s[SUMS];
      s[0] = sum_of_pair(sgd);
      if (LAYER) s[SUMS - 1] = sum_of_pair(sg);
      team_sum<M, SUMS>(s, a, tiles.rank, area, turn);
      if (M != LANES) tiles.fetch();
      // from the sum on: rs alone may leave fp32's range cubed
      const float c2 = -(s[0] * inv * rs * rs * rs);
      const float c1 = LAYER ? -rs * (s[SUMS - 1] * inv) : 0.f;
      const uint64_t c22 = f2pack(c2, c2), c12 = f2pack(c1, c1);
      if (on) {
        float o[EPT];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          uint64_t g = mul2(pair_of(dy, i), w[i]);
          g = LAYER ? fma2(g, rs2, c12) : mul2(g, rs2);
          f2unpack(fma2(deviation(i), c22, g), o[2 * i], o[2 * i + 1]);
        }
        share.store<T, V>(out + r * a.H, o);
      }
    }
    if (M == LANES) {
      __syncwarp();
      tiles.fetch();
    }
  }
  tiles.drain();
  let_next_begin();  // k_norm_join, which waits for this launch's end
  if (M == CLUSTER) cluster_sync();  // no block ends before its sums are read
  if (!a.part) return;
  if constexpr (M != LANES) {
    to_slab(again);
  } else {
    float* p = slab();
    float aw[EPT], ab[EPT];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      f2unpack(dw[i], aw[2 * i], aw[2 * i + 1]);
      f2unpack(db[i], ab[2 * i], ab[2 * i + 1]);
    }
    // the warp's teams that have the same columns by shuffles (of rows of odd
    // width in pairs every other team), then what is left one after the other
    const int kinds = V == 2 && (a.H & 1) && rows_at_once > 1 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      for (int o = kinds * team; o < 32; o <<= 1) {
        aw[i] += __shfl_xor_sync(ALL_LANES, aw[i], o);
        if (LAYER) ab[i] += __shfl_xor_sync(ALL_LANES, ab[i], o);
      }
    }
    for (int turn_of = 0; turn_of < TEAM_WARPS * kinds; ++turn_of) {
      if ((threadIdx.x >> 5) == turn_of / kinds && sub == turn_of % kinds) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const int j = share.column<V>(i, a.H);
          if (j < 0) continue;
          sums[j] = turn_of ? sums[j] + aw[i] : aw[i];
          if (LAYER)
            sums[32 * EPT + j] = turn_of ? sums[32 * EPT + j] + ab[i] : ab[i];
        }
      }
      __syncthreads();
    }
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      p[j] = sums[j];
      if (LAYER) p[a.H + j] = sums[32 * EPT + j];
    }
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

// The slabs' sums added in a fixed order: a thread takes every JOIN_RUNS-th
// slab of a column, then the runs in order. (By fp64 additions this took 23 us
// for 456 slabs of 2 x 2560 columns.)
constexpr int JOIN_RUNS = 32;
constexpr int JOIN_AHEAD = 16;  // loads of a thread under way
__global__ void __launch_bounds__(32 * JOIN_RUNS)
    k_norm_join(const float* __restrict__ part, int slabs, int H, void* dweight,
                void* dbias, int grad_f32) {
  __shared__ LongSum runs[JOIN_RUNS][32];
  const int col = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + col;
  void* out = blockIdx.y ? dbias : dweight;
  wait_for_earlier();
  if (!out) return;
  LongSum t;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * H + j;
  for (int s0 = run; s0 < slabs; s0 += JOIN_AHEAD * JOIN_RUNS) {
    float v[JOIN_AHEAD];
#pragma unroll
    for (int u = 0; u < JOIN_AHEAD; ++u) {
      const int s = s0 + u * JOIN_RUNS;
      v[u] = j < H && s < slabs ? p[static_cast<int64_t>(s) * 2 * H] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < JOIN_AHEAD; ++u) t.add(v[u]);
  }
  runs[run][col] = t;
  __syncthreads();
  if (run == 0 && j < H) {
#pragma unroll
    for (int q = 1; q < JOIN_RUNS; ++q) t.add(runs[q][col]);
    store_from_float(out, grad_f32, j, t.rounded());
  }
}

constexpr int64_t MAX_H = 1 << 20;
constexpr int64_t MAX_SLABS = 1024;
// Rows that a thread adds in fp32, as far as the slabs go, and since clusters
// are few (19 of eight blocks of 512 threads), no more than 48 and a 128th of
// all. More blocks or clusters than are resident take longer runs in turns;
// clusters whose rows are whole vectors add their registers to their slab
// instead. Either costs the other dearly: 16384 x 32768 bf16, RMS norm, 905 us
// as one run, 1159 in turns, 920 so; 20000 x 12345, layer norm, 720 as one run,
// 726 in turns, 867 with the slab (x and dy one tensor).
constexpr int64_t MAX_RUN = 1024;

// Rows of a run (MAX_RUN).
int64_t run_of(int64_t L) {
  const int64_t slack = L / 128 + 48;
  return slack < MAX_RUN ? slack : MAX_RUN;
}

// The most slabs of L rows. Blocks and clusters (H from 32 EPT to CLUSTER_H)
// are no more than 1024 threads of EPT columns on each SM (64 registers a
// thread, of the largest blocks), and the turns that their runs take: 69 MB for
// 16384 x 65536, where MAX_SLABS are 537.
int64_t slabs_of(int64_t L, int64_t H) {
  int64_t n = MAX_SLABS;
  if (H > 32 * EPT && H <= CLUSTER_H) {
    const int64_t resident = 152 * 1024 * EPT / H;
    const int64_t turns = resident + resident / 64 + 1 + L / run_of(L);
    if (n > turns) n = turns;
  }
  return n < L ? n : L > 0 ? L : 1;
}

constexpr int64_t RING_BYTES = 48 * 1024;  // of a block, as far as two stages

struct Geometry {
  Mode mode;
  bool exact;  // whole 16-byte vectors
  int threads;
  size_t smem;
};

// Team, tile and ring of rows of H elements, `arrays` of them read, `v` to a
// chunk. Tiles of lane teams are about 2 KB, so that a copy is worth its issue,
// where there are rows enough for all warps. A cluster's slices are 4096
// columns at first, as blocks of 256 threads share an SM with others, then
// 8192.
Geometry geometry(NormArgs& a, int v, int size, int arrays, bool may_be_big,
                  int num_sms) {
  Geometry g{};
  const bool exact = g.exact = v * size == 16;
  a.cluster = 1;
  a.slice = a.H;
  const bool big = may_be_big && v > 1 && a.H > BLOCK_H && a.H <= BIG_H;
  if (a.H > BLOCK_H && !big) {
    const int64_t columns = v == 2 ? round_up(a.H, 2) : a.H;  // whole pairs
    a.cluster = a.H <= 4 * 4096 ? 4 : MAX_CLUSTER;
    a.slice = static_cast<int>(round_up(ceil_div(columns, a.cluster), 16));
    a.cluster = static_cast<int>(ceil_div(columns, a.slice));
  }
  const int per = EPT / v, chunks = static_cast<int>(ceil_div(a.slice, v));
  const int need = static_cast<int>(ceil_div(chunks, per));
  g.mode = big                  ? BIG
           : a.H > BLOCK_H      ? CLUSTER
           : chunks > 32 * per ? BLOCK
                               : LANES;
  if (g.mode != LANES) {
    g.threads = static_cast<int>(round_up(need, 32));
    a.team = g.threads;
    a.tile_rows = 1;
  } else {
    g.threads = TEAM_WARPS * 32;
    a.team = 1;
    while (a.team < need) a.team *= 2;
    const int at_once = 32 / a.team;
    a.tile_rows = at_once;
    const bool alternate = v == 2 && a.H % 2 && at_once == 1;  // Share
    while (!alternate && a.tile_rows * a.H * size < 2048 && a.tile_rows < 32 &&
           a.L > static_cast<int64_t>(num_sms) * TEAM_WARPS * a.tile_rows * 2)
      a.tile_rows += at_once;
  }
  // with room for the units at both ends
  const int64_t bytes = static_cast<int64_t>(a.tile_rows) * a.slice * size;
  a.array_bytes = static_cast<uint32_t>(
      exact ? bytes : round_up(bytes, 16) + 16);
  const int64_t stage = static_cast<int64_t>(g.mode == LANES ? TEAM_WARPS : 1) *
                        arrays * a.array_bytes;
  a.stages = static_cast<int>(RING_BYTES / stage);
  a.stages = a.stages < 2 ? 2 : a.stages > MAX_STAGES ? MAX_STAGES : a.stages;
  g.smem = static_cast<size_t>(stage) * a.stages;
  return g;
}

// The most shared memory that any geometry asks for: two stages of two arrays,
// of a row of BLOCK_H fp32 (or one of BIG_H), or for each warp of a tile that a
// step of at most 2 KB brought to 2 KB; each with the units at its ends.
constexpr int MAX_NORM_SMEM = 2 * 2 * TEAM_WARPS * (4096 + 16);
static_assert(MAX_NORM_SMEM >= 2 * 2 * (BLOCK_H * 4 + 32), "a block's row");
static_assert(32 * EPT * 4 <= 2048, "the step of a tile");

// Launches a kernel over a.L rows; *teams: blocks, or clusters, of the launch,
// as many as are resident at once, or a multiple of that.
template <class K>
cudaError_t launch_rows(K kern, NormArgs& a, const Geometry& g, int num_sms,
                        cudaStream_t s, int* teams) {
  a.run = static_cast<int>(run_of(a.L));
  cudaError_t e;
  if (g.smem > 40 * 1024) {  // with the static part, up to 5 KB
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             MAX_NORM_SMEM);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(g.threads);
  cfg.dynamicSmemBytes = g.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.mode == CLUSTER ? 1 : 0;
  const int64_t tiles = ceil_div(a.L, a.tile_rows);
  int64_t n = ceil_div(tiles, g.mode == LANES ? TEAM_WARPS : 1);
  if (n > num_sms / a.cluster) {
    int most = 0;
    if (g.mode == CLUSTER) {
      cfg.gridDim = dim3(a.cluster);
      e = cudaOccupancyMaxActiveClusters(&most, kern, &cfg);
    } else {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&most, kern, g.threads,
                                                        g.smem);
      most *= num_sms;
    }
    if (e != cudaSuccess) return e;
    if (most < 1) return cudaErrorLaunchOutOfResources;
    if (n > most) n = most;
  }
  if (a.part) {
    // the slabs' sums are written and read again: no more than the rows' own
    // bytes, as far as there are SMs
    const int64_t most = a.L * a.size * 3 / 16;
    if (n > most) n = most > num_sms ? most : num_sms;
    if (n > a.L) n = a.L;
    const int64_t slabs = slabs_of(a.L, a.H);
    if (n > slabs) n = slabs;
    // longer runs of rows are taken in turns
    const int64_t at_once = g.mode == LANES ? TEAM_WARPS * 32 / a.team : 1;
    const int64_t turns = ceil_div(ceil_div(a.L, n * at_once), a.run);
    if (g.mode != CLUSTER || !g.exact)
      n *= turns < slabs / n ? turns : slabs / n;
  }
  // rows of a team that has several are of one parity (Share)
  if (g.mode != LANES && a.H % 2 && n < tiles) n = n < 2 ? 2 : n & ~1ll;
  *teams = static_cast<int>(n);
  cfg.gridDim = dim3(static_cast<unsigned>(n * a.cluster));
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, int V, bool LAYER>
cudaError_t rows_fwd(NormArgs& a, int num_sms, cudaStream_t s) {
  const Geometry g = geometry(a, V, sizeof(T), 1, true, num_sms);
  auto kern = g.mode == LANES   ? k_norm_fwd<T, V, LANES, LAYER>
              : g.mode == BLOCK ? k_norm_fwd<T, V, BLOCK, LAYER>
                                : k_norm_fwd<T, V, CLUSTER, LAYER>;
  if constexpr (V > 1) {
    if (g.mode == BIG) kern = k_norm_fwd<T, V, BIG, LAYER>;
  }
  int teams;
  return launch_rows(kern, a, g, num_sms, s, &teams);
}
template <typename T, int V, bool LAYER>
cudaError_t rows_bwd(NormArgs& a, int num_sms, cudaStream_t s) {
  // two stages of two rows of BIG_H bf16 fit; a layer norm's registers do not
  constexpr bool MAY_BE_BIG = V > 1 && sizeof(T) == 2 && !LAYER;
  const Geometry g = geometry(a, V, sizeof(T), 2, MAY_BE_BIG, num_sms);
  a.size = sizeof(T);
  auto kern = g.mode == LANES   ? k_norm_bwd<T, V, LANES, LAYER>
              : g.mode == BLOCK ? k_norm_bwd<T, V, BLOCK, LAYER>
                                : k_norm_bwd<T, V, CLUSTER, LAYER>;
  if (g.mode == BLOCK && g.threads > 256 && g.threads <= PAIRED)
    kern = k_norm_bwd<T, V, BLOCK, LAYER, PAIRED>;
  if constexpr (MAY_BE_BIG) {
    if (g.mode == BIG) kern = k_norm_bwd<T, V, BIG, LAYER, 1024>;
  }
  return launch_rows(kern, a, g, num_sms, s, &a.slabs);
}

// Elements to a chunk: 16 bytes where every row of every array begins on them;
// else two where a row begins alike in all arrays, on a pair's address if it is
// of even width; else one.
template <typename T>
int chunk_of(int H, const void* x, const void* p, const void* q) {
  constexpr int V = 16 / sizeof(T);
  if (H % V == 0 && aligned_to(x, 16) && aligned_to(p, 16) && aligned_to(q, 16))
    return V;
  auto element = [](const void* t) {
    return reinterpret_cast<uintptr_t>(t) / sizeof(T) & 1;
  };
  const uintptr_t start = element(x);
  if (element(p) != start || (q && element(q) != start)) return 1;
  return H % 2 == 0 && start != 0 ? 1 : 2;
}

template <typename T, bool LAYER>
cudaError_t forward(NormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (a.H <= CLUSTER_H) {
    switch (chunk_of<T>(a.H, a.x, a.y, nullptr)) {
      case V: return rows_fwd<T, V, LAYER>(a, num_sms, s);
      case 2: return rows_fwd<T, 2, LAYER>(a, num_sms, s);
      default: return rows_fwd<T, 1, LAYER>(a, num_sms, s);
    }
  }
  const int64_t most = num_sms * 8;
  k_norm_fwd_wide<T, LAYER>
      <<<static_cast<unsigned>(a.L < most ? a.L : most), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool LAYER>
cudaError_t backward(NormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  if (a.H <= CLUSTER_H) {
    switch (chunk_of<T>(a.H, a.x, a.dy, a.y)) {
      case V: return rows_bwd<T, V, LAYER>(a, num_sms, s);
      case 2: return rows_bwd<T, 2, LAYER>(a, num_sms, s);
      default: return rows_bwd<T, 1, LAYER>(a, num_sms, s);
    }
  }
  if (a.part) {
    a.slabs = static_cast<int>(slabs_of(a.L, a.H));
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
  return static_cast<size_t>(slabs_of(L, H)) * 2 * H * sizeof(float);
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
  const uintptr_t elt = dt == LCE_F32 ? 4 : 2;
  const uintptr_t gelt = grad_dt == LCE_F32 ? 4 : 2;
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
    e = launch_early(k_norm_join,
                     dim3(static_cast<unsigned>(ceil_div(H, 32)), dbias ? 2 : 1),
                     dim3(32 * JOIN_RUNS), 0, s, a.part, a.slabs, a.H, dweight,
                     dbias, grad_dt == LCE_F32 ? 1 : 0);
  }
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "norm_bwd");
}

}  // extern "C"
