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
// Bound: the bytes of the logits (read in each direction) and dlogits. A team
// of lanes holds a row, 8 elements to a lane up to 256 experts, so that a warp
// has several rows of few experts; a lane has the same experts in every row
// and adds their scores in registers. Exponentials and reciprocals are the
// approximate instructions, the rounding of the exponential's argument put back
// (2^-21 of a score, however far from zero or below the row's largest, but for
// the rounding of z - max; 131072 x 256: 1 to 3 us of a pass).
//
// Measured alone, 131072 x 256 fp32 sigmoid: forward 36 us (3.9 TB/s; 68% of
// the issue slots at 46% of the warps: instructions and their latency
// together), joining 608 blocks' sums 11 us (a cold L2), backward 46 us (5.9
// TB/s).
#include <cooperative_groups.h>
#include <math.h>

#include <utility>

#include "lce_host.h"
#include "lce_vec.cuh"

namespace lce {
namespace {

constexpr int MAX_E = 1024;
constexpr int WARPS = 8;
constexpr int64_t SMS = 152;
constexpr int JOIN_BLOCKS = 8;  // of one cluster
constexpr int JOIN_THREADS = 1024;
constexpr int JOIN_AHEAD = 10;  // loads of a thread under way

struct BalanceArgs {
  const void* logits;
  const int32_t* experts;
  const uint8_t* mask;
  int64_t L;
  int E, K;
  int team;  // lanes of a row
  float coef;
  float* loss;
  int32_t* counts;
  float* slopes;
  const float* dloss;
  void* dlogits;
  float* part_p;  // [blocks][E] sums of p
  int* part_n;    // [blocks][E + 1] slots of each expert, tokens
  int blocks;
  unsigned* err;
};

// Over a row's team; `team` is the same for all of a launch.
__device__ __forceinline__ float team_max(float v, int team) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < team) v = fmaxf(v, __shfl_xor_sync(ALL_LANES, v, o));
  return v;
}
__device__ __forceinline__ float team_sum(float v, int team) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < team) v += __shfl_xor_sync(ALL_LANES, v, o);
  return v;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint64_t both(float v) { return f2pack(v, v); }
__device__ __forceinline__ uint64_t ex2_of_pair(uint64_t v) {
  float lo, hi;
  f2unpack(v, lo, hi);
  return f2pack(ex2(lo), ex2(hi));
}

// v (or -v) within [LEAST_EXP, MOST_EXP]; NaN stays. There e^v is 0 and 1 / (1
// + e^v) is 0, what lies below 2^-126 being 0 to both instructions; beyond it
// the correction below would meet infinities.
constexpr float LEAST_EXP = -104.f, MOST_EXP = 88.5f;
template <bool NEGATE>
__device__ __forceinline__ float clamped(float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;"
      : "=f"(r)
      : "f"(NEGATE ? -v : v), "f"(LEAST_EXP));
  if (NEGATE)
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(MOST_EXP));
  return r;
}

// e^v of a pair of v <= 0, or e^-v of any pair, to 2^-22 of itself. The
// argument h of 2^h is rounded, which alone is an error that grows with |v|
// (3e-6 at 60); v - h ln 2, exact but for its own last place, says by how much,
// and e^(v - h ln 2) is 1 + (v - h ln 2) to 2^-35.
constexpr float LN2_HIGH = 0.693147180559945309, LN2_LOW =
    0.693147180559945309 - LN2_HIGH;
template <bool NEGATE>
__device__ __forceinline__ uint64_t exp_of_pair(uint64_t v) {
  float lo, hi;
  f2unpack(v, lo, hi);
  v = f2pack(clamped<NEGATE>(lo), clamped<NEGATE>(hi));
  const uint64_t h = mul2(v, both(LOG2E)), r = ex2_of_pair(h);
  const uint64_t off =
      fma2(h, both(-LN2_LOW), fma2(h, both(-LN2_HIGH), v));
  return fma2(r, off, r);
}

// The largest of a row's logits, 0 for a row without one above -inf.
template <int P>
__device__ __forceinline__ float row_max(const uint64_t (&z)[P], int team) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float lo, hi;
    f2unpack(z[i], lo, hi);
    m = max3(m, lo, hi);
  }
  m = team_max(m, team);
  return m == -INFINITY ? 0.f : m;
}

// Below this a row's sigmoid scores are taken relative to the largest: s is e^z
// and 1 - s is 1, both to less than half a step of fp32, and none is lost to
// fp32's range that is more than 1e-30 of the sum.
constexpr float LEAST_SUM = 1e-8f;

// A row's scores in place of its logits, not yet divided by their sum, which
// is returned; with SLOPE 1 - s of sigmoid scores (for softmax not written).
// Two elements to an instruction where there is one. s = 1 / (1 + q), 1 - s = q
// s with q = e^-z; where s is 0, 1 - s is too, which is of no account.
// Should all sigmoid scores be small, s e^-m = e^(z - m) and 1 - s = 1.
template <int P, bool SIGMOID, bool SLOPE>
__device__ __forceinline__ float scores(uint64_t (&z)[P], uint64_t (&slope)[P],
                                        int team) {
  uint64_t t = 0;
  if (!SIGMOID) {
    const uint64_t minus = both(-row_max(z, team));
#pragma unroll
    for (int i = 0; i < P; ++i) {
      z[i] = exp_of_pair<false>(add2(z[i], minus));
      t = add2(t, z[i]);
    }
    return team_sum(sum_of_pair(t), team);
  }
  const uint64_t one = both(1.f);
  uint64_t s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint64_t q = exp_of_pair<true>(z[i]);
    float lo, hi;
    f2unpack(add2(q, one), lo, hi);
    s[i] = f2pack(reciprocal(lo), reciprocal(hi));
    if (SLOPE) slope[i] = mul2(q, s[i]);
    t = add2(t, s[i]);
  }
  float sum = team_sum(sum_of_pair(t), team);
  // the vote is the warp's: its teams take the shuffles together
  if (__any_sync(ALL_LANES, sum < LEAST_SUM)) {
    const uint64_t minus = both(-row_max(z, team));
    uint64_t far = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      z[i] = exp_of_pair<false>(add2(z[i], minus));
      if (sum < LEAST_SUM) {
        s[i] = z[i];
        if (SLOPE) slope[i] = one;
      }
      far = add2(far, z[i]);
    }
    const float all = team_sum(sum_of_pair(far), team);
    if (sum < LEAST_SUM) sum = all;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) z[i] = s[i];
  return sum;
}

// The rows of a lane: its row's elements, runs of V, a row every `step`; the
// next is under way while one is computed. Rows that take no part are not read
// and leave the last one's elements; elements beyond E are -inf throughout.
template <typename T, int N, int V>
struct Rows {
  const int id, team, E, L, step;
  const T* next;         // the row that is loaded next
  const uint8_t* masks;  // of the row after it
  int row;               // that row
  int64_t leap;
  bool on, on_next;
  Chunk<T, V> q[N / V];

  __device__ __forceinline__ Rows(const BalanceArgs& a, int id_, int first,
                                  int step_)
      : id(id_),
        team(a.team),
        E(a.E),
        L(static_cast<int>(a.L)),
        step(step_),
        next(static_cast<const T*>(a.logits) +
             static_cast<int64_t>(first) * a.E + id_ * V),
        masks(a.mask ? a.mask + first : nullptr),
        row(first),
        leap(static_cast<int64_t>(step_) * a.E) {
    float off[V];
#pragma unroll
    for (int i = 0; i < V; ++i) off[i] = -INFINITY;
#pragma unroll
    for (int c = 0; c < N / V; ++c) q[c].pack(off);
    look();
    load();
  }
  __device__ __forceinline__ void look() {
    on_next = row < L;
    if (masks) {
      if (on_next) on_next = *masks != 0;
      masks += step;
    }
    row += step;
  }
  __device__ __forceinline__ void load() {
    on = on_next;
#pragma unroll
    for (int c = 0; c < N / V; ++c)
      if (on && (id + team * c) * V < E)
        q[c] = load_chunk<T, V>(next + team * c * V);
    next += leap;
    look();
  }
  __device__ __forceinline__ void unpack(uint64_t (&z)[N / 2]) const {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) z[i] = pair_of(q, i);
  }
};

// Blocks of an SM that the registers leave room for. (131072 x 256 fp32, us of
// a forward and a backward pass: 85 with 4 blocks of one row under way, 90 with
// 3, 121 with 5, 143 with 6, where registers spill; with 3 blocks of two rows
// under way 6 more than with 4 of one.)
constexpr int blocks_per_sm(int n) { return n <= 8 ? 4 : n <= 16 ? 2 : 1; }
static_assert(SMS * 4 <= JOIN_THREADS, "a thread to a block's tokens");

// Slots of tokens [t0, t1) into hist, a few loads under way at a time.
__device__ __forceinline__ void count_slots(const int32_t* experts,
                                            const uint8_t* mask, int64_t t0,
                                            int64_t t1, int K, int E, int* hist,
                                            unsigned* err) {
  constexpr int AHEAD = 8;
  const int64_t end = t1 * K;
  for (int64_t i0 = t0 * K + threadIdx.x; i0 < end;
       i0 += AHEAD * static_cast<int64_t>(blockDim.x)) {
    int e[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int64_t i = i0 + u * static_cast<int64_t>(blockDim.x);
      e[u] = -1;
      if (i < end && (!mask || mask[static_cast<uint32_t>(i) / K]))
        e[u] = experts[i];
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (static_cast<unsigned>(e[u]) < static_cast<unsigned>(E))
        atomicAdd(&hist[e[u]], 1);
      else if (e[u] != -1)
        atomicOr(err, ERRBIT_EXPERT_RANGE);
    }
  }
}

// What the sums over tokens give for expert e: its term of the loss / coef.
// f - 1 = (E counts - N K) / (N K), whose numerator is exact.
__device__ __forceinline__ double finish(const BalanceArgs& a, int e, int count,
                                         double p, int tokens) {
  const int64_t slots = static_cast<int64_t>(tokens) * a.K;
  const int64_t load = static_cast<int64_t>(count) * a.E;
  const double inv = slots > 0 ? 1.0 / static_cast<double>(slots) : 0.0;
  a.counts[e] = count;
  a.slopes[e] = static_cast<float>(static_cast<double>(a.coef) * a.K * inv *
                                   (static_cast<double>(load - slots) * inv));
  return static_cast<double>(load) * inv * (p * inv * a.K);
}

// Block b counts the slots of tokens [b, b + 1) L / blocks; the rows of logits
// go to the warps of all blocks in turn.
template <typename T, int N, int V, bool SIGMOID>
__global__ void __launch_bounds__(WARPS * 32, blocks_per_sm(N))
    k_balance(const BalanceArgs a) {
  constexpr int P = N / 2;
  extern __shared__ float sums[];                       // [WARPS][E]
  int* hist = reinterpret_cast<int*>(sums + WARPS * a.E);  // [E + 1]
  __shared__ double part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int id = lane & (a.team - 1), sub = lane / a.team;
  const int at_once = 32 / a.team;
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  // the next rows are under way while some are computed, their masks before
  const int step = gridDim.x * WARPS * at_once;
  const int first = (blockIdx.x * WARPS + warp) * at_once;
  Rows<T, N, V> rows(a, id, first + sub, step);
  count_slots(a.experts, a.mask, a.L * blockIdx.x / a.blocks,
              a.L * (blockIdx.x + 1) / a.blocks, a.K, a.E, hist, a.err);
  uint64_t pairs[P];
#pragma unroll
  for (int i = 0; i < P; ++i) pairs[i] = 0;
  int tokens = 0;
  for (int t0 = first; t0 < a.L; t0 += step) {
    uint64_t z[P], unused[P];
    rows.unpack(z);
    const bool on = rows.on;
    tokens += on;
    rows.load();
    const float t = scores<P, SIGMOID, false>(z, unused, a.team);
    const uint64_t inv = both(t == 0.f ? 0.f : reciprocal(t));
    if (on) {
#pragma unroll
      for (int i = 0; i < P; ++i) pairs[i] = fma2(z[i], inv, pairs[i]);
    }
  }
  float acc[N];
#pragma unroll
  for (int i = 0; i < P; ++i) f2unpack(pairs[i], acc[2 * i], acc[2 * i + 1]);
  let_next_begin();  // k_balance_join, which waits for this launch's end
  if (id == 0 && tokens) atomicAdd(&hist[a.E], tokens);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    for (int o = a.team; o < 32; o <<= 1)
      acc[i] += __shfl_xor_sync(ALL_LANES, acc[i], o);
    const int j = (id + a.team * (i / V)) * V + i % V;
    if (sub == 0 && j < a.E) sums[warp * a.E + j] = acc[i];
  }
  __syncthreads();
  double term = 0.0;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float s = 0.f;
    for (int w = 0; w < WARPS; ++w) s += sums[w * a.E + e];
    if (gridDim.x == 1) {
      term += finish(a, e, hist[e], s, hist[a.E]);
    } else {
      a.part_n[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + e] = hist[e];
      a.part_p[static_cast<int64_t>(blockIdx.x) * a.E + e] = s;
    }
  }
  if (gridDim.x == 1) {
    term = block_total(term, part);
    if (threadIdx.x == 0) *a.loss = static_cast<float>(term * a.coef);
  } else if (threadIdx.x == 0) {
    a.part_n[static_cast<int64_t>(blockIdx.x) * (a.E + 1) + a.E] = hist[a.E];
  }
}

// The blocks' sums: block r of the cluster has the experts 32 r + 256 i + lane,
// its warps the blocks in turn.
__global__ void __launch_bounds__(JOIN_THREADS)
    k_balance_join(const BalanceArgs a) {
  namespace cg = cooperative_groups;
  constexpr int RUNS = JOIN_THREADS / 32;
  __shared__ int tokens_of[32];
  __shared__ LongSum sums[RUNS][32];
  __shared__ int counts[RUNS][32];
  __shared__ double terms[JOIN_BLOCKS];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  // every block has begun before another writes its shared memory
  auto begun = cluster.barrier_arrive();
  wait_for_earlier();
  int n = threadIdx.x < a.blocks
              ? a.part_n[static_cast<int64_t>(threadIdx.x) * (a.E + 1) + a.E]
              : 0;
  double term = 0.0;
  for (int e0 = 32 * blockIdx.x; e0 < a.E; e0 += 32 * JOIN_BLOCKS) {
    const int e = e0 + lane;
    int c = 0;
    LongSum p;
    for (int b0 = run; b0 < a.blocks; b0 += JOIN_AHEAD * RUNS) {
      float v[JOIN_AHEAD];
      int k[JOIN_AHEAD];
#pragma unroll
      for (int u = 0; u < JOIN_AHEAD; ++u) {
        const int b = b0 + u * RUNS;
        const bool has = e < a.E && b < a.blocks;
        v[u] = has ? a.part_p[static_cast<int64_t>(b) * a.E + e] : 0.f;
        k[u] = has ? a.part_n[static_cast<int64_t>(b) * (a.E + 1) + e] : 0;
      }
#pragma unroll
      for (int u = 0; u < JOIN_AHEAD; ++u) {
        p.add(v[u]);
        c += k[u];
      }
    }
    if (e0 == 32 * blockIdx.x) n = block_sum(n, tokens_of);
    sums[run][lane] = p;
    counts[run][lane] = c;
    __syncthreads();
    if (run == 0 && e < a.E) {
#pragma unroll
      for (int q = 1; q < RUNS; ++q) {
        p.add(sums[q][lane]);
        c += counts[q][lane];
      }
      term += finish(a, e, c, p.value(), n);
    }
    __syncthreads();
  }
  if (run == 0) term = lanes_sum(term);
  cluster.barrier_wait(std::move(begun));
  if (threadIdx.x == 0)
    *cluster.map_shared_rank(&terms[blockIdx.x], 0) = term;
  cluster.sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    double loss = 0.0;
    for (int r = 0; r < JOIN_BLOCKS; ++r) loss += terms[r];
    *a.loss = static_cast<float>(loss * a.coef);
  }
}

template <typename T, int N, int V, bool SIGMOID>
__global__ void __launch_bounds__(WARPS * 32, blocks_per_sm(N))
    k_balance_bwd(const BalanceArgs a) {
  constexpr int P = N / 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int id = lane & (a.team - 1), sub = lane / a.team;
  const int at_once = 32 / a.team;
  const int step = gridDim.x * WARPS * at_once;
  const int first = (blockIdx.x * WARPS + warp) * at_once;
  Rows<T, N, V> rows(a, id, first + sub, step);
  T* out = static_cast<T*>(a.dlogits) +
           static_cast<int64_t>(first + sub) * a.E + id * V;
  const float d = *a.dloss;
  uint64_t f[P];
  auto slope_of = [&](int i) {
    const int j = (id + a.team * (i / V)) * V + i % V;
    return j < a.E ? a.slopes[j] * d : 0.f;
  };
#pragma unroll
  for (int i = 0; i < P; ++i)
    f[i] = f2pack(slope_of(2 * i), slope_of(2 * i + 1));
  for (int t0 = first; t0 < a.L; t0 += step) {
    uint64_t z[P], slope[P], dots = 0;
    rows.unpack(z);
    const bool on = rows.on;
    rows.load();
    const float t = scores<P, SIGMOID, true>(z, slope, a.team);
    const float inv = t == 0.f ? 0.f : reciprocal(t);
#pragma unroll
    for (int i = 0; i < P; ++i) dots = fma2(f[i], z[i], dots);
    const float dot = team_sum(sum_of_pair(dots), a.team) * inv;
    if (t0 + sub < a.L) {
      float o[N];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        uint64_t v = mul2(mul2(z[i], both(inv)), add2(f[i], both(-dot)));
        if (SIGMOID) v = mul2(v, slope[i]);
        f2unpack(on ? v : 0, o[2 * i], o[2 * i + 1]);
      }
#pragma unroll
      for (int c = 0; c < N / V; ++c)
        if ((id + a.team * c) * V < a.E)
          store_chunk<T, V>(out + a.team * c * V, &o[c * V]);
    }
    out += rows.leap;
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

// Elements of a row that a lane holds, and the lanes of its team.
int held(int64_t E) { return E <= 256 ? 8 : E <= 512 ? 16 : 32; }
int team_of(int64_t E) {
  int team = 1;
  while (team * held(E) < E) team *= 2;
  return team;
}

// Blocks of a forward pass. One alone, without a join, up to 8 rows to a team:
// 128 x 128 takes 7.3 us on the GPU so and 7.6 in several blocks, 256 x 128 (16
// rows) 10.4 and 7.8. Else two rows to a team as long as the SMs have no more
// than a block, then four, since every block's sums have to be joined: 4099 x
// 60 takes 8.8 us with two and 9.6 with four, 16384 x 128 12.1 and 10.5.
int blocks_of(int64_t L, int64_t E) {
  const int64_t rows = WARPS * 32 / team_of(E);  // of a block at a time
  if (L <= 8 * rows) return 1;
  const int64_t two = ceil_div(L, 2 * rows), four = ceil_div(L, 4 * rows);
  const int64_t most = SMS * blocks_per_sm(held(E));
  return static_cast<int>(two <= SMS ? two
                          : four <= SMS ? SMS : four < most ? four : most);
}

bool sizes_ok(int64_t L, int64_t E) {
  return L >= 0 && L <= (1ll << 30) && E >= 1 && E <= MAX_E;
}
bool slots_ok(int64_t L, int64_t K) {
  return K >= 1 && K <= 32 && L * K <= (1ll << 30);
}

template <typename T, int N, int V>
cudaError_t forward(const BalanceArgs& a, bool sigmoid, cudaStream_t s) {
  // at most 9 * 1024 + 1 words, below what needs no attribute
  const size_t smem = (WARPS * a.E + a.E + 1) * sizeof(float);
  auto kern = sigmoid ? k_balance<T, N, V, true> : k_balance<T, N, V, false>;
  kern<<<a.blocks, WARPS * 32, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.blocks == 1) return e;
  return launch_early_cluster(k_balance_join, dim3(JOIN_BLOCKS),
                              dim3(JOIN_THREADS), 0, s, JOIN_BLOCKS, a);
}

template <typename T, int N, int V>
cudaError_t backward(const BalanceArgs& a, bool sigmoid, int num_sms,
                     cudaStream_t s) {
  const int64_t need = ceil_div(a.L, WARPS * 32 / a.team);
  const int64_t most = num_sms * blocks_per_sm(N);
  const int grid = static_cast<int>(need < most ? need : most);
  auto kern = sigmoid ? k_balance_bwd<T, N, V, true>
                      : k_balance_bwd<T, N, V, false>;
  kern<<<grid, WARPS * 32, 0, s>>>(a);
  return cudaGetLastError();
}

// Calls f.run<T, N, V>(): by type, row length and alignment.
template <typename T, class F>
cudaError_t by_size(int64_t E, bool wide, F&& f) {
  constexpr int V = 16 / sizeof(T);
  switch (held(E)) {
    case 8: return wide ? f.template run<T, 8, V>() : f.template run<T, 8, 1>();
    case 16:
      return wide ? f.template run<T, 16, V>() : f.template run<T, 16, 1>();
    default:
      return wide ? f.template run<T, 32, V>() : f.template run<T, 32, 1>();
  }
}
template <class F>
cudaError_t by_type(lce_dtype dt, int64_t E, bool aligned, F&& f) {
  if (dt == LCE_F32) return by_size<float>(E, aligned && E % 4 == 0, f);
  return by_size<__nv_bfloat16>(E, aligned && E % 8 == 0, f);
}

struct Forward {
  const BalanceArgs& a;
  bool sigmoid;
  cudaStream_t s;
  template <typename T, int N, int V>
  cudaError_t run() {
    return forward<T, N, V>(a, sigmoid, s);
  }
};
struct Backward {
  const BalanceArgs& a;
  bool sigmoid;
  int num_sms;
  cudaStream_t s;
  template <typename T, int N, int V>
  cudaError_t run() {
    return backward<T, N, V>(a, sigmoid, num_sms, s);
  }
};

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_balance_workspace_size(int64_t L, int64_t E) {
  if (!sizes_ok(L, E)) return 0;
  return static_cast<size_t>(blocks_of(L, E)) * (2 * E + 1) * 4;
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
  a.team = team_of(E);
  a.coef = coef;
  a.loss = loss;
  a.counts = counts;
  a.slopes = slopes;
  a.blocks = blocks_of(L, E);
  a.part_p = static_cast<float*>(ws);
  a.part_n = reinterpret_cast<int*>(a.part_p + a.blocks * E);
  a.err = dev->err;
  ProfScope ps(LCE_K_BALANCE, s);
  const cudaError_t e = by_type(dt, E, aligned_to(logits, 16),
                                Forward{a, scoring == LCE_SIGMOID, s});
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
  a.team = team_of(E);
  a.slopes = const_cast<float*>(slopes);
  a.dloss = dloss;
  a.dlogits = dlogits;
  ProfScope ps(LCE_K_BALANCE_BWD, s);
  const cudaError_t e = by_type(
      dt, E, aligned_to(logits, 16) && aligned_to(dlogits, 16),
      Backward{a, scoring == LCE_SIGMOID, dev->num_sms, s});
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
