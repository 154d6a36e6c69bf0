// The norm of many gradients together, and their clipping (lce_grad_norm /
// lce_clip_grads / lce_clip_grad_norm).
//
// norm = sqrt(sum of all g^2), out = min(1, max_norm / (norm + 1e-6)) g. A
// launch takes a table of tensors as its argument. The 16-byte vectors of a
// tensor are cut into chunks of 32 KB, and a block takes every gridDim-th
// chunk; elements before the first and behind the last whole vector go with
// the tensor's first chunk.
//
// Squares of four vectors (16 or 32 elements) are added in fp32, groups in
// fp64. A group whose sum leaves the range in which fp32 squares are exact to
// their rounding is added again in fp64 from the elements, so gradients far
// below 1e-19 or above 1e19 count in full.
//
// Bound: the bytes of the gradients, read for the norm, read and written for
// the clipping, which starts from the end, where the first pass has left them
// in L2. Measured alone on 3.0 GB: the squares 418 us (7.3 TB/s), the clipping
// 899 us (6.7 TB/s).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <new>
#include <tuple>
#include <utility>

#include "lce_host.h"
#include "lce_vec.cuh"

namespace lce {
namespace {

constexpr int TABLE = 256;  // tensors of a launch
constexpr int GRAD_BLOCKS = 608;
constexpr int GRAD_THREADS = 256;
constexpr int UNROLL = 8;  // vectors of a chunk that a thread holds
constexpr int CHUNK = GRAD_THREADS * UNROLL;  // vectors
constexpr int GROUP = 4;   // vectors whose squares are added in fp32

struct GradTable {
  const void* grad[TABLE];
  void* out[TABLE];
  int64_t size[TABLE];
  int first[TABLE + 1];  // chunks before a tensor's own
  uint8_t f32[TABLE];
  int count;
};

// A chunk of a table: vectors [v0, v1) of its tensor's whole ones, which begin
// `head` elements into it.
struct Piece {
  int k;
  bool f32, ends;  // ends: with the elements outside the whole vectors
  int64_t head, whole, v0, v1;
};

__device__ __forceinline__ Piece piece_of(const GradTable& t, int chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  Piece p;
  p.k = lo;
  p.f32 = t.f32[lo];
  const int shift = p.f32 ? 2 : 1;
  const uintptr_t a = reinterpret_cast<uintptr_t>(t.grad[lo]);
  const int64_t n = t.size[lo];
  p.head = static_cast<int64_t>((16 - (a & 15)) & 15) >> shift;
  p.head = min(p.head, n);
  p.whole = (n - p.head) >> (4 - shift);
  const int64_t c = chunk - t.first[lo];
  p.ends = c == 0;
  p.v0 = c * CHUNK;
  p.v1 = min(p.v0 + CHUNK, p.whole);
  return p;
}

__device__ __forceinline__ void unpack(uint4 q, bool f32, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(f32 ? w[i] : w[i] << 16);
    v[2 * i + 1] = f32 ? 0.f : __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ bool in_range(float s) {
  return s >= 1e-28f && s <= 1e37f;
}

__device__ __forceinline__ double square64(float v) {
  return static_cast<double>(v) * static_cast<double>(v);
}

// Squares of a group; 0 stands for absent elements.
__device__ __forceinline__ void add_squares(const uint4 (&q)[GROUP], bool f32,
                                            double& sum) {
  float s = 0.f;
  uint32_t any = 0;
#pragma unroll
  for (int g = 0; g < GROUP; ++g) {
    const uint32_t w[4] = {q[g].x, q[g].y, q[g].z, q[g].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      any |= w[i];
      if (f32) {
        const float v = __uint_as_float(w[i]);
        s = fmaf(v, v, s);
      } else {
        const float a = __uint_as_float(w[i] << 16);
        const float b = __uint_as_float(w[i] & 0xffff0000u);
        s = fmaf(a, a, s);
        s = fmaf(b, b, s);
      }
    }
  }
  if (in_range(s)) {
    sum += static_cast<double>(s);
  } else if (any & (f32 ? 0x7fffffffu : 0x7fff7fffu)) {
#pragma unroll
    for (int g = 0; g < GROUP; ++g) {
      float v[8];
      unpack(q[g], f32, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += square64(v[i]);
    }
  }
}

// A block's share of the squares, blocks taking chunks first, first + step...
__device__ __forceinline__ double squares(const GradTable& t, int first,
                                          int step) {
  double sum = 0.0;
  for (int c = first; c < t.first[t.count]; c += step) {
    const Piece p = piece_of(t, c);
    const uint4* v = reinterpret_cast<const uint4*>(
        static_cast<const char*>(t.grad[p.k]) + p.head * (p.f32 ? 4 : 2));
    uint4 q[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int64_t i = p.v0 + u * GRAD_THREADS + threadIdx.x;
      q[u] = i < p.v1 ? v[i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; u += GROUP) {
      uint4 g[GROUP];
#pragma unroll
      for (int i = 0; i < GROUP; ++i) g[i] = q[u + i];
      if (p.f32)
        add_squares(g, true, sum);
      else
        add_squares(g, false, sum);
    }
    if (p.ends) {
      const int64_t body = p.whole * (p.f32 ? 4 : 8);
      const int64_t rest = t.size[p.k] - body;  // before and behind
      if (threadIdx.x < rest) {
        const int64_t i =
            threadIdx.x < p.head ? threadIdx.x : threadIdx.x + body;
        sum += square64(load_as_float(t.grad[p.k], p.f32, i));
      }
    }
  }
  return sum;
}

// The factor of a norm: NaN for a norm that is NaN, whatever the limit; 1 for
// any other under an infinite limit.
__device__ __forceinline__ float factor(float norm, float max_norm) {
  if (isnan(norm)) return norm;
  const double r =
      static_cast<double>(max_norm) / (static_cast<double>(norm) + 1e-6);
  return isinf(max_norm) || r >= 1.0 ? 1.f : static_cast<float>(r);
}

__device__ __forceinline__ uint4 scaled(uint4 q, bool f32, float scale) {
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = f32 ? __float_as_uint(__uint_as_float(w[i]) * scale)
               : pack_bf16x2(__uint_as_float(w[i] << 16) * scale,
                             __uint_as_float(w[i] & 0xffff0000u) * scale);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements [0, head) and [tail, n) of a tensor, fewer than a block's threads.
__device__ __forceinline__ void clip_ends(const void* grad, void* out, bool f32,
                                          int64_t head, int64_t tail, int64_t n,
                                          float scale) {
  const int64_t i = threadIdx.x < head ? threadIdx.x
                                       : threadIdx.x - head + tail;
  if (i < n)
    store_from_float(out, f32, i, load_as_float(grad, f32, i) * scale);
}

// 16 bytes from byte `shift` (not 0, a multiple of 2) of two vectors on.
__device__ __forceinline__ uint4 joined(uint4 a, uint4 b, int shift) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (shift & 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Chunks from the last one down. An output that does not lie like its gradient
// relative to 16 bytes is written in its own whole vectors, each joined from
// the two of the gradient that hold it; those whose two reach past the
// gradient go with the ends.
__device__ __forceinline__ void clip(const GradTable& t, int first, int step,
                                     float scale) {
  const int chunks = t.first[t.count];
  for (int c = chunks - 1 - first; c >= 0; c -= step) {
    const Piece p = piece_of(t, c);
    const void* grad = t.grad[p.k];
    void* out = t.out[p.k];
    if (scale == 1.f && out == grad) continue;
    const int64_t n = t.size[p.k];
    const int lsize = p.f32 ? 2 : 1;  // an element's bytes, as a shift
    const uintptr_t from = reinterpret_cast<uintptr_t>(grad);
    const uintptr_t to = reinterpret_cast<uintptr_t>(out);
    if (((from ^ to) & 15) == 0) {
      const uint4* v =
          reinterpret_cast<const uint4*>(from + (p.head << lsize));
      uint4* o = reinterpret_cast<uint4*>(to + (p.head << lsize));
      uint4 q[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int64_t i = p.v0 + u * GRAD_THREADS + threadIdx.x;
        if (i < p.v1) q[u] = __ldcs(v + i);
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int64_t i = p.v0 + u * GRAD_THREADS + threadIdx.x;
        if (i < p.v1) __stcs(o + i, scaled(q[u], p.f32, scale));
      }
      if (p.ends)
        clip_ends(grad, out, p.f32, p.head,
                  p.head + (p.whole << (4 - lsize)), n, scale);
      continue;
    }
    // head: to the output's first whole vector whose bytes in the gradient
    // begin at its first vector or behind it
    int64_t head = static_cast<int64_t>((16 - (to & 15)) & 15) >> lsize;
    const int shift = static_cast<int>((from + (head << lsize)) & 15);
    if ((head << lsize) < shift) head += 16 >> lsize;
    const int64_t bytes = ((n - head) << lsize) - (16 - shift);
    int64_t whole = bytes > 0 ? bytes >> 4 : 0;
    const int64_t most =
        static_cast<int64_t>(t.first[p.k + 1] - t.first[p.k]) * CHUNK;
    whole = min(whole, most);
    if (whole == 0) head = 0;
    const uint4* v = reinterpret_cast<const uint4*>(
        (from + (head << lsize)) & ~static_cast<uintptr_t>(15));
    uint4* o = reinterpret_cast<uint4*>(to + (head << lsize));
    const int64_t v1 = min(p.v0 + CHUNK, whole);
#pragma unroll
    for (int u0 = 0; u0 < UNROLL; u0 += 4) {
      uint4 q[4], r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = p.v0 + (u0 + u) * GRAD_THREADS + threadIdx.x;
        if (i < v1) {
          q[u] = v[i];
          r[u] = v[i + 1];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = p.v0 + (u0 + u) * GRAD_THREADS + threadIdx.x;
        if (i < v1)
          __stcs(o + i, scaled(joined(q[u], r[u], shift), p.f32, scale));
      }
    }
    if (p.ends)
      clip_ends(grad, out, p.f32, head, head + (whole << (4 - lsize)), n,
                scale);
  }
}

__global__ void __launch_bounds__(GRAD_THREADS)
    k_grad_squares(const __grid_constant__ GradTable t, double* part) {
  __shared__ double warps[32];
  const double mine = squares(t, blockIdx.x, gridDim.x);
  let_next_begin();  // what reads the parts, which waits for this launch's end
  const double sum = block_total(mine, warps);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The norm of all blocks' squares, in thread 0: the same bits in any block.
__device__ __forceinline__ float norm_of(const double* part, int64_t n,
                                         double* warps) {
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += GRAD_THREADS) sum += part[i];
  sum = block_total(sum, warps);
  return threadIdx.x == 0 ? static_cast<float>(sqrt(sum)) : 0.f;
}

// Thread 0's factor for the block.
__device__ __forceinline__ float shared_factor(float norm, float max_norm) {
  __shared__ float scale;
  if (threadIdx.x == 0) scale = factor(norm, max_norm);
  __syncthreads();
  return scale;
}

__global__ void __launch_bounds__(GRAD_THREADS)
    k_grad_norm(const double* part, int64_t n, float* norm) {
  __shared__ double warps[32];
  wait_for_earlier();
  const float v = norm_of(part, n, warps);
  if (threadIdx.x == 0) *norm = v;
}

__global__ void __launch_bounds__(GRAD_THREADS)
    k_clip(const __grid_constant__ GradTable t, const float* norm,
           float max_norm) {
  clip(t, blockIdx.x, gridDim.x, shared_factor(*norm, max_norm));
}

// Clipping behind k_grad_squares: every block forms the norm for itself.
__global__ void __launch_bounds__(GRAD_THREADS)
    k_norm_clip(const __grid_constant__ GradTable t, const double* part,
                int64_t n, float max_norm, float* norm) {
  __shared__ double warps[32];
  wait_for_earlier();
  const float v = norm_of(part, n, warps);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  clip(t, blockIdx.x, gridDim.x, shared_factor(v, max_norm));
}

// Few chunks: one cluster does it all, its blocks' sums passed through
// distributed shared memory.
constexpr int SMALL_BLOCKS = 8;
__global__ void __launch_bounds__(GRAD_THREADS)
    k_clip_small(const __grid_constant__ GradTable t, float max_norm,
                 float* norm) {
  namespace cg = cooperative_groups;
  __shared__ double warps[32];
  __shared__ double sums[SMALL_BLOCKS];
  cg::cluster_group cluster = cg::this_cluster();
  // every block has begun before another writes its shared memory
  auto begun = cluster.barrier_arrive();
  const double sum = block_total(squares(t, blockIdx.x, SMALL_BLOCKS), warps);
  cluster.barrier_wait(std::move(begun));
  if (threadIdx.x == 0) {
    for (int i = 0; i < SMALL_BLOCKS; ++i)
      *cluster.map_shared_rank(&sums[blockIdx.x], i) = sum;
  }
  cluster.sync();
  float v = 0.f;
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int i = 0; i < SMALL_BLOCKS; ++i) all += sums[i];
    v = static_cast<float>(sqrt(all));
    if (blockIdx.x == 0) *norm = v;
  }
  // the chunks that this block has read: those it takes from the end are
  // another's, whose reads the cluster's barrier has ended
  clip(t, blockIdx.x, SMALL_BLOCKS, shared_factor(v, max_norm));
}

constexpr int64_t MAX_ELEMENTS = 1ll << 40;

int64_t bytes_of(lce_dtype dt, int64_t n) { return n * (dt == LCE_F32 ? 4 : 2); }

lce_status check(const void* const* grads, const lce_dtype* dts,
                 const int64_t* sizes, int64_t n) {
  if (n < 0 || n > (1 << 20)) return LCE_ERR_INVALID_ARG;
  if (n > 0 && (!grads || !dts || !sizes)) return LCE_ERR_INVALID_ARG;
  int64_t total = 0;  // chunks are counted in 32 bits
  for (int64_t i = 0; i < n; ++i) {
    if (dts[i] != LCE_BF16 && dts[i] != LCE_F32) return LCE_ERR_UNSUPPORTED;
    if (sizes[i] < 0 || sizes[i] > MAX_ELEMENTS - total)
      return LCE_ERR_INVALID_ARG;
    total += sizes[i];
    if (sizes[i] > 0 &&
        (!grads[i] || !aligned_to(grads[i], dts[i] == LCE_F32 ? 4 : 2)))
      return LCE_ERR_INVALID_ARG;
  }
  return LCE_OK;
}

// What is written must not be read or written through another tensor: the
// outputs are disjoint, a gradient is its own output or apart from all, the
// norm is apart from the outputs and, where it is written, from the gradients.
lce_status check_disjoint(const void* const* grads, void* const* outs,
                          const lce_dtype* dts, const int64_t* sizes, int64_t n,
                          const float* norm, bool norm_written) {
  struct Range {
    uintptr_t a, b;
  };
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
  for (int64_t i = 0; norm_written && i < n; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]);
    if (sizes[i] > 0 && a < at + sizeof(float) &&
        at < a + bytes_of(dts[i], sizes[i]))
      return LCE_ERR_INVALID_ARG;
  }
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

lce_status check_outputs(const void* const* grads, void* const* outs,
                         const lce_dtype* dts, const int64_t* sizes, int64_t n,
                         const float* norm, bool norm_written,
                         float max_norm) {
  if (n > 0 && !outs) return LCE_ERR_INVALID_ARG;
  if (!norm || !aligned_to(norm, 4) || !(max_norm >= 0.f))
    return LCE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n; ++i)
    if (sizes[i] > 0 &&
        (!outs[i] || !aligned_to(outs[i], dts[i] == LCE_F32 ? 4 : 2)))
      return LCE_ERR_INVALID_ARG;
  return check_disjoint(grads, outs, dts, sizes, n, norm, norm_written);
}

// Chunks of a tensor, one at least.
int64_t chunks_of(const void* grad, lce_dtype dt, int64_t n) {
  const int64_t size = dt == LCE_F32 ? 4 : 2;
  const int64_t head =
      (16 - (reinterpret_cast<uintptr_t>(grad) & 15)) % 16 / size;
  const int64_t whole = n > head ? (n - head) / (16 / size) : 0;
  return whole > CHUNK ? ceil_div(whole, CHUNK) : 1;
}

// Calls launch(table, blocks) for every table of up to TABLE tensors.
template <class F>
cudaError_t each_table(const void* const* grads, void* const* outs,
                       const lce_dtype* dts, const int64_t* sizes, int64_t n,
                       F&& launch) {
  GradTable t;
  t.count = 0;
  t.first[0] = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (sizes[i] > 0) {
      const int64_t chunks = chunks_of(grads[i], dts[i], sizes[i]);
      const int k = t.count++;
      t.grad[k] = grads[i];
      t.out[k] = outs ? outs[i] : nullptr;
      t.size[k] = sizes[i];
      t.f32[k] = dts[i] == LCE_F32;
      t.first[k + 1] = t.first[k] + static_cast<int>(chunks);
    }
    if (t.count == TABLE || (i == n - 1 && t.count > 0)) {
      const int chunks = t.first[t.count];
      const cudaError_t e =
          launch(t, chunks < GRAD_BLOCKS ? chunks : GRAD_BLOCKS);
      if (e != cudaSuccess) return e;
      t.count = 0;
    }
  }
  return cudaSuccess;
}

// Chunks up to which one cluster takes them all. On the GPU 8 chunks take 5.1
// us in one launch and 6.3 in two, 16 take 6.8 and 6.3, 32 take 9.7 and 6.3; a
// launch less saves the host 2 us.
constexpr int64_t SMALL_CHUNKS = 16;

// Launches a kernel whose first argument is a table: `early` while the kernel
// before it still runs (it waits for it itself), or its blocks as one cluster.
enum class Launch { plain, early, cluster };
template <class... P, class... A>
cudaError_t launch_table(void (*kern)(GradTable, P...), Launch how, int blocks,
                         cudaStream_t s, const GradTable& t, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(GRAD_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (how == Launch::early) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = how == Launch::plain ? 0 : 1;
  std::tuple<P...> rest(static_cast<P>(args)...);
  return std::apply(
      [&](auto&... r) {
        void* ptrs[] = {const_cast<GradTable*>(&t), static_cast<void*>(&r)...};
        return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kern),
                                   ptrs);
      },
      rest);
}

// The squares of every table, a part for each of its blocks.
cudaError_t launch_squares(const void* const* grads, const lce_dtype* dts,
                           const int64_t* sizes, int64_t n, double* part,
                           int64_t* parts, cudaStream_t s) {
  return each_table(grads, nullptr, dts, sizes, n,
                    [&](const GradTable& t, int grid) {
                      double* to = part + *parts;
                      *parts += grid;
                      return launch_table(k_grad_squares, Launch::plain, grid,
                                          s, t, to);
                    });
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
  cudaError_t e = launch_squares(grads, dts, sizes, n, part, &parts, s);
  if (e == cudaSuccess)
    e = launch_early(k_grad_norm, dim3(1), dim3(GRAD_THREADS), 0, s, part,
                     parts, norm);
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "grad_norm");
}

lce_status lce_clip_grads(const void* const* grads, void* const* outs,
                          const lce_dtype* dts, const int64_t* sizes, int64_t n,
                          const float* norm, float max_norm, void* stream) {
  LCE_TRY(check(grads, dts, sizes, n));
  LCE_TRY(check_outputs(grads, outs, dts, sizes, n, norm, false, max_norm));
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ProfScope ps(LCE_K_CLIP_GRADS, s);
  const cudaError_t e = each_table(
      grads, outs, dts, sizes, n, [&](const GradTable& t, int grid) {
        return launch_table(k_clip, Launch::plain, grid, s, t, norm, max_norm);
      });
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "clip_grads");
}

lce_status lce_clip_grad_norm(const void* const* grads, void* const* outs,
                              const lce_dtype* dts, const int64_t* sizes,
                              int64_t n, float max_norm, float* norm, void* ws,
                              size_t ws_bytes, void* stream) {
  LCE_TRY(check(grads, dts, sizes, n));
  LCE_TRY(check_outputs(grads, outs, dts, sizes, n, norm, true, max_norm));
  if (!ws || !aligned_to(ws, 16)) return LCE_ERR_INVALID_ARG;
  if (ws_bytes < lce_grad_norm_workspace_size(n)) return LCE_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int64_t parts = 0, chunks = 0, tensors = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (sizes[i] == 0) continue;
    ++tensors;
    chunks += chunks_of(grads[i], dts[i], sizes[i]);
  }
  cudaError_t e = cudaSuccess;
  ProfScope ps(LCE_K_CLIP_GRADS, s);
  if (tensors > 0 && tensors <= TABLE && chunks <= SMALL_CHUNKS) {
    e = each_table(grads, outs, dts, sizes, n, [&](const GradTable& t, int) {
      return launch_table(k_clip_small, Launch::cluster, SMALL_BLOCKS, s, t,
                          max_norm, norm);
    });
  } else {
    e = launch_squares(grads, dts, sizes, n, part, &parts, s);
    bool first = true;
    if (e == cudaSuccess && tensors == 0)
      e = launch_early(k_grad_norm, dim3(1), dim3(GRAD_THREADS), 0, s, part,
                       parts, norm);
    if (e == cudaSuccess)
      e = each_table(grads, outs, dts, sizes, n,
                     [&](const GradTable& t, int grid) {
                       float* to = first ? norm : nullptr;
                       first = false;
                       return launch_table(k_norm_clip, Launch::early, grid, s,
                                           t, part, parts, max_norm, to);
                     });
  }
  ps.done(0);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, "clip_grad_norm");
}

}  // extern "C"
