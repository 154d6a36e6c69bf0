// Grouped tensor-core contractions of the experts' gated MLP. Rows are the
// padded segments of the plan (lce_experts.h); an expert's rows meet only
// its own weights. One persistent kernel template, five uses:
//   UP    a = silu(g) u, g | u = x[token] (Wg_e | Wu_e)^T           K = H
//   DOWN  rows = a Wd_e^T                                           K = I
//   DGU   da' = dy[token] Wd_e beside g and u again, all three in tensor
//         memory at once; the epilogue forms da = w da', dg, du, w a and
//         the row's share of dw = da' . a without rounding g, u or da'
//   DX    rows = [dg | du] [Wg_e ; Wu_e]                            K = 2 I
//   GRAD  dWd_e = dy[token]^T (w a), dWg_e = dg^T x[token],
//         dWu_e = du^T x[token]                           K = rows of e
// x[token] and dy[token] are copies of the token rows in plan order, made
// once for all contractions that read them. Gathering them into the stages by
// TMA instead (four rows to an instruction, one instruction to a lane) needs
// no copy but held every contraction to 37 ns an instruction per SM, 32 of
// them a stage: UP ran at 540 TFLOP/s (L = 32768, H = 2048, I = 768, E = 128,
// top 8), from copies at 1690; gathering by the threads at 418 (16-byte
// asynchronous copies of four warps, three stages ahead) and at 685 (loads of
// eight warps into registers, four K blocks ahead).
//
// Work: units are 128 x 256 output tiles (UP and DGU 128 x 128 of a, whose
// accumulator columns are g | u), walked in a static stride by one CTA per
// SM with the roles of k_gemm: producer warp, MMA lane, epilogue warps; or 256
// x 256 tiles by CTA pairs (PAIR). A unit's accumulation is split into parts,
// each with its own columns, number of buffers and K loop.
//
// Rates, at L = 32768, H = 2048, I = 768, E = 128, top 8 (on pairs): UP 1690
// TFLOP/s, GRAD 1590, DX 1520, DOWN 1440 (K = 768), DGU 1344 (its da' part has
// half the columns for the same rows). With a quarter of the experts and
// tokens the tensor pipe is active in 80, 78, 69, 64 and 60% of the cycles and
// the SMs take 13.6, 13.0, 12.0, 11.4 and 12.3 TB/s of operands, at half of
// L2's peak rate. UP and GRAD are near what a plain product sustains under the
// power limit (1727 TFLOP/s); what holds the others below it is neither the
// tensor pipe nor L2's rate, and has not been found.
#include <cuda_fp16.h>

#include "lce_device.cuh"
#include "lce_experts.h"
#include "lce_host.h"

namespace lce {
namespace {

constexpr unsigned FULL = 0xffffffffu;

struct Maps {
  CUtensorMap a0, a1;       // A operands
  CUtensorMap b0, b1, b2;   // B operands
  CUtensorMap s0, s1, s2;   // store maps (32 x 32 boxes)
};

struct Geom {
  const PlanHead* head;
  const RowTile* tile;
  const int2* seg;
  const int* slot;
  int H, I, E;
  int kb_h, kb_i;   // 64-wide K blocks of H and I
  int num_n;        // column tiles of a row tile
  int d_tiles, d_n;    // tiles of dWd_e (0: not wanted), and column tiles
  int gu_tiles, gu_n;  // of dWg_e, and of dWu_e
  int tile_m;       // output rows of a unit: 128, or 256 of a CTA pair
  int rank;         // of this CTA in its pair (set by the kernel)
  uint64_t timeout_ns;
};

struct Unit {
  int e;        // expert
  int row0;     // first row (row tiles) or first K row (weight gradients)
  int rows;     // padded rows of this CTA's part of the tile, or the K extent
  int both;     // row tiles: padded rows of the whole tile
  int m, n;     // tile of the output
  int which;    // weight gradients: 0 dWd, 1 dWg, 2 dWu
};

// ---- loads -------------------------------------------------------------------
// PAIR: on CTA pairs (cta_group::2, tiles of 256 rows). Each CTA stages its
// 128 rows of A and its half of B's columns; completion is counted on the
// leader's barrier (bar: its cluster address).
template <bool PAIR>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* tm,
                                        int c0, int c1, uint32_t bar) {
  if (PAIR)
    tma_load_2d_pair(dst, tm, c0, c1, bar);
  else
    tma_load_2d(dst, tm, c0, c1, bar);
}
template <bool PAIR>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* tm,
                                        int c0, int c1, int c2, uint32_t bar) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile."
        "mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2),
        "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::"
        "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2),
        "r"(bar)
        : "memory");
}

// K-major A rows of this CTA's part of a tile: 0, 64 or 128 rows.
template <bool PAIR>
__device__ __forceinline__ void load_rows(uint32_t sa, const CUtensorMap* tm,
                                          const Unit& u, int c0, uint32_t bar) {
  if (u.rows > 0) load_2d<PAIR>(sa, tm, c0, u.row0, bar);
  if (u.rows > 64) load_2d<PAIR>(sa + 8192, tm, c0, u.row0 + 64, bar);
}

// 64 rows from r0 as the K index of an MN-major operand: BOXES boxes of 64
// columns from c0.
template <bool PAIR, int BOXES>
__device__ __forceinline__ void load_cols(uint32_t dst, const CUtensorMap* tm,
                                          int c0, int r0, uint32_t bar) {
#pragma unroll
  for (int j = 0; j < BOXES; ++j)
    load_2d<PAIR>(dst + j * 8192, tm, c0 + 64 * j, r0, bar);
}
template <bool PAIR, int BOXES>
__device__ __forceinline__ void load_cols_of(uint32_t dst,
                                             const CUtensorMap* tm, int c0,
                                             int r0, int e, uint32_t bar) {
#pragma unroll
  for (int j = 0; j < BOXES; ++j)
    load_3d<PAIR>(dst + j * 8192, tm, c0 + 64 * j, r0, e, bar);
}

// ---- the uses ----------------------------------------------------------------
constexpr int GROUP_N = 8;

struct RowUnits {
  __device__ static int units(const Geom& g) {
    return g.head->tiles * g.num_n;
  }
  // An expert's units in groups of GROUP_N column tiles, its row tiles inside
  // a group: what runs at once then reads some 8 panels of weights and 10 of
  // rows, where a row tile after the other would stream all of a wide
  // expert's weights once per row tile. L = 8192, H = 4096, I = 8192, E = 8,
  // top 2 (134 MB of Wg_e and Wu_e): UP 1386 -> 1202 us.
  __device__ static Unit unit(const Geom& g, int u) {
    const int4 x = reinterpret_cast<const int4*>(g.tile)[u / g.num_n];
    const int first = x.y, row0 = x.z, rows = x.w;
    const int tiles = (rows + g.tile_m - 1) / g.tile_m;
    const int r = u - first * g.num_n;
    const int n0 = r / (tiles * GROUP_N) * GROUP_N;
    const int in = r - n0 * tiles;
    const int width = min(GROUP_N, g.num_n - n0);
    const int m = in / width;
    const int both = min(g.tile_m, rows - m * g.tile_m);
    return Unit{x.x,
                row0 + m * g.tile_m + g.rank * BM,
                min(max(both - g.rank * BM, 0), BM),
                both,
                m,
                n0 + in - m * width,
                0};
  }
};
struct GradUnits {
  __device__ static int units(const Geom& g) {
    return g.E * (g.d_tiles + 2 * g.gu_tiles);
  }
  __device__ static Unit unit(const Geom& g, int u) {
    const int per = g.d_tiles + 2 * g.gu_tiles;
    const int e = u / per;
    int r = u - e * per;
    const int2 s = g.seg[e];
    if (r < g.d_tiles)
      return Unit{e, s.x, s.y, 0, r / g.d_n, r % g.d_n, 0};
    r -= g.d_tiles;
    const int which = r >= g.gu_tiles ? 2 : 1;
    if (which == 2) r -= g.gu_tiles;
    return Unit{e, s.x, s.y, 0, r / g.gu_n, r % g.gu_n, which};
  }
};

template <int N_, int COL_, int BUFS_, bool A_MN_, bool B_MN_>
struct Part {
  static constexpr int N = N_, COL = COL_, BUFS = BUFS_;
  static constexpr bool A_MN = A_MN_, B_MN = B_MN_;
};

// blocks: K blocks of a part; bytes: what a K block's loads of all CTAs of the
// unit bring; load: this CTA's loads of one K block.
struct OpUp : RowUnits {
  static constexpr int PARTS = 1;
  using P0 = Part<256, 0, 2, false, false>;
  using P1 = P0;
  template <int P>
  __device__ static int blocks(const Geom& g, const Unit&) { return g.kb_h; }
  template <int P>
  __device__ static uint32_t bytes(const Geom&, const Unit& u) {
    return u.both * 128u + 32768u;
  }
  template <int P, bool PAIR>
  __device__ static void load(const Maps& m, const Geom& g, const Unit& u,
                              int kb, uint32_t sa, uint32_t sb, uint32_t bar) {
    load_rows<PAIR>(sa, &m.a0, u, kb * BK, bar);
    if (PAIR) {  // the leader stages Wg's rows, its peer Wu's
      load_3d<PAIR>(sb, g.rank ? &m.b1 : &m.b0, kb * BK, u.n * 128, u.e, bar);
    } else {
      load_3d<PAIR>(sb, &m.b0, kb * BK, u.n * 128, u.e, bar);
      load_3d<PAIR>(sb + 16384, &m.b1, kb * BK, u.n * 128, u.e, bar);
    }
  }
};

struct OpDown : RowUnits {
  static constexpr int PARTS = 1;
  using P0 = Part<256, 0, 2, false, false>;
  using P1 = P0;
  template <int P>
  __device__ static int blocks(const Geom& g, const Unit&) { return g.kb_i; }
  template <int P>
  __device__ static uint32_t bytes(const Geom&, const Unit& u) {
    return u.both * 128u + 32768u;
  }
  template <int P, bool PAIR>
  __device__ static void load(const Maps& m, const Geom& g, const Unit& u,
                              int kb, uint32_t sa, uint32_t sb, uint32_t bar) {
    load_rows<PAIR>(sa, &m.a0, u, kb * BK, bar);
    // boxes of 256 rows of Wd_e, of 128 on a pair
    load_3d<PAIR>(sb, &m.b0, kb * BK, u.n * 256 + g.rank * 128, u.e, bar);
  }
};

struct OpDx : RowUnits {
  static constexpr int PARTS = 1;
  using P0 = Part<256, 0, 2, false, true>;
  using P1 = P0;
  template <int P>
  __device__ static int blocks(const Geom& g, const Unit&) {
    return 2 * g.kb_i;
  }
  template <int P>
  __device__ static uint32_t bytes(const Geom&, const Unit& u) {
    return u.both * 128u + 32768u;
  }
  template <int P, bool PAIR>
  __device__ static void load(const Maps& m, const Geom& g, const Unit& u,
                              int kb, uint32_t sa, uint32_t sb, uint32_t bar) {
    const bool second = kb >= g.kb_i;  // du and Wu after dg and Wg
    const int k0 = (second ? kb - g.kb_i : kb) * BK;
    load_rows<PAIR>(sa, second ? &m.a1 : &m.a0, u, k0, bar);
    load_cols_of<PAIR, PAIR ? 2 : 4>(sb, second ? &m.b1 : &m.b0,
                                     u.n * 256 + g.rank * 128, k0, u.e, bar);
  }
};

// da' first (two buffers of 128 columns), then g | u (one of 256): while the
// epilogue reads a tile, the next tile's da' is already being accumulated.
struct OpDgu : RowUnits {
  static constexpr int PARTS = 2;
  using P0 = Part<128, 256, 2, false, true>;
  using P1 = Part<256, 0, 1, false, false>;
  template <int P>
  __device__ static int blocks(const Geom& g, const Unit&) { return g.kb_h; }
  template <int P>
  __device__ static uint32_t bytes(const Geom&, const Unit& u) {
    return u.both * 128u + (P == 0 ? 16384u : 32768u);
  }
  template <int P, bool PAIR>
  __device__ static void load(const Maps& m, const Geom& g, const Unit& u,
                              int kb, uint32_t sa, uint32_t sb, uint32_t bar) {
    if (P == 0) {
      load_rows<PAIR>(sa, &m.a1, u, kb * BK, bar);
      load_cols_of<PAIR, PAIR ? 1 : 2>(sb, &m.b2, u.n * 128 + g.rank * 64,
                                       kb * BK, u.e, bar);
    } else {
      OpUp::load<0, PAIR>(m, g, u, kb, sa, sb, bar);
    }
  }
};

// The three weight gradients in one launch: units of an expert are the tiles
// of dWd_e (A dy, B w a), then of dWg_e and dWu_e (A dg or du, B x).
struct OpGrad : GradUnits {
  static constexpr int PARTS = 1;
  using P0 = Part<256, 0, 2, true, true>;
  using P1 = P0;
  template <int P>
  __device__ static int blocks(const Geom&, const Unit& u) {
    return u.rows / SEG_ROWS;
  }
  template <int P>
  __device__ static uint32_t bytes(const Geom& g, const Unit&) {
    return g.tile_m * 128u + 32768u;
  }
  template <int P, bool PAIR>
  __device__ static void load(const Maps& m, const Geom& g, const Unit& u,
                              int kb, uint32_t sa, uint32_t sb, uint32_t bar) {
    const int k0 = u.row0 + kb * BK;
    const CUtensorMap* ta = u.which == 0 ? &m.b0 : u.which == 1 ? &m.a0 : &m.a1;
    const CUtensorMap* tb = u.which == 0 ? &m.b1 : &m.b2;
    load_cols<PAIR, 2>(sa, ta, u.m * g.tile_m + g.rank * BM, k0, bar);
    load_cols<PAIR, PAIR ? 2 : 4>(sb, tb, u.n * BN + g.rank * 128, k0, bar);
  }
};

// ---- epilogues ---------------------------------------------------------------
// Each runs on a warp's 32 rows and its half of the columns of a finished
// unit (eight epilogue warps: two to each lane quarter of tensor memory;
// taddr is the quarter). Against four warps DGU 1906 -> 1873 us, dWd 600 ->
// 582 us (L = 32768, H = 2048, I = 768, E = 128, top 8).

// A unit's accumulators go back to the MMA as soon as the warp has read them
// (release(), once per unit), before the last values are worked on and stored.
template <int PARTS, bool PAIR>
struct Release {
  uint32_t bar0, bar1;
  bool done;
  __device__ __forceinline__ void operator()() {
    if (done) return;
    done = true;
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31u) == 0) {
      if (PAIR) {
        mbar_arrive_cluster(mapa_shared(bar0, 0));
        if (PARTS == 2) mbar_arrive_cluster(mapa_shared(bar1, 0));
      } else {
        mbar_arrive(bar0);
        if (PARTS == 2) mbar_arrive(bar1);
      }
    }
  }
};

// a = silu(g) u in bf16.
struct EpiUp : EpiBase {
  struct Params {
    int unused;
  };
  template <class R>
  __device__ __forceinline__ void tile(const Params&, const Maps& m,
                                       const Geom& g, const Unit& u,
                                       uint32_t taddr, int r, int half,
                                       int i, R& release) {
    const int wr = r & ~31;
    if (wr >= u.rows) return;
    const uint32_t t0 = taddr + (i & 1) * 256;
#pragma unroll 1
    for (int c = 2 * half; c < 2 * half + 2; ++c) {
      const int j0 = u.n * 128 + c * 32;
      if (j0 >= g.I) break;
      float gv[32], uv[32];
      tmem_ld32(t0 + c * 32, gv);
      tmem_ld32(t0 + 128 + c * 32, uv);
      if (c == 2 * half + 1) release();
#pragma unroll
      for (int k = 0; k < 32; ++k) uv[k] *= gv[k] * sigmoid_fast(gv[k]);
      store_box(uv, j0, u.row0 + wr, &m.s0);
    }
  }
};

// Rows of H columns for the sum over a token's slots, in fp16 under a power
// of two for each row and 128 columns: the largest finite value of the
// piece lands in [2^14, 2^15), so a value is off by 2^-11 of itself at most
// (below 2^-14, where fp16's steps stay 2^-24, by 2^-39 of the piece's
// largest), an eighth of a bf16 rounding, at half the bytes of fp32.
// Infinities and NaN stay what they are. Against fp32
// rows stored straight from registers: DOWN 1149 -> 592 us, DX 1303 ->
// 1079 us, the two sums 694 -> 477 us (L = 32768, H = 2048, I = 768, E =
// 128, top 8).
struct EpiRows : EpiBase {
  struct Params {
    float* scale;  // [max_rows][2 num_n]
  };
  template <class R>
  __device__ __forceinline__ void tile(const Params& p, const Maps& m,
                                       const Geom& g, const Unit& u,
                                       uint32_t taddr, int r, int half,
                                       int i, R& release) {
    const int wr = r & ~31;
    if (wr >= u.rows) return;
    const int c0 = u.n * 256 + half * 128;
    if (c0 >= g.H) return;
    te = &m.s0;
    const uint32_t t0 = taddr + (i & 1) * 256 + half * 128;
    float v[2][64];  // columns past H are zero
    tmem_ld64(t0, v[0]);
    tmem_ld64(t0 + 64, v[1]);
    release();
    float mx = 0.f;
#pragma unroll
    for (int k = 0; k < 64; ++k)
      mx = fmaxf(fmaxf(mx, fabsf(v[0][k])), fabsf(v[1][k]));
    if (__any_sync(FULL, mx > 3.4028235e38f)) {  // infinities: the others' max
      mx = 0.f;
#pragma unroll
      for (int k = 0; k < 64; ++k) {
        const float x = fabsf(v[0][k]), y = fabsf(v[1][k]);
        if (x <= 3.4028235e38f) mx = fmaxf(mx, x);
        if (y <= 3.4028235e38f) mx = fmaxf(mx, y);
      }
    }
    // 2^(exponent - 14), kept normal; 1 for a piece of zeros
    const int e = static_cast<int>(__float_as_uint(mx) >> 23);  // mx >= 0
    const int se = mx == 0.f ? 127 : max(e - 14, 1);
    const float scale = __uint_as_float(static_cast<uint32_t>(se) << 23);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - se) << 23);
    p.scale[static_cast<int64_t>(u.row0 + r) * (2 * g.num_n) + 2 * u.n + half] =
        scale;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int j0 = c0 + c * 64;
      if (j0 >= g.H) break;
      uint32_t w0[16], w1[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const __half2 x = __floats2half2_rn(v[c][2 * k] * inv,
                                            v[c][2 * k + 1] * inv);
        const __half2 y = __floats2half2_rn(v[c][32 + 2 * k] * inv,
                                            v[c][33 + 2 * k] * inv);
        w0[k] = *reinterpret_cast<const uint32_t*>(&x);
        w1[k] = *reinterpret_cast<const uint32_t*>(&y);
      }
      store_box_pair(w0, w1, j0, u.row0 + wr, j0 + 32 < g.H);
    }
  }
};

// dg, du, w a and the row's part of da' . a (this tile's columns).
struct EpiDgu : EpiBase {
  struct Params {
    const void* w;
    int w_f32;
    float* part;
    int64_t stride;
  };
  template <class R>
  __device__ __forceinline__ void tile(const Params& p, const Maps& m,
                                       const Geom& g, const Unit& u,
                                       uint32_t taddr, int r, int half,
                                       int i, R& release) {
    const int wr = r & ~31;
    if (wr >= u.rows) return;
    const int slot = g.slot[u.row0 + r];
    float w = 0.f;
    if (slot >= 0)
      w = p.w_f32 ? __ldg(static_cast<const float*>(p.w) + slot)
                  : static_cast<float>(
                        static_cast<const __nv_bfloat16*>(p.w)[slot]);
    const uint32_t tda = taddr + 256 + (i & 1) * 128;
    float dot = 0.f;
#pragma unroll 1
    for (int c = 2 * half; c < 2 * half + 2; ++c) {
      const int j0 = u.n * 128 + c * 32;
      if (j0 >= g.I) break;
      float gv[32], uv[32], da[32];
      tmem_ld32(taddr + c * 32, gv);
      tmem_ld32(taddr + 128 + c * 32, uv);
      tmem_ld32(tda + c * 32, da);
      if (c == 2 * half + 1) release();
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float s = sigmoid_fast(gv[k]);
        const float sil = gv[k] * s;     // silu(g)
        const float a = sil * uv[k];
        dot = fmaf(da[k], a, dot);
        const float d = w * da[k];
        // silu'(g) = s (1 + g (1 - s))
        const float dg = d * uv[k] * s * (1.f + gv[k] * (1.f - s));
        gv[k] = dg;
        da[k] = d * sil;                 // du
        uv[k] = w * a;
      }
      if (slot < 0) {  // a padding row adds nothing to a weight gradient
#pragma unroll           // (0 times an infinite weight is NaN)
        for (int k = 0; k < 32; ++k) gv[k] = da[k] = uv[k] = 0.f;
      }
      store_box(gv, j0, u.row0 + wr, &m.s0);
      store_box(da, j0, u.row0 + wr, &m.s1);
      store_box(uv, j0, u.row0 + wr, &m.s2);
    }
    p.part[(2 * u.n + half) * p.stride + u.row0 + r] = dot;
  }
};

// An expert's weight gradient, bf16 or fp32, zero where it has no rows. fp32
// goes straight from registers, a row to a lane, which costs more than its
// twice the bytes: against bf16 GRAD takes 1860 and 1580 us (L = 32768, H =
// 2048, I = 768, E = 128, top 8), 216 and 126 us (L = 8192, H = 1024, I = 512,
// E = 64, top 6), 39 and 23 us (L = 1537, H = 1000, I = 424, E = 10, top 2).
struct EpiWeights : EpiBase {
  struct Params {
    float* out[3];  // fp32 gradients: dWd [E][H][I], dWg and dWu [E][I][H];
                    // NULL: bf16, through the store maps
  };
  // Box of this warp's 32 rows and 32 columns of expert e's gradient (as
  // store_box; the map drops what lies past the expert's rows and columns).
  __device__ __forceinline__ void store_box_of(const float (&v)[32],
                                               const CUtensorMap* map, int j0,
                                               int row0, int e) {
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t buf = stage + (nstored & 1u) * EPI_BUF_BYTES;
    if (lane == 0 && nstored >= 2) bulk_wait_read1();
    __syncwarp();
    const uint32_t rowa = buf + lane * 64u;
    const uint32_t sw = (lane >> 1) & 3u;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      st_shared_v4(rowa + ((static_cast<uint32_t>(q) ^ sw) << 4),
                   pack_bf16x2(v[8 * q], v[8 * q + 1]),
                   pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                   pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                   pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      asm volatile(
          "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, "
          "%3, %4}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
          "r"(buf), "r"(j0), "r"(row0), "r"(e)
          : "memory");
      bulk_commit();
    }
    ++nstored;
  }

  template <class R>
  __device__ __forceinline__ void tile(const Params& p, const Maps& m,
                                       const Geom& g, const Unit& u,
                                       uint32_t taddr, int r, int half,
                                       int i, R& release) {
    float* base = u.which == 0 ? p.out[0] : u.which == 1 ? p.out[1] : p.out[2];
    const CUtensorMap* map =
        u.which == 0 ? &m.s0 : u.which == 1 ? &m.s1 : &m.s2;
    const int rows = u.which == 0 ? g.H : g.I;
    const int cols = u.which == 0 ? g.I : g.H;
    const int row = u.m * g.tile_m + g.rank * BM + r;
    if (row - (r & 31) >= rows) return;  // the same for the warp
    const int64_t at = (static_cast<int64_t>(u.e) * rows + row) * cols;
#pragma unroll 1
    for (int c = 4 * half; c < 4 * half + 4; ++c) {
      const int j0 = u.n * BN + c * 32;
      if (j0 >= cols) break;
      float v[32];
      if (u.rows > 0) {
        tmem_ld32(taddr + (i & 1) * 256 + c * 32, v);
        if (c == 4 * half + 3) release();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = 0.f;
      }
      if (base == nullptr) {
        store_box_of(v, map, j0, row - (r & 31), u.e);
        continue;
      }
      if (row >= rows) continue;
      float4* d = reinterpret_cast<float4*>(base + at + j0);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (j0 + 4 * q < cols)  // cols % 8 == 0
          d[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2],
                             v[4 * q + 3]);
    }
  }
};

// ---- roles -------------------------------------------------------------------
// Ring of stages by form: one CTA stages 128 rows of A and 256 columns of B,
// a CTA of a pair 128 and 128.
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;

template <bool PAIR>
struct Form {
  static constexpr int STAGES_ = PAIR ? STAGES2 : STAGES;
  static constexpr int A_BYTES = A_STAGE_BYTES;
  static constexpr int B_BYTES = PAIR ? B2_STAGE_BYTES : B_STAGE_BYTES;
  static constexpr int RING_BYTES = STAGES_ * (A_BYTES + B_BYTES);
  static constexpr int SMEM =
      1024 + RING_BYTES + 1024 + EPI_WARPS * 2 * EPI_BUF_BYTES;
};

// Barriers: full / empty per stage; tfull[2]: a unit's accumulators are
// ready (by unit parity); tempty[part][2]: a part's buffer may be overwritten.
// On a pair, full and tempty live in the leader, empty and tfull in both.
template <bool PAIR>
struct Bars {
  static constexpr int S = Form<PAIR>::STAGES_;
  static constexpr int COUNT = 2 * S + 7;
  uint32_t base;
  __device__ uint32_t full(int s) const { return base + 8u * s; }
  __device__ uint32_t empty(int s) const { return base + 8u * (S + s); }
  __device__ uint32_t tfull(int b) const { return base + 8u * (2 * S + b); }
  __device__ uint32_t tempty(int part, int b) const {
    return base + 8u * (2 * S + 2 + 2 * part + b);
  }
  __device__ uint32_t drain() const { return base + 8u * (2 * S + 6); }
};

template <bool PAIR>
struct Ring {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == Form<PAIR>::STAGES_) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

template <class Op, int P, bool PAIR>
__device__ __forceinline__ bool produce(const Maps& m, const Geom& g,
                                        const Unit& u, uint32_t sa,
                                        uint32_t sb, const Bars<PAIR>& bars,
                                        Ring<PAIR>& ring, uint32_t& issued,
                                        const WaitCtx& ctx) {
  const int n = Op::template blocks<P>(g, u);
  for (int kb = 0; kb < n; ++kb) {
    if (!mbar_wait(bars.empty(ring.stage), ring.phase ^ 1u, ctx, true))
      return false;
    uint32_t fb = bars.full(ring.stage);
    if (!PAIR || g.rank == 0)
      mbar_arrive_expect_tx(fb, Op::template bytes<P>(g, u));
    if (PAIR) fb = mapa_shared(fb, 0);
    Op::template load<P, PAIR>(m, g, u, kb,
                               sa + ring.stage * Form<PAIR>::A_BYTES,
                               sb + ring.stage * Form<PAIR>::B_BYTES, fb);
    ++issued;
    ring.next();
  }
  return true;
}

template <bool A_MN, bool B_MN, int N, bool PAIR>
__device__ __forceinline__ constexpr uint32_t idesc_n() {
  return (1u << 4) | (1u << 7) | (1u << 10) |
         (static_cast<uint32_t>(A_MN) << 15) |
         (static_cast<uint32_t>(B_MN) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>((PAIR ? 2 * BM : BM) >> 4) << 24);
}

template <class Op, int P, class PT, bool PAIR>
__device__ __forceinline__ bool multiply(const Geom& g, const Unit& u, int i,
                                         uint32_t sa, uint32_t sb,
                                         const Bars<PAIR>& bars,
                                         Ring<PAIR>& ring, uint32_t tmem,
                                         const WaitCtx& ctx) {
  constexpr uint32_t IDESC = idesc_n<PT::A_MN, PT::B_MN, PT::N, PAIR>();
  constexpr uint32_t MN_LBO = 64 * BK * 2;
  const int buf = PT::BUFS == 2 ? (i & 1) : 0;
  const uint32_t turn = PT::BUFS == 2 ? (i >> 1) : i;
  if (!mbar_wait(bars.tempty(P, buf), (turn & 1u) ^ 1u, ctx, true))
    return false;
  tc_fence_after();
  const uint32_t d = tmem + PT::COL + buf * PT::N;
  const int n = Op::template blocks<P>(g, u);
  for (int kb = 0; kb < n; ++kb) {
    if (!mbar_wait(bars.full(ring.stage), ring.phase, ctx, true)) return false;
    tc_fence_after();
    const uint32_t a = sa + ring.stage * Form<PAIR>::A_BYTES;
    const uint32_t b = sb + ring.stage * Form<PAIR>::B_BYTES;
#pragma unroll
    for (int k = 0; k < BK / 16; ++k) {
      const uint64_t ad = PT::A_MN ? sdesc_sw128(a + k * 2048, MN_LBO, 1024)
                                   : sdesc_sw128(a + k * 32, 16, 1024);
      const uint64_t bd = PT::B_MN ? sdesc_sw128(b + k * 2048, MN_LBO, 1024)
                                   : sdesc_sw128(b + k * 32, 16, 1024);
      const uint32_t more = (kb > 0 || k > 0) ? 1u : 0u;
      if (PAIR)
        tc_mma_pair(d, ad, bd, IDESC, more);
      else
        tc_mma(d, ad, bd, IDESC, more);
    }
    if (PAIR)
      tc_commit_pair_both(bars.empty(ring.stage));
    else
      tc_commit(bars.empty(ring.stage));
    ring.next();
  }
  return true;
}

template <class Op, class Epi, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1)
    k_experts(const __grid_constant__ Maps maps, Geom g,
              const typename Epi::Params p, unsigned* err) {
  extern __shared__ uint8_t smem_raw[];
  using F = Form<PAIR>;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t sa = base, sb = base + F::STAGES_ * F::A_BYTES;
  const Bars<PAIR> bars{base + F::RING_BYTES};
  uint8_t* misc = smem_raw + (bars.base - raw) + 8 * Bars<PAIR>::COUNT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  g.rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < F::STAGES_; ++s) {
      mbar_init(bars.full(s), 1);
      mbar_init(bars.empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bars.tfull(b), 1);
      // one arrival per epilogue warp
      for (int q = 0; q < 2; ++q) mbar_init(bars.tempty(q, b), EPI_WARPS * (PAIR ? 2 : 1));
    }
    mbar_init(bars.drain(), 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  // both CTAs' barriers exist before either CTA signals the other's
  if (PAIR) cluster_sync_all();
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx ctx{abort_flag, err, g.timeout_ns};
  begin_early();  // all above touches no global memory
  const int units = Op::units(g);
  const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int stride = PAIR ? gridDim.x >> 1 : gridDim.x;

  if (warp == 0) {
    if (lane == 0) {
      Ring<PAIR> ring;
      uint32_t issued = 0;
      bool ok = true;
      for (int u = first; ok && u < units; u += stride) {
        const Unit t = Op::unit(g, u);
        ok = produce<Op, 0, PAIR>(maps, g, t, sa, sb, bars, ring, issued, ctx);
        if (Op::PARTS == 2 && ok)
          ok = produce<Op, Op::PARTS - 1, PAIR>(maps, g, t, sa, sb, bars, ring,
                                                issued, ctx);
      }
      // every copy issued must have landed before the CTA may exit (the
      // leader's full barriers count both CTAs' copies)
      if (!PAIR || g.rank == 0)
        for (int s = 0; s < F::STAGES_; ++s) {
          const uint32_t cnt =
              issued / F::STAGES_ +
              (static_cast<uint32_t>(s) < issued % F::STAGES_ ? 1u : 0u);
          if (cnt) mbar_wait(bars.full(s), (cnt - 1u) & 1u, ctx, false);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && g.rank == 0) {
      Ring<PAIR> ring;
      bool ok = true;
      int i = 0;  // units accumulated so far
      for (int u = first; ok && u < units; u += stride, ++i) {
        const Unit t = Op::unit(g, u);
        ok = multiply<Op, 0, typename Op::P0, PAIR>(g, t, i, sa, sb, bars,
                                                    ring, tmem, ctx);
        if (Op::PARTS == 2 && ok)
          ok = multiply<Op, Op::PARTS - 1, typename Op::P1, PAIR>(
              g, t, i, sa, sb, bars, ring, tmem, ctx);
        if (ok) {
          if (PAIR)
            tc_commit_pair_both(bars.tfull(i & 1));
          else
            tc_commit(bars.tfull(i & 1));
        }
      }
      if (PAIR)
        tc_commit_pair_local(bars.drain());
      else
        tc_commit(bars.drain());
      mbar_wait(bars.drain(), 0, ctx, false);
    }
    __syncwarp();
  } else {
    const int q = warp & 3;  // the lane quarter this warp may access
    const int half = (warp - 2) >> 2;
    const int r = q * 32 + lane;
    Epi epi;
    epi.stage = base + F::RING_BYTES + 1024 +
                static_cast<uint32_t>(warp - 2) * 2u * EPI_BUF_BYTES;
    int i = 0;
    for (int u = first; u < units; u += stride, ++i) {
      const Unit t = Op::unit(g, u);
      const bool got = mbar_wait(bars.tfull(i & 1), (i >> 1) & 1, ctx, true);
      if (!__all_sync(FULL, got)) break;
      tc_fence_after();
      Release<Op::PARTS, PAIR> release{
          bars.tempty(0, Op::P0::BUFS == 2 ? (i & 1) : 0),
          bars.tempty(1, Op::P1::BUFS == 2 ? (i & 1) : 0), false};
      epi.tile(p, maps, g, t, tmem + (static_cast<uint32_t>(q * 32) << 16), r,
               half, i, release);
      release();
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA frees its memory while the pair's MMAs or the peer's barrier
  // traffic may still touch it
  if (PAIR) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, TMEM_COLS);
    else
      tmem_dealloc(tmem, TMEM_COLS);
  }
}

// ---- host side ---------------------------------------------------------------
constexpr CUtensorMapDataType BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr CUtensorMapSwizzle SW128 = CU_TENSOR_MAP_SWIZZLE_128B;

// [rows][cols] bf16, boxes of box_c x box_r.
lce_status map2(CUtensorMap* m, const void* p, int64_t cols, int64_t rows,
                uint32_t box_c, uint32_t box_r,
                CUtensorMapSwizzle swz = SW128) {
  const uint64_t d[2] = {static_cast<uint64_t>(cols),
                         static_cast<uint64_t>(rows)};
  const uint64_t st[1] = {static_cast<uint64_t>(cols) * 2};
  const uint32_t b[2] = {box_c, box_r};
  return make_tmap_nd(m, BF, 2, p, d, st, b, swz);
}
// [E][rows][cols] bf16, boxes inside one expert.
lce_status map3(CUtensorMap* m, const void* p, int64_t cols, int64_t rows,
                int64_t E, uint32_t box_c, uint32_t box_r,
                CUtensorMapSwizzle swz = SW128) {
  const uint64_t d[3] = {static_cast<uint64_t>(cols),
                         static_cast<uint64_t>(rows),
                         static_cast<uint64_t>(E)};
  const uint64_t st[2] = {static_cast<uint64_t>(cols) * 2,
                          static_cast<uint64_t>(cols) * rows * 2};
  const uint32_t b[3] = {box_c, box_r, 1};
  return make_tmap_nd(m, BF, 3, p, d, st, b, swz);
}
lce_status store_map(CUtensorMap* m, const void* p, int64_t cols,
                     int64_t rows) {
  return map2(m, p, cols, rows, EPI_BOX, EPI_BOX, CU_TENSOR_MAP_SWIZZLE_64B);
}

Geom geom(const ExpertsArgs& a, bool pair) {
  Geom g{};
  g.head = a.plan.head;
  g.tile = a.plan.tile;
  g.seg = a.plan.seg;
  g.slot = a.plan.slot;
  g.H = static_cast<int>(a.H);
  g.I = static_cast<int>(a.I);
  g.E = a.E;
  g.kb_h = static_cast<int>(ceil_div(a.H, BK));
  g.kb_i = static_cast<int>(ceil_div(a.I, BK));
  g.tile_m = BM * (pair ? 2 : 1);
  g.timeout_ns = a.timeout_ns;
  return g;
}

template <class Op, class Epi>
lce_status launch(const char* what, const Maps& m, const Geom& g,
                  const typename Epi::Params& p, const ExpertsArgs& a,
                  cudaStream_t s) {
  const bool pair = g.tile_m > BM;
  auto kern = pair ? k_experts<Op, Epi, true> : k_experts<Op, Epi, false>;
  const int smem = pair ? Form<true>::SMEM : Form<false>::SMEM;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = launch_early_cluster(kern, pair ? 2 * a.pair_slots : a.num_sms,
                             THREADS, smem, s, pair ? 2 : 1, m, g, p, a.err);
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, what);
}

}  // namespace

lce_status launch_experts_up(const ExpertsArgs& a, cudaStream_t s) {
  Maps m{};
  LCE_TRY(map2(&m.a0, a.xr, a.H, a.max_rows, BK, 64));
  LCE_TRY(map3(&m.b0, a.Wg, a.H, a.I, a.E, BK, 128));
  LCE_TRY(map3(&m.b1, a.Wu, a.H, a.I, a.E, BK, 128));
  LCE_TRY(store_map(&m.s0, a.a, a.I, a.max_rows));
  Geom g = geom(a, a.pair);
  g.num_n = static_cast<int>(ceil_div(a.I, 128));
  return launch<OpUp, EpiUp>("experts_up", m, g, {0}, a, s);
}

lce_status launch_experts_down(const ExpertsArgs& a, cudaStream_t s) {
  Maps m{};
  LCE_TRY(map2(&m.a0, a.a, a.I, a.max_rows, BK, 64));
  LCE_TRY(map3(&m.b0, a.Wd, a.I, a.H, a.E, BK, a.pair ? 128 : 256));
  Geom g = geom(a, a.pair);
  LCE_TRY(store_map(&m.s0, a.rows_out, a.H, a.max_rows));
  g.num_n = static_cast<int>(ceil_div(a.H, 256));
  return launch<OpDown, EpiRows>("experts_down", m, g, {a.rows_scale}, a, s);
}

lce_status launch_experts_dgu(const ExpertsArgs& a, cudaStream_t s) {
  Maps m{};
  LCE_TRY(map2(&m.a0, a.xr, a.H, a.max_rows, BK, 64));
  LCE_TRY(map2(&m.a1, a.dyr, a.H, a.max_rows, BK, 64));
  LCE_TRY(map3(&m.b0, a.Wg, a.H, a.I, a.E, BK, 128));
  LCE_TRY(map3(&m.b1, a.Wu, a.H, a.I, a.E, BK, 128));
  LCE_TRY(map3(&m.b2, a.Wd, a.I, a.H, a.E, 64, BK));
  LCE_TRY(store_map(&m.s0, a.dg, a.I, a.max_rows));
  LCE_TRY(store_map(&m.s1, a.du, a.I, a.max_rows));
  LCE_TRY(store_map(&m.s2, a.a, a.I, a.max_rows));
  Geom g = geom(a, a.pair);
  g.num_n = static_cast<int>(ceil_div(a.I, 128));
  return launch<OpDgu, EpiDgu>(
      "experts_dgu", m, g, {a.w, a.wdt == LCE_F32, a.part, a.max_rows}, a, s);
}

lce_status launch_experts_dx(const ExpertsArgs& a, cudaStream_t s) {
  Maps m{};
  LCE_TRY(map2(&m.a0, a.dg, a.I, a.max_rows, BK, 64));
  LCE_TRY(map2(&m.a1, a.du, a.I, a.max_rows, BK, 64));
  LCE_TRY(map3(&m.b0, a.Wg, a.H, a.I, a.E, 64, BK));
  LCE_TRY(map3(&m.b1, a.Wu, a.H, a.I, a.E, 64, BK));
  Geom g = geom(a, a.pair);
  LCE_TRY(store_map(&m.s0, a.rows_out, a.H, a.max_rows));
  g.num_n = static_cast<int>(ceil_div(a.H, 256));
  return launch<OpDx, EpiRows>("experts_dx", m, g, {a.rows_scale}, a, s);
}

lce_status launch_experts_grads(const ExpertsArgs& a, cudaStream_t s) {
  // 256-row tiles unless a gradient's rows fit one of 128
  Geom g = geom(a, a.use_pairs && a.H > BM && a.I > BM);
  const int h_m = static_cast<int>(ceil_div(a.H, g.tile_m));
  const int i_m = static_cast<int>(ceil_div(a.I, g.tile_m));
  g.d_n = static_cast<int>(ceil_div(a.I, BN));
  g.gu_n = static_cast<int>(ceil_div(a.H, BN));
  g.d_tiles = a.dWd ? h_m * g.d_n : 0;
  g.gu_tiles = a.dWg ? i_m * g.gu_n : 0;
  Maps m{};
  LCE_TRY(map2(&m.a0, a.dg, a.I, a.max_rows, 64, BK));
  LCE_TRY(map2(&m.a1, a.du, a.I, a.max_rows, 64, BK));
  LCE_TRY(map2(&m.b0, a.dyr, a.H, a.max_rows, 64, BK));
  LCE_TRY(map2(&m.b1, a.a, a.I, a.max_rows, 64, BK));
  LCE_TRY(map2(&m.b2, a.xr, a.H, a.max_rows, 64, BK));
  EpiWeights::Params p{};
  if (a.gdt == LCE_F32) {
    p.out[0] = static_cast<float*>(a.dWd);
    p.out[1] = static_cast<float*>(a.dWg);
    p.out[2] = static_cast<float*>(a.dWu);
  } else {
    constexpr CUtensorMapSwizzle SW64 = CU_TENSOR_MAP_SWIZZLE_64B;
    if (a.dWd) LCE_TRY(map3(&m.s0, a.dWd, a.I, a.H, a.E, 32, 32, SW64));
    if (a.dWg) LCE_TRY(map3(&m.s1, a.dWg, a.H, a.I, a.E, 32, 32, SW64));
    if (a.dWg) LCE_TRY(map3(&m.s2, a.dWu, a.H, a.I, a.E, 32, 32, SW64));
  }
  return launch<OpGrad, EpiWeights>("experts_grads", m, g, p, a, s);
}

}  // namespace lce
