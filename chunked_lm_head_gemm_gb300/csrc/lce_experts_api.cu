// Host layer of the experts' gated MLP (lce_experts_forward /
// lce_experts_backward): argument checks, workspace carving and the launch
// sequence.
#include <algorithm>
#include <cmath>

#include "lce_experts.h"
#include "lce_host.h"

namespace lce {
namespace {

struct Sizes {
  int64_t L, H, I, E, K;
};

// Whether the forward takes its slots one by one on the CUDA cores
// (launch_token), each reading its expert's weights, instead of planning tiles
// for the tensor cores, which read the weights of every expert hit once but
// cost about 18 us of small launches. That is what some 100 MB take to read,
// so the border is where as much is read again: slots - (experts hit)
// experts' weights, with the slots falling evenly. At H = 2048, I = 768, E =
// 128 the two take 60 and 70 us for 32 slots (302 MB slot by slot), 112 and 92
// us for 64 (604 MB); at H = 2048, I = 4096, E = 8 they take 47 and 59 us for
// 4 slots (201 MB), 80 and 77 us for 8 (403 MB). (At most 64 slots: their fp32
// activations fit the bf16 rows of a planned call.)
bool takes_tokens(const Sizes& z) {
  const double n = static_cast<double>(z.L) * z.K;
  if (n > 64) return false;
  const double hit = z.E * (1.0 - std::pow(1.0 - 1.0 / z.E, n));
  return (n - hit) * 6.0 * z.H * z.I <= 100e6;
}

// Rows an expert has on average from which the row tiles are 256 rows on CTA
// pairs: they halve the weights that L2 hands out, but pad more. At 2048 rows
// (H = 4096, I = 8192) UP takes 1608 us on single CTAs and 1402 us on pairs, at
// 768 (H = 1024, I = 512) the forward's and backward's row contractions 395
// and 388 us, at 256 (H = 2048, I = 768) UP and DOWN 317 and 322 us.
constexpr int64_t PAIR_ROWS = 512;

bool sizes_ok(const Sizes& z) {
  if (z.L < 0 || z.E < 1 || z.E > MAX_EXPERTS || z.K < 1 || z.K > 32)
    return false;
  if (z.H < 8 || z.I < 8 || z.H % 8 || z.I % 8 || z.H > (1 << 20) ||
      z.I > (1 << 20))
    return false;
  // rows and slots are 32-bit indices
  return z.L <= (1ll << 30) && z.L * z.K <= (1ll << 30);
}

int64_t max_rows(const Sizes& z) {
  const int64_t n = z.L * z.K;
  return round_up(n + (SEG_ROWS - 1) * std::min(z.E, n), SEG_ROWS);
}
int64_t max_tiles(const Sizes& z) {
  const int64_t n = z.L * z.K;
  return n / BM + std::min(z.E, n);
}

struct Layout {
  size_t head, tile, seg, slot, row, hist;
  size_t xr, dyr, a, dg, du, rows, scale, part, total;
};

Layout layout(const Sizes& z, bool backward) {
  Layout w{};
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t o = off;
    off = static_cast<size_t>(round_up(static_cast<int64_t>(off) + bytes, 256));
    return o;
  };
  const int64_t n = z.L * z.K, P = max_rows(z);
  w.head = take(sizeof(PlanHead));
  w.tile = take(max_tiles(z) * static_cast<int64_t>(sizeof(RowTile)));
  w.seg = take(z.E * 8);
  w.slot = take(P * 4);
  w.row = take(n * 4);
  w.hist = take(z.E * ceil_div(n, PLAN_CHUNK) * 4);
  w.xr = take(P * z.H * 2);
  w.a = take(P * z.I * 2);
  if (backward) {
    w.dyr = take(P * z.H * 2);
    w.dg = take(P * z.I * 2);
    w.du = take(P * z.I * 2);
    w.part = take(P * 2 * ceil_div(z.I, 128) * 4);
  }
  w.rows = take(P * z.H * 2);
  w.scale = take(P * 2 * ceil_div(z.H, 256) * 4);
  w.total = off;
  return w;
}

lce_status check(const Sizes& z, const void* x, const void* Wg, const void* Wu,
                 const void* Wd, const void* weights, lce_dtype wdt,
                 const int32_t* experts, const void* ws) {
  if (!sizes_ok(z)) return LCE_ERR_INVALID_ARG;
  if (wdt != LCE_BF16 && wdt != LCE_F32) return LCE_ERR_UNSUPPORTED;
  if (!Wg || !Wu || !Wd || !ws || !aligned_to(Wg, 16) || !aligned_to(Wu, 16) ||
      !aligned_to(Wd, 16) || !aligned_to(ws, 256))
    return LCE_ERR_INVALID_ARG;
  if (z.L == 0) return LCE_OK;
  if (!x || !weights || !experts || !aligned_to(x, 16) ||
      !aligned_to(experts, 4) || !aligned_to(weights, wdt == LCE_F32 ? 4 : 2))
    return LCE_ERR_INVALID_ARG;
  return LCE_OK;
}

ExpertsArgs arguments(const Sizes& z, const Layout& w, uint8_t* ws,
                      const DeviceInfo& dev) {
  ExpertsArgs a{};
  a.plan.head = reinterpret_cast<PlanHead*>(ws + w.head);
  a.plan.tile = reinterpret_cast<RowTile*>(ws + w.tile);
  a.plan.seg = reinterpret_cast<int2*>(ws + w.seg);
  a.plan.slot = reinterpret_cast<int*>(ws + w.slot);
  a.plan.row = reinterpret_cast<int*>(ws + w.row);
  a.plan.hist = reinterpret_cast<int*>(ws + w.hist);
  a.H = z.H;
  a.I = z.I;
  a.E = static_cast<int>(z.E);
  a.timeout_ns = wait_timeout_ns();
  a.err = dev.err;
  a.num_sms = dev.num_sms;
  a.pair_slots = dev.pair_slots;
  a.use_pairs = lce_get_cta_pair() != 0 && dev.pair_slots > 0;
  a.pair = a.use_pairs && z.L * z.K >= PAIR_ROWS * z.E;
  a.xr = reinterpret_cast<uint16_t*>(ws + w.xr);
  a.dyr = reinterpret_cast<uint16_t*>(ws + w.dyr);
  a.a = reinterpret_cast<uint16_t*>(ws + w.a);
  a.dg = reinterpret_cast<uint16_t*>(ws + w.dg);
  a.du = reinterpret_cast<uint16_t*>(ws + w.du);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.rows_out = reinterpret_cast<uint16_t*>(ws + w.rows);
  a.rows_scale = reinterpret_cast<float*>(ws + w.scale);
  a.max_rows = max_rows(z);
  return a;
}

lce_status cuda_try(cudaError_t e, const char* where) {
  return e == cudaSuccess ? LCE_OK : cuda_fail(e, where);
}

template <class F>
lce_status timed(int kind, double flops, cudaStream_t s, F&& f) {
  ProfScope ps(kind, s);
  const lce_status st = f();
  ps.done(flops);
  return st;
}

// The plan, and the token rows of x (and dy) in its order.
lce_status make_plan(const Sizes& z, const int32_t* experts, const void* x,
                     const void* dy, const ExpertsArgs& a, cudaStream_t s) {
  LCE_TRY(timed(LCE_K_EXPERTS_PLAN, 0, s, [&] {
    return cuda_try(launch_plan(experts, z.L * z.K, a.E, a.pair ? 2 * BM : BM,
                                a.plan, a.err, s),
                    "experts_plan");
  }));
  return timed(LCE_K_EXPERTS_GATHER, 0, s, [&] {
    return cuda_try(launch_gather(a.plan, z.L, static_cast<int>(z.K), a.E, z.H,
                                  x, a.xr, dy, a.dyr, dy != nullptr, s),
                    "experts_gather");
  });
}

}  // namespace
}  // namespace lce

using namespace lce;

extern "C" {

size_t lce_experts_workspace_size(int64_t L, int64_t H, int64_t I, int64_t E,
                                  int64_t top_k, int backward) {
  const Sizes z{L, H, I, E, top_k};
  if (!sizes_ok(z) || (backward != 0 && backward != 1)) return 0;
  return layout(z, backward != 0).total;
}

lce_status lce_experts_forward(const void* x, const void* Wg, const void* Wu,
                               const void* Wd, const void* weights,
                               lce_dtype weights_dt, const int32_t* experts,
                               int64_t L, int64_t H, int64_t I, int64_t E,
                               int64_t top_k, void* y, void* ws,
                               size_t ws_bytes, void* stream) {
  const Sizes z{L, H, I, E, top_k};
  LCE_TRY(check(z, x, Wg, Wu, Wd, weights, weights_dt, experts, ws));
  if (L > 0 && (!y || !aligned_to(y, 16))) return LCE_ERR_INVALID_ARG;
  const Layout w = layout(z, false);
  if (ws_bytes < w.total) return LCE_ERR_WORKSPACE;
  if (L == 0) return LCE_OK;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ExpertsArgs a = arguments(z, w, static_cast<uint8_t*>(ws), *dev);
  a.Wg = Wg;
  a.Wu = Wu;
  a.Wd = Wd;
  const double slot_flops = 2.0 * L * top_k * H * I;
  if (takes_tokens(z))
    return timed(LCE_K_EXPERTS_TOKEN, 3 * slot_flops, s, [&] {
      return cuda_try(
          launch_token(x, Wg, Wu, Wd, weights, weights_dt, experts, L,
                       static_cast<int>(top_k), H, I, a.E,
                       reinterpret_cast<float*>(a.a), y, a.err, s),
          "experts_token");
    });
  LCE_TRY(make_plan(z, experts, x, nullptr, a, s));
  LCE_TRY(timed(LCE_K_EXPERTS_UP, 2 * slot_flops, s,
                [&] { return launch_experts_up(a, s); }));
  LCE_TRY(timed(LCE_K_EXPERTS_DOWN, slot_flops, s,
                [&] { return launch_experts_down(a, s); }));
  return timed(LCE_K_EXPERTS_COMBINE, 0, s, [&] {
    return cuda_try(launch_combine(a.rows_out, a.rows_scale, a.plan.row,
                                   weights, weights_dt, L,
                                   static_cast<int>(top_k), H, y, s),
                    "experts_combine");
  });
}

lce_status lce_experts_backward(const void* x, const void* Wg, const void* Wu,
                                const void* Wd, const void* weights,
                                lce_dtype weights_dt, const int32_t* experts,
                                const void* dy, int64_t L, int64_t H,
                                int64_t I, int64_t E, int64_t top_k,
                                lce_dtype grad_dt, void* dx, void* dWg,
                                void* dWu, void* dWd, void* dweights, void* ws,
                                size_t ws_bytes, void* stream) {
  const Sizes z{L, H, I, E, top_k};
  LCE_TRY(check(z, x, Wg, Wu, Wd, weights, weights_dt, experts, ws));
  if (grad_dt != LCE_BF16 && grad_dt != LCE_F32) return LCE_ERR_UNSUPPORTED;
  if (!dWg != !dWu || (!dx && !dWg && !dWd && !dweights) ||
      !aligned_to(dx, 16) || !aligned_to(dWg, 16) || !aligned_to(dWu, 16) ||
      !aligned_to(dWd, 16) ||
      !aligned_to(dweights, weights_dt == LCE_F32 ? 4 : 2))
    return LCE_ERR_INVALID_ARG;
  if (L > 0 && (!dy || !aligned_to(dy, 16))) return LCE_ERR_INVALID_ARG;
  const Layout w = layout(z, true);
  if (ws_bytes < w.total) return LCE_ERR_WORKSPACE;
  DeviceInfo* dev = nullptr;
  LCE_TRY(device_info(&dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (L == 0) {  // no token reaches an expert: the weights' gradients are 0
    const size_t bytes =
        static_cast<size_t>(E) * H * I * (grad_dt == LCE_F32 ? 4 : 2);
    for (void* p : {dWg, dWu, dWd})
      if (p) LCE_TRY(cuda_try(cudaMemsetAsync(p, 0, bytes, s), "zero"));
    return LCE_OK;
  }
  ExpertsArgs a = arguments(z, w, static_cast<uint8_t*>(ws), *dev);
  a.Wg = Wg;
  a.Wu = Wu;
  a.Wd = Wd;
  a.w = weights;
  a.wdt = weights_dt;
  a.gdt = grad_dt;
  const double slot_flops = 2.0 * L * top_k * H * I;
  const int K = static_cast<int>(top_k);
  LCE_TRY(make_plan(z, experts, x, dy, a, s));
  LCE_TRY(timed(LCE_K_EXPERTS_DGU, 3 * slot_flops, s,
                [&] { return launch_experts_dgu(a, s); }));
  if (dx)
    LCE_TRY(timed(LCE_K_EXPERTS_DX, 2 * slot_flops, s,
                  [&] { return launch_experts_dx(a, s); }));
  if (dx || dweights)
    LCE_TRY(timed(LCE_K_EXPERTS_COMBINE, 0, s, [&] {
      return cuda_try(
          launch_backward_sums(a.rows_out, a.rows_scale, a.plan.row, L, K, H,
                               dx, a.part, a.max_rows,
                               2 * static_cast<int>(ceil_div(I, 128)),
                               weights_dt, dweights, s),
          "experts_combine");
    }));
  if (dWd || dWg) {
    a.dWg = dWg;
    a.dWu = dWu;
    a.dWd = dWd;
    const double flops = (dWd ? 1.0 : 0.0) + (dWg ? 2.0 : 0.0);
    LCE_TRY(timed(LCE_K_EXPERTS_GRADS, flops * slot_flops, s,
                  [&] { return launch_experts_grads(a, s); }));
  }
  return LCE_OK;
}

}  // extern "C"
