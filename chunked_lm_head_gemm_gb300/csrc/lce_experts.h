// Internal declarations of the experts' gated MLP: the plan that groups the
// slots (token, choice) by expert, and the launch wrappers of its kernels.
//
// Rows: the slots of an expert, in slot order, form one segment of rows;
// segments start at multiples of SEG_ROWS and are padded to one with rows
// that hold no slot.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/lce.h"

namespace lce {

// Programmatic dependent launch (launch_early): every kernel of a call but its
// first begins early, waits here before its first access to global memory,
// and lets the next one begin. What the kernels before it wrote is read by
// plain loads, never by the read-only path, whose loads the compiler may move
// up past the wait.
__device__ __forceinline__ void begin_early() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

constexpr int SEG_ROWS = 64;     // one K block of the weight gradients
constexpr int MAX_EXPERTS = 1024;
constexpr int PLAN_CHUNK = 2048; // slots of one counting block
constexpr int PLAN_SMALL = 4096; // up to here one block makes the plan

struct PlanHead {
  int tiles;  // row tiles of at most tile_m rows (launch_plan)
  int rows;   // padded rows
};

// What a row tile (of at most tile_m rows) knows of its expert: the first of
// the expert's tiles, and its segment's first row and padded rows.
struct RowTile {
  int expert, first, row0, rows;
};

// The plan, in device memory.
struct Plan {
  PlanHead* head;
  RowTile* tile;  // [max_tiles]
  int2* seg;      // [E]: first row, padded rows
  int* slot;      // [max_rows]: slot of a row, -1 for a padding row
  int* row;       // [n]: row of a slot, -1 where it is dropped
  int* hist;      // [E][chunks]: slots of an expert in a chunk, then before it
};

// Queues the plan of the slots experts[n], in row tiles of tile_m. Deterministic:
// integer counts and positions that follow slot order.
cudaError_t launch_plan(const int32_t* experts, int64_t n, int E, int tile_m,
                        const Plan& p, unsigned* err, cudaStream_t s);

// out[row of (t, k)][:] = x[t][:] for every slot of the plan, bf16 of H
// columns; with y also out_y from y. With `zero` the padding rows become 0:
// the weight gradients sum over them; elsewhere what they hold reaches no
// result.
cudaError_t launch_gather(const Plan& p, int64_t L, int K, int E, int64_t H,
                          const void* x, uint16_t* out, const void* y,
                          uint16_t* out_y, bool zero, cudaStream_t s);

// out[t][:] = sum_k w[t][k] rows[row(t, k)][:] in bf16, k in order, dropped
// slots left out. rows: fp16 times the scale of each row and 128 columns.
cudaError_t launch_combine(const uint16_t* rows, const float* scale,
                           const int* row, const void* w, lce_dtype wdt,
                           int64_t L, int K, int64_t H, void* out,
                           cudaStream_t s);
// The backward's sums, in one launch: dx likewise with weights 1 (NULL: none),
// and dweights[slot] = sum over the column pieces of part[piece][row], in order
// (NULL: none).
cudaError_t launch_backward_sums(const uint16_t* rows, const float* scale,
                                 const int* row, int64_t L, int K, int64_t H,
                                 void* dx, const float* part, int64_t stride,
                                 int pieces, lce_dtype wdt, void* dweights,
                                 cudaStream_t s);

// The forward of few slots without a plan (a: fp32 [L K][I] scratch).
cudaError_t launch_token(const void* x, const void* Wg, const void* Wu,
                         const void* Wd, const void* weights, lce_dtype wdt,
                         const int32_t* experts, int64_t L, int K, int64_t H,
                         int64_t I, int E, float* a, void* y, unsigned* err,
                         cudaStream_t s);

// ---- grouped contractions ----------------------------------------------------
struct ExpertsArgs {
  Plan plan;
  int64_t H, I;
  int E;
  uint64_t timeout_ns;
  unsigned* err;
  int num_sms, pair_slots;
  bool use_pairs;          // CTA pairs may be used (lce_set_cta_pair)
  bool pair;               // row tiles of 256, contracted on CTA pairs
  // operand maps by use; each kernel takes the ones it names
  const void *Wg, *Wu, *Wd;
  uint16_t *xr, *dyr;      // [max_rows][H]: token rows in plan order
  uint16_t *a, *dg, *du;   // [max_rows][I]
  int64_t max_rows;
  uint16_t* rows_out;      // [max_rows][H] fp16 (DOWN, DX) ...
  float* rows_scale;       // ... times [max_rows][2 ceil(H / 256)]
  const void* w;           // routing weights of the slots
  lce_dtype wdt;
  float* part;             // [2 ceil(I / 128)][max_rows] of da' . a
  void *dWg, *dWu, *dWd;   // weight gradients, or NULL
  lce_dtype gdt;
};

lce_status launch_experts_up(const ExpertsArgs& a, cudaStream_t s);
lce_status launch_experts_down(const ExpertsArgs& a, cudaStream_t s);
lce_status launch_experts_dgu(const ExpertsArgs& a, cudaStream_t s);
lce_status launch_experts_dx(const ExpertsArgs& a, cudaStream_t s);
lce_status launch_experts_grads(const ExpertsArgs& a, cudaStream_t s);

}  // namespace lce
