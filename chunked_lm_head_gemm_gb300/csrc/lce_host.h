// Host-side helpers shared by the translation units that implement the C
// ABI: device lookup, the thread's last CUDA error text, tensor maps, and
// per-kernel timing. Defined in lce_api.cu. Not part of the C ABI.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/lce.h"
#include "lce_internal.h"

// Returns a status that is not LCE_OK to the caller.
#define LCE_TRY(call)              \
  do {                             \
    const lce_status st_ = (call); \
    if (st_ != LCE_OK) return st_; \
  } while (0)

namespace lce {

struct DeviceInfo {
  bool ready = false;
  bool supported = false;
  int num_sms = 0;
  int pair_slots = 0;       // co-resident CTA pairs of the pair kernels
  unsigned* err = nullptr;  // device address of the error word
};

// The current device (LCE_ERR_UNSUPPORTED unless it is sm_103).
lce_status device_info(DeviceInfo** out);

// Keeps the error's text for lce_last_cuda_error; returns LCE_ERR_CUDA.
lce_status cuda_fail(cudaError_t e, const char* where);

// Limit of one bounded wait inside a kernel.
uint64_t wait_timeout_ns();

// Tensor map of rank 2 or 3 over a row-major array of 2- or 4-byte elements:
// dims and box innermost first, strides in bytes of dimensions 1 and 2.
// Out-of-range elements of a box read as zero and are not written.
lce_status make_tmap_nd(CUtensorMap* tm, CUtensorMapDataType type, int rank,
                        const void* base, const uint64_t* dims,
                        const uint64_t* strides, const uint32_t* box,
                        CUtensorMapSwizzle swz);

// Brackets one launch with two events while lce_profile_start is on:
// construct before the launch, call done(flops) after it.
struct ProfScope {
  int kind;
  cudaStream_t s;
  cudaEvent_t e0 = nullptr;
  ProfScope(int k, cudaStream_t st);
  void done(double flops);
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Launches a kernel that may begin while the kernel before it on the stream
// still runs (programmatic dependent launch): it has to execute
// griddepcontrol.wait before it touches what earlier kernels read or write.
template <class... P, class... A>
cudaError_t launch_early_cluster(void (*kern)(P...), dim3 grid, dim3 block,
                                 size_t smem, cudaStream_t s, unsigned cluster,
                                 A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}
template <class... P, class... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, dim3 block,
                         size_t smem, cudaStream_t s, A... args) {
  return launch_early_cluster(kern, grid, block, smem, s, 1u, args...);
}

}  // namespace lce
