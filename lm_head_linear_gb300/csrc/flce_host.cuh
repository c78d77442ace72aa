// Host-side pieces every translation unit of the library shares: error text,
// argument helpers, the launch bracket of the timing aid, the limit of the
// kernels' bounded waits and the TMA tensor-map encoder.  Defined in
// flce_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <nvtx3/nvToolsExt.h>

#include <cstddef>
#include <cstdint>

#include "flce.h"

namespace flce {
namespace host {

// Records the text flce_last_error() returns on this host thread; returns `st`.
flce_status fail(flce_status st, const char* fmt, ...);

#define CUDA_TRY(expr)                                                                            \
  do {                                                                                            \
    cudaError_t e_ = (expr);                                                                      \
    if (e_ != cudaSuccess) return fail(FLCE_ERR_CUDA, "%s: %s", #expr, cudaGetErrorString(e_));  \
  } while (0)

constexpr size_t kHeaderBytes = 256;  // status word and spare scalars at the start of each workspace
// T and V bound: tile coordinates (block * 128 + row) stay inside int32 with room to spare.
constexpr int64_t kMaxRows = int64_t(1) << 30;

// Limit of the bounded waits of one GEMM launch whose longest tile has a K loop of `k_max`.
uint64_t wait_limit_ns(int64_t k_max);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The kernels read and write the per-token arrays with plain typed loads and
// stores, so each pointer must carry its type's natural alignment (checked on the
// host: a misaligned access would fault the device instead of returning an error).
template <typename E>
bool misaligned(const E* p) {
  return (reinterpret_cast<uintptr_t>(p) % alignof(E)) != 0;
}

// The current device's SM count and its `slot` (ordinal, < 64), after checking
// that the library's kernels run on it.
flce_status current_device(int* slot, int* sms);

// cuTensorMapEncodeTiled, once get_encoder() has returned FLCE_OK.
extern PFN_cuTensorMapEncodeTiled_v12000 g_encode;
flce_status get_encoder();

// ------------------------------------------------------------------ profiling
struct LaunchRecord {
  int kind;
  cudaEvent_t start, stop;
  double flops, bytes;
  // Launches over the backward's row list add rows * (flops, bytes) per row, the
  // rows read from the workspace when the records are collected.
  const int32_t* rows_dev;
  int64_t index0, cap;
  double flops_per_row, bytes_per_row;
};

// Brackets one launch with an NVTX range named after the kernel (seen by any
// attached profiler) and, while profiling is enabled, with events on its stream.
struct KernelScope {
  bool on = false;
  bool nvtx = true;
  LaunchRecord rec{};
  cudaStream_t stream;
  KernelScope(int kind, cudaStream_t s, double flops, double bytes, const int32_t* rows_dev = nullptr,
              int64_t index0 = 0, int64_t cap = 0, double flops_per_row = 0.0, double bytes_per_row = 0.0);
  ~KernelScope();
  void done();

 private:
  void release_events();  // caller holds the records' mutex
};

flce_status check_launch(const char* what);

// Launches a kernel that may be dispatched, and set itself up, while the kernel before it
// on the stream is still finishing.  Every thread of it waits (griddepcontrol.wait)
// before it touches global memory; policy_main_kernel alone reads inputs earlier, which
// an ordinary launch before it (policy_count_kernel) has made complete.
template <typename... Params, typename... Args>
flce_status launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              const Args&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at, cfg.numAttrs = 1;
  CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
  return FLCE_OK;
}

}  // namespace host
}  // namespace flce
