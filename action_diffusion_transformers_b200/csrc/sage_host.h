// sage_host.h - host-side helpers shared by the C-ABI implementation files
// (sage_api.cu: quantized attention and projections; serve_api.cu: rotary
// positions, the quantized KV cache and the attention that reads it): status
// codes with a thread-local message, the per-device setup, launches.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sage.h"

namespace sage_host {

constexpr int kMaxDevices = 64;

// Records a printf-style message for sage_last_error() and returns `st`.
sage_status fail(sage_status st, const char* fmt, ...);
sage_status cuda_fail(cudaError_t e, const char* what);
// Reads (and clears) this thread's last CUDA error after a call's launches.
sage_status launch_check(const char* what);

// The device's two error words: [0] a kernel gave up a bounded wait, [1] a
// kernel met an index outside its cache and skipped it.  Both are reported and
// cleared by sage_check().
sage_status device_setup(int* dev_out, int** err_out, int* sm_count_out = nullptr);

int64_t wait_timeout_ns();

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled, valid after a device_setup() that returned SAGE_OK.
EncodeTiledFn encode_tiled();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Launches with programmatic stream serialization allowed: the kernel may be
// scheduled while the previous kernel in the stream is still running; every
// kernel of this library begins with pdl_enter(), which waits for that kernel
// to complete (and its writes to be visible) before anything is read.
// kEarly = false: an ordinary launch (after the previous kernel has finished),
// used for the attention kernel: with its blocks scheduled early beside the
// last quantization pass it measured 0.35% slower on one B200 and the same on
// another, for a gain of a few microseconds per step at most.
template <bool kEarly = true, typename... KArgs, typename... Args>
void pdl_launch_clusters(void (*kernel)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (kEarly) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = static_cast<unsigned>(n);
  // A failed launch is also recorded as this thread's last CUDA error, which
  // launch_check() reads after the call's launches.
  (void)cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

template <bool kEarly = true, typename... KArgs, typename... Args>
void pdl_launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args) {
  pdl_launch_clusters<kEarly>(kernel, 1, grid, block, smem, stream, args...);
}

}  // namespace sage_host

#define SAGE_NEED(p, name)                                                              \
  do {                                                                                  \
    if (!(p)) return sage_host::fail(SAGE_ERR_INVALID_ARG, "%s is NULL", name);         \
    if (!sage_host::aligned16(p))                                                       \
      return sage_host::fail(SAGE_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);    \
  } while (0)
