// gg_launch.cuh — launch helpers that the translation units share (host side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "gg_internal.h"

namespace gg {

// Launch with programmatic stream serialisation: the kernel may start while
// the one ahead of it in the stream runs, and must call grid_dependency_wait()
// before it touches anything that kernel writes or reads.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// TMA map of a row-major tensor (dims and box innermost first, up to three
// dimensions, rows `strides` bytes apart); false when the driver refuses it.
inline bool encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int rank,
                       const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                       CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (fn == nullptr) return false;
  const cuuint32_t elem_strides[3] = {1, 1, 1};
  return fn(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box,
            elem_strides, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch of a persistent kernel in clusters of two CTAs, one CTA per SM: as
// many clusters as can be resident at once (at most `most`), found once per
// device and kernel (`resident`: kMaxDevices entries of the kernel's own,
// zero before the first call; host threads may race, every writer stores the
// same value).
template <typename... Params, typename... Args>
cudaError_t launch_pairs(void (*kernel)(Params...), std::atomic<int>* resident, int threads,
                         size_t smem, int most, const DeviceInfo& dev, cudaStream_t stream,
                         Args... args) {
  if (dev.device < 0 || dev.device >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = resident[dev.device].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count / 2 * 2));
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (n > dev.sm_count / 2) n = dev.sm_count / 2;
    if (n <= 0) return cudaErrorInvalidConfiguration;
    resident[dev.device].store(n, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (n < most ? n : most)));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace gg
