// swin_calls.cuh -- what the entry points without a plan share on the host.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/swin_attn.h"

namespace swin {

// SMs of the current device (asked once per device: the calls are short).
inline int sm_count(int *sms) {
  static std::atomic<int> known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return SWIN_ERR_CUDA;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return SWIN_OK;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SWIN_ERR_CUDA;
  if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return SWIN_OK;
}

inline bool mis(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// A launch that may start while the kernel before it in the stream still runs;
// the kernel waits (griddepcontrol.wait) before it reads what that one wrote.
template <typename... P>
int launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                     const std::common_type_t<P> &...args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  void *ptrs[] = {const_cast<void *>(static_cast<const void *>(&args))...};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(kernel), ptrs) == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

}  // namespace swin
