// diff_launch_impl.cuh -- definition of launch_diff, included by the
// translation units that instantiate it (diff_bf16.cu, diff_fp16.cu).
#pragma once
#include "diff_kernel.cuh"
#include "diff_launch.h"

namespace fi {

template <typename T, bool kMask>
cudaError_t launch_diff(const DiffParams& dp, int num_ctas, cudaStream_t stream) {
  static bool configured[kMaxDevices] = {};
  auto kern = diff_attention_kernel<T, kMask>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !configured[dev]) {
    // both phases move registers between warpgroups (see launch_run)
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kDiffRegsLaunch) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kDiffSmemBytes));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) configured[dev] = true;
  }
  kern<<<num_ctas, kDiffThreads, kDiffSmemBytes, stream>>>(dp);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_behind_run(diff_merge_kernel<T>, 2 * num_ctas, 256, stream, dp) : e;
}

}  // namespace fi
