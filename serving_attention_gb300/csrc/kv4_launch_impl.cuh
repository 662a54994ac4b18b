// kv4_launch_impl.cuh -- definition of launch_kv4, included by the translation
// units that instantiate it (kv4_bf16.cu, kv4_fp16.cu).
#pragma once
#include "kv4_kernel.cuh"

namespace fi {

template <typename T>
cudaError_t launch_kv4(const Kv4Params& kp, int num_ctas, cudaStream_t stream) {
  static bool configured[kMaxDevices] = {};
  auto kern = kv4_attention_kernel<T>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !configured[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kKv4SmemBytes));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) configured[dev] = true;
  }
  kern<<<num_ctas, kKv4Threads, kKv4SmemBytes, stream>>>(kp);
  return cudaGetLastError();
}

}  // namespace fi
