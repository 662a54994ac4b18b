// kv4_launch_impl.cuh -- definition of launch_kv4, included by the translation
// units that instantiate it (kv4_bf16.cu, kv4_fp16.cu).
#pragma once
#include "kv4_kernel.cuh"

namespace fi {

template <typename T, int kB>
cudaError_t launch_kv4_block(const Kv4Params& kp, int num_ctas, cudaStream_t stream) {
  static bool configured[kMaxDevices] = {};
  auto kern = kv4_attention_kernel<T, kB>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !configured[dev]) {
    // warpgroups exchange registers (see launch_run)
    cudaFuncAttributes fa{};
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < kKv4RegsLaunch) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kKv4SmemBytes));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) configured[dev] = true;
  }
  kern<<<num_ctas, kKv4Threads, kKv4SmemBytes, stream>>>(kp);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_kv4(const Kv4Params& kp, int num_ctas, cudaStream_t stream) {
  return kp.block_slots == 32   ? launch_kv4_block<T, 32>(kp, num_ctas, stream)
         : kp.block_slots == 16 ? launch_kv4_block<T, 16>(kp, num_ctas, stream)
                                : launch_kv4_block<T, 0>(kp, num_ctas, stream);
}

}  // namespace fi
