// kv4_bf16.cu -- bf16 kernels of attention over the 4-bit cache.
#include "kv4_launch_impl.cuh"

namespace fi {

template cudaError_t launch_kv4<__nv_bfloat16>(const Kv4Params&, int, cudaStream_t);

}  // namespace fi
