// kv4_fp16.cu -- fp16 kernels of attention over the 4-bit cache.
#include "kv4_launch_impl.cuh"

namespace fi {

template cudaError_t launch_kv4<__half>(const Kv4Params&, int, cudaStream_t);

}  // namespace fi
