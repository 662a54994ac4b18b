// diff_bf16.cu -- bf16 kernels of differential attention.
#include "diff_launch_impl.cuh"

namespace fi {

template cudaError_t launch_diff<__nv_bfloat16, false>(const DiffParams&, int, cudaStream_t);
template cudaError_t launch_diff<__nv_bfloat16, true>(const DiffParams&, int, cudaStream_t);

}  // namespace fi
