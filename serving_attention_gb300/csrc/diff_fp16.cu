// diff_fp16.cu -- fp16 kernels of differential attention.
#include "diff_launch_impl.cuh"

namespace fi {

template cudaError_t launch_diff<__half, false>(const DiffParams&, int, cudaStream_t);
template cudaError_t launch_diff<__half, true>(const DiffParams&, int, cudaStream_t);

}  // namespace fi
