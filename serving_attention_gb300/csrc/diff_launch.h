// diff_launch.h -- launch of differential attention, one instantiation per
// element type and window / sink mask, in translation units of their own.
#pragma once
#include "diff_params.h"
#include "launch.h"

namespace fi {

// The run on the plan's grid, then the merge of split units behind it.
template <typename T, bool kMask>
cudaError_t launch_diff(const DiffParams& dp, int num_ctas, cudaStream_t stream);

}  // namespace fi
