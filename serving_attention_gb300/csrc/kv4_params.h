// kv4_params.h -- parameters of the attention kernel over the 4-bit cache, and
// its launch (one instantiation per element type, in translation units of
// their own).
#pragma once
#include "attention.cuh"
#include "launch.h"

namespace fi {

struct Kv4Params {
  RunParams run;
  const uint8_t* cache;
  int64_t page_stride, head_stride;  // bytes
  int32_t block_slots, log2_block, block_bytes;
};

template <typename T>
cudaError_t launch_kv4(const Kv4Params& kp, int num_ctas, cudaStream_t stream);

}  // namespace fi
