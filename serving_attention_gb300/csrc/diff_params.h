// diff_params.h -- parameters of the differential attention kernels.
#pragma once
#include "attention.cuh"

namespace fi {

struct DiffParams {
  RunParams run;
  const float* lambda;  // [num_qo_heads]
  const float* norm_w;  // [128] or null: no norm
  float norm_eps, out_scale;
  const uint16_t* k;    // the cache, for pages that are copied row by row
  const uint16_t* v;
  int64_t k_strides[3], v_strides[3];  // page, slot, head (elements)
};

}  // namespace fi
