// Arguments of the head norm + rotation kernels and their backward.
#pragma once

#include "common.h"

namespace gnf4 {

struct RopeArgs {
  const uint16_t *q, *k;                       // bf16 [T][H][D], token strides in elements
  int64_t q_stride, k_stride;
  const uint16_t *dq, *dk;                     // backward: gradients of the results
  int64_t dq_stride, dk_stride;
  uint16_t *q_out, *k_out;                     // results, or gradients of q and k
  int64_t q_out_stride, k_out_stride;
  int32_t T, Hq, Hk, D;
  const uint16_t *wq, *wk;                     // bf16 [D] or NULL
  float eps;
  int32_t rot, interleaved;
  const float *inv_freq;
  float mscale;
  const int32_t *positions;
  float *part;                                 // backward: [blocks][2][D] parts of the weight gradients
  float *dwq, *dwk;
};

int32_t rope_dx_blocks(int32_t T);
hipError_t launch_norm_rope(const RopeArgs &a, hipStream_t s);
hipError_t launch_norm_rope_dx(const RopeArgs &a, hipStream_t s);

}  // namespace gnf4
