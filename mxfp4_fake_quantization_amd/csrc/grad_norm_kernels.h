// grad_norm_kernels.h -- host-side launch descriptors of the gradient norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxfp4.h"

namespace mxfp4 {

using GradTensor = mxfp4_grad_item_t;  // grad, out (clipping: may be grad), count, dtype

struct GradNormLaunch {
  const GradTensor *tensors;
  int n, order;        // order: 1, 2, or 0 for the largest magnitude
  double *workspace;   // grad_norm_workspace(n, elements) doubles
  float *norm;
  bool clip;           // write the clipped gradients too
  bool given;          // norm is an input
  float max_norm;
};
int64_t grad_norm_workspace(int64_t n, int64_t elements);
hipError_t launch_grad_norm(const GradNormLaunch &L, hipStream_t stream);

}  // namespace mxfp4
