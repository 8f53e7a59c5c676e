// What the kernels of grads.hip share with the ABI: the gradients of a step as one list of tensors.
#pragma once

#include "elem.h"

namespace beam {

// One tensor; types are ElemType.  out null: none is written.
struct GradTensor {
  const void* p;
  void* out;
  int64_t n;
  int type, out_type;
};

// Every element's gradient counts `scale` times.  norm_in null: the norm is computed.
struct ClipArgs {
  double scale, max_norm, eps;
  const float* norm_in;
  float* norm;  // null: not written
};

// Partial sums that the norm of `count` tensors needs.
int grad_partials(int count);
// norm = |scale| sqrt(sum of squares)
hipError_t launch_grad_norm(const GradTensor* t, int count, double scale, double* part, float* norm, hipStream_t st);
// out = g scale min(1, max_norm / (norm + eps))
hipError_t launch_clip_grads(const GradTensor* t, int count, const ClipArgs& a, double* part, hipStream_t st);

}  // namespace beam
