// What the kernels of grads.hip share with the ABI: the gradients of a step as one list of tensors.
#pragma once

#include "elem.h"

namespace beam {

// One tensor; types are ElemType.  out null: none is written.
struct GradTensor {
  const void* p;
  void* out;
  int64_t n;
  uint32_t end;  // chunks of the list up to this tensor's last; the launches set it
  uint8_t type, out_type;
};
static_assert(sizeof(GradTensor) == 32, "a table's entry");

// Every element's gradient counts `scale` times.  norm_in null: the norm is computed.
struct ClipArgs {
  double scale, max_norm, eps;
  const float* norm_in;
  float* norm;  // null: not written
};

// Workspace of both calls for `count` tensors.
size_t grad_workspace(int count);
// norm = |scale| sqrt(sum of squares).  Tensors without elements are left out of the list before.
hipError_t launch_grad_norm(GradTensor* t, int count, double scale, void* ws, float* norm, hipStream_t st);
// out = g scale min(1, max_norm / (norm + eps))
hipError_t launch_clip_grads(GradTensor* t, int count, const ClipArgs& a, void* ws, hipStream_t st);

}  // namespace beam
