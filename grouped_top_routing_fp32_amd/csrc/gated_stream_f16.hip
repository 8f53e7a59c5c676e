// The large product of a gated layer on fp16 operands (gfx950).
#include "stream.h"

namespace beam {

hipError_t launch_gated_stream_f16(const GatedArgs& g, int grid, int mt, int nt, hipStream_t st) {
  if (g.out_type == kElemF32)
    hipLaunchKernelGGL((stream_kernel<GatedArgs, true, F32>), dim3(grid), dim3(512), 0, st, g, mt, nt);
  else
    hipLaunchKernelGGL((stream_kernel<GatedArgs, true, F16>), dim3(grid), dim3(512), 0, st, g, mt, nt);
  return hipGetLastError();
}

}  // namespace beam
