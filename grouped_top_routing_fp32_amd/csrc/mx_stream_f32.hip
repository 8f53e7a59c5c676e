// The large product of 4-bit operands with fp32 results (gfx950).
#include "stream.h"

namespace beam {

hipError_t launch_mx_stream_f32(const MxArgs& g, int mt, int nt, int grid, hipStream_t st) {
  hipLaunchKernelGGL((stream_kernel<MxArgs, false, F32>), dim3(grid), dim3(512), 0, st, g, mt, nt);
  return hipGetLastError();
}

}  // namespace beam
