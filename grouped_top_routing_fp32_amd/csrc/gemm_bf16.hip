// The tiled product on bf16 operands (gfx950).
#include "gemm_tiles.h"

namespace beam {

hipError_t launch_gemm_bf16(const GemmArgs& g, const GemmPlan& p, float* part, int64_t ldpart, hipStream_t st) {
  return launch_gemm_tiles<false>(g, p, part, ldpart, st);
}

hipError_t launch_gemm_pair_bf16(const GemmArgs& dx, const GemmArgs& dw, hipStream_t st) {
  return launch_gemm_pair<false>(dx, dw, st);
}

}  // namespace beam
