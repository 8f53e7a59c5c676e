// The tiled product on bf16 operands (gfx950).
#include "gemm_tiles.h"

namespace beam {

hipError_t launch_gemm_bf16(const GemmArgs& g, const GemmSplit& s, int tile, hipStream_t st) {
  return launch_gemm_tiles<false>(g, s, tile, st);
}

hipError_t launch_gemm_pair_bf16(const GemmArgs& dx, const GemmSplit& sx, const GemmArgs& dw, const GemmSplit& sw,
                                 int tile, hipStream_t st) {
  return tile == 128 ? launch_gemm_pair<false, 128>(dx, sx, dw, sw, st) : launch_gemm_pair<false, 64>(dx, sx, dw, sw, st);
}

}  // namespace beam
