// The tiled products of a gated layer on fp16 operands (gfx950).
#include "gemm_tiles.h"

namespace beam {

hipError_t launch_gated_f16(const GatedArgs& g, const GemmSplit& s, int tile, hipStream_t st) {
  return launch_gemm_tiles<true>(g, s, tile, st);
}

hipError_t launch_gated_pair_f16(const GatedArgs& dx, const GemmSplit& sx, const GatedArgs& dw, const GemmSplit& sw,
                                 int tile, hipStream_t st) {
  if (tile == 256) return launch_gemm_pair<true, 256>(dx, sx, dw, sw, st);
  return tile == 128 ? launch_gemm_pair<true, 128>(dx, sx, dw, sw, st) : launch_gemm_pair<true, 64>(dx, sx, dw, sw, st);
}

}  // namespace beam
