// The tiled products of 4-bit operands, and of 16-bit rows with 4-bit weights (gfx950).
#include "gemm_tiles.h"

namespace beam {

hipError_t launch_mx_tiles(const MxArgs& g, const GemmSplit& s, int tile, bool half, hipStream_t st) {
  const int mt = (g.M + tile - 1) / tile, nt = (g.N + tile - 1) / tile, total = mt * nt * s.splits;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(total), dim3(256), 0, st, g, mt, nt, total, s.k_per_split, s.part, s.ld);
    return hipGetLastError();
  };
  auto of = [&](auto h) {
    constexpr bool kHalf = decltype(h)::value;
    if (tile == 128) return go(gemm_kernel<kHalf, false, false, 128, 128, 2, 2, true, false, MxArgs>);
    return go(gemm_kernel<kHalf, false, false, 64, 64, 2, 2, true, false, MxArgs>);
  };
  return half ? of(std::true_type{}) : of(std::false_type{});
}

hipError_t launch_code_tiles(const CodeArgs& g, const GemmSplit& s, int tile, hipStream_t st) {
  const int mt = (g.M + tile - 1) / tile, nt = (g.N + tile - 1) / tile, total = mt * nt * s.splits;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(total), dim3(256), 0, st, g, mt, nt, total, s.k_per_split, s.part, s.ld);
    return hipGetLastError();
  };
  auto of = [&](auto h) {
    constexpr bool kHalf = decltype(h)::value;
    if (tile == 128) return go(gemm_kernel<kHalf, false, false, 128, 128, 2, 2, true, true, CodeArgs>);
    return go(gemm_kernel<kHalf, false, false, 64, 64, 2, 2, true, true, CodeArgs>);
  };
  return g.type == kElemF16 ? of(std::true_type{}) : of(std::false_type{});
}

}  // namespace beam
