// A matrix product with weights, or both operands, in microscaled 4 bits, with bias, activation and residual in its
// epilogue (gfx950).
//
//   y = keep res + add act(x w^T + bias)
//
// Few rows are bound by reading w, a quarter of its 16-bit bytes: one kernel takes codes and scales straight from
// memory ([1, 5120] x [2560, 5120], 7 MB, 6.5 us, of which some 5 are a launch and one trip to memory).
// With both operands in 4 bits the products run on scaled matrix instructions, four times the 16-bit rate for the
// same bytes in LDS: small ones in the tiled product, large ones in a persistent kernel ([16384, 2560] x [5120,
// 2560] 149 us, 2.9 PFLOP/s).  With x of 16 bits, products of few tiles turn codes into x's type on their way into
// LDS ([64, 2560] x [5120, 2560] 11.1 us and 5.0 for the join of the splits; 23.9 with w laid out first); larger ones
// lay w out as x's type in the workspace first and run the plain product.
#include <algorithm>
#include <cmath>

#include "mxfp4.h"

namespace beam {
namespace {

int ceil_div(int a, int b) { return (a + b - 1) / b; }
constexpr int kCUs = 256;

// Few rows (M <= 16).  A workgroup takes `cols` <= 16 columns and its 16 waves share K in pieces of 128: a lane
// (row l % 16, block l / 16) takes one block of 32 codes, 16 bytes, and its scale.  With x of 16 bits the
// products' K runs over the four blocks' first 8 elements, then their second 8, and so on, which is the same
// sum.  The waves' sums are joined in LDS in wave order.
template <bool HALF, bool FOUR>
__global__ __launch_bounds__(64 * kSkinnyWaves) void mx_skinny_kernel(MxLinear a, int cols) {
  __shared__ f32x4 sum[kSkinnyWaves][64];
  const GemmArgs& g = a.g;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, gr = lane >> 4;
  const int n0 = blockIdx.x * cols, n1 = min(g.N, n0 + cols), row = min(n0 + l16, n1 - 1), xr = min(l16, g.M - 1);
  const uint8_t* wrow = a.w + row * a.ldw;
  const uint8_t* wscale = a.w_scales + row * a.ldws;
  const uint16_t* xrow = static_cast<const uint16_t*>(a.x) + xr * a.ldx;
  const uint8_t* xcodes = static_cast<const uint8_t*>(a.x) + xr * a.ldx;
  const uint8_t* xscale = FOUR ? a.x_scales + xr * a.ldxs : nullptr;
  const int blocks = (g.K + kMxBlock - 1) / kMxBlock;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int b = 4 * wave + gr; b - gr < blocks; b += 4 * kSkinnyWaves) {
    u32x4 w = {0u, 0u, 0u, 0u};
    uint32_t ws = 0, xs = 0;
    u32x4 x[4] = {};
    if (b < blocks) {
      w = ldg16(wrow + 16 * b);
      ws = wscale[b];
      if constexpr (FOUR) {
        x[0] = ldg16(xcodes + 16 * b);
        xs = xscale[b];
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = chunk_of_row(xrow, 32 * b + 8 * s, g.K);
      }
    }
    if constexpr (FOUR) {
      acc = mfma_mx<0, 0>(w, x[0], acc, ws, xs);
    } else {
      const float scale = mx_scale(ws);
#pragma unroll
      for (int s = 0; s < 4; ++s) acc = mfma<HALF>(codes_to_16<HALF>(w[s], scale), x[s], acc);
    }
  }
  sum[wave][lane] = acc;
  __syncthreads();
  if (wave > 0) return;
  f32x4 z = acc;
#pragma unroll
  for (int w = 1; w < kSkinnyWaves; ++w) {
    const f32x4 v = sum[w][lane];
#pragma unroll
    for (int q = 0; q < 4; ++q) z[q] += v[q];
  }
  const int n = n0 + 4 * gr;
  if (l16 >= g.M || n >= n1) return;
  by_act(g.act, [&](auto act) { epilogue4<decltype(act)::value>(g, g.add, l16, n, n1, z); });
}

// Two operands in 4 bits, K of `units` of four codes.  A long K of few tiles is split as any product's.  Else the
// tile with the least of these estimates, in microseconds with S the stages of K; they meet 21 shapes of 256 to 16384
// rows, 512 to 5120 columns and K of 200 to 5120 to some 15%, and nearer where the choice is close:
// - 64: t (0.003 + 0.0013 S) + 3 ([512, 5120] x [5120, 5120], 640 tiles, 20.2 us; 22.6 in 128-row tiles, 41.9 in 256)
// - 128: rounds of 512 tiles of 4 + 1.45 S, + 3 ([2000, 2000] x [3000, 2000], 384 tiles, 19.8; 21.8 and 28.0)
// - 256: rounds of 256 tiles of 5.5 + 1.9 S, + 6.5, the scales' launch among it ([16384, 2560] x [5120, 2560], 1280
//   tiles, 132 us; 180 in 128-row tiles; [2048, 5120] x [5120, 5120], 160 tiles, 48.8 and 54.6, but [8192, 5120] x
//   [1024, 5120], 128, 46.5 and 38.2)
GemmPlan plan_mx_tiles(int M, int N, int units, bool wide_rows) {
  GemmPlan p = plan_tiles(M, N, units);
  if (p.splits > 1) return p;
  const double S = ceil_div(units, 64);
  auto tiles = [&](int t) { return (double)ceil_div(M, t) * ceil_div(N, t); };
  const double small = tiles(64) * (0.003 + 0.0013 * S) + 3.;
  const double middle = std::ceil(tiles(128) / 512) * (4. + 1.45 * S) + 3.;
  const double large = std::ceil(tiles(256) / 256) * (5.5 + 1.9 * S) + 6.5;
  p.tile = !wide_rows && large <= std::min(small, middle) ? 256 : small <= middle ? 64 : 128;
  if (tiles(64) > 1 << 20) p.tile = wide_rows ? 128 : 256;  // threads of a grid fit 32 bits
  p.total = p.tile == 256 ? mx_stream_bytes(M, N, units) : 0;
  return p;
}

}  // namespace

MxPlan plan_mx(int M, int N, int K, bool four, int64_t ldx, int64_t ldw) {
  MxPlan p{};
  if (M <= kSkinnyRows) return p;
  const int blocks = (int)mx_blocks(K);
  if (four) {
    // 256 rows of an operand span less than 2^31 bytes in the large product
    p.gemm = plan_mx_tiles(M, N, 8 * blocks, std::max(ldx, ldw) >= int64_t(1) << 23);
    p.total = p.gemm.total;
    return p;
  }
  p.gemm = plan_tiles(M, N, (int)up8(K));
  p.fused = few_tiles(p.gemm, (int64_t)ceil_div(M, p.gemm.tile) * ceil_div(N, p.gemm.tile), K);
  if (p.fused) {
    p.total = p.gemm.total;
    return p;
  }
  p.copy_x = !regular_rows(ldx, K);
  p.off_w = p.copy_x ? up256(padded_bytes(M, K)) : 0;
  p.off_gemm = p.off_w + up256((size_t)N * blocks * kMxBlock * 2);
  p.total = p.off_gemm + p.gemm.total;
  return p;
}

hipError_t launch_linear_mx(const MxLinear& a, const MxPlan& p, void* ws, hipStream_t st) {
  const int blocks = (int)mx_blocks(a.g.K);
  const bool half = a.g.type == kElemF16;
  char* base = static_cast<char*>(ws);
  if (p.gemm.kind == GemmPlan::kSkinny) {
    const int rounds = ceil_div(a.g.N, 16 * kCUs), cols = std::max(4, ceil_div(a.g.N, rounds * kCUs));
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(ceil_div(a.g.N, cols)), dim3(64 * kSkinnyWaves), 0, st, a, cols);
      return hipGetLastError();
    };
    if (a.four) return go(mx_skinny_kernel<false, true>);
    return half ? go(mx_skinny_kernel<true, false>) : go(mx_skinny_kernel<false, false>);
  }
  hipError_t e;
  if (a.four) {
    MxArgs g{a.g, a.x_scales, a.w_scales, a.ldxs, a.ldws};
    g.a = a.x;
    g.lda = a.ldx / 2;
    g.b = a.w;
    g.ldb = a.ldw / 2;
    g.K = 8 * blocks;
    if (p.gemm.tile == 256) return launch_mx_stream(g, base, st);
    const GemmSplit s = split_of(p.gemm, g.N, base);
    e = launch_mx_tiles(g, s, p.gemm.tile, half, st);
    return e != hipSuccess ? e : launch_join_one(g, s, st);
  }
  if (p.fused) {
    CodeArgs g{a.g, a.w_scales, a.ldws, blocks};
    g.a = a.x;
    g.lda = a.ldx;
    g.b = a.w;
    g.ldb = a.ldw;
    const GemmSplit s = split_of(p.gemm, g.N, base);
    e = launch_code_tiles(g, s, p.gemm.tile, st);
    return e != hipSuccess ? e : launch_join_one(g, s, st);
  }
  GemmArgs g = a.g;
  g.a = a.x;
  g.lda = a.ldx;
  if (p.copy_x) {
    const PadJob j{a.x, a.ldx, g.M, g.K, base};
    if ((e = launch_pad(j, {}, {}, st)) != hipSuccess) return e;
    g.a = j.dst;
    g.lda = up8(g.K);
  }
  g.b = base + p.off_w;
  g.ldb = blocks * kMxBlock;
  g.K = (int)up8(g.K);
  e = launch_dequantize_mx(a.w, a.ldw, a.w_scales, a.ldws, base + p.off_w, g.type, g.ldb, g.N, blocks * kMxBlock, st);
  return e != hipSuccess ? e : launch_gemm(g, p.gemm, base + p.off_gemm, st);
}

}  // namespace beam
