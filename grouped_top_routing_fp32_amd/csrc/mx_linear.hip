// A matrix product with weights, or both operands, in microscaled 4 bits, with bias, activation and residual in its
// epilogue (gfx950).
//
//   y = keep res + add act(x w^T + bias)
//
// Few rows are bound by reading w, a quarter of its 16-bit bytes: one kernel takes codes and scales straight from memory
// to registers ([1, 5120] x [2560, 5120], 7 MB, 6.5 us, of which some 5 are a launch and one trip to memory).
// With both operands in 4 bits the products run on scaled matrix instructions, four times the 16-bit rate for the
// same bytes in LDS: small ones in the tiled product, large ones in a persistent kernel ([16384, 2560] x [5120,
// 2560] 123 to 131 us in calls, 3.3 to 3.5 PFLOP/s).  With x of 16 bits, some rows go through tiles that hold codes in LDS and turn them into
// x's type on their way to the matrix instructions ([64, 2560] x [5120, 2560] 9.8 us and 4.0 for the join of its splits;
// [64, 5120] x [32768, 5120] 39 us, 2.3 TB/s of codes and scales).  Where rows are no whole chunks, products of few
// tiles do so on the codes' way into LDS; larger ones lay w out as x's type in the workspace first and run the plain
// product.
#include <algorithm>
#include <cmath>

#include "mxfp4.h"

namespace beam {
namespace {

template <class A>
A ceil_div(A a, int b) {
  return (a + b - 1) / b;
}
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

// 16-bit rows in tiles of 64 rows, 32 where there are no more, and 128 columns (launch_code_rows): a workgroup to a CU,
// rounds of them of 4 us and some 0.75 (0.6 of 32 rows) for each stage of 128 of K, 26 KB (18) at what a CU gets from
// its L2.  K is split where that saves more than the launch that joins the sums, 4.5 us.  Taken where this estimate is
// below the other form's:
// - up to 16 rows the kernel for few, which reads w evenly, 15 bytes a nanosecond and CU, but x once for each 16
//   columns of a CU ([16, 5120] x [10240, 5120] 22.6 us, 15.8 here; [8, 5120] x [5120, 5120] 11.6 and 12.6; [1, 5120] x
//   [32768, 5120] 29 both)
// - above, w turned into 16 bits, in its tiles or in memory, and the product at 1.15 PFLOP/s ([256, 2560] x [5120, 2560]
//   27.5 us, 18.9 here; [512, 5120] x [2560, 5120] 31 and 33.6; [64, 5120] x [32768, 5120] 161 and 39)
bool plan_mx_rows(MxPlan* p, int M, int N, int K) {
  const int rows = M <= 32 ? 32 : 64, stages = ceil_div(K, 128);
  const int64_t tiles = (int64_t)ceil_div(M, rows) * ceil_div(N, 128);
  if (tiles < 1 || tiles > 1 << 20) return false;
  const double stage = rows == 32 ? 0.6 : 0.75, weights = (double)N * K;
  int s = tiles <= kCUs ? std::max(1, std::min({kCUs / (int)tiles, stages / 4, 16})) : 1;
  if ((stages - ceil_div(stages, s)) * stage < 4.5) s = 1;
  const int per = ceil_div(stages, s);
  const double here = (double)ceil_div(tiles * s, kCUs) * (4. + stage * per) + (s > 1 ? 5.5 : 1.);
  const double rounds = ceil_div(N, 16 * kCUs);
  const double few = 4. + weights * 0.53 / kCUs / 15e3 + rounds * (0.5 + M * (double)K * 2 / 42e3);
  const double other = 10. + weights * 2.53 / 4.5e6 + weights * M * 2 / 1.15e9;
  if (here >= (M <= kSkinnyRows ? few : other)) return false;
  p->rows = rows;
  p->gemm.kind = GemmPlan::kTiles;
  p->gemm.k_per_split = per * 128;
  p->gemm.splits = ceil_div(K, p->gemm.k_per_split);
  p->gemm.total = p->gemm.splits > 1 ? up256((size_t)p->gemm.splits * M * ((N + 3) / 4 * 4) * sizeof(float)) : 0;
  p->total = p->gemm.total;
  return true;
}

}  // namespace

MxPlan plan_mx(int M, int N, int K, bool four, int64_t ldx, int64_t ldw) {
  MxPlan p{};
  if (!four && regular_rows(ldx, K) && plan_mx_rows(&p, M, N, K)) return p;
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
  if (p.fused || p.rows) {
    CodeArgs g{a.g, a.w_scales, a.ldws, blocks};
    g.a = a.x;
    g.lda = a.ldx;
    g.b = a.w;
    g.ldb = a.ldw;
    const GemmSplit s = split_of(p.gemm, g.N, base);
    e = p.rows ? launch_code_rows(g, s, p.rows, st) : launch_code_tiles(g, s, p.gemm.tile, st);
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
