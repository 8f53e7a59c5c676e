// The large product of two operands in microscaled 4 bits (gfx950): the scales' order and the launch.
#include <algorithm>

#include "stream.h"

namespace beam {
namespace {

// One operand's scales by tile, stage and 64 rows: byte (g, l, s, i) of 512 is block 8 stage + 4 s + g of row
// 16 i + l; 0 past the row's blocks.  A thread has four rows' eight blocks of a stage.
struct ScaleJob {
  const uint8_t* from;
  int64_t ld;
  int rows;
  uint8_t* to;
  int threads;
};
__global__ __launch_bounds__(256) void mx_scales_kernel(ScaleJob first, ScaleJob second, int groups, int blocks) {
  const bool other = (int)blockIdx.x >= groups;
  const ScaleJob j = other ? second : first;
  const int stages = (blocks + 7) / 8, t = (blockIdx.x - (other ? groups : 0)) * 256 + threadIdx.x;
  if (t >= j.threads) return;
  const int l = t & 15, quarter = (t >> 4) & 3, at = t >> 6, stage = at % stages, tile = at / stages;
  using Stage = ScaleStage<kT>;
  uint64_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = min(tile * kT + quarter * 64 + 16 * i + l, j.rows - 1);
    v[i] = Stage::load(j.from + r * j.ld, 8 * stage, blocks);
  }
  uint8_t* to = j.to + (int64_t)at * (kScales / 2) + quarter * 512 + l * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (blocks >= 8) v[i] >>= 8 * max(8 * stage + 8 - blocks, 0);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    u32x2 w = {0u, 0u};
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[s] |= (uint32_t)(uint8_t)(v[i] >> (8 * (4 * s + g))) << (8 * i);
    *reinterpret_cast<u32x2*>(to + g * 128) = w;
  }
}

int tiles_of(int n) { return (n + kT - 1) / kT; }

}  // namespace

hipError_t launch_mx_stream_bf16(const MxArgs& g, int mt, int nt, int grid, hipStream_t st);
hipError_t launch_mx_stream_f16(const MxArgs& g, int mt, int nt, int grid, hipStream_t st);
hipError_t launch_mx_stream_f32(const MxArgs& g, int mt, int nt, int grid, hipStream_t st);

size_t mx_stream_bytes(int M, int N, int K) {
  return (size_t)(tiles_of(M) + tiles_of(N)) * ((K + 63) / 64) * (kScales / 2);
}

hipError_t launch_mx_stream(const MxArgs& args, void* ws, hipStream_t st) {
  MxArgs g = args;
  const int mt = tiles_of(g.M), nt = tiles_of(g.N), blocks = g.K / 8, stages = (blocks + 7) / 8;
  uint8_t* a = static_cast<uint8_t*>(ws);
  uint8_t* b = a + (int64_t)mt * stages * (kScales / 2);
  const ScaleJob ja{g.sa, g.ldsa, g.M, a, mt * stages * 64}, jb{g.sb, g.ldsb, g.N, b, nt * stages * 64};
  const int ga = (ja.threads + 255) / 256, gb = (jb.threads + 255) / 256;
  hipLaunchKernelGGL(mx_scales_kernel, dim3(ga + gb), dim3(256), 0, st, ja, jb, ga, blocks);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  g.sa = a;
  g.sb = b;
  const int grid = std::min((mt * nt + 7) / 8 * 8, 256);  // a workgroup to a CU
  if (g.out_type == kElemF32) return launch_mx_stream_f32(g, mt, nt, grid, st);
  return g.out_type == kElemF16 ? launch_mx_stream_f16(g, mt, nt, grid, st) : launch_mx_stream_bf16(g, mt, nt, grid, st);
}

}  // namespace beam
