// A matrix product with bias, activation and residual in its epilogue, and the
// gradients that go with it (gfx950).
//
//   y  = keep res + add act(x w^T + bias)
//   dz = add dy act'(z),  dx = dz w,  dw = dz^T x,  dbias = sum_m dz,  dres = keep dy
//
// Products run on 16-bit MFMA with FP32 accumulation; the epilogue is FP32 and
// rounds once to the output's type.
#include "linear.h"

namespace beam {

constexpr int kLinTile = 64;  // rows and columns of an output tile
constexpr int kLinK = 32;     // K per step
constexpr int kLinPad = 8;    // LDS rows of 80 bytes: 16-byte reads of 16 rows fall on distinct banks

// Element (i, k) of an operand, 0 past its ends.
__device__ __forceinline__ uint16_t operand_at(const void* p, int64_t ld, bool trans, int i, int k, int ni, int nk) {
  if (i >= ni || k >= nk) return 0;
  return static_cast<const uint16_t*>(p)[trans ? (int64_t)k * ld + i : (int64_t)i * ld + k];
}

// grid (ceil(N / 64), ceil(M / 64)), 4 waves as 2 x 2, each 32 x 32 of the tile.
__global__ __launch_bounds__(256) void gemm_simple_kernel(GemmArgs g) {
  __shared__ __align__(16) uint16_t sa[kLinTile][kLinK + kLinPad], sb[kLinTile][kLinK + kLinPad];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int m0 = blockIdx.y * kLinTile, n0 = blockIdx.x * kLinTile;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x4 acc[2][2] = {};
  for (int k0 = 0; k0 < g.K; k0 += kLinK) {
    __syncthreads();
    for (int i = tid; i < kLinTile * kLinK; i += 256) {
      // consecutive threads along the operand's contiguous axis
      const int ar = g.at ? i % kLinTile : i / kLinK, ak = g.at ? i / kLinTile : i % kLinK;
      sa[ar][ak] = operand_at(g.a, g.lda, g.at, m0 + ar, k0 + ak, g.M, g.K);
      const int br = g.bt ? i % kLinTile : i / kLinK, bk = g.bt ? i / kLinTile : i % kLinK;
      sb[br][bk] = operand_at(g.b, g.ldb, g.bt, n0 + br, k0 + bk, g.N, g.K);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4 fa = *reinterpret_cast<const u32x4*>(&sa[wm + 16 * i + (lane & 15)][8 * (lane >> 4)]);
        const u32x4 fb = *reinterpret_cast<const u32x4*>(&sb[wn + 16 * j + (lane & 15)][8 * (lane >> 4)]);
        acc[i][j] = g.type == kElemBF16 ? mfma16x16x32(fa, fb, acc[i][j]) : mfma16x16x32_f16(fa, fb, acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = m0 + wm + 16 * i + 4 * (lane >> 4) + r, n = n0 + wn + 16 * j + (lane & 15);
        if (m < g.M && n < g.N) epilogue(g, m, n, acc[i][j][r]);
      }
}

// dz[m, n] = add dy act'(z), rounded to the products' 16-bit type (the rounding that a
// gradient kept between two layers has anyway); part[u][n] = the unit's sum of the
// unrounded dz; dres = keep dy.  grid (ceil(N / 256), units), one column to a thread.
__global__ __launch_bounds__(256) void linear_dz_kernel(const void* __restrict__ dy, int dy_type, int64_t lddy,
                                                        const void* __restrict__ z, int64_t ldz, int act, float keep,
                                                        float add, uint16_t* __restrict__ dz, int64_t lddz, int type,
                                                        float* __restrict__ part, void* __restrict__ dres,
                                                        int64_t lddres, int M, int N, int rows) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  const int m0 = blockIdx.y * rows, m1 = min(M, m0 + rows);
  float s = 0.f;
  for (int m = m0; m < m1; ++m) {
    const float d = load_elem(dy, (int64_t)m * lddy + n, dy_type);
    float v = add * d;
    if (act != kActNone) v *= act_slope_f32(load_elem(z, (int64_t)m * ldz + n, type), act);
    if (dz) store_elem(dz, (int64_t)m * lddz + n, type, v);
    if (dres) store_elem(dres, (int64_t)m * lddres + n, dy_type, keep * d);
    s += v;
  }
  if (part) part[(int64_t)blockIdx.y * N + n] = s;
}

hipError_t launch_gemm(const GemmArgs& g, hipStream_t st) {
  hipLaunchKernelGGL(gemm_simple_kernel, dim3((g.N + kLinTile - 1) / kLinTile, (g.M + kLinTile - 1) / kLinTile),
                     dim3(256), 0, st, g);
  return hipGetLastError();
}

int linear_dz_units(int M) { return M < 128 ? M : 128; }

hipError_t launch_linear_dz(const void* dy, int dy_type, int64_t lddy, const void* z, int64_t ldz, int act, float keep,
                            float add, uint16_t* dz, int64_t lddz, int type, float* part, void* dres, int64_t lddres,
                            int M, int N, hipStream_t st) {
  const int units = linear_dz_units(M), rows = (M + units - 1) / units;
  hipLaunchKernelGGL(linear_dz_kernel, dim3((N + 255) / 256, units), dim3(256), 0, st, dy, dy_type, lddy, z, ldz, act,
                     keep, add, dz, lddz, type, part, dres, lddres, M, N, rows);
  return hipGetLastError();
}

}  // namespace beam
