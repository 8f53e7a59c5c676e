// A matrix product with bias, activation and residual in its epilogue, and the
// gradients that go with it (gfx950).
//
//   y  = keep res + add act(x w^T + bias)
//   dz = add dy act'(z),  dx = dz w,  dw = dz^T x,  dbias = sum_m dz,  dres = keep dy
//
// All three products are one kernel over operands whose contiguous axis is K (x and w
// of the forward product, dz in dx) or the output's (w in dx, both in dw); products
// run on 16-bit MFMA with FP32 accumulation; the epilogue is FP32 and rounds once to
// the output's type.
#include <type_traits>

#include "linear.h"

namespace beam {

// out from the partial sums of the splits, added in order: four columns to a thread.
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs g, const float* __restrict__ part, int64_t ldpart,
                                                        int splits) {
  const int quads = (int)(ldpart / 4);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)g.M * quads) return;
  const int m = (int)(i / quads), n = (int)(i % quads) * 4;
  f32x4 z = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < splits; ++s) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(part + ((int64_t)s * g.M + m) * ldpart + n);
#pragma unroll
    for (int q = 0; q < 4; ++q) z[q] += v[q];
  }
  const bool wide = epilogue_wide(g);
  by_act(g.act, [&](auto act) { epilogue4<decltype(act)::value>(g, wide, m, n, z); });
}

// Few rows (M <= 16, both operands K contiguous): bound by reading w once.  A workgroup
// takes 16 columns; its 8 waves share K in pieces of 128, straight from memory into
// MFMA operands (a wave reads 256 contiguous bytes of 16 rows of w), and their sums are
// joined in LDS in wave order.
constexpr int kSkinnyWaves = 8;

template <bool HALF, bool WIDE>
__global__ __launch_bounds__(64 * kSkinnyWaves) void gemm_skinny_kernel(GemmArgs g) {
  __shared__ f32x4 sum[kSkinnyWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, gr = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const uint16_t* wrow = static_cast<const uint16_t*>(g.b) + (int64_t)min(n0 + l16, g.N - 1) * g.ldb;
  const uint16_t* xrow = static_cast<const uint16_t*>(g.a) + (int64_t)min(l16, g.M - 1) * g.lda;
  auto chunk = [&](const uint16_t* row, int k) {  // 8 elements from k, 0 past K
    if constexpr (WIDE) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (k < g.K) v = ldg16(row + k);
      return v;
    } else {
      uint16_t e[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) e[q] = k + q < g.K ? row[k + q] : 0;
      u32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = e[2 * q] | ((uint32_t)e[2 * q + 1] << 16);
      return v;
    }
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int k = 128 * wave; k < g.K; k += 128 * kSkinnyWaves) {
    u32x4 fw[4], fx[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      fw[s] = chunk(wrow, k + 32 * s + 8 * gr);
      fx[s] = chunk(xrow, k + 32 * s + 8 * gr);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = mfma<HALF>(fw[s], fx[s], acc);
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
  if (l16 >= g.M || n >= g.N) return;
  const bool wide = epilogue_wide(g);
  by_act(g.act, [&](auto act) { epilogue4<decltype(act)::value>(g, wide, l16, n, z); });
}

// Lays one or two operands out anew, the first with blocks workgroups and the second with
// the rest: one launch for what a product or both gradients need.
__global__ __launch_bounds__(256) void pad_rows_kernel(PadJob first, PadJob second, int blocks) {
  const bool other = (int)blockIdx.x >= blocks;
  const PadJob j = other ? second : first;
  const int64_t threads = 256 * (int64_t)(other ? gridDim.x - blocks : blocks);
  const int chunks = (j.cols + 7) / 8;
  const int64_t n = (int64_t)j.rows * chunks;
  for (int64_t i = (int64_t)(blockIdx.x - (other ? blocks : 0)) * 256 + threadIdx.x; i < n; i += threads) {
    const int r = (int)(i / chunks), c = (int)(i % chunks) * 8;
    const uint16_t* s = static_cast<const uint16_t*>(j.src) + (int64_t)r * j.ld;
    u32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t lo = c + 2 * q < j.cols ? s[c + 2 * q] : 0, hi = c + 2 * q + 1 < j.cols ? s[c + 2 * q + 1] : 0;
      v[q] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(j.dst) + ((int64_t)r * chunks + c / 8) * 8) = v;
  }
}

// dz[m, n] = add dy act'(z), rounded to the products' 16-bit type (the rounding that a
// gradient kept between two layers has anyway); part[u][n] = the unit's sum of the
// unrounded dz; dres = keep dy.  grid (ceil(N / VEC / 64), units), block (64, 4): thread
// (c, r) takes chunk c of VEC columns in rows r, r + 4, ... of the unit.  dz rows are
// lddz long, a multiple of 8, with zeros past N.
template <int VEC>
__global__ __launch_bounds__(256) void linear_dz_kernel(const void* __restrict__ dy, int dy_type, int64_t lddy,
                                                        const void* __restrict__ z, int64_t ldz, int act, float keep,
                                                        float add, uint16_t* __restrict__ dz, int64_t lddz, int type,
                                                        float* __restrict__ part, void* __restrict__ dres,
                                                        int64_t lddres, int M, int N, int rows) {
  __shared__ float sums[4][64][VEC];
  const int n = (blockIdx.x * 64 + threadIdx.x) * VEC, y = threadIdx.y;
  const int m1 = min(M, (int)(blockIdx.y + 1) * rows);
  float s[VEC] = {};
  if (n < (dz ? lddz : N)) {
    auto load = [&](const void* p, int64_t i, int ty, float* v) {
      if constexpr (VEC == 1) {
        v[0] = load_elem(p, i, ty);
      } else if (ty == kElemF32) {
        load_n<F32, VEC>(static_cast<const float*>(p) + i, v);
      } else if (ty == kElemBF16) {
        load_n<BF16, VEC>(static_cast<const uint16_t*>(p) + i, v);
      } else {
        load_n<F16, VEC>(static_cast<const uint16_t*>(p) + i, v);
      }
    };
    auto store = [&](void* p, int64_t i, int ty, const float* v) {
      if constexpr (VEC == 1) {
        store_elem(p, i, ty, v[0]);
      } else if (ty == kElemF32) {
        store_n<F32, VEC>(static_cast<float*>(p) + i, v);
      } else if (ty == kElemBF16) {
        store_n<BF16, VEC>(static_cast<uint16_t*>(p) + i, v);
      } else {
        store_n<F16, VEC>(static_cast<uint16_t*>(p) + i, v);
      }
    };
    by_act(act, [&](auto a) {
      constexpr int ACT = decltype(a)::value;
#pragma unroll 4
      for (int m = blockIdx.y * rows + y; m < m1; m += 4) {
        float d[VEC] = {}, v[VEC] = {}, zz[VEC] = {};
        if (n < N) {  // VEC = 8 only where N holds whole chunks
          load(dy, (int64_t)m * lddy + n, dy_type, d);
          if constexpr (ACT != kActNone) load(z, (int64_t)m * ldz + n, type, zz);
#pragma unroll
          for (int q = 0; q < VEC; ++q) {
            v[q] = add * d[q] * act_slope_f32<ACT>(zz[q]);
            s[q] += v[q];
            d[q] *= keep;
          }
          if (dres) store(dres, (int64_t)m * lddres + n, dy_type, d);
        }
        if (dz) store(dz, (int64_t)m * lddz + n, type, v);
      }
    });
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < VEC; ++q) sums[y][threadIdx.x][q] = s[q];
  __syncthreads();
  for (int i = y * 64 + threadIdx.x; i < 64 * VEC; i += 256) {
    const int c = i / VEC, q = i % VEC, col = (blockIdx.x * 64 + c) * VEC + q;
    if (col < N) part[(int64_t)blockIdx.y * N + col] = (sums[0][c][q] + sums[1][c][q]) + (sums[2][c][q] + sums[3][c][q]);
  }
}

// ---------------------------------------------------------------------------
// plans and launches
// ---------------------------------------------------------------------------
namespace {

constexpr int kBK = 64;  // K per stage of the tiled kernel
constexpr int kCUs = 256;
// Up to here the skinny kernel: 2560 columns, K 5120: 11.3 us at 16 rows against 12.8 in
// tiles; its form for 32 rows took 15.9 against 12.8.
constexpr int kSkinnyRows = 16;
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int ceil_div(int a, int b) { return (a + b - 1) / b; }
}  // namespace

GemmPlan plan_gemm(int M, int N, int K, bool at, bool bt, int64_t lda, int64_t ldb, bool padded) {
  GemmPlan p{};
  p.splits = 1;
  p.k_per_split = K > 0 ? ceil_div(K, kBK) * kBK : kBK;
  if (!at && !bt && M <= kSkinnyRows) {
    p.kind = GemmPlan::kSkinny;
    return p;
  }
  p.kind = GemmPlan::kTiles;
  p.copy_a = !padded && !regular_rows(lda, at ? M : K);
  p.copy_b = !padded && !regular_rows(ldb, bt ? N : K);
  // 256-row tiles from 160 of them on ([4096, 5120] x [2560, 5120], 160 tiles: 125 us, 134
  // in 128-row tiles; [3000, ...], 120 tiles: 91 and 90).  Below, 128-row tiles with K
  // split until two workgroups a CU (what LDS holds) have work, in at least 8 stages each;
  // under 24 stages the join costs what a split gains.  64-row tiles where even split
  // 128-row tiles would leave CUs without work: [1000, 1000] x [1000, 1000] forward and
  // back 32 us, 41 in 128-row tiles; but [512, 5120] x [2560, 5120] 42 us, 28 in those.
  const int stages = ceil_div(K, kBK);
  int tiles = ceil_div(M, 256) * ceil_div(N, 256);
  p.tile = 256;
  if (tiles < 160) {
    p.tile = 128;
    tiles = ceil_div(M, 128) * ceil_div(N, 128);
    if (tiles * (stages / 8 + 1) < kCUs) {
      p.tile = 64;
      tiles = ceil_div(M, 64) * ceil_div(N, 64);
    }
    int s = tiles > 0 ? 2 * kCUs / tiles : 1;
    s = s < stages / 8 ? s : stages / 8;
    s = s < 16 ? s : 16;
    if (s > 1 && stages >= 24) {
      p.k_per_split = ceil_div(stages, s) * kBK;
      p.splits = ceil_div(K, p.k_per_split);
    }
  }
  size_t off = 0;
  p.off_a = off;
  if (p.copy_a) off = up256(off + padded_bytes(at ? K : M, at ? M : K));
  p.off_b = off;
  if (p.copy_b) off = up256(off + padded_bytes(bt ? K : N, bt ? N : K));
  p.off_part = off;
  if (p.splits > 1) off = up256(off + (size_t)p.splits * M * ((N + 3) / 4 * 4) * sizeof(float));
  p.total = off;
  return p;
}

namespace {

template <bool HALF>
hipError_t launch_skinny(const GemmArgs& g, hipStream_t st) {
  const bool wide = regular_rows(g.lda, g.K) && regular_rows(g.ldb, g.K);
  const dim3 grid(ceil_div(g.N, 16)), block(64 * kSkinnyWaves);
  if (wide)
    hipLaunchKernelGGL((gemm_skinny_kernel<HALF, true>), grid, block, 0, st, g);
  else
    hipLaunchKernelGGL((gemm_skinny_kernel<HALF, false>), grid, block, 0, st, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pad(const PadJob& first, const PadJob& second, hipStream_t st) {
  auto blocks = [](const PadJob& j) {
    const int64_t n = (j.rows * (up8(j.cols) / 8) + 255) / 256;
    return (int)(n < (1 << 20) ? n : 1 << 20);
  };
  const int a = blocks(first), b = blocks(second);
  if (a + b == 0) return hipSuccess;
  hipLaunchKernelGGL(pad_rows_kernel, dim3(a + b), dim3(256), 0, st, first, second, a);
  return hipGetLastError();
}

hipError_t launch_gemm(const GemmArgs& args, const GemmPlan& p, void* ws, hipStream_t st) {
  GemmArgs g = args;
  char* base = static_cast<char*>(ws);
  hipError_t e;
  PadJob ja{}, jb{};
  if (p.copy_a) {
    ja = {g.a, g.lda, g.at ? g.K : g.M, g.at ? g.M : g.K, base + p.off_a};
    g.a = ja.dst;
    g.lda = up8(ja.cols);
  }
  if (p.copy_b) {
    jb = {g.b, g.ldb, g.bt ? g.K : g.N, g.bt ? g.N : g.K, base + p.off_b};
    g.b = jb.dst;
    g.ldb = up8(jb.cols);
  }
  if ((e = launch_pad(ja, jb, st)) != hipSuccess) return e;
  const int64_t ldpart = (g.N + 3) / 4 * 4;
  float* part = p.splits > 1 ? reinterpret_cast<float*>(base + p.off_part) : nullptr;
  const bool half = g.type == kElemF16;
  if (p.kind == GemmPlan::kSkinny) return half ? launch_skinny<true>(g, st) : launch_skinny<false>(g, st);
  e = half ? launch_gemm_f16(g, p, part, ldpart, st) : launch_gemm_bf16(g, p, part, ldpart, st);
  if (e != hipSuccess || !part) return e;
  const int64_t quads = (int64_t)g.M * (ldpart / 4);
  hipLaunchKernelGGL(gemm_join_kernel, dim3((uint32_t)((quads + 255) / 256)), dim3(256), 0, st, g, part, ldpart,
                     p.splits);
  return hipGetLastError();
}

hipError_t launch_gemm_pair(const GemmArgs& dx, const GemmPlan& px, const GemmArgs& dw, const GemmPlan& pw, void* ws,
                            hipStream_t st) {
  auto whole = [](const GemmPlan& p) { return p.kind == GemmPlan::kTiles && p.tile == 64 && p.splits == 1; };
  if (dx.M > 0 && whole(px) && whole(pw))
    return dx.type == kElemF16 ? launch_gemm_pair_f16(dx, dw, st) : launch_gemm_pair_bf16(dx, dw, st);
  if (dx.M > 0) {
    const hipError_t e = launch_gemm(dx, px, ws, st);
    if (e != hipSuccess) return e;
  }
  return launch_gemm(dw, pw, ws, st);
}

// Rows of partial sums of dbias: 16 rows or more to each.
int linear_dz_units(int M) { return M < 32 ? 1 : M / 16 < 256 ? M / 16 : 256; }

hipError_t launch_linear_dz(const void* dy, int dy_type, int64_t lddy, const void* z, int64_t ldz, int act, float keep,
                            float add, uint16_t* dz, int64_t lddz, int type, float* part, void* dres, int64_t lddres,
                            int M, int N, hipStream_t st) {
  const int units = linear_dz_units(M), rows = ceil_div(M, units);
  const bool wide = N % 8 == 0 && lddy % 8 == 0 && (act == kActNone || ldz % 8 == 0) && (!dres || lddres % 8 == 0);
  const int cols = dz ? (int)lddz : N;
  auto go = [&](auto kernel, int vec) {
    hipLaunchKernelGGL(kernel, dim3(ceil_div(ceil_div(cols, vec), 64), units), dim3(64, 4), 0, st, dy, dy_type, lddy,
                       z, ldz, act, keep, add, dz, lddz, type, part, dres, lddres, M, N, rows);
  };
  if (wide)
    go(linear_dz_kernel<8>, 8);
  else
    go(linear_dz_kernel<1>, 1);
  return hipGetLastError();
}

}  // namespace beam
