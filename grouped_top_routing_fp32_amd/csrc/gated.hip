// The two projections of a gated layer with activation and product, and the gradients that go with them (gfx950).
//
//   zg = x wg^T + bg,  zu = x wu^T + bu,  h = act(zg) zu
//   dzg = dh zu act'(zg),  dzu = dh act(zg)
//   dx = dzg wg + dzu wu,  dwg = dzg^T x,  dwu = dzu^T x,  dbg = sum_m dzg,  dbu = sum_m dzu
//
// The forward pass is one product of x with the rows of both weights in turn, so that a lane's sums hold both
// arguments of an element and neither projection goes to memory.  dz_gate and dz_up lie side by side in one
// buffer: dx is one product over K = both halves, dw another whose rows are both weights'.  The kernels are
// those of the plain product, with its tiles and plans; the forward pass in 256-row tiles has the persistent one
// ([16384, 5120] x [2560, 5120] bf16 670 us, 1280 TFLOP/s; 683 in the tiled one).
#include <algorithm>
#include <type_traits>

#include "gated.h"

namespace beam {
namespace {

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
constexpr int kCUs = 256;

// One element of h, or both arguments of it too.
template <int ACT>
__device__ __forceinline__ void gated1(const GatedArgs& g, int m, int n, float zg, float zu) {
  if (g.bias) zg += g.bias[n];
  if (g.bias2) zu += g.bias2[n];
  if (g.pre) store_elem(g.pre, (int64_t)m * g.ldp + n, g.type, zg);
  if (g.pre2) store_elem(g.pre2, (int64_t)m * g.ldp2 + n, g.type, zu);
  store_elem(g.out, (int64_t)m * g.ldo + n, g.out_type, act_f32<ACT>(zg) * zu);
}

// Columns n .. n + 3 of row m, those from `end` on left alone.
template <int ACT>
__device__ __forceinline__ void gated4(const GatedArgs& g, int m, int n, int end, f32x4 zg, f32x4 zu) {
  if (n + 4 <= end) {
    auto bias = [&](const float* b, f32x4& z) {
      if (!b) return;
      const f32x4 v = *reinterpret_cast<const f32x4_any*>(b + n);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] += v[q];
    };
    bias(g.bias, zg);
    bias(g.bias2, zu);
    if (g.pre) store_elem4(g.pre, (int64_t)m * g.ldp + n, g.type, zg);
    if (g.pre2) store_elem4(g.pre2, (int64_t)m * g.ldp2 + n, g.type, zu);
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = act_f32<ACT>(zg[q]) * zu[q];
    store_elem4(g.out, (int64_t)m * g.ldo + n, g.out_type, v);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < end) gated1<ACT>(g, m, n + q, zg[q], zu[q]);
  }
}

// h from the partial sums of the splits, added in order: four columns to a thread.
__global__ __launch_bounds__(256) void gated_join_kernel(GatedArgs g, GemmSplit sp) {
  const int quads = (int)(sp.ld / 8);
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)g.M * quads) return;
  const int m = (int)(i / quads), n = (int)(i % quads) * 4;
  f32x4 zg = {0.f, 0.f, 0.f, 0.f}, zu = zg;
  for (int s = 0; s < sp.splits; ++s) {
    const float* p = sp.part + ((int64_t)s * g.M + m) * sp.ld + n;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + sp.ld / 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      zg[q] += a[q];
      zu[q] += b[q];
    }
  }
  by_act(g.act, [&](auto act) { gated4<decltype(act)::value>(g, m, n, g.N, zg, zu); });
}

// The gradients' from theirs; the first has `blocks` workgroups.
__global__ __launch_bounds__(256) void gated_gradient_join_kernel(GatedArgs gx, GemmSplit sx, GatedArgs gw, GemmSplit sw,
                                                                  int blocks) {
  const bool other = (int)blockIdx.x >= blocks;
  const GatedArgs& g = other ? gw : gx;
  const GemmSplit& sp = other ? sw : sx;
  const float add = add_of(g);
  const int quads = (int)(sp.ld / 4);
  const int64_t i = (int64_t)(blockIdx.x - (other ? blocks : 0)) * 256 + threadIdx.x;
  if (i >= (int64_t)g.M * quads) return;
  const int m = (int)(i / quads), n = (int)(i % quads) * 4;
  f32x4 z = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < sp.splits; ++s) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(sp.part + ((int64_t)s * g.M + m) * sp.ld + n);
#pragma unroll
    for (int q = 0; q < 4; ++q) z[q] += v[q];
  }
  gradient4(g, add, m, n, z);
}

// Few rows (M <= 16): bound by reading both weights once ([1, 5120] x [2560, 5120], 52 MB, 11.4 us, 4.6 TB/s with
// the launch).  As the plain product's kernel for few rows, with two rows of weights to a lane and a sum of each.
template <bool HALF>
__global__ __launch_bounds__(64 * kSkinnyWaves) void gated_skinny_kernel(GatedArgs g, int cols) {
  __shared__ f32x4 sum[2][kSkinnyWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, gr = lane >> 4;
  const int n0 = blockIdx.x * cols, n1 = min(g.N, n0 + cols), row = min(n0 + l16, n1 - 1);
  const uint16_t* grow = static_cast<const uint16_t*>(g.b) + (int64_t)row * g.ldb;
  const uint16_t* urow = static_cast<const uint16_t*>(g.b2) + (int64_t)row * g.ldb2;
  const uint16_t* xrow = static_cast<const uint16_t*>(g.a) + (int64_t)min(l16, g.M - 1) * g.lda;
  f32x4 ag = {0.f, 0.f, 0.f, 0.f}, au = ag;
  // whole pieces without a test, so that all of their loads are in flight together
  int k = 128 * wave;
  for (; k + 128 <= g.K; k += 128 * kSkinnyWaves) {
    u32x4 fg[4], fu[4], fx[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      fg[s] = *reinterpret_cast<const u32x4_any*>(grow + k + 32 * s + 8 * gr);
      fu[s] = *reinterpret_cast<const u32x4_any*>(urow + k + 32 * s + 8 * gr);
      fx[s] = *reinterpret_cast<const u32x4_any*>(xrow + k + 32 * s + 8 * gr);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      ag = mfma<HALF>(fg[s], fx[s], ag);
      au = mfma<HALF>(fu[s], fx[s], au);
    }
  }
  if (k < g.K) {  // K's last piece, one wave's
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int ks = k + 32 * s + 8 * gr;
      const u32x4 fx = chunk_of_row(xrow, ks, g.K);
      ag = mfma<HALF>(chunk_of_row(grow, ks, g.K), fx, ag);
      au = mfma<HALF>(chunk_of_row(urow, ks, g.K), fx, au);
    }
  }
  sum[0][wave][lane] = ag;
  sum[1][wave][lane] = au;
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 1; w < kSkinnyWaves; ++w) {
    const f32x4 a = sum[0][w][lane], b = sum[1][w][lane];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      ag[q] += a[q];
      au[q] += b[q];
    }
  }
  const int n = n0 + 4 * gr;
  if (l16 >= g.M || n >= n1) return;
  by_act(g.act, [&](auto act) { gated4<decltype(act)::value>(g, l16, n, n1, ag, au); });
}

// Eight elements of both gradients.  An infinite argument stands for one past the type's range: the activation at it
// is its limit, and 0 times an infinite argument or activation is 0, as times the finite one.  Where d zu leaves FP32's
// range the slope, which is small or 0 there, is taken first.  All of these come out infinite or NaN as the formulas stand,
// and only then are looked at.
template <int ACT>
__device__ __forceinline__ void gated_slopes(const float* d, const float* zg, const float* zu, float* dg, float* du) {
  float odd = 0.f;  // NaN if one is not finite
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    dg[q] = d[q] * zu[q] * act_slope_f32<ACT>(zg[q]);
    du[q] = d[q] * act_f32<ACT>(zg[q]);
    odd = fmaf(du[q], 0.f, fmaf(dg[q], 0.f, odd));
  }
  if (odd == 0.f) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float p = d[q] * act_slope_f32<ACT>(zg[q]), a = act_limit_f32<ACT>(zg[q]);
    if (!__builtin_isfinite(dg[q])) dg[q] = p == 0.f && __builtin_isinf(zu[q]) ? 0.f : p * zu[q];
    du[q] = d[q] == 0.f && __builtin_isinf(a) ? 0.f : d[q] * a;
  }
}

// peaks[b] = the bits of the largest finite |dzg| or |dzu| in a workgroup's part, for the scale of an fp16 dz.
// Threads as in gated_dz_kernel, at most kMaxPeaks workgroups ([517, 1003] 8 us, latency); behind them those that lay
// operands out anew, which so do not wait.
template <class DT, class T>
__global__ __launch_bounds__(256) void gated_peak_kernel(GatedDz a, int units, int rows, PadJobs pad) {
  __shared__ uint32_t top[4];
  const int wide = ceil_div(a.N, 512), bx = blockIdx.x % wide, unit = blockIdx.x / wide, y = threadIdx.y;
  if (unit >= units) return pad_rows(pad, blockIdx.x - wide * units, y * 64 + threadIdx.x);
  const int n = (bx * 64 + threadIdx.x) * 8, cols = min(8, a.N - n);  // <= 0: none
  const int m1 = min(a.M, (unit + 1) * rows);
  uint32_t best = 0;
  if (cols > 0) {
    by_act(a.act, [&](auto act) {
      for (int m = unit * rows + y; m < m1; m += 4) {
        float d[8], zg[8], zu[8], dg[8], du[8];
        load8<DT>(static_cast<const typename DT::S*>(a.dh) + (int64_t)m * a.lddh + n, cols, d);
        load8<T>(static_cast<const typename T::S*>(a.zg) + (int64_t)m * a.ldzg + n, cols, zg);
        load8<T>(static_cast<const typename T::S*>(a.zu) + (int64_t)m * a.ldzu + n, cols, zu);
        gated_slopes<decltype(act)::value>(d, zg, zu, dg, du);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t b = __float_as_uint(dg[q]) & 0x7fffffffu, c = __float_as_uint(du[q]) & 0x7fffffffu;
          best = b < 0x7f800000u && b > best ? b : best;
          best = c < 0x7f800000u && c > best ? c : best;
        }
      }
    });
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, off));
  if (threadIdx.x == 0) top[y] = best;
  __syncthreads();
  if (threadIdx.x == 0 && y == 0) a.peaks[blockIdx.x] = max(max(top[0], top[1]), max(top[2], top[3]));
}

// dz = (dzg | dzu), each row two halves of gated_half(N) columns with zeros past N, in the products' 16-bit type: the
// matrix cores take no wider operands at this rate, two terms of dz would double both products, and a gradient kept between two
// layers has that rounding anyway.  The results are 2.35e-3 off in bf16 and 2.9e-4 in fp16, 1.7e-3 and 2.1e-4 without it.
// part[u] = the unit's sums of the unrounded dzg and dzu, N columns of each.  An fp16 dz is held times a
// power of two, as the plain product's is.  grid ceil(N / 512) * units, block (64, 4): thread (c, r) takes 8
// columns in rows r, r + 4, ... of the unit.  Bound by HBM ([8192, 2560] bf16, 210 MB, 38 us, 5.5 TB/s).
template <class DT, class T>
__global__ __launch_bounds__(256) void gated_dz_kernel(GatedDz a, int peak_count, int units, int rows, PadJobs pad) {
  __shared__ float sums[4][64][8];
  const int half = gated_half(a.N), wide = ceil_div(half, 512);
  const int bx = blockIdx.x % wide, unit = blockIdx.x / wide, y = threadIdx.y;
  if (unit >= units) return pad_rows(pad, blockIdx.x - wide * units, y * 64 + threadIdx.x);
  const int n = (bx * 64 + threadIdx.x) * 8, cols = min(8, a.N - n);  // <= 0: none
  const int m1 = min(a.M, (unit + 1) * rows);
  [[maybe_unused]] float up = 1.f;
  if constexpr (std::is_same_v<T, F16>) {
    if (a.dz) {
      up = dz_scale(a.peaks, peak_count, 1.0);
      if (blockIdx.x == 0 && threadIdx.x == 0 && y == 0) *a.unscale = 1.f / up;
    }
  }
  float sg[8] = {}, su[8] = {};
  if (n < half) {
    by_act(a.act, [&](auto act) {
#pragma unroll 2
      for (int m = unit * rows + y; m < m1; m += 4) {
        float d[8], zg[8], zu[8], dg[8], du[8];
        load8<DT>(static_cast<const typename DT::S*>(a.dh) + (int64_t)m * a.lddh + n, cols, d);  // zeros past N
        load8<T>(static_cast<const typename T::S*>(a.zg) + (int64_t)m * a.ldzg + n, cols, zg);
        load8<T>(static_cast<const typename T::S*>(a.zu) + (int64_t)m * a.ldzu + n, cols, zu);
        gated_slopes<decltype(act)::value>(d, zg, zu, dg, du);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          sg[q] += dg[q];
          su[q] += du[q];
          if constexpr (std::is_same_v<T, F16>) {
            dg[q] *= up;
            du[q] *= up;
          }
        }
        if (a.dz) {
          store8<T>(a.dz + (int64_t)m * 2 * half + n, 8, dg);
          store8<T>(a.dz + (int64_t)m * 2 * half + half + n, 8, du);
        }
      }
    });
  }
  if (!a.part) return;
  auto put = [&](const float* s, int64_t first) {
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[y][threadIdx.x][q] = s[q];
    __syncthreads();
    for (int i = y * 64 + threadIdx.x; i < 512; i += 256) {
      const int c = i / 8, q = i % 8, col = bx * 512 + i;
      if (col < a.N)
        a.part[(int64_t)unit * 2 * a.N + first + col] = (sums[0][c][q] + sums[1][c][q]) + (sums[2][c][q] + sums[3][c][q]);
    }
    __syncthreads();
  };
  put(sg, 0);
  put(su, a.N);
}

__global__ __launch_bounds__(256) void gated_sums_kernel(SumJob j) {
  __shared__ float s[256];
  sum_columns(s, j, blockIdx.x);
}

hipError_t launch_tiles(const GatedArgs& g, const GemmSplit& s, int tile, hipStream_t st) {
  return g.type == kElemF16 ? launch_gated_f16(g, s, tile, st) : launch_gated_bf16(g, s, tile, st);
}

hipError_t launch_gradient_join(const GatedArgs& dx, const GemmSplit& sx, const GatedArgs& dw, const GemmSplit& sw,
                                hipStream_t st) {
  auto blocks = [](const GatedArgs& g, const GemmSplit& s) { return s.part ? (int)((g.M * (s.ld / 4) + 255) / 256) : 0; };
  const int a = blocks(dx, sx), b = blocks(dw, sw);
  if (a + b == 0) return hipSuccess;
  hipLaunchKernelGGL(gated_gradient_join_kernel, dim3(a + b), dim3(256), 0, st, dx, sx, dw, sw, a);
  return hipGetLastError();
}

}  // namespace

GatedPlan plan_gated(int M, int N, int K, int64_t ldx, int64_t ldg, int64_t ldu) {
  GatedPlan p{};
  if (M <= kSkinnyRows) return p;  // kSkinny
  p.gemm = plan_tiles(M, 2 * N, K);
  p.copy_x = !regular_rows(ldx, K);
  p.copy_gate = !regular_rows(ldg, K);
  p.copy_up = !regular_rows(ldu, K);
  if ((p.copy_x || p.copy_gate || p.copy_up) &&
      few_tiles(p.gemm, (int64_t)ceil_div(M, p.gemm.tile) * ceil_div(2 * N, p.gemm.tile), K)) {
    p.copy_x = p.copy_gate = p.copy_up = false;
    p.gemm.regs = true;
  }
  p.stream = p.gemm.tile == 256 && K % 64 == 0 && std::max({ldx, ldg, ldu}) < int64_t(1) << 22;
  p.off_gate = p.copy_x ? up256(padded_bytes(M, K)) : 0;
  p.off_up = p.off_gate + (p.copy_gate ? up256(padded_bytes(N, K)) : 0);
  p.off_gemm = p.off_up + (p.copy_up ? up256(padded_bytes(N, K)) : 0);
  // a column of gate and one of up to each of h, both in whole groups of four
  p.gemm.total = p.gemm.splits > 1 ? (size_t)p.gemm.splits * M * (2 * ((N + 3) / 4 * 4)) * sizeof(float) : 0;
  p.total = p.off_gemm + p.gemm.total;
  return p;
}

hipError_t launch_gated(const GatedArgs& args, const GatedPlan& p, void* ws, hipStream_t st) {
  GatedArgs g = args;
  char* base = static_cast<char*>(ws);
  hipError_t e;
  PadJob jx{}, jg{}, ju{};
  auto copy = [&](PadJob& j, const void*& m, int64_t& ld, int rows, size_t off) {
    j = {m, ld, rows, g.K, base + off};
    m = j.dst;
    ld = up8(g.K);
  };
  if (p.copy_x) copy(jx, g.a, g.lda, g.M, 0);
  if (p.copy_gate) copy(jg, g.b, g.ldb, g.N, p.off_gate);
  if (p.copy_up) copy(ju, g.b2, g.ldb2, g.N, p.off_up);
  if ((e = launch_pad(jx, jg, ju, st)) != hipSuccess) return e;
  if (p.gemm.kind == GemmPlan::kSkinny) {
    // as many columns as share the weights evenly among the CUs
    const int rounds = ceil_div(g.N, 16 * kCUs), cols = std::max(4, ceil_div(g.N, rounds * kCUs));
    hipLaunchKernelGGL(g.type == kElemF16 ? gated_skinny_kernel<true> : gated_skinny_kernel<false>,
                       dim3(ceil_div(g.N, cols)), dim3(64 * kSkinnyWaves), 0, st, g, cols);
    return hipGetLastError();
  }
  if (p.stream) {
    const int mt = ceil_div(g.M, 256), nt = ceil_div(g.N, 128), grid = std::min((mt * nt + 7) / 8 * 8, kCUs);
    return g.type == kElemF16 ? launch_gated_stream_f16(g, grid, mt, nt, st) : launch_gated_stream_bf16(g, grid, mt, nt, st);
  }
  g.regs = p.gemm.regs;
  const GemmSplit s = split_of(p.gemm, 2 * ((g.N + 3) / 4 * 4), base + p.off_gemm);
  e = launch_tiles(g, s, p.gemm.tile, st);
  if (e != hipSuccess || !s.part) return e;
  hipLaunchKernelGGL(gated_join_kernel, dim3((unsigned)((g.M * (s.ld / 8) + 255) / 256)), dim3(256), 0, st, g, s);
  return hipGetLastError();
}

void plan_gated_gradients(int rows, int N, int inner, GemmPlan* dx, GemmPlan* dw) {
  const int wide = 2 * gated_half(N);
  plan_gradients(rows, wide, inner, dx, dw);
  if (dx->paired || dx->tile != 256 || dw->tile != 256) return;
  // 256-row tiles for both: in one launch, those with the longer K first, where together they end sooner by this
  // count of stages ([8192, 5120] x [2560, 5120], 640 tiles of 80 and 400 of 128, 448 stages against 496, 810 us
  // against 870; [12712, 4352] x [1664, 4352] 680 against 735; where the counts are near each other so are the times)
  const int tx = ceil_div(rows, 256) * ceil_div(inner, 256), tw = ceil_div(wide, 256) * ceil_div(inner, 256);
  const int lx = ceil_div(wide, 64), lw = ceil_div(rows, 64);
  const int64_t together = lx >= lw ? pair_stages(tx, lx, tw, lw, kCUs) : pair_stages(tw, lw, tx, lx, kCUs);
  const int64_t apart = (int64_t)ceil_div(tx, kCUs) * lx + (int64_t)ceil_div(tw, kCUs) * lw;
  dx->paired = dw->paired = (double)together < 0.97 * (double)apart;
}

size_t gated_peak_bytes() { return kMaxPeaks * sizeof(uint32_t); }

int gated_dz_units(int M) { return M < 8 ? 1 : M / 4 < 256 ? M / 4 : 256; }

hipError_t launch_gated_dz(const GatedDz& d, PadJobs pad, hipStream_t st) {
  const int units = gated_dz_units(d.M), rows = ceil_div(d.M, units);
  const int wide = ceil_div(gated_half(d.N), 512), wide_peaks = ceil_div(d.N, 512);
  int few = 0;
  auto go = [&](auto dt, auto t) -> hipError_t {
    using DT = decltype(dt);
    using T = decltype(t);
    if (d.dz && std::is_same_v<T, F16>) {
      few = units * wide_peaks <= kMaxPeaks ? units : kMaxPeaks / wide_peaks;  // wide_peaks <= 256
      hipLaunchKernelGGL((gated_peak_kernel<DT, T>), dim3(few * wide_peaks + pad.total()), dim3(64, 4), 0, st, d, few,
                         ceil_div(d.M, few), pad);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      pad = PadJobs{};
    }
    hipLaunchKernelGGL((gated_dz_kernel<DT, T>), dim3(wide * units + pad.total()), dim3(64, 4), 0, st, d, few * wide_peaks,
                       units, rows, pad);
    return hipGetLastError();
  };
  if (d.type == kElemF16) return d.dh_type == kElemF32 ? go(F32{}, F16{}) : go(F16{}, F16{});
  return d.dh_type == kElemF32 ? go(F32{}, BF16{}) : go(BF16{}, BF16{});
}

hipError_t launch_gated_sums(const SumJob& j, hipStream_t st) {
  hipLaunchKernelGGL(gated_sums_kernel, dim3(ceil_div(j.cols, 16)), dim3(256), 0, st, j);
  return hipGetLastError();
}

hipError_t launch_gated_gradients(const GatedArgs& dx, const GemmPlan& px, const GatedArgs& dw, const GemmPlan& pw,
                                  void* ws, hipStream_t st) {
  char* base = static_cast<char*>(ws);
  hipError_t e = hipSuccess;
  if (dx.out && dw.out && px.paired) {
    const GemmSplit sx = split_of(px, dx.N, base), sw = split_of(pw, dw.N, base + px.total);
    e = dx.type == kElemF16 ? launch_gated_pair_f16(dx, sx, dw, sw, px.tile, st)
                            : launch_gated_pair_bf16(dx, sx, dw, sw, px.tile, st);
    return e != hipSuccess ? e : launch_gradient_join(dx, sx, dw, sw, st);
  }
  auto one = [&](const GatedArgs& g, const GemmPlan& p) {
    if (!g.out || e != hipSuccess) return;
    const GemmSplit s = split_of(p, g.N, base);
    e = launch_tiles(g, s, p.tile, st);
    if (e == hipSuccess) e = launch_gradient_join(g, s, g, GemmSplit{}, st);
  };
  one(dx, px);
  one(dw, pw);
  return e;
}

}  // namespace beam
