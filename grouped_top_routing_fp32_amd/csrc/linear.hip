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
#include <algorithm>
#include <type_traits>

#include "linear.h"

namespace beam {

// out from the partial sums of the splits, added in order: four columns to a thread; of one
// product or of two, the first with `blocks` workgroups.
struct JoinJob {
  GemmArgs g;
  GemmSplit s;
};
__global__ __launch_bounds__(256) void gemm_join_kernel(JoinJob first, JoinJob second, int blocks) {
  const bool other = (int)blockIdx.x >= blocks;
  const GemmArgs& g = other ? second.g : first.g;
  const GemmSplit& sp = other ? second.s : first.s;
  const float add = add_of(g);  // requested before the sums, which hide it
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
  by_act(g.act, [&](auto act) { epilogue4<decltype(act)::value>(g, add, m, n, g.N, z); });
}

// Few rows (M <= 16, both operands K contiguous): bound by reading w once, and one CU
// takes no more than some 22 bytes a nanosecond from beyond its L2.  So a workgroup takes
// `cols` <= 16 columns, as many as share w evenly among the CUs; its 16 waves share K in
// pieces of 128, straight from memory into MFMA operands (a wave reads 256 contiguous
// bytes of a row of w; operand rows past cols repeat the last), and their sums are joined
// in LDS in wave order.
constexpr int kSkinnyWaves = 16;

template <bool HALF>
__global__ __launch_bounds__(64 * kSkinnyWaves) void gemm_skinny_kernel(GemmArgs g, int cols) {
  __shared__ f32x4 sum[kSkinnyWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, gr = lane >> 4;
  const int n0 = blockIdx.x * cols, n1 = min(g.N, n0 + cols);
  const uint16_t* wrow = static_cast<const uint16_t*>(g.b) + (int64_t)min(n0 + l16, n1 - 1) * g.ldb;
  const uint16_t* xrow = static_cast<const uint16_t*>(g.a) + (int64_t)min(l16, g.M - 1) * g.lda;
  auto chunk = [&](const uint16_t* row, int k) {  // 8 elements from k, 0 past K
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k + 8 <= g.K) {
      v = *reinterpret_cast<const u32x4_any*>(row + k);
    } else if (k < g.K) {
      Raw8<F16> part;  // the bits alone matter
      part.load_part(row + k, g.K - k);
      v = part.w[0];
    }
    return v;
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  // whole pieces without a test, so that all of their loads are in flight together
  int k = 128 * wave;
  for (; k + 128 <= g.K; k += 128 * kSkinnyWaves) {
    u32x4 fw[4], fx[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      fw[s] = *reinterpret_cast<const u32x4_any*>(wrow + k + 32 * s + 8 * gr);
      fx[s] = *reinterpret_cast<const u32x4_any*>(xrow + k + 32 * s + 8 * gr);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = mfma<HALF>(fw[s], fx[s], acc);
  }
  if (k < g.K) {  // K's last piece, one wave's
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int ks = k + 32 * s + 8 * gr;
      acc = mfma<HALF>(chunk(wrow, ks), chunk(xrow, ks), acc);
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

// Lays one or two operands out anew, the first with `blocks` workgroups of 256 threads and the
// second with the rest: one launch for what a product or both gradients need.  b is the
// workgroup's place among `total`.
struct PadJobs {
  PadJob first, second;
  int blocks, total;
};
__device__ __forceinline__ void pad_rows(const PadJobs& p, int b, int tid) {
  const bool other = b >= p.blocks;
  const PadJob j = other ? p.second : p.first;
  const int64_t threads = 256 * (int64_t)(other ? p.total - p.blocks : p.blocks);
  const int chunks = (j.cols + 7) / 8;
  const int64_t n = (int64_t)j.rows * chunks;
  for (int64_t i = (int64_t)(b - (other ? p.blocks : 0)) * 256 + tid; i < n; i += threads) {
    const int r = (int)(i / chunks), c = (int)(i % chunks) * 8;
    const uint16_t* s = static_cast<const uint16_t*>(j.src) + (int64_t)r * j.ld + c;
    Raw8<F16> v;  // the bits alone matter
    if (c + 8 <= j.cols)
      v.load(s);
    else
      v.load_part(s, j.cols - c);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(j.dst) + 8 * i) = v.w[0];
  }
}

__global__ __launch_bounds__(256) void pad_rows_kernel(PadJobs p) { pad_rows(p, blockIdx.x, threadIdx.x); }

// peaks[g] = the bits of the largest finite |dy| in a workgroup's part, for the scale of an fp16
// dz.  grid ceil(N / 512) * units, block (64, 4), over the rows as in linear_dz_kernel, and behind
// them the workgroups that lay operands out anew, so that those do not wait for it.
constexpr int kMaxPeaks = 1024;
template <class DT>
__global__ __launch_bounds__(256) void linear_peak_kernel(const typename DT::S* __restrict__ dy, int64_t lddy,
                                                          uint32_t* __restrict__ peaks, int M, int N, int units,
                                                          int rows, PadJobs pad) {
  __shared__ uint32_t top[4];
  const int wide = (N + 511) / 512, bx = blockIdx.x % wide, unit = blockIdx.x / wide, y = threadIdx.y;
  if (unit >= units) return pad_rows(pad, blockIdx.x - wide * units, y * 64 + threadIdx.x);
  const int n = (bx * 64 + threadIdx.x) * 8, cols = min(8, N - n);  // <= 0: none
  const int m1 = min(M, (unit + 1) * rows);
  uint32_t best = 0;
  if (cols > 0) {
#pragma unroll 4
    for (int m = unit * rows + y; m < m1; m += 4) {
      float d[8];
      load8<DT>(dy + (int64_t)m * lddy + n, cols, d);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t b = __float_as_uint(d[q]) & 0x7fffffffu;
        best = b < 0x7f800000u && b > best ? b : best;
      }
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, off));
  if (threadIdx.x == 0) top[y] = best;
  __syncthreads();
  if (threadIdx.x == 0 && y == 0) peaks[blockIdx.x] = max(max(top[0], top[1]), max(top[2], top[3]));
}

// The power of two that takes a bound of the finite |dz|, 1.13 |add| max |dy| (no activation's
// slope is larger), into [2^14, 2^15).  Between 2^-126 and 2^126, so that its reciprocal is as
// exact; past those no result fits fp16.  By a whole workgroup of 256.
__device__ __forceinline__ float dz_scale(const uint32_t* __restrict__ peaks, int count, float add) {
  __shared__ uint32_t top[4];
  const int tid = threadIdx.y * 64 + threadIdx.x;
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < kMaxPeaks; i += 256)
    if (i + tid < count) best = max(best, peaks[i + tid]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) best = max(best, (uint32_t)__shfl_xor((int)best, off));
  if (threadIdx.x == 0) top[threadIdx.y] = best;
  __syncthreads();
  best = max(max(top[0], top[1]), max(top[2], top[3]));
  const double bound = 1.13 * fabs((double)add) * __uint_as_float(best);  // inside FP64's range
  if (bound == 0.0) return 1.f;
  const int e = (int)(__builtin_bit_cast(uint64_t, bound) >> 52) - 1022;  // bound < 2^e
  return __uint_as_float((uint32_t)(min(max(15 - e, -126), 126) + 127) << 23);
}

// dz[m, n] = add dy act'(z), rounded to the products' 16-bit type (the rounding that a
// gradient kept between two layers has anyway).  A gradient may well lie below fp16's range or
// above: there dz is held times dz_scale's power of two, whose reciprocal goes to *unscale and
// into the products' results, so that an element is off by half a step, or by 2^-39 of the
// bound, whatever their size.  part[u][n] = the unit's sum of the unscaled,
// unrounded dz; dres = keep dy.  grid ceil(N / 512) * units, block (64, 4): thread (c, r)
// takes 8 columns in rows r, r + 4, ... of the unit.  Behind them the workgroups that lay the
// products' other operands out anew, which would leave most of the card idle in a launch of
// their own.  dz rows are lddz long, a multiple of
// 8, with zeros past N.  Bound by HBM and, with a smooth activation, its arithmetic:
// [8192, 2560] bf16 SiLU 26 us for 126 MB.
template <class DT, class T>
__global__ __launch_bounds__(256) void linear_dz_kernel(const typename DT::S* __restrict__ dy, int64_t lddy,
                                                        const typename T::S* __restrict__ z, int64_t ldz, int act,
                                                        float keep, float add, const uint32_t* __restrict__ peaks,
                                                        int peak_count, float* __restrict__ unscale,
                                                        typename T::S* __restrict__ dz, int64_t lddz, float* __restrict__ part,
                                                        typename DT::S* __restrict__ dres, int64_t lddres, int M, int N,
                                                        int units, int rows, PadJobs pad) {
  __shared__ float sums[4][64][8];
  const int wide = (N + 511) / 512, bx = blockIdx.x % wide, unit = blockIdx.x / wide;
  if (unit >= units) return pad_rows(pad, blockIdx.x - wide * units, threadIdx.y * 64 + threadIdx.x);
  const int n = (bx * 64 + threadIdx.x) * 8, y = threadIdx.y;
  const int cols = min(8, N - n);  // <= 0: none
  const int m1 = min(M, (unit + 1) * rows);
  [[maybe_unused]] float up = 1.f;
  if constexpr (std::is_same_v<T, F16>) {
    if (dz) {
      up = dz_scale(peaks, peak_count, add);
      if (blockIdx.x == 0 && threadIdx.x == 0 && y == 0) *unscale = 1.f / up;
    }
  }
  float s[8] = {};
  if (cols > 0) {
    by_act(act, [&](auto a) {
      constexpr int ACT = decltype(a)::value;
#pragma unroll 4
      for (int m = unit * rows + y; m < m1; m += 4) {
        float d[8], v[8], zz[8] = {};
        load8<DT>(dy + (int64_t)m * lddy + n, cols, d);  // zeros past N
        if constexpr (ACT != kActNone) load8<T>(z + (int64_t)m * ldz + n, cols, zz);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] = add * d[q] * act_slope_f32<ACT>(zz[q]);
          s[q] += v[q];
          d[q] *= keep;
        }
        if (dres) store8<DT>(dres + (int64_t)m * lddres + n, cols, d);
        if constexpr (std::is_same_v<T, F16>) {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] *= up;
        }
        if (dz) store8<T>(dz + (int64_t)m * lddz + n, 8, v);
      }
    });
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) sums[y][threadIdx.x][q] = s[q];
  __syncthreads();
  for (int i = y * 64 + threadIdx.x; i < 512; i += 256) {
    const int c = i / 8, q = i % 8, col = bx * 512 + i;
    if (col < N)
      part[(int64_t)unit * N + col] = (sums[0][c][q] + sums[1][c][q]) + (sums[2][c][q] + sums[3][c][q]);
  }
}

// ---------------------------------------------------------------------------
// plans and launches
// ---------------------------------------------------------------------------
namespace {

constexpr int kBK = 64;  // K per stage of the tiled kernel
constexpr int kCUs = 256;
// Up to here the skinny kernel: 2560 columns, K 5120: 10.4 us at 16 rows against 12.7 in
// tiles; a form of it for 32 rows took 15.9 against 12.8.
constexpr int kSkinnyRows = 16;
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
int ceil_div(int a, int b) { return (a + b - 1) / b; }

constexpr int kMaxSplits = 16;

// Splits of a K of `stages` for `tiles` workgroups where `room` of them run at once.
int splits_of(int tiles, int stages, int room) {
  int s = tiles > 0 && stages >= 24 ? room / tiles : 1;
  s = s < stages / 8 ? s : stages / 8;
  s = s < kMaxSplits ? s : kMaxSplits;
  return s > 1 ? s : 1;
}

void split_plan(GemmPlan& p, int s, int K) {
  p.splits = 1;
  p.k_per_split = K > 0 ? ceil_div(K, kBK) * kBK : kBK;
  if (s > 1) {
    p.k_per_split = ceil_div(ceil_div(K, kBK), s) * kBK;
    p.splits = ceil_div(K, p.k_per_split);
  }
}

size_t split_bytes(const GemmPlan& p, int M, int N) {
  return p.splits > 1 ? up256((size_t)p.splits * M * ((N + 3) / 4 * 4) * sizeof(float)) : 0;
}

// A product of operands whose rows are whole chunks on 16 bytes.
GemmPlan plan_tiles(int M, int N, int K) {
  GemmPlan p{};
  p.kind = GemmPlan::kTiles;
  // The tile is chosen by how full the card's rounds are: a round is 256 workgroups of
  // 256-row tiles (one a CU) or 512 of 128-row ones (two, each filling the other's gaps),
  // and full rounds of the smaller reach 0.85 of the larger's rate up to 24 stages, then
  // 0.8 ([16384, 2560] x [5120, 2560], full rounds of both: 391 us, 465 in 128-row tiles;
  // [8192, 2560] x [2560, 2560], 1.25 rounds and 2.5: 137 and 118; [8192, 1024] x [5120,
  // 1024], 2.5 and 5: 112 and 106, but 220 and 240 with K 2560).  128-row tiles split K until
  // two workgroups a CU have work, in at least 8 stages each; under 24 stages the join costs
  // what a split gains.  64-row tiles where 128-row ones, in as many splits as K allows, make no
  // more than a workgroup a CU ([2048, 1472] x [1024, 1472], 128 of those, 15.2 us against 21.4;
  // [4096, 1024] x [1024, 1024], 256, 16.1 against 17.3; [300, 16384] x [300, 16384], 9 in 16
  // splits, 19.4 against 23.2; [512, 9216] x [512, 9216], 16 in 16, 19.7 against 22.5, but 38.4
  // against 35.3 with K 32768; [2048, 1024] x [2560, 1024], 320, 23.7 against 20.3; [512, 5120] x
  // [2560, 5120], 80 in six, 42 against 28), and for one or two stages, where the result's stores
  // are most of the work ([3000, 128] x [3000, 128] 12.7 us against 15.7).
  const int stages = ceil_div(K, kBK);
  const int t256 = ceil_div(M, 256) * ceil_div(N, 256), t128 = ceil_div(M, 128) * ceil_div(N, 128);
  auto fill = [](int64_t n, int round) { return (double)n / (double)((n + round - 1) / round * round); };
  auto splits = [&](int tiles) { return splits_of(tiles, stages, 2 * kCUs); };
  if (t128 > 1 << 20)  // so large a grid of smaller tiles would pass 2^32 threads
    p.tile = 256;
  else if (stages <= 2 || (int64_t)t128 * (stages >= 24 ? std::min(stages / 8 + 1, kMaxSplits) : 1) <= kCUs)
    p.tile = 64;
  else
    p.tile = fill(t256, kCUs) >= (stages <= 24 ? 0.85 : 0.8) * fill((int64_t)t128 * splits(t128), 2 * kCUs) ? 256 : 128;
  split_plan(p, p.tile == 256 ? 1 : splits(p.tile == 128 ? t128 : ceil_div(M, 64) * ceil_div(N, 64)), K);
  p.total = split_bytes(p, M, N);
  return p;
}
}  // namespace

GemmPlan plan_linear(int M, int N, int K, int64_t ldx, int64_t ldw) {
  if (M <= kSkinnyRows) return GemmPlan{};  // kSkinny
  GemmPlan p = plan_tiles(M, N, K);
  p.copy_a = !regular_rows(ldx, K);
  p.copy_b = !regular_rows(ldw, K);
  // Rows that are no whole chunks go through registers where that costs less than laying them
  // out anew, a launch and their bytes twice: [500, 640] x [1000, 640] 8.0 us against 10.6,
  // [8000, 1401] x [300, 1401], 625 x 22 stages of 64-row tiles, 26.3 against 30.9, but [4000,
  // 1401] x [1000, 1401], 1008 x 22, 38.0 against 30.5, and [8000, 100] x [2500, 100], 5000 x
  // 2, 30.8 against 24.1; [500, 5003] x [2500, 5003], 80 128-row tiles, 34.6 against 39.7, but
  // [1000, 2560] x [2500, 2560], 160, 33.0 against 31.7.
  const int64_t tiles = (int64_t)ceil_div(M, p.tile) * ceil_div(N, p.tile);
  const bool few = p.tile == 64 ? tiles <= 4 * kCUs && tiles * ceil_div(K, kBK) <= 56 * kCUs
                                : p.tile == 128 && tiles <= kCUs / 2;
  if (few && (p.copy_a || p.copy_b)) {
    p.copy_a = p.copy_b = false;
    p.regs = true;
  }
  p.off_b = p.copy_a ? up256(padded_bytes(M, K)) : 0;
  p.off_part = p.off_b + (p.copy_b ? up256(padded_bytes(N, K)) : 0);
  p.total += p.off_part;
  return p;
}

namespace {

hipError_t launch_skinny(const GemmArgs& g, hipStream_t st) {
  // [1, 5120] x [5120, 5120], 320 workgroups of 16 columns 16.5 us, 512 of 10 13.1 us; below
  // 4 columns x is read more often than w
  const int rounds = ceil_div(g.N, 16 * kCUs);
  int cols = ceil_div(g.N, rounds * kCUs);
  cols = cols < 4 ? 4 : cols;
  hipLaunchKernelGGL(g.type == kElemF16 ? gemm_skinny_kernel<true> : gemm_skinny_kernel<false>,
                     dim3(ceil_div(g.N, cols)), dim3(64 * kSkinnyWaves), 0, st, g, cols);
  return hipGetLastError();
}

}  // namespace

static GemmSplit split_of(const GemmArgs& g, const GemmPlan& p, char* base) {
  return {p.splits > 1 ? reinterpret_cast<float*>(base + p.off_part) : nullptr, (g.N + 3) / 4 * 4, p.splits,
          p.k_per_split};
}

// The results of those that were split.
static hipError_t launch_join(const JoinJob& first, const JoinJob& second, hipStream_t st) {
  auto blocks = [](const JoinJob& j) { return j.s.part ? (int)((j.g.M * (j.s.ld / 4) + 255) / 256) : 0; };
  const int a = blocks(first), b = blocks(second);
  if (a + b == 0) return hipSuccess;
  hipLaunchKernelGGL(gemm_join_kernel, dim3(a + b), dim3(256), 0, st, first, second, a);
  return hipGetLastError();
}

static PadJobs pad_jobs(const PadJob& first, const PadJob& second) {
  auto blocks = [](const PadJob& j) {
    const int64_t n = (j.rows * (up8(j.cols) / 8) + 255) / 256;
    return (int)(n < (1 << 20) ? n : 1 << 20);
  };
  const int a = blocks(first), b = blocks(second);
  return {first, second, a, a + b};
}

hipError_t launch_pad(const PadJob& first, const PadJob& second, hipStream_t st) {
  const PadJobs p = pad_jobs(first, second);
  if (p.total == 0) return hipSuccess;
  hipLaunchKernelGGL(pad_rows_kernel, dim3(p.total), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_gemm(const GemmArgs& args, const GemmPlan& p, void* ws, hipStream_t st) {
  GemmArgs g = args;
  char* base = static_cast<char*>(ws);
  hipError_t e;
  PadJob ja{}, jb{};
  if (p.copy_a) {
    ja = {g.a, g.lda, g.M, g.K, base};
    g.a = ja.dst;
    g.lda = up8(g.K);
  }
  if (p.copy_b) {
    jb = {g.b, g.ldb, g.N, g.K, base + p.off_b};
    g.b = jb.dst;
    g.ldb = up8(g.K);
  }
  if ((e = launch_pad(ja, jb, st)) != hipSuccess) return e;
  if (p.kind == GemmPlan::kSkinny) return launch_skinny(g, st);
  g.regs = p.regs;
  const GemmSplit s = split_of(g, p, base);
  e = g.type == kElemF16 ? launch_gemm_f16(g, s, p.tile, st) : launch_gemm_bf16(g, s, p.tile, st);
  return e != hipSuccess ? e : launch_join({g, s}, {}, st);
}

// Stages until n workgroups of `len` stages each and, started after them, m of l <= len are
// done, where `room` run at once.
static int64_t pair_stages(int64_t n, int64_t len, int64_t m, int64_t l) {
  constexpr int64_t room = 2 * kCUs;
  const int64_t rounds = n / room * len, late = n % room, soon = room - late;
  if (late == 0) return rounds + (m + room - 1) / room * l;
  // soon places take the m from the start on, the late ones from len on
  int64_t a = len / l, b = 0, t = len;
  if (m > soon * a + 8 * room) {  // whole rounds of both
    b = (m - soon * a) / room - 4;
    a += b;
    t += b * l;
  }
  while (soon * a + late * b < m) {
    const bool next_soon = (a + 1) * l <= len + (b + 1) * l;
    t = next_soon ? ++a * l : len + ++b * l;
  }
  return rounds + t;
}

void plan_gradients(int rows, int cols, int inner, GemmPlan* dx, GemmPlan* dw) {
  // dz rows are whole chunks with zeros past cols, and the other operands' are made so
  *dx = plan_tiles(rows, inner, cols);
  *dw = plan_tiles(cols, inner, rows);
  if (rows == 0 || rows > 1 << 17 || cols > 1 << 17 || inner > 1 << 17) return;  // far from the tiles' limits
  if (dx->tile == 64 && dw->tile == 64) {
    dx->paired = dw->paired = true;
    return;
  }
  auto tiles = [](int m, int n) { return ceil_div(m, 128) * ceil_div(n, 128); };
  const int tx = tiles(rows, inner), tw = tiles(cols, inner);
  const int lx = ceil_div(cols, kBK), lw = ceil_div(rows, kBK);
  // 128-row tiles for both, and of the splits of both those that end first: a stage is about a
  // microsecond where two workgroups share a CU, a join some 3 and its partial sums' bytes.
  // Gradients of [1000, 2500] x [1700, 2500] 49.7 us one product after the other, 40.2 so; [7000,
  // 640] x [900, 640] 43.8 and 40.7; [3600, 640] x [2560, 640] 46.1 and 37.4.
  auto join = [&](int s, int m) { return s > 1 ? (double)s * m * inner * 8 / 4e6 : 0.; };
  auto cost = [&](int sx, int sw) {
    const int ax = ceil_div(lx, sx), aw = ceil_div(lw, sw);
    const int64_t t = ax >= aw ? pair_stages((int64_t)tx * sx, ax, (int64_t)tw * sw, aw)
                           : pair_stages((int64_t)tw * sw, aw, (int64_t)tx * sx, ax);
    return t + join(sx, rows) + join(sw, cols) + (sx > 1 || sw > 1 ? 3. : 0.);
  };
  constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12};
  int bx = 1, bw = 1;
  double best = 1e30;
  for (int sx : kSplits) {
    if (sx > 1 && (lx < 24 || sx > lx / 8)) break;
    for (int sw : kSplits) {
      if (sw > 1 && (lw < 24 || sw > lw / 8)) break;
      const double c = cost(sx, sw);
      if (c < best) best = c, bx = sx, bw = sw;
    }
  }
  // Where one takes 256-row tiles, which run one to a CU for 1.7 of a 128-row tile's stages (see
  // plan_tiles), both stay as they are unless together they end first by this count, which is
  // good to some 10%: of 23 sizes with 1000 rows and more and cols and inner from 512 on those
  // that counted 0.90 to 0.94 of alone were 0 to 14% faster together and those at 0.945 to 0.99 1
  // to 4% slower, while of 28 with 200 to 700 rows, or cols or inner of 64 to 200, those at 0.94
  // to 0.97 were 24% faster to 3% slower ([2000, 2560] x [4000, 2560], 0.78, 114.6 us by themselves,
  // 89.3 together; [4096, 5120] x [5120, 5120], 0.936, 474 and 433; [35712, 64] x [512, 64], 47.9
  // and 38.9; [8192, 5120] x [2560, 5120], 0.977, 433 and 449).
  if (dx->tile == 256 || dw->tile == 256) {
    auto alone = [&](const GemmPlan& p, int m) {
      const int64_t n = (int64_t)ceil_div(m, p.tile) * ceil_div(inner, p.tile) * p.splits;
      const int64_t room = p.tile == 256 ? kCUs : p.tile == 128 ? 2 * kCUs : 5 * kCUs;  // as LDS holds
      return (double)((n + room - 1) / room) * (p.k_per_split / kBK) * (p.tile == 256 ? 1.7 : 1.) + join(p.splits, m);
    };
    if (best > 0.97 * (alone(*dx, rows) + alone(*dw, cols) + 4.)) return;
  }
  dx->paired = dw->paired = true;
  dx->tile = dw->tile = 128;
  split_plan(*dx, bx, cols);
  split_plan(*dw, bw, rows);
  dx->total = split_bytes(*dx, rows, inner);
  dw->total = split_bytes(*dw, cols, inner);
}

hipError_t launch_gemm_pair(const GemmArgs& dx, const GemmPlan& px, const GemmArgs& dw, const GemmPlan& pw, void* ws,
                            hipStream_t st) {
  if (!px.paired) {
    const hipError_t e = launch_gemm(dx, px, ws, st);
    return e != hipSuccess ? e : launch_gemm(dw, pw, ws, st);
  }
  char* base = static_cast<char*>(ws);
  const GemmSplit sx = split_of(dx, px, base), sw = split_of(dw, pw, base + px.total);
  const hipError_t e = dx.type == kElemF16 ? launch_gemm_pair_f16(dx, sx, dw, sw, px.tile, st)
                                           : launch_gemm_pair_bf16(dx, sx, dw, sw, px.tile, st);
  return e != hipSuccess ? e : launch_join({dx, sx}, {dw, sw}, st);
}

size_t linear_peak_bytes() { return kMaxPeaks * sizeof(uint32_t); }

// Rows of partial sums of dbias: a unit of linear_dz_kernel has 4 rows (one to each row of
// its threads) until there are 256 units.  At 16 rows GELU's arithmetic alone took 10 us
// of [517, 1003].
int linear_dz_units(int M) { return M < 8 ? 1 : M / 4 < 256 ? M / 4 : 256; }

hipError_t launch_linear_dz(const void* dy, int dy_type, int64_t lddy, const void* z, int64_t ldz, int act, float keep,
                            float add, uint32_t* peaks, float* unscale, uint16_t* dz, int64_t lddz, int type,
                            float* part, void* dres, int64_t lddres, int M, int N, const PadJob& first,
                            const PadJob& second, hipStream_t st) {
  const int units = linear_dz_units(M), rows = ceil_div(M, units), wide = ceil_div(N, 512);
  PadJobs pad = pad_jobs(first, second);
  int peak_count = 0;
  if (dz && type == kElemF16) {
    const int few = units * wide <= kMaxPeaks ? units : kMaxPeaks / wide;  // wide <= 512
    peak_count = few * wide;
    auto peak = [&](auto dt) {
      using DT = decltype(dt);
      hipLaunchKernelGGL((linear_peak_kernel<DT>), dim3(peak_count + pad.total), dim3(64, 4), 0, st,
                         static_cast<const typename DT::S*>(dy), lddy, peaks, M, N, few, ceil_div(M, few), pad);
    };
    dy_type == kElemF32 ? peak(F32{}) : peak(F16{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    pad = PadJobs{};
  }
  auto go = [&](auto dt, auto t) {
    using DT = decltype(dt);
    using T = decltype(t);
    hipLaunchKernelGGL((linear_dz_kernel<DT, T>), dim3(wide * units + pad.total), dim3(64, 4), 0, st,
                       static_cast<const typename DT::S*>(dy), lddy, static_cast<const typename T::S*>(z), ldz, act,
                       keep, add, peaks, peak_count, unscale, dz, lddz, part, static_cast<typename DT::S*>(dres),
                       lddres, M, N, units, rows, pad);
  };
  if (type == kElemF16)
    dy_type == kElemF32 ? go(F32{}, F16{}) : go(F16{}, F16{});
  else
    dy_type == kElemF32 ? go(F32{}, BF16{}) : go(BF16{}, BF16{});
  return hipGetLastError();
}

}  // namespace beam
