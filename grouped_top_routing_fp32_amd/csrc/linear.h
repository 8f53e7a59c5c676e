// What the kernels of linear.hip share with the ABI: a matrix product's operands
// and its epilogue.
#pragma once

#include <type_traits>

#include "elem.h"

namespace beam {

// Values of the ABI's activation argument (BEAM_MOE_ACT_*).
enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

// out[h] = sum_u part[u][h]; out null: nothing to do.
struct SumJob {
  const float* part;
  float* out;
  int units, cols;
  float* out2;  // the sums of the second half of the columns; null: all go to out
  __device__ void put(int h, float v) const {
    if (out2 && 2 * h >= cols)
      out2[h - cols / 2] = v;
    else
      out[h] = v;
  }
};

// out[m, n] = keep res[m, n] + add act(sum_k a(m, k) b(n, k) + bias[n]), pre[m, n] = the
// activation's argument.  a(m, k) is at a + m * lda + k, or with at (A transposed) at
// a + k * lda + m; b the same with n.  Types are ElemType; a, b and pre share one of two bytes.
struct GemmArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  bool at, bt;
  bool regs;  // the operands, neither transposed, go through registers: rows start at any element
  int M, N, K;
  int type;
  const float* bias;  // null: none
  int act;
  const void* res;  // out's type; null: none
  int64_t ldr;
  float keep, add;
  const float* add_at;  // a gradient's add, on the device; null: add
  void* out;
  int out_type;
  int64_t ldo;
  void* pre;  // null: not written
  int64_t ldp;
  SumJob sums;  // runs beside a product of transposed b alone (dx)
};

// The products of a gated layer.  Forward: b and b2 are both weights, the result act(a b + bias) (a b2 + bias2),
// N its columns, pre and pre2 the two sums.  dx = dz_gate w_gate + dz_up w_up: a holds `half` columns (a multiple of
// 64, zeros past the `valid` of them that are a weight's rows) of dz_gate and then of dz_up, K is 2 half.
// dw: a transposed is the same, out the first half's rows and out2 the second's, `valid` of each.
struct GatedArgs : GemmArgs {
  const void* b2;
  int64_t ldb2;
  const float* bias2;
  void* pre2;
  int64_t ldp2;
  void* out2;
  int64_t ldo2;
  int half, valid;
};

// The product of two operands in microscaled 4 bits, both K contiguous: a, b, their leading dimensions and K count
// units of 16 bits, four codes each; K is whole blocks of 8 units.  A row has a scale byte to a block.
struct MxArgs : GemmArgs {
  const uint8_t *sa, *sb;
  int64_t ldsa, ldsb;
};

// The product of 16-bit rows with weights in microscaled 4 bits: b are the codes, ldb their row stride in bytes, and a
// row has `blocks` of 32 codes and as many scales.
struct CodeArgs : GemmArgs {
  const uint8_t* sb;
  int64_t ldsb;
  int blocks;
};

// Up to here the skinny kernel: 2560 columns, K 5120: 10.4 us at 16 rows against 12.7 in
// tiles; a form of it for 32 rows took 15.9 against 12.8.
constexpr int kSkinnyRows = 16;
constexpr int kSkinnyWaves = 16;
// Workgroups that look for the largest element of an fp16 gradient, at most.
constexpr int kMaxPeaks = 1024;

// How a product runs: which kernel, and the workspace it needs (bytes from its start).
struct GemmPlan {
  enum Kind { kSkinny, kTiles } kind;
  int tile;            // kTiles: 256, 128 or 64, rows and columns of an output tile
  int splits;          // of K; above 1 the partial sums go through the workspace
  int k_per_split;     // multiple of 64
  bool copy_a, copy_b; // the operand is laid out anew in the workspace
  bool regs;           // operands go through registers
  bool paired;         // runs with the other gradient's product
  size_t off_b, off_part, total;  // the first operand lies at the start
};
// Where the partial sums of a product's splits go: [splits][M][ld] (null: one split, the result itself).
struct GemmSplit {
  float* part;
  int64_t ld;  // a multiple of four
  int splits, k_per_split;
};
// Operand shapes and leading dimensions decide alone, so a size query and its call agree.
GemmPlan plan_tiles(int M, int N, int K);  // rows are whole chunks on 16 bytes
// Whether rows that are no whole chunks go through registers: where that costs less than laying them
// out anew, a launch and their bytes twice.  [500, 640] x [1000, 640] 8.0 us against 10.6,
// [8000, 1401] x [300, 1401], 625 x 22 stages of 64-row tiles, 26.3 against 30.9, but [4000,
// 1401] x [1000, 1401], 1008 x 22, 38.0 against 30.5, and [8000, 100] x [2500, 100], 5000 x
// 2, 30.8 against 24.1; [500, 5003] x [2500, 5003], 80 128-row tiles, 34.6 against 39.7, but
// [1000, 2560] x [2500, 2560], 160, 33.0 against 31.7.
bool few_tiles(const GemmPlan& p, int64_t tiles, int K);
GemmPlan plan_linear(int M, int N, int K, int64_t ldx, int64_t ldw);
GemmSplit split_of(const GemmPlan& p, int N, char* base);
hipError_t launch_join_one(const GemmArgs& g, const GemmSplit& s, hipStream_t st);  // where it was split
hipError_t launch_gemm(const GemmArgs& g, const GemmPlan& p, void* ws, hipStream_t st);
// Both gradients' products, planned together.  Where they are paired (run in one launch) their workspaces lie one
// behind the other, dx's first, else in the same place.
void plan_gradients(int rows, int cols, int inner, GemmPlan* dx, GemmPlan* dw);
// Stages until n workgroups of `len` stages each and, started after them, m of l <= len are
// done, where `room` run at once.
int64_t pair_stages(int64_t n, int64_t len, int64_t m, int64_t l, int64_t room);
hipError_t launch_gemm_pair(const GemmArgs& dx, const GemmPlan& px, const GemmArgs& dw, const GemmPlan& pw, void* ws,
                            hipStream_t st);
hipError_t launch_column_sums(const float* part, float* out0, float* out1, int units, int H, hipStream_t st);

// A matrix to be laid out anew: dst rows of up8(cols) elements, zeros past cols.
struct PadJob {
  const void* src;
  int64_t ld;
  int rows, cols;  // rows 0: nothing to do
  void* dst;
};
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
inline int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
// Whether the tiled kernel's copies can take rows as they are: whole chunks of 8 elements on 16 bytes.
inline bool regular_rows(int64_t ld, int cols) { return ld % 8 == 0 && cols % 8 == 0; }
// Up to three operands to be laid out anew in one launch, or in workgroups of 256 threads behind another's: those from
// start[k] to start[k + 1] - 1 have job k.
struct PadJobs {
  PadJob job[3];
  int start[4];
  __host__ __device__ int total() const { return start[3]; }
};
PadJobs pad_jobs(const PadJob& first, const PadJob& second, const PadJob& third);
inline size_t padded_bytes(int rows, int cols) { return (size_t)rows * up8(cols) * 2; }
hipError_t launch_pad(const PadJob& first, const PadJob& second, const PadJob& third, hipStream_t st);
hipError_t launch_gemm_bf16(const GemmArgs& g, const GemmSplit& s, int tile, hipStream_t st);
hipError_t launch_gemm_f16(const GemmArgs& g, const GemmSplit& s, int tile, hipStream_t st);
// In tiles of 64 or 32 rows and 128 columns, K split by 128; rows of a are whole chunks.
hipError_t launch_code_rows(const CodeArgs& g, const GemmSplit& s, int rows, hipStream_t st);
// In tiles of 128 or 64.
hipError_t launch_code_tiles(const CodeArgs& g, const GemmSplit& s, int tile, hipStream_t st);
// The same; `half`: a result of 16 bits is fp16, not bf16.
hipError_t launch_mx_tiles(const MxArgs& g, const GemmSplit& s, int tile, bool half, hipStream_t st);
// In 256-row tiles, with the scales laid out in ws; 256 rows of either operand span less than 2^31 bytes.
size_t mx_stream_bytes(int M, int N, int K);
hipError_t launch_mx_stream(const MxArgs& g, void* ws, hipStream_t st);
hipError_t launch_gated_bf16(const GatedArgs& g, const GemmSplit& s, int tile, hipStream_t st);
hipError_t launch_gated_f16(const GatedArgs& g, const GemmSplit& s, int tile, hipStream_t st);
// A gated layer's forward product in 256-row tiles: K whole stages of 64, strides below 2^22.
hipError_t launch_gated_stream_bf16(const GatedArgs& g, int grid, int mt, int nt, hipStream_t st);
hipError_t launch_gated_stream_f16(const GatedArgs& g, int grid, int mt, int nt, hipStream_t st);
hipError_t launch_gated_pair_bf16(const GatedArgs& dx, const GemmSplit& sx, const GatedArgs& dw, const GemmSplit& sw,
                                  int tile, hipStream_t st);
hipError_t launch_gated_pair_f16(const GatedArgs& dx, const GemmSplit& sx, const GatedArgs& dw, const GemmSplit& sw,
                                 int tile, hipStream_t st);
hipError_t launch_gemm_pair_bf16(const GemmArgs& dx, const GemmSplit& sx, const GemmArgs& dw, const GemmSplit& sw,
                                 int tile, hipStream_t st);
hipError_t launch_gemm_pair_f16(const GemmArgs& dx, const GemmSplit& sx, const GemmArgs& dw, const GemmSplit& sw,
                                int tile, hipStream_t st);

template <bool HALF>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return HALF ? mfma16x16x32_f16(a, b, c) : mfma16x16x32(a, b, c);
}

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 x 16 outputs from 128 codes of each row, a block of 32 to a lane; SA and SB pick the scale's byte.
template <int SA, int SB>
__device__ __forceinline__ f32x4 mfma_mx(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 wa = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 wb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  constexpr int kE2M1 = 4;
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, kE2M1, kE2M1, SA, (int)sa, SB, (int)sb);
}

// A scale byte of 32 codes as the FP32 that the converting instructions take.  They read its exponent field alone: 0
// is 2^-127 to them, and 255 makes every result NaN.
__device__ __forceinline__ float mx_scale(uint32_t e) { return __uint_as_float(e << 23); }

// Eight codes as eight 16-bit values.
template <bool HALF>
__device__ __forceinline__ u32x4 codes_to_16(uint32_t c, float s) {
  if constexpr (HALF)
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3))};
  else
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3))};
}

// 1 / (1 + e^-z) from the hardware base-2 exponential and reciprocal, about 1 ulp each.
// The rounded exponent -z log2 e makes e^-z up to |z| half steps off; the result moves by
// s (1 - s) of that, and z s by at most 0.6 half steps of 1.
__device__ __forceinline__ float sigmoid_f32(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

// The normal distribution function at z, and e^(-z^2 / 2) with it.  At -|z| it is that
// exponential times a polynomial in t = 1 / (1 + 0.35 |z|) (Hastings' form), fitted in 64 bits to
// the scaled complementary error function on |z| <= 14.5, where the exponential vanishes: 4.5e-8
// of itself with these constants, 4e-7 at most as evaluated in FP32, far below zero too, where
// 1 + erf(z / sqrt 2) cancels.  The exponent's two roundings and its constant's add up to three
// half steps of z^2 / 2; below z = -13 the exponential is subnormal.  Fewer instructions than erff
// and expf: [8192, 1024] x [2560, 1024] with GELU 62 us, 68.5 with those, its gradients 135 and 144.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.35f, fabsf(z), 1.f));
  e = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
  float p = -0.029157998f;
  p = fmaf(p, t, 0.14403148f);
  p = fmaf(p, t, -0.255840153f);
  p = fmaf(p, t, 0.159320995f);
  p = fmaf(p, t, -0.0232132431f);
  p = fmaf(p, t, 0.105552875f);
  p = fmaf(p, t, 0.119821198f);
  p = fmaf(p, t, 0.139863521f);
  p = fmaf(p, t, 0.139621302f);
  const float low = p * t * e;
  return z > 0.f ? 1.f - low : low;
}

template <int ACT>
__device__ __forceinline__ float act_f32(float z) {
  if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;  // NaN stays NaN
  if constexpr (ACT == kActSilu) return z * sigmoid_f32(z);
  if constexpr (ACT == kActGelu) {
    float e;
    return z * normal_cdf(z, e);
  }
  return z;
}

// The same with the limit 0 at minus infinity, where SiLU's and GELU's factor z meets a 0: z is held from -128 on, where
// that factor has been 0 for long (the same bits for every finite z).  NaN comes through sigmoid or distribution function.
template <int ACT>
__device__ __forceinline__ float act_limit_f32(float z) {
  const float f = fmaxf(z, -128.f);
  if constexpr (ACT == kActSilu) return f * sigmoid_f32(z);
  if constexpr (ACT == kActGelu) {
    float e;
    return f * normal_cdf(z, e);
  }
  return act_f32<ACT>(z);
}

// d act / dz.  The factor z is held within +-128, where what it multiplies is 0 or takes the
// rest to 0, so that an infinite z (a pre past fp16's range) has the slope's limit, 0 or 1, and
// not 0 times infinity.  NaN comes through sigmoid or distribution function.
template <int ACT>
__device__ __forceinline__ float act_slope_f32(float z) {
  const float f = __builtin_amdgcn_fmed3f(z, -128.f, 128.f);
  if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid_f32(z);
    return s * (1.f + f * (1.f - s));
  }
  if constexpr (ACT == kActGelu) {
    float e;
    const float cdf = normal_cdf(z, e);
    return fmaf(f * 0.39894228040143268f, e, cdf);
  }
  return 1.f;
}

// f(integral_constant<int, act>) for a run-time activation.
template <class F>
__device__ __forceinline__ void by_act(int act, F f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    default: f(std::integral_constant<int, kActNone>{});
  }
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int type) {
  if (type == kElemF32) return static_cast<const float*>(p)[i];
  const uint16_t v = static_cast<const uint16_t*>(p)[i];
  return type == kElemBF16 ? BF16::up(v) : F16::up(v);
}

__device__ __forceinline__ void store_elem(void* p, int64_t i, int type, float f) {
  if (type == kElemF32)
    static_cast<float*>(p)[i] = f;
  else
    static_cast<uint16_t*>(p)[i] = type == kElemBF16 ? BF16::down(f) : F16::down(f);
}

// Four consecutive elements from any one.
__device__ __forceinline__ f32x4 load_elem4(const void* p, int64_t i, int type) {
  if (type == kElemF32) return *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + i);
  const u32x2 r = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(p) + i);
  f32x4 v;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint16_t h = (uint16_t)(r[q / 2] >> (16 * (q % 2)));
    v[q] = type == kElemBF16 ? BF16::up(h) : F16::up(h);
  }
  return v;
}

__device__ __forceinline__ void store_elem4(void* p, int64_t i, int type, f32x4 v) {
  if (type == kElemF32) {
    *reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + i) = v;
    return;
  }
  uint32_t h[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) h[q] = type == kElemBF16 ? BF16::down(v[q]) : F16::down(v[q]);
  *reinterpret_cast<u32x2_any*>(static_cast<uint16_t*>(p) + i) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
}

// The power of two that takes a bound of the finite |dz|, `times` the largest of the values whose
// bits are in peaks, into [2^14, 2^15).  Between 2^-126 and 2^126, so that its reciprocal is as
// exact; past those no result fits fp16.  By a whole workgroup of 256.
__device__ __forceinline__ float dz_scale(const uint32_t* __restrict__ peaks, int count, double times) {
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
  const double bound = times * __uint_as_float(best);  // inside FP64's range
  if (bound == 0.0) return 1.f;
  const int e = (int)(__builtin_bit_cast(uint64_t, bound) >> 52) - 1022;  // bound < 2^e
  return __uint_as_float((uint32_t)(min(max(15 - e, -126), 126) + 127) << 23);
}

// b is the workgroup's place among the jobs'.
__device__ __forceinline__ void pad_rows(const PadJobs& p, int b, int tid) {
  const int k = (b >= p.start[1]) + (b >= p.start[2]);
  const PadJob j = k == 0 ? p.job[0] : k == 1 ? p.job[1] : p.job[2];
  const int first = k == 0 ? 0 : k == 1 ? p.start[1] : p.start[2];
  const int64_t threads = 256 * (int64_t)((k == 0 ? p.start[1] : k == 1 ? p.start[2] : p.start[3]) - first);
  const int chunks = (j.cols + 7) / 8;
  const int64_t n = (int64_t)j.rows * chunks;
  for (int64_t i = (int64_t)(b - first) * 256 + tid; i < n; i += threads) {
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

// Eight elements of a row of K from k on, zeros past K.
__device__ __forceinline__ u32x4 chunk_of_row(const uint16_t* row, int k, int K) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k + 8 <= K) {
    v = *reinterpret_cast<const u32x4_any*>(row + k);
  } else if (k < K) {
    Raw8<F16> part;  // the bits alone matter
    part.load_part(row + k, K - k);
    v = part.w[0];
  }
  return v;
}

// The column sums that run beside dx's product, in workgroups behind its tiles: b's are those
// of 16 columns, thread (c, g) adds the rows g, g + 16, ... of column c, and a column's 16
// sums are added in order, in FP64.  As a launch of their own they take 3 to 5 us, mostly
// latency.
__device__ __forceinline__ void sum_columns(float* s, const SumJob& j, int b) {
  const int tid = threadIdx.x, c = tid & 15, h = b * 16 + c;
  float v = 0.f;
  if (tid < 256 && h < j.cols)
#pragma unroll 16
    for (int u = tid >> 4; u < j.units; u += 16) v += j.part[(int64_t)u * j.cols + h];
  s[tid] = v;
  __syncthreads();
  if (tid < 16 && h < j.cols) {
    double a = 0.0;
#pragma unroll
    for (int g = 0; g < 16; ++g) a += s[16 * g + c];
    j.put(h, (float)a);
  }
}
// A product's `add`; read once, before its results.
__device__ __forceinline__ float add_of(const GemmArgs& g) { return g.add_at ? *g.add_at : g.add; }

// One element of the result from its sum over k.
template <int ACT>
__device__ __forceinline__ void epilogue1(const GemmArgs& g, float add, int m, int n, float z) {
  if (g.bias) z += g.bias[n];
  if (g.pre) store_elem(g.pre, (int64_t)m * g.ldp + n, g.type, z);
  float v = add * act_f32<ACT>(z);
  if (g.res) v += g.keep * load_elem(g.res, (int64_t)m * g.ldr + n, g.out_type);
  store_elem(g.out, (int64_t)m * g.ldo + n, g.out_type, v);
}

// Columns n .. n + 3 of row m, those from `end` on left alone.
template <int ACT>
__device__ __forceinline__ void epilogue4(const GemmArgs& g, float add, int m, int n, int end, f32x4 z) {
  if (n + 4 <= end) {
    if (g.bias) {
      const f32x4 b = *reinterpret_cast<const f32x4_any*>(g.bias + n);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] += b[q];
    }
    if (g.pre) store_elem4(g.pre, (int64_t)m * g.ldp + n, g.type, z);
    f32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = add * act_f32<ACT>(z[q]);
    if (g.res) {
      const f32x4 r = load_elem4(g.res, (int64_t)m * g.ldr + n, g.out_type);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += g.keep * r[q];
    }
    store_elem4(g.out, (int64_t)m * g.ldo + n, g.out_type, v);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < end) epilogue1<ACT>(g, add, m, n + q, z[q]);
  }
}

// The same of a gradient, which has the sums alone.
__device__ __forceinline__ void gradient4(const GemmArgs& g, float add, int m, int n, f32x4 z);

// A gated layer's: rows of dw belong to either weight, those of dz's filling to none.
__device__ __forceinline__ void gradient4(const GatedArgs& g, float add, int m, int n, f32x4 z) {
  GemmArgs of = g;
  if (g.at) {
    if (m >= g.half) {
      m -= g.half;
      of.out = g.out2;
      of.ldo = g.ldo2;
    }
    if (m >= g.valid) return;
  }
  gradient4(of, add, m, n, z);
}

__device__ __forceinline__ void gradient4(const GemmArgs& g, float add, int m, int n, f32x4 z) {
#pragma unroll
  for (int q = 0; q < 4; ++q) z[q] *= add;
  const int64_t i = (int64_t)m * g.ldo + n;
  if (n + 4 <= g.N) {
    store_elem4(g.out, i, g.type, z);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < g.N) store_elem(g.out, i + q, g.type, z[q]);
  }
}

}  // namespace beam
