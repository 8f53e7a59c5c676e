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
GemmPlan plan_linear(int M, int N, int K, int64_t ldx, int64_t ldw);
hipError_t launch_gemm(const GemmArgs& g, const GemmPlan& p, void* ws, hipStream_t st);
// Both gradients' products, planned together.  Where they are paired (run in one launch) their workspaces lie one
// behind the other, dx's first, else in the same place.
void plan_gradients(int rows, int cols, int inner, GemmPlan* dx, GemmPlan* dw);
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
inline int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
// Whether the tiled kernel's copies can take rows as they are: whole chunks of 8 elements on 16 bytes.
inline bool regular_rows(int64_t ld, int cols) { return ld % 8 == 0 && cols % 8 == 0; }
inline size_t padded_bytes(int rows, int cols) { return (size_t)rows * up8(cols) * 2; }
hipError_t launch_pad(const PadJob& first, const PadJob& second, hipStream_t st);
hipError_t launch_gemm_bf16(const GemmArgs& g, const GemmSplit& s, int tile, hipStream_t st);
hipError_t launch_gemm_f16(const GemmArgs& g, const GemmSplit& s, int tile, hipStream_t st);
hipError_t launch_gemm_pair_bf16(const GemmArgs& dx, const GemmSplit& sx, const GemmArgs& dw, const GemmSplit& sw,
                                 int tile, hipStream_t st);
hipError_t launch_gemm_pair_f16(const GemmArgs& dx, const GemmSplit& sx, const GemmArgs& dw, const GemmSplit& sw,
                                int tile, hipStream_t st);

template <bool HALF>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return HALF ? mfma16x16x32_f16(a, b, c) : mfma16x16x32(a, b, c);
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
