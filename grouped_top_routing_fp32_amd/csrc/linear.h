// What the kernels of linear.hip share with the ABI: a matrix product's operands
// and its epilogue.
#pragma once

#include "elem.h"

namespace beam {

// Values of the ABI's activation argument (BEAM_MOE_ACT_*).
enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

// out[m, n] = keep res[m, n] + add act(sum_k a(m, k) b(n, k) + bias[n]), pre[m, n] = the
// activation's argument.  a(m, k) is at a + m * lda + k, or with at at a + k * lda + m;
// b the same with n.  Types are ElemType; a, b and pre share one of two bytes.
struct GemmArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  bool at, bt;
  int M, N, K;
  int type;
  const float* bias;  // null: none
  int act;
  const void* res;  // out's type; null: none
  int64_t ldr;
  float keep, add;
  void* out;
  int out_type;
  int64_t ldo;
  void* pre;  // null: not written
  int64_t ldp;
};

__device__ __forceinline__ float act_f32(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case kActSilu: return z / (1.f + expf(-z));
    case kActGelu: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    default: return z;
  }
}

// d act / dz
__device__ __forceinline__ float act_slope_f32(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f ? 1.f : 0.f;
    case kActSilu: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    case kActGelu:
      return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.39894228040143268f * expf(-0.5f * z * z);
    default: return 1.f;
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

// One element of the result from its sum over k.
__device__ __forceinline__ void epilogue(const GemmArgs& g, int m, int n, float z) {
  if (g.bias) z += g.bias[n];
  if (g.pre) store_elem(g.pre, (int64_t)m * g.ldp + n, g.type, z);
  float v = g.add * act_f32(z, g.act);
  if (g.res) v += g.keep * load_elem(g.res, (int64_t)m * g.ldr + n, g.out_type);
  store_elem(g.out, (int64_t)m * g.ldo + n, g.out_type, v);
}

}  // namespace beam
