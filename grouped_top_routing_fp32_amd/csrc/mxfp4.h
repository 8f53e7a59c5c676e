// Microscaled 4-bit floating point (OCP MX v1.0): E2M1 elements, 32 of them sharing a power of two.
//
// A code's bits are sign, two of exponent (bias 1), one of mantissa: 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Two codes
// to a byte, the first in the low half.  A scale byte e stands for 2^(e - 127), 255 for NaN.
#pragma once

#include "linear.h"

namespace beam {

constexpr int kMxBlock = 32;
typedef float f32x2 __attribute__((ext_vector_type(2)));

inline int64_t mx_blocks(int64_t cols) { return (cols + kMxBlock - 1) / kMxBlock; }

// The scale byte of a block whose largest magnitude has the bits `top` (FP32): 2^(floor(log2) - 2),
// so that the largest lies in [4, 8) of it.  Subnormals are floored to FP32's least normal.  An infinity or NaN
// among the 32 makes it NaN.
__device__ __forceinline__ uint32_t mx_scale_of(uint32_t top) {
  const int e = (int)(top >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

hipError_t launch_quantize_mx(const void* x, int type, int64_t ldx, uint8_t* codes, int64_t ldc, uint8_t* scales,
                              int64_t lds, int rows, int cols, hipStream_t st);
hipError_t launch_dequantize_mx(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, void* y, int type,
                                int64_t ldy, int rows, int cols, hipStream_t st);

// y = keep res + add act(x w^T + bias), w in 4 bits; x of one of the 16-bit types, or in 4 bits too.
struct MxLinear {
  GemmArgs g;                // M, N, K and the epilogue; type is the 16-bit type of x, or of a 16-bit result
  bool four;                 // x is codes
  const void* x;
  int64_t ldx;               // elements; codes: bytes
  const uint8_t* x_scales;
  int64_t ldxs;
  const uint8_t* w;
  int64_t ldw;               // bytes
  const uint8_t* w_scales;
  int64_t ldws;
};
struct MxPlan {
  GemmPlan gemm;
  int rows;                  // of launch_code_rows' tiles; 0: not those
  bool fused;                // codes become x's type on their way into LDS; else:
  bool copy_x;               // x is laid out anew in the workspace, and w as x's type behind it
  size_t off_w, off_gemm, total;
};
MxPlan plan_mx(int M, int N, int K, bool four, int64_t ldx, int64_t ldw);
hipError_t launch_linear_mx(const MxLinear& a, const MxPlan& p, void* ws, hipStream_t st);

}  // namespace beam
