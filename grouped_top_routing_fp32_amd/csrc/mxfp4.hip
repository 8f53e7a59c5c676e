// Microscaled 4-bit floating point: values to codes and scales, and back (gfx950).
//
//   scale = 2^(floor(log2 max |x|) - 2) of each 32,  code = x / scale to the nearest E2M1 value, ties to even, 6 at most
//
// Bound by HBM.  A lane takes 8 elements, 16 bytes of a 16-bit type, and four lanes a block: the largest
// magnitude is found among their bits in two DPP moves, and the codes leave as 4 bytes a lane, both in whole lines.
// [16384, 5120] bf16: to codes 47 to 51 us (212 MB, 4.2 to 4.5 TB/s), back 32 (codes out of the Infinity Cache).
#include "mxfp4.h"

namespace beam {
namespace {

// The largest of four neighbouring lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
}

// The codes of 8 elements and, for all four lanes of a block, its scale byte.
__device__ __forceinline__ uint32_t to_codes(const float* v, uint32_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) top = max(top, __float_as_uint(v[q]) & 0x7fffffffu);
  const uint32_t e = mx_scale_of(quad_max(top));
  *scale = e;
  if (e == 255u) return 0;
  const float s = mx_scale(e);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
}

// The values of 8 codes.
__device__ __forceinline__ void from_codes(uint32_t c, uint32_t e, float* v) {
  const float s = mx_scale(e);
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2), f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
  const float r[8] = {a[0], a[1], b[0], b[1], d[0], d[1], f[0], f[1]};
#pragma unroll
  for (int q = 0; q < 8; ++q) v[q] = r[q];
}

// A workgroup's 256 threads are `wide` (a power of two, from 4 on) along a row and the rest down the
// rows, kRows of them to a thread so that as many loads are in flight.
constexpr int kRows = 4;

template <class T>
__global__ __launch_bounds__(256) void quantize_mx_kernel(const typename T::S* __restrict__ x, int64_t ldx,
                                                          uint8_t* __restrict__ codes, int64_t ldc,
                                                          uint8_t* __restrict__ scales, int64_t lds, int rows, int cols,
                                                          int log_wide) {
  const int wide = 1 << log_wide, down = 256 >> log_wide;
  const int r0 = blockIdx.x * (down * kRows) + (threadIdx.x >> log_wide);
  const int chunks = (cols + kMxBlock - 1) / kMxBlock * 4;
  const int c = blockIdx.y * wide + (threadIdx.x & (wide - 1));
  if (c >= chunks) return;  // with the other three of its block
  Raw8<T> raw[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = r0 + u * down, n = cols - 8 * c;
    if (r < rows && n >= 8)
      raw[u].load(x + (int64_t)r * ldx + 8 * c);
    else
      raw[u].load_part(x + (int64_t)r * ldx + 8 * c, r < rows ? n : 0);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = r0 + u * down;
    if (r >= rows) break;
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = raw[u][q];
    uint32_t e;
    const uint32_t w = to_codes(v, &e);
    *reinterpret_cast<uint32_t*>(codes + (int64_t)r * ldc + 4 * c) = w;
    if (c % 4 == 0) scales[(int64_t)r * lds + c / 4] = (uint8_t)e;
  }
}

template <class T>
__global__ __launch_bounds__(256) void dequantize_mx_kernel(const uint8_t* __restrict__ codes, int64_t ldc,
                                                            const uint8_t* __restrict__ scales, int64_t lds,
                                                            typename T::S* __restrict__ y, int64_t ldy, int rows,
                                                            int cols, int log_wide) {
  const int wide = 1 << log_wide, down = 256 >> log_wide;
  const int r0 = blockIdx.x * (down * kRows) + (threadIdx.x >> log_wide);
  const int c = blockIdx.y * wide + (threadIdx.x & (wide - 1));
  if (8 * c >= cols) return;
  uint32_t w[kRows], e[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = min(r0 + u * down, rows - 1);
    w[u] = *reinterpret_cast<const uint32_t*>(codes + (int64_t)r * ldc + 4 * c);
    e[u] = scales[(int64_t)r * lds + c / 4];
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = r0 + u * down;
    if (r >= rows) break;
    float v[8];
    from_codes(w[u], e[u], v);
    store8<T>(y + (int64_t)r * ldy + 8 * c, cols - 8 * c, v);
  }
}

// f(grid, log_wide) for rows of `chunks` chunks of 8.
template <class F>
hipError_t by_shape(int rows, int chunks, F f) {
  int log_wide = 2;
  while (log_wide < 8 && 1 << log_wide < chunks) ++log_wide;
  const int tall = (256 >> log_wide) * kRows;
  f(dim3((rows + tall - 1) / tall, (chunks + (1 << log_wide) - 1) >> log_wide), log_wide);
  return hipGetLastError();
}

template <class F>
hipError_t by_elem(int type, F f) {
  return type == kElemF32 ? f(F32{}) : type == kElemF16 ? f(F16{}) : f(BF16{});
}

}  // namespace

hipError_t launch_quantize_mx(const void* x, int type, int64_t ldx, uint8_t* codes, int64_t ldc, uint8_t* scales,
                              int64_t lds, int rows, int cols, hipStream_t st) {
  return by_elem(type, [&](auto t) {
    using T = decltype(t);
    return by_shape(rows, (int)mx_blocks(cols) * 4, [&](dim3 grid, int log_wide) {
      hipLaunchKernelGGL((quantize_mx_kernel<T>), grid, dim3(256), 0, st, static_cast<const typename T::S*>(x), ldx,
                         codes, ldc, scales, lds, rows, cols, log_wide);
    });
  });
}

hipError_t launch_dequantize_mx(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, void* y, int type,
                                int64_t ldy, int rows, int cols, hipStream_t st) {
  return by_elem(type, [&](auto t) {
    using T = decltype(t);
    return by_shape(rows, (cols + 7) / 8, [&](dim3 grid, int log_wide) {
      hipLaunchKernelGGL((dequantize_mx_kernel<T>), grid, dim3(256), 0, st, codes, ldc, scales, lds,
                         static_cast<typename T::S*>(y), ldy, rows, cols, log_wide);
    });
  });
}

}  // namespace beam
