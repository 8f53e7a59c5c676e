// Element types of the operators around the block (layer norm, linear and their
// backward passes): storage, loads and stores of 1 or 8 consecutive elements as
// FP32, and wave reductions.
#pragma once

#include "common.h"

namespace beam {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Vectors in global memory that start at any element: this target's wide loads and
// stores need no more than that, so rows of any stride are moved 16 bytes at a time.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// Values of the ABI's element type arguments (BEAM_MOE_BF16, _F16, _F32).
enum ElemType { kElemBF16 = 0, kElemF16 = 1, kElemF32 = 2 };

// Stores round once, to nearest even, in the hardware converters (NaN stays NaN).
struct BF16 {
  using S = uint16_t;
  __device__ static float up(S v) { return __uint_as_float((uint32_t)v << 16); }
  __device__ static S down(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};
struct F16 {
  using S = uint16_t;
  __device__ static float up(S v) { return (float)__builtin_bit_cast(_Float16, v); }
  __device__ static S down(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};
struct F32 {
  using S = float;
  __device__ static float up(S v) { return v; }
  __device__ static S down(float f) { return f; }
};

// Eight consecutive elements as they lie in memory (so that a load can be requested
// before its values are wanted), read as FP32.
template <class T>
struct Raw8 {
  static constexpr int kWords = sizeof(typename T::S) / 2;  // of 16 bytes: 1 or 2
  u32x4 w[kWords];
  __device__ __forceinline__ void load(const typename T::S* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const u32x4_any*>(p)[i];
  }
  // n < 8 elements, zeros after them
  __device__ __forceinline__ void load_part(const typename T::S* p, int n) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (sizeof(typename T::S) == 4)
          w[i / 4][i % 4] = __float_as_uint(p[i]);
        else
          w[0][i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
      }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(typename T::S) == 4)
      return __uint_as_float(w[i / 4][i % 4]);
    else
      return T::up((uint16_t)(w[0][i / 2] >> (16 * (i % 2))));
  }
};

// n >= 8: eight elements, else the first n, and zeros.
template <class T>
__device__ __forceinline__ void load8(const typename T::S* p, int n, float* v) {
  Raw8<T> r;
  if (n >= 8)
    r.load(p);
  else
    r.load_part(p, n);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r[i];
}

template <class T>
__device__ __forceinline__ void store8(typename T::S* p, int n, const float* v) {
  if (n >= 8) {
    if constexpr (sizeof(typename T::S) == 4) {
      reinterpret_cast<f32x4_any*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
      reinterpret_cast<f32x4_any*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      u32x4 r;
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = T::down(v[2 * q]) | ((uint32_t)T::down(v[2 * q + 1]) << 16);
      *reinterpret_cast<u32x4_any*>(p) = r;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = T::down(v[i]);
  }
}

// Sum over each 16 lanes, then over the wave (every lane gets it), in DPP moves and
// readlanes: a tenth of the latency of shuffles through LDS.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float row16_sum(float v) {
  v = dpp_add<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v = dpp_add<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v = dpp_add<0x124>(v);  // row_ror 4
  return dpp_add<0x128>(v);  // row_ror 8
}
__device__ __forceinline__ float wave_sum(float v) {
  const int r = __builtin_bit_cast(int, row16_sum(v));
  const float a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 0));
  const float b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 16));
  const float c = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 32));
  const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 48));
  return (a + b) + (c + d);
}

}  // namespace beam
