// Argument checks and workspace carving shared by the C ABI's source files.
#pragma once

#include "../../include/beam_moe.h"

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

namespace beam {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename Tp>
Tp* at(void* ws, size_t off) {
  return reinterpret_cast<Tp*>(static_cast<char*>(ws) + off);
}

inline int check_ptrs(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return BEAM_MOE_ERR_INVALID_ARG;
  return BEAM_MOE_OK;
}

// Pointers that may be null.
inline int check_optional(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned16(p)) return BEAM_MOE_ERR_INVALID_ARG;
  return BEAM_MOE_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? BEAM_MOE_OK : BEAM_MOE_ERR_HIP; }

constexpr int64_t kMaxLd = int64_t(1) << 40;  // row offsets stay far inside 64 bits

inline bool type_ok(int t) { return t == BEAM_MOE_BF16 || t == BEAM_MOE_F16 || t == BEAM_MOE_F32; }
inline bool half_type(int t) { return t == BEAM_MOE_BF16 || t == BEAM_MOE_F16; }
inline bool act_ok(int act) { return act >= BEAM_MOE_ACT_NONE && act <= BEAM_MOE_ACT_GELU; }
inline bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxLd; }

// The block's dims and batch size (abi.cpp).
int check_block(const beam_moe_dims* d, int32_t T);

}  // namespace beam
