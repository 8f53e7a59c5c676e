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

// The block's dims and batch size (abi.cpp).
int check_block(const beam_moe_dims* d, int32_t T);

}  // namespace beam
