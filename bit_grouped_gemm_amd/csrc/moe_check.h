// moe_check.h -- argument checks shared by the ABI of the row-major operators
// (host code only).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <utility>

#include "../../include/moe.h"

namespace moe {

constexpr int kMaxRows = 0x7FFFFFFF - 1023;  // a row count rounded up to a tile stays an int32

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// (pointer, required)
using PtrList = std::initializer_list<std::pair<const void*, bool>>;
inline int null_ptrs(PtrList ps) {
  for (auto& p : ps)
    if (p.second && !p.first) return MOE_ERR_NULL_ARG;
  return MOE_OK;
}
// tensors on 16 bytes, index arrays (a slice of a longer one, say) on 4
inline int misaligned_ptrs(std::initializer_list<const void*> tensors,
                           std::initializer_list<const int32_t*> indices = {}) {
  for (auto p : tensors)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return MOE_ERR_MISALIGNED;
  for (auto p : indices)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

}  // namespace moe
