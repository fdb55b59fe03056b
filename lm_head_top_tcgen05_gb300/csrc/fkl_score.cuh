// What the scoring operators share: the given tokens, whose ids are 32 or 64 bits wide.
#pragma once

#include <cstdint>

namespace fkl {

struct TokenIds {
  const void* p;
  int32_t bytes;  // 4 or 8
  // The token at `at`, or -1 where it is outside [0, V).
  __device__ __forceinline__ int get(int64_t at, int V) const {
    const int64_t v = bytes == 8 ? static_cast<const int64_t*>(p)[at] : static_cast<const int32_t*>(p)[at];
    return v >= 0 && v < V ? static_cast<int>(v) : -1;
  }
};

}  // namespace fkl
