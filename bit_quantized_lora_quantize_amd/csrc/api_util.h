// api_util.h -- what the host sides of libqlora's entry points (api.cpp,
// api_train.cpp) share: size limits, alignment checks, workspace carving.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "qlora.h"

namespace qlora {

// Layer sizes and token counts per call: every device byte offset the kernels
// form within one tile, split or transposed copy then stays below 2^31.
constexpr int64_t kMaxLinearDim = int64_t(1) << 21;
constexpr int64_t kMaxTokens = int64_t(1) << 21;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? QLORA_OK : QLORA_ERR_HIP; }

// Sequential carving of a workspace into 256-byte aligned pieces; with a null
// base it only measures.
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <class T>
  T* take(int64_t count) {
    off = (off + 255) & ~size_t(255);
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += size_t(std::max<int64_t>(count, 0)) * sizeof(T);
    return p;
  }
};

}  // namespace qlora
