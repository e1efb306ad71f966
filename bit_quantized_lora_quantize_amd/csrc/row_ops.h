// row_ops.h -- element access and workgroup reductions shared by the kernels
// that work on rows (norm.hip, logits.hip).
#pragma once

#include "qlora.h"
#include "qlora_device.h"

namespace qlora {

// Element types of a row: float or uint16_t (BF16 bits).
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void from_f32(float v, float& out) { out = v; }
__device__ __forceinline__ void from_f32(float v, uint16_t& out) {
  out = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
}

// Sum over a wavefront; every lane gets it.
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int half = 32; half >= 1; half >>= 1) v += __shfl_xor(v, half, 64);
  return v;
}

// Sum over a workgroup of THREADS; every thread gets it.  `lds` holds one
// value per wavefront and may be used again after the next barrier.
template <int THREADS, typename V>
__device__ __forceinline__ V block_sum(V v, V* lds) {
  v = wave_sum(v);
  if constexpr (THREADS == 64) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  V s = lds[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) s += lds[w];
  return s;
}

}  // namespace qlora
