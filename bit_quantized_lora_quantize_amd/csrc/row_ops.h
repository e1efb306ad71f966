// row_ops.h -- element access and reductions shared by the kernels that work
// on rows (norm.hip, logits.hip).
//
// Rows are taken in 16-byte vectors that need not be aligned: a row of odd
// length starts anywhere, and one wavefront's access still covers 1 KB without
// gaps.  Measured on 65536-element BF16 rows, a read and a copy run as fast at
// 4-byte alignment as at 16-byte; off it, a read loses 17 % (5.8 to 4.8 TB/s).
// Rows of logits therefore start their vectors at the first 4-byte boundary
// (RowCut).
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

// Elements of a 16-byte vector.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// A 16-byte vector at the alignment of an element.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
template <typename T>
struct VecAt {
  typedef u32x4_at4 type;
};
template <>
struct VecAt<uint16_t> {
  typedef u32x4_at2 type;
};
template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T* p) {
  return *reinterpret_cast<const typename VecAt<T>::type*>(p);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, u32x4 v) {
  *reinterpret_cast<typename VecAt<T>::type*>(p) = v;
}
// The same past the caches' retention, for data that no kernel here reads
// again.
template <typename T>
__device__ __forceinline__ u32x4 load_vec_once(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const typename VecAt<T>::type*>(p));
}
template <typename T>
__device__ __forceinline__ void store_vec_once(T* p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<typename VecAt<T>::type*>(p));
}

template <typename T>
__device__ __forceinline__ void unpack(u32x4 v, float* f) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16lo_to_f32(v[j]);
      f[2 * j + 1] = bf16hi_to_f32(v[j]);
    }
  }
}
template <typename T>
__device__ __forceinline__ u32x4 pack(const float* f) {
  u32x4 v;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
  }
  return v;
}

// A row of `size` elements as `nvec` vectors from element `head` on and single
// elements for the first lanes: `edge` is the calling lane's, -1 without.
template <typename T>
struct RowCut {
  int head, nvec, edge;
  __device__ __forceinline__ RowCut(const T* p, int size, int lane) {
    head = sizeof(T) == 2 ? (int)(reinterpret_cast<uintptr_t>(p) >> 1 & 1) : 0;
    const int body = size - head;
    nvec = body / kVec<T>;
    const int tail = body - nvec * kVec<T>;
    edge = lane < tail ? size - tail + lane : (lane == tail && head ? 0 : -1);
  }
  // The first element of vector v.
  __device__ __forceinline__ int at(int v) const { return head + v * kVec<T>; }
};

// A vector of -inf.
template <typename T>
__device__ __forceinline__ u32x4 vec_neg_inf() {
  const uint32_t w = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
  return u32x4{w, w, w, w};
}

// Values moved between the lanes of a wavefront inside the VALU (data-parallel
// primitives): lane i takes lane i - 1, 2, 4 or 8 of its row of 16, then rows
// 1 and 3 take lane 15 of the row before them and rows 2 and 3 lane 31.  Lanes
// without a source take `none`.  After the six steps lane 63 has combined all.
constexpr int kRowShr1 = 0x111, kRowShr2 = 0x112, kRowShr4 = 0x114, kRowShr8 = 0x118;
constexpr int kRowBcast15 = 0x142, kRowBcast31 = 0x143;

template <int CTRL, int ROWS, typename V>
__device__ __forceinline__ V lane_move(V none, V v) {
  constexpr int W = sizeof(V) / 4;
  struct Words {
    int w[W];
  };
  const Words n = __builtin_bit_cast(Words, none);
  Words x = __builtin_bit_cast(Words, v);
#pragma unroll
  for (int i = 0; i < W; ++i)
    x.w[i] = __builtin_amdgcn_update_dpp(n.w[i], x.w[i], CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(V, x);
}
template <typename V>
__device__ __forceinline__ V from_lane(V v, int lane) {
  constexpr int W = sizeof(V) / 4;
  struct Words {
    int w[W];
  };
  Words x = __builtin_bit_cast(Words, v);
#pragma unroll
  for (int i = 0; i < W; ++i) x.w[i] = __builtin_amdgcn_readlane(x.w[i], lane);
  return __builtin_bit_cast(V, x);
}

// Sum over a wavefront, all of whose lanes are active; every lane gets it.
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
  v += lane_move<kRowShr1, 0xF>(V(0), v);
  v += lane_move<kRowShr2, 0xF>(V(0), v);
  v += lane_move<kRowShr4, 0xF>(V(0), v);
  v += lane_move<kRowShr8, 0xF>(V(0), v);
  v += lane_move<kRowBcast15, 0xA>(V(0), v);
  v += lane_move<kRowBcast31, 0xC>(V(0), v);
  return from_lane(v, 63);
}
// Sum over the first 16 lanes; every lane gets it.
template <typename V>
__device__ __forceinline__ V row16_sum(V v) {
  v += lane_move<kRowShr1, 0xF>(V(0), v);
  v += lane_move<kRowShr2, 0xF>(V(0), v);
  v += lane_move<kRowShr4, 0xF>(V(0), v);
  v += lane_move<kRowShr8, 0xF>(V(0), v);
  return from_lane(v, 15);
}
__device__ __forceinline__ float wave_max(float v) {
  const float none = -__builtin_huge_valf();
  v = fmaxf(v, lane_move<kRowShr1, 0xF>(none, v));
  v = fmaxf(v, lane_move<kRowShr2, 0xF>(none, v));
  v = fmaxf(v, lane_move<kRowShr4, 0xF>(none, v));
  v = fmaxf(v, lane_move<kRowShr8, 0xF>(none, v));
  v = fmaxf(v, lane_move<kRowBcast15, 0xA>(none, v));
  v = fmaxf(v, lane_move<kRowBcast31, 0xC>(none, v));
  return from_lane(v, 63);
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
template <int THREADS>
__device__ __forceinline__ float block_max(float v, float* lds) {
  v = wave_max(v);
  if constexpr (THREADS == 64) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float m = lds[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) m = fmaxf(m, lds[w]);
  return m;
}

}  // namespace qlora
