// pack8.hip -- activations in 8 bits: blocks of 64 values of a row share one
// FP32 scale (gfx950).
//
//   a = max |x| over the block,  scale = RN(a / 127), kept below overflow
//   code = the integer nearest to 127 x / a (ties to even), |code| <= 127
//   restored x = RN_type(RN_fp32(code * scale))
//
// The nearest integer is decided exactly.  t = RN(x * RN(127 / a)) is within
// 2^-23 t of 127 x / a.
//   BF16 x, a: a quotient that is no half integer is 2^-17 t or more away from
//     every one (the difference is a multiple of the last place of x over 2 a,
//     8-bit numbers both).  So t rounded to 20 bits is a half integer where the
//     quotient is one, and on the quotient's side of it elsewhere.
//   FP32: within 4e-5 of a half integer the sign of |127 x - k a| - a / 2 is
//     taken in FP64, where both products (31 and 32 bits) and their difference
//     are exact; where the quotients are spread, one vector of 1500 gets there.
// (In FP64 for every value the kernel was bound by its arithmetic: 44 us for
// 4096 x 11008 BF16.)
//
// Blocks whose a is below 2^-119, where 127 / a leaves FP32's range, restore as
// zeros; a block that holds an infinity or a NaN restores as NaN.
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

constexpr float kTiny = 0x1p-119f;
constexpr float kMostScale = 0x1.020406p+121f;   // the largest whose 127-fold is finite

// Eight neighbouring lanes hold a block, eight values each.  The largest |x| of
// eight lanes', as FP32 bits, of which a NaN's are the largest.
__device__ __forceinline__ uint32_t max8(uint32_t v) {
  // lanes within eight: swap neighbours, pairs, then fours (row_half_mirror)
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  return v;
}

// Integers nearest to 127 x / a of eight values, as FP32.
template <typename T>
__device__ __forceinline__ void nearest_codes(const float* x, float inv, float a, float* k) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = x[j] * inv, c = t * 17.0f;   // 20 of 24 bits kept
      k[j] = __builtin_rintf(c - (c - t));
    }
  } else {
    bool near = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float t = x[j] * inv;
      k[j] = __builtin_rintf(t);
      near |= fabsf(t - k[j]) > 0.5f - 4e-5f;
    }
    if (near) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = 127.0 * (double)x[j] - (double)k[j] * (double)a;
        const double past = 2.0 * fabs(d) - (double)a;
        // past the border, or on it with an odd k
        if (past > 0.0 || (past == 0.0 && ((int)k[j] & 1))) k[j] += d > 0.0 ? 1.0f : -1.0f;
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t col, int64_t d, float* f) {
  if (col + 8 <= d) {
#pragma unroll
    for (int j = 0; j < 8; j += kVec<T>) unpack<T>(load_vec(row + col + j), f + j);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = col + j < d ? to_f32(row[col + j]) : 0.0f;
}

// A workgroup takes 32 rows of four neighbouring blocks, a thread eight values
// of four of the rows (their loads together): 128 bytes of scales of each block
// column are written by one workgroup.
constexpr int kPackRows = 4;

template <typename T>
__global__ __launch_bounds__(256) void k_pack8(const T* __restrict__ X, int64_t M, int64_t d,
                                               uint8_t* __restrict__ codes,
                                               float* __restrict__ scale) {
  const int64_t nb = (d + 63) / 64;
  const int sub = threadIdx.x & 7;              // eight values of the block
  const int bcol = (threadIdx.x >> 3) & 3;      // block within the workgroup's four
  const int rsub = threadIdx.x >> 5;
  const int64_t cgroups = (nb + 3) / 4;
  const int64_t rgroups = (M + 8 * kPackRows - 1) / (8 * kPackRows);
  for (int64_t w = blockIdx.x; w < cgroups * rgroups; w += gridDim.x) {
    const int64_t b = (w % cgroups) * 4 + bcol, m0 = (w / cgroups) * 8 * kPackRows + rsub;
    if (b >= nb) continue;                      // (the same for a block's eight lanes)
    float f[kPackRows][8];
#pragma unroll
    for (int i = 0; i < kPackRows; ++i) {
      const int64_t m = m0 + 8 * i < M ? m0 + 8 * i : M - 1;
      load8(X + m * d, b * 64 + 8 * sub, d, f[i]);
    }
#pragma unroll
    for (int i = 0; i < kPackRows; ++i) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[i][j]) & 0x7FFFFFFFu);
      top = max8(top);
      const float a = __uint_as_float(top);
      float s = fminf(a / 127.0f, kMostScale);
      uint32_t c[2] = {0, 0};
      if (!(a < INFINITY)) {
        s = __uint_as_float(0x7FC00000u);
      } else if (a < kTiny) {
        s = 0.0f;
      } else {
        float k[8];
        nearest_codes<T>(f[i], 127.0f / a, a, k);
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j >> 2] |= ((uint32_t)(int)k[j] & 0xFFu) << (8 * (j & 3));
      }
      const int64_t m = m0 + 8 * i;
      if (m >= M) continue;
      *reinterpret_cast<uint2*>(codes + (m * nb + b) * 64 + 8 * sub) = make_uint2(c[0], c[1]);
      if (sub == 0) scale[b * M + m] = s;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_unpack8(const uint8_t* __restrict__ codes,
                                                 const float* __restrict__ scale, int64_t M,
                                                 int64_t d, T* __restrict__ X) {
  const int64_t nb = (d + 63) / 64;
  const int sub = threadIdx.x & 7, bcol = (threadIdx.x >> 3) & 3, rsub = threadIdx.x >> 5;
  const int64_t cgroups = (nb + 3) / 4;
  const int64_t rgroups = (M + 7) / 8;
  for (int64_t w = blockIdx.x; w < cgroups * rgroups; w += gridDim.x) {
    const int64_t b = (w % cgroups) * 4 + bcol, m = (w / cgroups) * 8 + rsub;
    const int64_t col = b * 64 + 8 * sub;
    if (b >= nb || m >= M || col >= d) continue;
    const uint2 c = *reinterpret_cast<const uint2*>(codes + (m * nb + b) * 64 + 8 * sub);
    const float s = scale[b * M + m];
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = (float)(int8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3))) * s;
    T* row = X + m * d;
    if (col + 8 <= d) {
      if constexpr (sizeof(T) == 2) {
        store_vec(row + col, pack<T>(f));
      } else {
        store_vec(row + col, pack<T>(f));
        store_vec(row + col + 4, pack<T>(f + 4));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < d) from_f32(f[j], row[col + j]);
    }
  }
}

unsigned pack_grid(int64_t M, int64_t d, int rows) {
  const int64_t wgs = ((d + 255) / 256) * ((M + rows - 1) / rows);
  return (unsigned)std::min<int64_t>(wgs, int64_t(1) << 20);
}

}  // namespace

hipError_t launch_pack8(int type, const void* X, int64_t M, int64_t d, uint8_t* codes,
                        float* scale, hipStream_t st) {
  if (type == QLORA_F32)
    hipLaunchKernelGGL(k_pack8<float>, dim3(pack_grid(M, d, 8 * kPackRows)), dim3(256), 0, st,
                       static_cast<const float*>(X), M, d, codes, scale);
  else
    hipLaunchKernelGGL(k_pack8<uint16_t>, dim3(pack_grid(M, d, 8 * kPackRows)), dim3(256), 0, st,
                       static_cast<const uint16_t*>(X), M, d, codes, scale);
  return hipGetLastError();
}

hipError_t launch_unpack8(const uint8_t* codes, const float* scale, int64_t M, int64_t d, int type,
                          void* X, hipStream_t st) {
  if (type == QLORA_F32)
    hipLaunchKernelGGL(k_unpack8<float>, dim3(pack_grid(M, d, 8)), dim3(256), 0, st, codes, scale, M,
                       d, static_cast<float*>(X));
  else
    hipLaunchKernelGGL(k_unpack8<uint16_t>, dim3(pack_grid(M, d, 8)), dim3(256), 0, st, codes, scale,
                       M, d, static_cast<uint16_t*>(X));
  return hipGetLastError();
}

}  // namespace qlora
