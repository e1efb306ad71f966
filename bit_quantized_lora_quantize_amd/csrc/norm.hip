// norm.hip -- layer norm and RMS norm over the last axis, forward (with the
// residual addition) and backward (gfx950).
//
//   forward   H = RN(X + R);  Y = (H - mean) * rstd * gamma + beta
//   backward  n = (H - mean) * rstd,  u = dY * gamma,
//             dX = (u - sum(u)/d - n * sum(u n)/d) * rstd + dH,
//             dgamma = sum_rows dY n,  dbeta = sum_rows dY
// with mean = 0 (and no sum(u) term) for the RMS norm.
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

__device__ __forceinline__ float load_w(const void* w, int w_type, int64_t i) {
  return w_type == QLORA_F32 ? static_cast<const float*>(w)[i]
                             : to_f32(static_cast<const uint16_t*>(w)[i]);
}

}  // namespace

// One workgroup per row.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_fwd(NormFwdArgs a) {
  __shared__ float lds[2][4];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.d;
  const T* r = a.r ? static_cast<const T*>(a.r) + row * a.d : nullptr;
  T* h = a.r ? static_cast<T*>(a.h) + row * a.d : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.d;
  const bool layer = a.kind == QLORA_NORM_LAYER;
  float sum = 0.0f;
  for (int64_t i = threadIdx.x; i < a.d; i += 256) {
    float v = to_f32(x[i]);
    if (r) {
      T t;
      from_f32(v + to_f32(r[i]), t);
      h[i] = t;
      v = to_f32(t);
    }
    sum += v;
  }
  const T* s = r ? h : x;
  const float mean = layer ? block_sum<256>(sum, lds[0]) / (float)a.d : 0.0f;
  float sq = 0.0f;
  for (int64_t i = threadIdx.x; i < a.d; i += 256) {
    const float c = to_f32(s[i]) - mean;
    sq += c * c;
  }
  const float var = block_sum<256>(sq, lds[1]) / (float)a.d;
  const float rstd = 1.0f / sqrtf(var + a.eps);
  for (int64_t i = threadIdx.x; i < a.d; i += 256) {
    float v = (to_f32(s[i]) - mean) * rstd * load_w(a.gamma, a.w_type, i);
    if (a.beta) v += load_w(a.beta, a.w_type, i);
    from_f32(v, y[i]);
  }
  if (threadIdx.x == 0) {
    if (a.mean && layer) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_bwd(NormBwdArgs a) {
  __shared__ float lds[2][4];
  const int64_t row = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy) + row * a.d;
  const T* h = static_cast<const T*>(a.h) + row * a.d;
  const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.d : nullptr;
  T* dx = static_cast<T*>(a.dx) + row * a.d;
  const bool layer = a.kind == QLORA_NORM_LAYER;
  const float mean = layer ? a.mean[row] : 0.0f, rstd = a.rstd[row];
  float su = 0.0f, sn = 0.0f;
  for (int64_t i = threadIdx.x; i < a.d; i += 256) {
    const float u = to_f32(dy[i]) * load_w(a.gamma, a.w_type, i);
    su += u;
    sn += u * ((to_f32(h[i]) - mean) * rstd);
  }
  const float mu = layer ? block_sum<256>(su, lds[0]) / (float)a.d : 0.0f;
  const float mn = block_sum<256>(sn, lds[1]) / (float)a.d;
  for (int64_t i = threadIdx.x; i < a.d; i += 256) {
    const float u = to_f32(dy[i]) * load_w(a.gamma, a.w_type, i);
    const float n = (to_f32(h[i]) - mean) * rstd;
    float v = (u - mu - n * mn) * rstd;
    if (dh) v += to_f32(dh[i]);
    from_f32(v, dx[i]);
  }
}

// Weight gradients of one row group: a thread per column.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_wgrad(NormBwdArgs a, int64_t per) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.d) return;
  const int64_t r0 = (int64_t)blockIdx.y * per, r1 = min(a.rows, r0 + per);
  float g = 0.0f, b = 0.0f;
  for (int64_t row = r0; row < r1; ++row) {
    const float mean = a.kind == QLORA_NORM_LAYER ? a.mean[row] : 0.0f;
    const float dy = to_f32(static_cast<const T*>(a.dy)[row * a.d + i]);
    const float n = (to_f32(static_cast<const T*>(a.h)[row * a.d + i]) - mean) * a.rstd[row];
    g += dy * n;
    b += dy;
  }
  a.part[(2 * (int64_t)blockIdx.y) * a.d + i] = g;
  a.part[(2 * (int64_t)blockIdx.y + 1) * a.d + i] = b;
}

__global__ __launch_bounds__(256) void k_norm_wgrad_finish(const float* part, int parts, int64_t d,
                                                           float* dgamma, float* dbeta) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= d) return;
  float g = 0.0f, b = 0.0f;
  for (int p = 0; p < parts; ++p) {
    g += part[(2 * (int64_t)p) * d + i];
    b += part[(2 * (int64_t)p + 1) * d + i];
  }
  if (dgamma) dgamma[i] = g;
  if (dbeta) dbeta[i] = b;
}

int norm_parts(int64_t rows, int64_t) {
  return (int)std::min<int64_t>(rows, 64);
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.rows);
  if (a.type == QLORA_BF16) hipLaunchKernelGGL(k_norm_fwd<uint16_t>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_norm_fwd<float>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st) {
  const unsigned cols = (unsigned)((a.d + 255) / 256);
  int parts = 0;
  if ((a.dgamma || a.dbeta) && a.rows > 0) {
    // before dX, which may overwrite dY
    parts = norm_parts(a.rows, a.d);
    const int64_t per = (a.rows + parts - 1) / parts;
    const dim3 grid(cols, (unsigned)parts);
    if (a.type == QLORA_BF16)
      hipLaunchKernelGGL(k_norm_wgrad<uint16_t>, grid, dim3(256), 0, st, a, per);
    else hipLaunchKernelGGL(k_norm_wgrad<float>, grid, dim3(256), 0, st, a, per);
  }
  if (a.rows > 0) {
    const dim3 grid((unsigned)a.rows);
    if (a.type == QLORA_BF16) hipLaunchKernelGGL(k_norm_bwd<uint16_t>, grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(k_norm_bwd<float>, grid, dim3(256), 0, st, a);
  }
  if (a.dgamma || a.dbeta)
    hipLaunchKernelGGL(k_norm_wgrad_finish, dim3(cols), dim3(256), 0, st, a.part, parts, a.d,
                       a.dgamma, a.dbeta);
  return hipGetLastError();
}

}  // namespace qlora
