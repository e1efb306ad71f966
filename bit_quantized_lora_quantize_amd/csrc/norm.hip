// norm.hip -- layer norm and RMS norm over the last axis, forward (with the
// residual addition) and backward (gfx950).
//
//   forward   H = RN(X + R);  Y = (H - mean) * rstd * gamma + beta
//   backward  n = (H - mean) * rstd,  u = dY * gamma,
//             dX = (u - sum(u)/d - n * sum(u n)/d) * rstd + dH,
//             dgamma = sum_rows dY n,  dbeta = sum_rows dY
// with mean = 0 (and no sum(u) term) for the RMS norm.
//
// Every kernel is bound by memory.  A row is held in the registers of the
// ROW threads that own it, E values each, so every array is read once; the
// variance is summed from the centred values, which costs no second read.
// ROW and E are the smallest that hold the row (by_width); wider rows take
// the looping kernels below, which read them again from the caches.
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

__device__ __forceinline__ float load_w(const void* w, int w_type, int64_t i) {
  return w_type == QLORA_F32 ? static_cast<const float*>(w)[i]
                             : to_f32(static_cast<const uint16_t*>(w)[i]);
}

// N weights from element i on.
template <int N>
__device__ __forceinline__ void load_w_vec(const void* w, int w_type, int64_t i, float* f) {
  if (w_type == QLORA_F32) {
    const float* p = static_cast<const float*>(w) + i;
#pragma unroll
    for (int q = 0; q < N / 4; ++q) unpack<float>(load_vec(p + 4 * q), f + 4 * q);
  } else if constexpr (N == 8) {
    unpack<uint16_t>(load_vec(static_cast<const uint16_t*>(w) + i), f);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = to_f32(static_cast<const uint16_t*>(w)[i + j]);
  }
}

// The part of a row that one of its ROW threads holds: V vectors, ROW apart,
// and at most one element of the last, partial vector (`rest`, -1 without).
template <typename T, int ROW, int E>
struct Part {
  static constexpr int N = kVec<T>, V = E / N;
  int lane, nvec, rest;
  __device__ __forceinline__ Part(int thread, int d) {
    lane = thread;
    nvec = d / N;
    const int i = nvec * N + thread;
    rest = i < d ? i : -1;
  }
  __device__ __forceinline__ bool has(int q) const { return lane + q * ROW < nvec; }
  __device__ __forceinline__ int64_t at(int q) const { return (int64_t)(lane + q * ROW) * N; }
};

template <bool ONCE, typename T, int ROW, int E>
__device__ __forceinline__ void load_part(const Part<T, ROW, E>& p, const T* x, u32x4* v, T& rest) {
#pragma unroll
  for (int q = 0; q < Part<T, ROW, E>::V; ++q) {
    v[q] = u32x4{0, 0, 0, 0};
    if (p.has(q)) v[q] = ONCE ? load_vec_once(x + p.at(q)) : load_vec(x + p.at(q));
  }
  rest = T(0);
  if (p.rest >= 0) rest = x[p.rest];
}

template <bool ONCE, typename T>
__device__ __forceinline__ void put_vec(T* p, u32x4 v) {
  if constexpr (ONCE) store_vec_once(p, v);
  else store_vec(p, v);
}

// The weights of a thread's part (0 past the row's end).
template <typename T, int ROW, int E>
__device__ __forceinline__ void weight_part(const Part<T, ROW, E>& p, const void* w, int w_type,
                                            float* f, float& rest) {
  constexpr int N = Part<T, ROW, E>::N;
#pragma unroll
  for (int q = 0; q < Part<T, ROW, E>::V; ++q) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[q * N + j] = 0.0f;
    if (p.has(q)) load_w_vec<N>(w, w_type, p.at(q), f + q * N);
  }
  rest = p.rest >= 0 ? load_w(w, w_type, p.rest) : 0.0f;
}

// Sums over the ROW threads of each row of a workgroup; the rows of a
// workgroup go through it together.
template <int ROW, int THREADS, int COUNT>
__device__ __forceinline__ void row_sums(float (&v)[COUNT], float (*lds)[COUNT]) {
#pragma unroll
  for (int c = 0; c < COUNT; ++c) v[c] = wave_sum(v[c]);
  if constexpr (ROW > 64) {
    constexpr int W = ROW / 64;
    const int wave = threadIdx.x / 64;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int c = 0; c < COUNT; ++c) lds[wave][c] = v[c];
    }
    __syncthreads();
    const int first = wave / W * W;
#pragma unroll
    for (int c = 0; c < COUNT; ++c) {
      v[c] = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[c] += lds[first + w][c];
    }
  }
}

// The sums of a workgroup's row groups, added in order, as one row of d
// partials: four columns a thread at a time, the groups meeting in LDS.
template <typename T, int ROW, int E, int THREADS>
__device__ __forceinline__ void write_partial(const Part<T, ROW, E>& p, int group, const float* v,
                                              float rest, float* part) {
  constexpr int G = THREADS / ROW, N = kVec<T>;
  if constexpr (G == 1) {
#pragma unroll
    for (int c = 0; c < E / 4; ++c)
      if (p.has(4 * c / N)) store_vec(part + p.at(4 * c / N) + 4 * c % N, pack<float>(v + 4 * c));
    if (p.rest >= 0) part[p.rest] = rest;
  } else {
    __shared__ f32x4 sum[THREADS];
#pragma unroll
    for (int c = 0; c <= E / 4; ++c) {
      const bool last = c == E / 4;            // the partial vector's element
      __syncthreads();
      if (last) sum[threadIdx.x].x = rest;
      else sum[threadIdx.x] = __builtin_bit_cast(f32x4, pack<float>(v + 4 * c));
      __syncthreads();
      if (group) continue;
      f32x4 t = sum[p.lane];
#pragma unroll
      for (int k = 1; k < G; ++k) t += sum[k * ROW + p.lane];
      if (last) {
        if (p.rest >= 0) part[p.rest] = t.x;
      } else if (p.has(4 * c / N)) {
        store_vec(part + p.at(4 * c / N) + 4 * c % N, __builtin_bit_cast(u32x4, t));
      }
    }
  }
}

constexpr int kBwdThreads = 1024;
constexpr int kFinishCols = 16;
// Arrays of this size and more go past the caches' retention: the two to four
// of a call would drive each other out of the 256 MB of the last level anyway.
// Backward of 16384 x 8192 BF16: 199 us kept, 187 us past; smaller outputs stay
// for the layer that reads them next.
constexpr int64_t kOnceBytes = int64_t(128) << 20;

}  // namespace

// THREADS / ROW rows per workgroup, each by ROW of its threads.
template <typename T, int ROW, int E, int THREADS, bool ONCE>
__global__ __launch_bounds__(THREADS) void k_norm_fwd(NormFwdArgs a) {
  __shared__ float lds[2][THREADS / 64][1];
  const int64_t row = (int64_t)blockIdx.x * (THREADS / ROW) + threadIdx.x / ROW;
  const bool live = row < a.rows;
  const int64_t base = (live ? row : a.rows - 1) * a.d;
  const Part<T, ROW, E> p(threadIdx.x % ROW, (int)a.d);
  constexpr int N = Part<T, ROW, E>::N, V = Part<T, ROW, E>::V;
  u32x4 v[V];
  T rest;
  load_part<ONCE>(p, static_cast<const T*>(a.x) + base, v, rest);
  float h[E], hr;
  if (a.r) {
    u32x4 w[V];
    T rr;
    load_part<ONCE>(p, static_cast<const T*>(a.r) + base, w, rr);
    T* out = static_cast<T*>(a.h) + base;
    float f[N];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      unpack<T>(v[q], h + q * N);
      unpack<T>(w[q], f);
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] += h[q * N + j];
      v[q] = pack<T>(f);                       // the one rounding of H
      if (live && p.has(q)) put_vec<ONCE>(out + p.at(q), v[q]);
    }
    from_f32(to_f32(rest) + to_f32(rr), rest);
    if (live && p.rest >= 0) out[p.rest] = rest;
  }
  float g[E], b[E], gr, br = 0.0f;
  weight_part(p, a.gamma, a.w_type, g, gr);
  if (a.beta) {
    weight_part(p, a.beta, a.w_type, b, br);
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) b[j] = 0.0f;
  }
#pragma unroll
  for (int q = 0; q < V; ++q) unpack<T>(v[q], h + q * N);
  hr = to_f32(rest);
  const float inv = 1.0f / (float)a.d;
  float mean = 0.0f;
  if (a.kind == QLORA_NORM_LAYER) {
    float s[1] = {hr};                         // 0 in threads without a rest
#pragma unroll
    for (int j = 0; j < E; ++j) s[0] += h[j];
    row_sums<ROW, THREADS>(s, lds[0]);
    mean = s[0] * inv;
    hr -= mean;
#pragma unroll
    for (int j = 0; j < E; ++j) h[j] -= mean;
  }
  float s[1] = {p.rest >= 0 ? hr * hr : 0.0f};
#pragma unroll
  for (int q = 0; q < V; ++q) {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) t += h[q * N + j] * h[q * N + j];
    if (p.has(q)) s[0] += t;
  }
  row_sums<ROW, THREADS>(s, lds[1]);
  const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
  if (!live) return;
  T* y = static_cast<T*>(a.y) + base;
#pragma unroll
  for (int q = 0; q < V; ++q) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = q * N + j;
      h[e] = h[e] * rstd * g[e] + b[e];
    }
    if (p.has(q)) put_vec<ONCE>(y + p.at(q), pack<T>(h + q * N));
  }
  if (p.rest >= 0) from_f32(hr * rstd * gr + br, y[p.rest]);
  if (p.lane == 0) {
    if (a.mean && a.kind == QLORA_NORM_LAYER) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// Input gradients, and with WEIGHTS the partial weight gradients of the rows
// that a workgroup takes: G = THREADS / ROW at a time, each by ROW threads
// that keep the sums of their own columns in registers; at the end the G
// sums of a column are added in order and written as one partial.
template <typename T, int ROW, int E, int THREADS, bool WEIGHTS, bool ONCE>
__global__ __launch_bounds__(THREADS) void k_norm_bwd(NormBwdArgs a, int parts) {
  constexpr int N = Part<T, ROW, E>::N, V = Part<T, ROW, E>::V, G = THREADS / ROW;
  __shared__ float lds[2][THREADS / 64][2];
  const Part<T, ROW, E> p(threadIdx.x % ROW, (int)a.d);
  const int group = threadIdx.x / ROW;
  const bool layer = a.kind == QLORA_NORM_LAYER;
  const float inv = 1.0f / (float)a.d;
  float g[E], gr;
  weight_part(p, a.gamma, a.w_type, g, gr);
  float dg[E], db[E], dgr = 0.0f, dbr = 0.0f;
  if constexpr (WEIGHTS) {
#pragma unroll
    for (int j = 0; j < E; ++j) dg[j] = db[j] = 0.0f;
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < a.rows; r0 += (int64_t)parts * G, turn ^= 1) {
    const int64_t row = r0 + group;
    const bool live = row < a.rows;
    const int64_t base = (live ? row : a.rows - 1) * a.d;
    const float mean = layer ? a.mean[live ? row : a.rows - 1] : 0.0f;
    const float rstd = a.rstd[live ? row : a.rows - 1];
    u32x4 vy[V], vh[V], vd[V];
    T ry, rh, rd = T(0);
    load_part<ONCE>(p, static_cast<const T*>(a.dy) + base, vy, ry);
    load_part<ONCE>(p, static_cast<const T*>(a.h) + base, vh, rh);
    if (a.dh) load_part<ONCE>(p, static_cast<const T*>(a.dh) + base, vd, rd);
    float s[2] = {0.0f, 0.0f};                 // sum(u), sum(u n)
    float y[N], n[N];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      unpack<T>(vy[q], y);
      unpack<T>(vh[q], n);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = q * N + j;
        n[j] = (n[j] - mean) * rstd;
        if constexpr (WEIGHTS) {
          dg[e] += live ? y[j] * n[j] : 0.0f;
          db[e] += live ? y[j] : 0.0f;
        }
        const float u = y[j] * g[e];           // 0 past the row's end
        s[0] += u;
        s[1] += u * n[j];
      }
    }
    const float yr = to_f32(ry), nr = (to_f32(rh) - mean) * rstd, ur = yr * gr;
    if constexpr (WEIGHTS) {
      dgr += live ? yr * nr : 0.0f;
      dbr += live ? yr : 0.0f;
    }
    s[0] += ur;
    s[1] += ur * nr;
    row_sums<ROW, THREADS>(s, lds[turn]);
    const float mu = layer ? s[0] * inv : 0.0f, mn = s[1] * inv;
    if (live) {
      T* dx = static_cast<T*>(a.dx) + base;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        unpack<T>(vy[q], y);
        unpack<T>(vh[q], n);
#pragma unroll
        for (int j = 0; j < N; ++j)
          y[j] = (y[j] * g[q * N + j] - mu - (n[j] - mean) * rstd * mn) * rstd;
        if (a.dh) {
          unpack<T>(vd[q], n);
#pragma unroll
          for (int j = 0; j < N; ++j) y[j] += n[j];
        }
        if (p.has(q)) put_vec<ONCE>(dx + p.at(q), pack<T>(y));
      }
      if (p.rest >= 0) from_f32((ur - mu - nr * mn) * rstd + to_f32(rd), dx[p.rest]);
    }
  }
  if constexpr (WEIGHTS) {
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
    if (a.dgamma) write_partial<T, ROW, E, THREADS>(p, group, dg, dgr, part);
    if (a.dbeta) write_partial<T, ROW, E, THREADS>(p, group, db, dbr, part + a.d);
  }
}

// Weight gradients from the partials: kFinishCols columns per workgroup, the
// partials in slices summed apart, eight loads in flight, and added
// in order.
__global__ __launch_bounds__(1024) void k_norm_wgrad_finish(const float* part, int parts,
                                                            int64_t d, float* dgamma,
                                                            float* dbeta) {
  constexpr int S = 1024 / kFinishCols, U = 8;
  __shared__ float lds[S][kFinishCols];
  const int col = threadIdx.x % kFinishCols, slice = threadIdx.x / kFinishCols;
  const int64_t i = (int64_t)blockIdx.x * kFinishCols + col;
  const bool beta = blockIdx.y == 1 || !dgamma;
  float* out = beta ? dbeta : dgamma;
  const float* src = part + (beta ? d : 0);
  float s = 0.0f;
  if (i < d) {
    for (int p0 = slice; p0 < parts; p0 += S * U) {
      float f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = p0 + u * S;
        f[u] = p < parts ? src[(int64_t)p * 2 * d + i] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) s += f[u];
    }
  }
  lds[slice][col] = s;
  __syncthreads();
  // the slices' sums: added by halves, in a fixed order
#pragma unroll
  for (int half = S / 2; half >= 1; half /= 2) {
    if (slice < half) lds[slice][col] += lds[slice + half][col];
    __syncthreads();
  }
  if (slice == 0 && i < d) out[i] = lds[0][col];
}

// ------------------------------------------------- rows of any width
// One workgroup per row, which loops over it.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_fwd_wide(NormFwdArgs a) {
  __shared__ float lds[2][16];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.d;
  const T* r = a.r ? static_cast<const T*>(a.r) + row * a.d : nullptr;
  T* h = a.r ? static_cast<T*>(a.h) + row * a.d : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.d;
  const bool layer = a.kind == QLORA_NORM_LAYER;
  float sum = 0.0f;
  for (int64_t i = threadIdx.x; i < a.d; i += 1024) {
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
  const float mean = layer ? block_sum<1024>(sum, lds[0]) / (float)a.d : 0.0f;
  float sq = 0.0f;
  for (int64_t i = threadIdx.x; i < a.d; i += 1024) {
    const float c = to_f32(s[i]) - mean;
    sq += c * c;
  }
  const float var = block_sum<1024>(sq, lds[1]) / (float)a.d;
  const float rstd = 1.0f / sqrtf(var + a.eps);
  for (int64_t i = threadIdx.x; i < a.d; i += 1024) {
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
__global__ __launch_bounds__(1024) void k_norm_bwd_wide(NormBwdArgs a) {
  __shared__ float lds[2][16];
  const int64_t row = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy) + row * a.d;
  const T* h = static_cast<const T*>(a.h) + row * a.d;
  const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.d : nullptr;
  T* dx = static_cast<T*>(a.dx) + row * a.d;
  const bool layer = a.kind == QLORA_NORM_LAYER;
  const float mean = layer ? a.mean[row] : 0.0f, rstd = a.rstd[row];
  float su = 0.0f, sn = 0.0f;
  for (int64_t i = threadIdx.x; i < a.d; i += 1024) {
    const float u = to_f32(dy[i]) * load_w(a.gamma, a.w_type, i);
    su += u;
    sn += u * ((to_f32(h[i]) - mean) * rstd);
  }
  const float mu = layer ? block_sum<1024>(su, lds[0]) / (float)a.d : 0.0f;
  const float mn = block_sum<1024>(sn, lds[1]) / (float)a.d;
  for (int64_t i = threadIdx.x; i < a.d; i += 1024) {
    const float u = to_f32(dy[i]) * load_w(a.gamma, a.w_type, i);
    const float n = (to_f32(h[i]) - mean) * rstd;
    float v = (u - mu - n * mn) * rstd;
    if (dh) v += to_f32(dh[i]);
    from_f32(v, dx[i]);
  }
}

// Weight gradients of one group of `per` rows: a thread per column.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_wgrad_wide(NormBwdArgs a, int64_t per) {
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

// ------------------------------------------------- launches
constexpr int64_t kFwdHeld = 32768;   // widest row held in registers, forward
constexpr int64_t kBwdHeld = 16384;   // backward: twice the arrays, and the sums

// Threads that hold a row of the backward: 8 values each (16 above 8192).
static int bwd_row_threads(int64_t d) {
  int row = 64;
  while (row < 1024 && (int64_t)row * 8 < d) row *= 2;
  return row;
}

int norm_parts(int64_t rows, int64_t d) {
  if (d > kBwdHeld) return (int)std::min<int64_t>(rows, 64);
  const int64_t g = kBwdThreads / bwd_row_threads(d);
  const int64_t turns = (rows + g - 1) / g;   // rounds of g rows
  // one workgroup on each of the 256 compute units at most (the
  // registers allow no second one)
  return (int)std::min<int64_t>(turns, 256);
}

template <typename T, int ROW, int E, int THREADS>
static void run_fwd(const NormFwdArgs& a, hipStream_t st) {
  constexpr int64_t g = THREADS / ROW;
  const dim3 grid((unsigned)((a.rows + g - 1) / g));
  if (a.rows * a.d * (int64_t)sizeof(T) < kOnceBytes)
    hipLaunchKernelGGL((k_norm_fwd<T, ROW, E, THREADS, false>), grid, dim3(THREADS), 0, st, a);
  else hipLaunchKernelGGL((k_norm_fwd<T, ROW, E, THREADS, true>), grid, dim3(THREADS), 0, st, a);
}

template <typename T>
static void fwd_by_width(const NormFwdArgs& a, hipStream_t st) {
  if (a.d <= 512) run_fwd<T, 64, 8, 256>(a, st);
  else if (a.d <= 1024) run_fwd<T, 128, 8, 256>(a, st);
  else if (a.d <= 2048) run_fwd<T, 256, 8, 256>(a, st);
  else if (a.d <= 4096) run_fwd<T, 512, 8, 512>(a, st);
  else if (a.d <= 8192) run_fwd<T, 1024, 8, 1024>(a, st);
  else if (a.d <= 16384) run_fwd<T, 1024, 16, 1024>(a, st);
  else if (a.d <= kFwdHeld) run_fwd<T, 1024, 32, 1024>(a, st);
  else
    hipLaunchKernelGGL(k_norm_fwd_wide<T>, dim3((unsigned)a.rows), dim3(1024), 0, st, a);
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t st) {
  if (a.type == QLORA_BF16) fwd_by_width<uint16_t>(a, st);
  else fwd_by_width<float>(a, st);
  return hipGetLastError();
}

template <typename T, int ROW, int E, bool ONCE>
static void run_bwd_as(const NormBwdArgs& a, hipStream_t st) {
  constexpr int64_t g = kBwdThreads / ROW;
  if (a.dgamma || a.dbeta) {
    const int parts = norm_parts(a.rows, a.d);
    hipLaunchKernelGGL((k_norm_bwd<T, ROW, E, kBwdThreads, true, ONCE>), dim3((unsigned)parts),
                       dim3(kBwdThreads), 0, st, a, parts);
  } else {
    const int grid = (int)((a.rows + g - 1) / g);
    hipLaunchKernelGGL((k_norm_bwd<T, ROW, E, kBwdThreads, false, ONCE>), dim3((unsigned)grid),
                       dim3(kBwdThreads), 0, st, a, grid);
  }
}

template <typename T, int ROW, int E>
static void run_bwd(const NormBwdArgs& a, hipStream_t st) {
  if (a.rows * a.d * (int64_t)sizeof(T) < kOnceBytes) run_bwd_as<T, ROW, E, false>(a, st);
  else run_bwd_as<T, ROW, E, true>(a, st);
}

template <typename T>
static void bwd_by_width(const NormBwdArgs& a, hipStream_t st) {
  switch (bwd_row_threads(a.d)) {
    case 64: return run_bwd<T, 64, 8>(a, st);
    case 128: return run_bwd<T, 128, 8>(a, st);
    case 256: return run_bwd<T, 256, 8>(a, st);
    case 512: return run_bwd<T, 512, 8>(a, st);
    default: break;
  }
  if (a.d <= 8192) return run_bwd<T, 1024, 8>(a, st);
  if (a.d <= kBwdHeld) return run_bwd<T, 1024, 16>(a, st);
  if (a.dgamma || a.dbeta) {   // before dX, which may overwrite dY
    const int parts = norm_parts(a.rows, a.d);
    hipLaunchKernelGGL(k_norm_wgrad_wide<T>,
                       dim3((unsigned)((a.d + 255) / 256), (unsigned)parts), dim3(256), 0, st, a,
                       (a.rows + parts - 1) / parts);
  }
  hipLaunchKernelGGL(k_norm_bwd_wide<T>, dim3((unsigned)a.rows), dim3(1024), 0, st, a);
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st) {
  if (a.rows > 0) {
    if (a.type == QLORA_BF16) bwd_by_width<uint16_t>(a, st);
    else bwd_by_width<float>(a, st);
  }
  if (a.dgamma || a.dbeta) {
    const int parts = a.rows > 0 ? norm_parts(a.rows, a.d) : 0;
    const dim3 grid((unsigned)((a.d + kFinishCols - 1) / kFinishCols), a.dgamma && a.dbeta ? 2 : 1);
    hipLaunchKernelGGL(k_norm_wgrad_finish, grid, dim3(1024), 0, st, a.part, parts, a.d, a.dgamma,
                       a.dbeta);
  }
  return hipGetLastError();
}

}  // namespace qlora
