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
// threads that own it, so every array is read once; the variance is summed
// from the centred values, which costs no second read.  A row takes as many
// wavefronts as it fills (at 8 or 16 values a thread, 32 in the widest
// forward), a workgroup as many rows as fit it, and the grid is persistent: a
// thread keeps its columns' weights, loads its part of the next row before it
// works on the present one, and in the backward sums its columns' weight
// gradients in registers.  Wider rows take the looping kernels below, which
// read them again from the caches (backward of 4096 x 18432 BF16: 269 us, 2.3
// TB/s; 388 with dgamma).
//
// Three shapes do not fit their registers and spill some: the layer norm's
// forward of 16385 to 32768 values a row (FP32 60 a thread: 125 us at 2048 x
// 32768, 4.3 TB/s, where the RMS norm, which spills 8, takes 102; BF16 8: 59
// us), and the layer norm's FP32 backward of 8193 to 16384 with weight gradients
// (15: 155 us at 4096 x 12288, 3.9 TB/s).
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

constexpr int kFinishCols = 16;
// Arrays of this size and more go past the caches' retention: the two to four
// of a call would drive each other out of the 256 MB of the last level anyway.
// Backward of 16384 x 8192 BF16: 199 us kept, 187 us past.  Forward with a
// residual: 193 and 181 us at 16384 x 8192, 98 and 90 at 8192 x 8192 (228 and
// 208 with the product that reads Y next).  Smaller outputs stay for the layer
// that reads them next.
constexpr int64_t kOnceBytes = int64_t(128) << 20;

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

template <bool ONCE, typename T>
__device__ __forceinline__ u32x4 get_vec(const T* p) {
  if constexpr (ONCE) return load_vec_once(p);
  else return load_vec(p);
}
template <bool ONCE, typename T>
__device__ __forceinline__ void put_vec(T* p, u32x4 v) {
  if constexpr (ONCE) store_vec_once(p, v);
  else store_vec(p, v);
}

// The part of a row that one of its `threads` threads holds: V vectors,
// `threads` apart, and at most one element of the last, partial vector
// (`rest`, -1 without).
template <typename T, int V>
struct Part {
  static constexpr int N = kVec<T>, E = V * N;
  int lane, threads, nvec, rest;
  __device__ __forceinline__ Part(int thread, int threads_, int d) {
    lane = thread;
    threads = threads_;
    nvec = d / N;
    const int i = nvec * N + thread;
    rest = i < d ? i : -1;
  }
  __device__ __forceinline__ bool has(int q) const { return lane + q * threads < nvec; }
  __device__ __forceinline__ int at(int q) const { return (lane + q * threads) * N; }
};

// A part's values of one array (0 past the row's end).
template <typename T, int V>
struct Held {
  u32x4 v[V];
  T rest;
};
template <bool ONCE, typename T, int V>
__device__ __forceinline__ void load_part(const Part<T, V>& p, const T* x, Held<T, V>& h) {
#pragma unroll
  for (int q = 0; q < V; ++q) {
    h.v[q] = u32x4{0, 0, 0, 0};
    if (p.has(q)) h.v[q] = get_vec<ONCE>(x + p.at(q));
  }
  h.rest = T(0);
  if (p.rest >= 0) h.rest = x[p.rest];
}

// Its weights (0 past the row's end).
template <typename T, int V>
__device__ __forceinline__ void weight_part(const Part<T, V>& p, const void* w, int w_type,
                                            float* f, float& rest) {
  constexpr int N = kVec<T>;
#pragma unroll
  for (int q = 0; q < V; ++q) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[q * N + j] = 0.0f;
    if (p.has(q)) load_w_vec<N>(w, w_type, p.at(q), f + q * N);
  }
  rest = p.rest >= 0 ? load_w(w, w_type, p.rest) : 0.0f;
}

// Sums over the `threads` threads (whole wavefronts, at most 16) of each row of
// a workgroup; the rows of a workgroup go through it together.
template <int COUNT>
__device__ __forceinline__ void row_sums(float (&v)[COUNT], int threads, float (*lds)[COUNT]) {
#pragma unroll
  for (int c = 0; c < COUNT; ++c) v[c] = wave_sum(v[c]);
  if (threads == 64) return;
  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63, W = threads / 64;
  if (lane == 0) {
#pragma unroll
    for (int c = 0; c < COUNT; ++c) lds[wave][c] = v[c];
  }
  lds_barrier();
  const int first = wave / W * W;
#pragma unroll
  for (int c = 0; c < COUNT; ++c) v[c] = row16_sum(lane < W ? lds[first + lane][c] : 0.0f);
}

// A thread's place: its row group of the workgroup, the same for its
// wavefront.
__device__ __forceinline__ int row_group(int row_threads) {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x / row_threads);
}

}  // namespace

// blockDim.x / row_threads rows per workgroup at a time, `stride` rows from
// one to the next.  RMS norm of 4096 x 4096 BF16 with a residual: 22 us, 6.1
// TB/s (64 us with three looping reads, 24.6 without the next row ahead).
template <typename T, int V, bool LAYER, bool ONCE>
__global__ __launch_bounds__(1024) void k_norm_fwd(NormFwdArgs a, int row_threads,
                                                   int64_t stride) {
  constexpr int N = kVec<T>, E = V * N;
  constexpr bool AHEAD = E <= 16;              // wider: no registers for the next row
  __shared__ float lds[2][2][16][1];
  const int group = row_group(row_threads), groups = blockDim.x / row_threads;
  const Part<T, V> p(threadIdx.x - group * row_threads, row_threads, (int)a.d);
  const T *xs = static_cast<const T*>(a.x), *rs = static_cast<const T*>(a.r);
  const float inv = 1.0f / (float)a.d;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  // rows past the end are those of a workgroup's idle groups: they read the last
  const auto base = [&](int64_t r) { return (r < a.rows ? r : a.rows - 1) * a.d; };
  Held<T, V> x, r;
  load_part<ONCE>(p, xs + base(row), x);
  if (rs) load_part<ONCE>(p, rs + base(row), r);
  const bool shifted = LAYER && a.beta;
  float g[AHEAD ? E : N], b[AHEAD ? E : N], gr, br = 0.0f;
  if constexpr (AHEAD) {
    weight_part(p, a.gamma, a.w_type, g, gr);
    if (shifted) weight_part(p, a.beta, a.w_type, b, br);
  } else {
    gr = p.rest >= 0 ? load_w(a.gamma, a.w_type, p.rest) : 0.0f;
    if (shifted && p.rest >= 0) br = load_w(a.beta, a.w_type, p.rest);
  }
  for (int turn = 0;; turn ^= 1, row += stride) {
    const bool live = row < a.rows, more = row - group + stride < a.rows;
    Held<T, V> xn, rn;
    if (AHEAD && more) {
      load_part<ONCE>(p, xs + base(row + stride), xn);
      if (rs) load_part<ONCE>(p, rs + base(row + stride), rn);
    }
    float h[E], hr;
    if (rs) {
      T* out = static_cast<T*>(a.h) + base(row);
      float f[N];
#pragma unroll
      for (int q = 0; q < V; ++q) {
        unpack<T>(x.v[q], h + q * N);
        unpack<T>(r.v[q], f);
#pragma unroll
        for (int j = 0; j < N; ++j) f[j] += h[q * N + j];
        x.v[q] = pack<T>(f);                   // the one rounding of H
        if (live && p.has(q)) put_vec<ONCE>(out + p.at(q), x.v[q]);
      }
      from_f32(to_f32(x.rest) + to_f32(r.rest), x.rest);
      if (live && p.rest >= 0) out[p.rest] = x.rest;
    }
#pragma unroll
    for (int q = 0; q < V; ++q) unpack<T>(x.v[q], h + q * N);
    hr = to_f32(x.rest);
    float mean = 0.0f;
    if constexpr (LAYER) {
      float s[1] = {hr};                       // 0 in threads without a rest
#pragma unroll
      for (int j = 0; j < E; ++j) s[0] += h[j];
      row_sums(s, row_threads, lds[turn][0]);
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
    row_sums(s, row_threads, lds[turn][1]);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    if (live) {
      T* y = static_cast<T*>(a.y) + base(row);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int w = AHEAD ? q * N : 0;       // the widest rows fetch their weights here
        if (!AHEAD && p.has(q)) {
          load_w_vec<N>(a.gamma, a.w_type, p.at(q), g);
          if (shifted) load_w_vec<N>(a.beta, a.w_type, p.at(q), b);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          h[q * N + j] = h[q * N + j] * rstd * g[w + j];
          if (shifted) h[q * N + j] += b[w + j];
        }
        if (p.has(q)) put_vec<ONCE>(y + p.at(q), pack<T>(h + q * N));
      }
      if (p.rest >= 0) from_f32(shifted ? hr * rstd * gr + br : hr * rstd * gr, y[p.rest]);
      if (p.lane == 0) {
        if (LAYER && a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
    if (!more) return;
    if constexpr (AHEAD) {
      x = xn;
      r = rn;
    } else {
      load_part<ONCE>(p, xs + base(row + stride), x);
      if (rs) load_part<ONCE>(p, rs + base(row + stride), r);
    }
  }
}

namespace {

// What the backward reads of one row.
template <typename T, int V>
struct BwdRow {
  Held<T, V> y, h, d;
  float mean, rstd;
};
template <bool LAYER, bool ONCE, typename T, int V>
__device__ __forceinline__ void load_row(const NormBwdArgs& a, const Part<T, V>& p, int64_t row,
                                         BwdRow<T, V>& o) {
  row = row < a.rows ? row : a.rows - 1;       // an idle group reads the last row
  const int64_t base = row * a.d;
  load_part<ONCE>(p, static_cast<const T*>(a.dy) + base, o.y);
  load_part<ONCE>(p, static_cast<const T*>(a.h) + base, o.h);
  if (a.dh) load_part<ONCE>(p, static_cast<const T*>(a.dh) + base, o.d);
  o.mean = LAYER ? a.mean[row] : 0.0f;
  o.rstd = a.rstd[row];
}

// The sums of a workgroup's row groups, added in order, as one row of d
// partials: four columns a thread at a time, the groups meeting in LDS.
template <typename T, int V>
__device__ __forceinline__ void write_partial(const Part<T, V>& p, int group, int groups,
                                              const float* v, float rest, float* part,
                                              f32x4* lds) {
  constexpr int N = kVec<T>, E = V * N;
  if (groups == 1) {
#pragma unroll
    for (int c = 0; c < E / 4; ++c)
      if (p.has(4 * c / N)) store_vec(part + p.at(4 * c / N) + 4 * c % N, pack<float>(v + 4 * c));
    if (p.rest >= 0) part[p.rest] = rest;
    return;
  }
#pragma unroll
  for (int c = 0; c <= E / 4; ++c) {
    const bool last = c == E / 4;              // the partial vector's element
    lds_barrier();
    if (last) lds[threadIdx.x].x = rest;
    else lds[threadIdx.x] = __builtin_bit_cast(f32x4, pack<float>(v + 4 * c));
    lds_barrier();
    if (group) continue;
    f32x4 t = lds[p.lane];
    for (int k = 1; k < groups; ++k) t += lds[k * p.threads + p.lane];
    if (last) {
      if (p.rest >= 0) part[p.rest] = t.x;
    } else if (p.has(4 * c / N)) {
      store_vec(part + p.at(4 * c / N) + 4 * c % N, __builtin_bit_cast(u32x4, t));
    }
  }
}

}  // namespace

// Input gradients, and with WEIGHTS the partial weight gradients of the rows
// that a workgroup takes.  gamma waits in LDS (four of a thread's columns side
// by side, so that a wavefront reads without bank conflicts).  Sums in FP32.
// RMS norm of 16384 x 8192 BF16 with dH and dgamma: 175 us, 6.1 TB/s, and 5 us
// for the partials; layer norm of 1003 x 5003 FP32: 14 and 6 us, where a
// workgroup has four rows and the 256 partials are a third of the traffic.
template <typename T, int V, bool LAYER, bool WEIGHTS, bool ONCE>
__global__ __launch_bounds__(1024) void k_norm_bwd(NormBwdArgs a, int row_threads,
                                                   int64_t stride) {
  constexpr int N = kVec<T>, E = V * N;
  // the next row's values need registers: of 16 a thread only beside few sums
  constexpr bool AHEAD = E <= 8 || (sizeof(T) == 2 && !(LAYER && WEIGHTS));
  __shared__ float lds[2][16][2];
  extern __shared__ f32x4 dyn[];               // gamma, later the groups' sums
  const int group = row_group(row_threads), groups = blockDim.x / row_threads;
  const Part<T, V> p(threadIdx.x - group * row_threads, row_threads, (int)a.d);
  const float inv = 1.0f / (float)a.d;
  int64_t row = (int64_t)blockIdx.x * groups + group;
  BwdRow<T, V> cur;
  load_row<LAYER, ONCE>(a, p, row, cur);
  float gr;
  {
    float g[E];
    weight_part(p, a.gamma, a.w_type, g, gr);
    if (group == 0) {
#pragma unroll
      for (int c = 0; c < E / 4; ++c)
        dyn[c * row_threads + p.lane] = __builtin_bit_cast(f32x4, pack<float>(g + 4 * c));
    }
    lds_barrier();
  }
  const f32x4* gam = dyn + p.lane;
  float dg[E], db[E], dgr = 0.0f, dbr = 0.0f;
  if constexpr (WEIGHTS) {
#pragma unroll
    for (int j = 0; j < E; ++j) dg[j] = db[j] = 0.0f;
  }
  for (int turn = 0;; turn ^= 1, row += stride) {
    const bool live = row < a.rows, more = row - group + stride < a.rows;
    BwdRow<T, V> next;
    if (AHEAD && more) load_row<LAYER, ONCE>(a, p, row + stride, next);
    const float mean = cur.mean, rstd = cur.rstd;
    float s[2] = {0.0f, 0.0f};                 // sum(u n), sum(u)
    float y[N], n[N];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      unpack<T>(cur.y.v[q], y);
      unpack<T>(cur.h.v[q], n);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int e = q * N + j;
        n[j] = (n[j] - mean) * rstd;
        if constexpr (WEIGHTS) {
          dg[e] += live ? y[j] * n[j] : 0.0f;
          if constexpr (LAYER) db[e] += live ? y[j] : 0.0f;
        }
        const float u = y[j] * gam[e / 4 * row_threads][e % 4];   // 0 past the row's end
        s[0] += u * n[j];
        if constexpr (LAYER) s[1] += u;
      }
    }
    const float yr = to_f32(cur.y.rest), nr = (to_f32(cur.h.rest) - mean) * rstd, ur = yr * gr;
    if constexpr (WEIGHTS) {
      dgr += live ? yr * nr : 0.0f;
      dbr += live ? yr : 0.0f;
    }
    s[0] += ur * nr;
    s[1] += ur;
    row_sums(s, row_threads, lds[turn]);
    const float mn = s[0] * inv, mu = LAYER ? s[1] * inv : 0.0f;
    if (live) {
      T* dx = static_cast<T*>(a.dx) + row * a.d;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        unpack<T>(cur.y.v[q], y);
        unpack<T>(cur.h.v[q], n);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int e = q * N + j;
          y[j] = (y[j] * gam[e / 4 * row_threads][e % 4] - mu - (n[j] - mean) * rstd * mn) * rstd;
        }
        if (a.dh) {
          unpack<T>(cur.d.v[q], n);
#pragma unroll
          for (int j = 0; j < N; ++j) y[j] += n[j];
        }
        if (p.has(q)) put_vec<ONCE>(dx + p.at(q), pack<T>(y));
      }
      if (p.rest >= 0)
        from_f32((ur - mu - nr * mn) * rstd + (a.dh ? to_f32(cur.d.rest) : 0.0f), dx[p.rest]);
    }
    if (!more) break;
    if constexpr (AHEAD) cur = next;
    else load_row<LAYER, ONCE>(a, p, row + stride, cur);
  }
  if constexpr (WEIGHTS) {
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.d;
    if (a.dgamma) write_partial(p, group, groups, dg, dgr, part, dyn);
    if constexpr (LAYER) {
      if (a.dbeta) write_partial(p, group, groups, db, dbr, part + a.d, dyn);
    }
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
constexpr int64_t kBwdHeld = 16384;   // backward: more arrays, and the sums

namespace {

// How a call takes its rows: threads a row, rows a workgroup, workgroups.
struct Shape {
  int row_threads, groups, grid;
};
// `held` values a thread, workgroups of at most `threads`, at most `waves`
// wavefronts on each of the 256 compute units.
Shape row_shape(int64_t rows, int64_t d, int held, int threads, int waves) {
  Shape s;
  s.row_threads = 64 * (int)((d + 64 * held - 1) / (64 * held));
  s.groups = std::max(1, threads / s.row_threads);
  const int64_t turns = (rows + s.groups - 1) / s.groups;
  const int64_t resident = 256 * std::max(1, waves * 64 / (s.groups * s.row_threads));
  s.grid = (int)std::min(turns, resident);
  return s;
}
// With weight gradients a workgroup costs a partial, and their sums registers:
// fewer of them.  Narrow rows meet in smaller workgroups, whose barriers wait
// for fewer (26090 x 566 BF16: 30.0 against 32.5 us).  Without weight gradients
// 24 wavefronts a compute unit are as fast as 16 or faster: 62.0 against 76.2 us
// at 8192 x 5120 BF16, 22.0 against 24.9 at 26090 x 566, 96.7 both at 16384 x
// 4096; a small batch of few turns loses (1003 x 5003 FP32 13.3 against 11.7).
Shape bwd_shape(int64_t rows, int64_t d, bool weights) {
  return row_shape(rows, d, d <= 8192 ? 8 : 16, d <= 1024 ? 512 : 1024, weights ? 16 : 24);
}

}  // namespace

int norm_parts(int64_t rows, int64_t d) {
  return d <= kBwdHeld ? bwd_shape(rows, d, true).grid : (int)std::min<int64_t>(rows, 64);
}

template <typename T, int V, bool LAYER>
static void run_fwd(const NormFwdArgs& a, int waves, hipStream_t st) {
  const Shape s = row_shape(a.rows, a.d, V * kVec<T>, 512, waves);
  const dim3 grid((unsigned)s.grid), block((unsigned)(s.row_threads * s.groups));
  const int64_t stride = (int64_t)s.grid * s.groups;
  if (a.rows * a.d * (int64_t)sizeof(T) < kOnceBytes)
    hipLaunchKernelGGL((k_norm_fwd<T, V, LAYER, false>), grid, block, 0, st, a, s.row_threads,
                       stride);
  else
    hipLaunchKernelGGL((k_norm_fwd<T, V, LAYER, true>), grid, block, 0, st, a, s.row_threads,
                       stride);
}

template <typename T, bool LAYER>
static void fwd_by_width(const NormFwdArgs& a, hipStream_t st) {
  constexpr int U = 8 / kVec<T>;   // vectors of 8 values
  // as many wavefronts as the registers allow (5123 x 7040 BF16: 28 us with
  // 32 a compute unit, 36 with 24)
  if (a.d <= 8192) run_fwd<T, U, LAYER>(a, sizeof(T) == 2 ? 32 : 24, st);
  else if (a.d <= 16384) run_fwd<T, 2 * U, LAYER>(a, 16, st);
  else if (a.d <= kFwdHeld) run_fwd<T, 4 * U, LAYER>(a, 16, st);
  else
    hipLaunchKernelGGL(k_norm_fwd_wide<T>, dim3((unsigned)a.rows), dim3(1024), 0, st, a);
}

template <typename T>
static void fwd_by_kind(const NormFwdArgs& a, hipStream_t st) {
  if (a.kind == QLORA_NORM_LAYER) fwd_by_width<T, true>(a, st);
  else fwd_by_width<T, false>(a, st);
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t st) {
  if (a.type == QLORA_BF16) fwd_by_kind<uint16_t>(a, st);
  else fwd_by_kind<float>(a, st);
  return hipGetLastError();
}

template <typename T, int V, bool LAYER, bool ONCE>
static void run_bwd(const NormBwdArgs& a, hipStream_t st) {
  const bool weights = a.dgamma || a.dbeta;
  const Shape s = bwd_shape(a.rows, a.d, weights);
  const dim3 grid((unsigned)s.grid), block((unsigned)(s.row_threads * s.groups));
  const int64_t stride = (int64_t)s.grid * s.groups;
  // gamma of a row's threads; then one 16-byte piece of every thread
  const size_t lds = 16 * std::max<size_t>(block.x, (size_t)s.row_threads * V * kVec<T> / 4);
  if (weights)
    hipLaunchKernelGGL((k_norm_bwd<T, V, LAYER, true, ONCE>), grid, block, lds, st, a,
                       s.row_threads, stride);
  else
    hipLaunchKernelGGL((k_norm_bwd<T, V, LAYER, false, ONCE>), grid, block, lds, st, a,
                       s.row_threads, stride);
}

template <typename T, int V, bool LAYER>
static void bwd_by_size(const NormBwdArgs& a, hipStream_t st) {
  if (a.rows * a.d * (int64_t)sizeof(T) < kOnceBytes) run_bwd<T, V, LAYER, false>(a, st);
  else run_bwd<T, V, LAYER, true>(a, st);
}

template <typename T>
static void bwd_by_width(const NormBwdArgs& a, hipStream_t st) {
  constexpr int U = 8 / kVec<T>;
  const bool layer = a.kind == QLORA_NORM_LAYER;
  if (a.d <= 8192) return layer ? bwd_by_size<T, U, true>(a, st) : bwd_by_size<T, U, false>(a, st);
  if (a.d <= kBwdHeld)
    return layer ? bwd_by_size<T, 2 * U, true>(a, st) : bwd_by_size<T, 2 * U, false>(a, st);
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
    const dim3 grid((unsigned)((a.d + kFinishCols - 1) / kFinishCols),
                    a.dgamma && a.dbeta ? 2 : 1);
    hipLaunchKernelGGL(k_norm_wgrad_finish, grid, dim3(1024), 0, st, a.part, parts, a.d, a.dgamma,
                       a.dbeta);
  }
  return hipGetLastError();
}

}  // namespace qlora
