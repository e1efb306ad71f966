// logits.hip -- log-probabilities of target tokens, the preference loss and
// the clipped policy loss, from a head's logits to their gradient (gfx950).
//
// Row i of the logits is softmax-distributed with inverse temperature
// `scale`.  With m its maximum and S = sum_j exp(scale (l_j - m)),
//   logp = scale (l_t - m) - log S,   lse = scale m + log S,
//   dlogits_j = scale dlogp ((j == t) - exp(scale (l_j - m) - log S)).
// The losses are functions of the logp of all tokens; see qlora.h.
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// Maximum and sum of exponentials (to the base 2 of x * k) of a set of
// logits; an empty set has m = -inf, s = 0.  A maximum of -inf is not
// subtracted (every term is then exp(-inf) = 0).
struct MaxSum {
  float m, s;
};

__device__ __forceinline__ float shift(float m) { return m == -kInf ? 0.0f : m; }

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float k) {
  const float m = fmaxf(a.m, b.m), z = shift(m);
  return {m, a.s * exp2_fast((a.m - z) * k) + b.s * exp2_fast((b.m - z) * k)};
}

template <int THREADS>
__device__ __forceinline__ MaxSum block_join(MaxSum v, float k, MaxSum* lds) {
#pragma unroll
  for (int half = 32; half >= 1; half >>= 1) {
    const MaxSum o{__shfl_xor(v.m, half, 64), __shfl_xor(v.s, half, 64)};
    v = join(v, o, k);
  }
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v = join(v, lds[w], k);
  return v;
}

// Rows of sequence s, clamped to [0, rows].
__device__ __forceinline__ void seq_rows(const int64_t* offsets, int64_t s, int64_t rows,
                                         int64_t& b, int64_t& e) {
  b = min(max(offsets[s], (int64_t)0), rows);
  e = min(max(offsets[s + 1], b), rows);
}

}  // namespace

// One workgroup per row.
template <typename T>
__global__ __launch_bounds__(256) void k_logp(LogitsArgs l, float* logp, float* lse,
                                              RowStat* stat) {
  __shared__ MaxSum lds[4];
  const int64_t row = blockIdx.x;
  const int64_t t = l.targets[row];
  if (t == l.ignore || t < 0 || t >= l.vocab) {
    const float v = t == l.ignore ? 0.0f : __builtin_nanf("");
    if (threadIdx.x == 0) {
      logp[row] = v;
      if (lse) lse[row] = v;
      if (stat) stat[row] = {v, v};
    }
    return;
  }
  const T* x = static_cast<const T*>(l.logits) + row * l.ld;
  const float k = l.scale * kLog2e;
  MaxSum v{-kInf, 0.0f};
  for (int64_t i = threadIdx.x; i < l.vocab; i += 256) v = join(v, {to_f32(x[i]), 1.0f}, k);
  v = block_join<256>(v, k, lds);
  if (threadIdx.x == 0) {
    const float m = shift(v.m), ls = logf(v.s);
    logp[row] = (to_f32(x[t]) - m) * l.scale - ls;
    if (lse) lse[row] = m * l.scale + ls;
    if (stat) stat[row] = {m, ls};
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_dlogits(LogitsArgs l, const RowStat* stat,
                                                 const float* lse, const float* dlogp, T* dlogits,
                                                 int64_t ldd) {
  const int64_t row = blockIdx.x;
  const int64_t t = l.targets[row];
  T* out = dlogits + row * ldd;
  float g = t == l.ignore ? 0.0f : dlogp[row] * l.scale;
  if (t != l.ignore && (t < 0 || t >= l.vocab) && g != 0.0f) g = __builtin_nanf("");
  T zero;
  from_f32(g == 0.0f ? 0.0f : g, zero);
  if (g == 0.0f || t < 0 || t >= l.vocab) {
    for (int64_t i = threadIdx.x; i < l.vocab; i += 256) out[i] = zero;
    return;
  }
  const T* x = static_cast<const T*>(l.logits) + row * l.ld;
  RowStat s;
  if (stat) {
    s = stat[row];
  } else {
    s.max = lse[row] / l.scale;
    s.logsum = lse[row] - s.max * l.scale;
  }
  const float k = l.scale * kLog2e, c = s.logsum * kLog2e;
  for (int64_t i = threadIdx.x; i < l.vocab; i += 256) {
    const float p = exp2_fast(__builtin_fmaf(to_f32(x[i]) - s.max, k, -c));
    from_f32(i == t ? g * (1.0f - p) : -g * p, out[i]);
  }
}

// One workgroup per pair: both sequences' sums in FP64, the loss and its
// slope, the gradient of every log-probability.  The first and the last
// workgroup also clear the rows before and after all sequences.
__global__ __launch_bounds__(256) void k_preference(PreferenceArgs a) {
  __shared__ double lds[6][4];
  const int64_t p = blockIdx.x;
  if (a.dlogp) {
    int64_t b0 = 0, e1 = 0, skip;
    if (a.pairs > 0) {
      seq_rows(a.offsets, 0, a.rows, b0, skip);
      seq_rows(a.offsets, 2 * a.pairs - 1, a.rows, skip, e1);
    }
    if (p == 0)
      for (int64_t i = threadIdx.x; i < b0; i += 256) a.dlogp[i] = 0.0f;
    if (p == gridDim.x - 1)
      for (int64_t i = e1 + threadIdx.x; i < a.rows; i += 256) a.dlogp[i] = 0.0f;
  }
  if (a.pairs == 0) return;
  double s[2], g[2], n[2];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    int64_t b, e;
    seq_rows(a.offsets, p + side * a.pairs, a.rows, b, e);
    double vs = 0.0, vg = 0.0, vn = 0.0;
    for (int64_t i = b + threadIdx.x; i < e; i += 256) {
      if (a.targets[i] == a.ignore) continue;
      const float lp = a.logp[i];
      vs += (double)lp;
      vg += a.ref ? (double)lp - (double)a.ref[i] : (double)lp;
      vn += 1.0;
    }
    s[side] = block_sum<256>(vs, lds[3 * side]);
    g[side] = block_sum<256>(vg, lds[3 * side + 1]);
    n[side] = block_sum<256>(vn, lds[3 * side + 2]);
    if (a.length_normalize) {
      n[side] = n[side] < 1.0 ? 1.0 : n[side];
      s[side] /= n[side];
      g[side] /= n[side];
    }
  }
  const double h = g[0] - g[1], beta = a.beta, z = beta * h - a.margin;
  double loss, slope;
  if (a.kind == QLORA_PREF_SIGMOID) {
    const double e = a.smoothing, x = exp(-fabs(z));
    const double low = log1p(x), tail = x / (1.0 + x);   // tail = sigmoid(-|z|)
    loss = (1.0 - e) * ((z < 0.0 ? -z : 0.0) + low);     // softplus(-z)
    if (e > 0.0) loss += e * ((z > 0.0 ? z : 0.0) + low);
    slope = beta * (z > 0.0 ? e - tail : tail - (1.0 - e));
  } else if (a.kind == QLORA_PREF_HINGE) {
    loss = z < 1.0 ? 1.0 - z : (z == z ? 0.0 : z);
    slope = z < 1.0 ? -beta : (z == z ? 0.0 : z);
  } else {
    const double off = h - 0.5 / beta;
    loss = off * off;
    slope = 2.0 * off;
  }
  if (threadIdx.x == 0) {
    a.loss[p] = (float)loss;
    a.seq_logp[p] = (float)s[0];
    a.seq_logp[p + a.pairs] = (float)s[1];
  }
  if (!a.dlogp) return;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    int64_t b, e;
    seq_rows(a.offsets, p + side * a.pairs, a.rows, b, e);
    double c = (side ? -slope : slope) * (double)a.weight;
    if (a.length_normalize) c /= n[side];
    for (int64_t i = b + threadIdx.x; i < e; i += 256)
      a.dlogp[i] = a.targets[i] == a.ignore ? 0.0f : (float)c;
  }
}

// One workgroup per sequence: the rows that count, and each row's sequence.
__global__ __launch_bounds__(256) void k_policy_count(LogitsArgs l, PolicyArgs a) {
  __shared__ int lds[4];
  const int64_t s = blockIdx.x;
  int64_t b0 = 0, e1 = 0, skip;
  if (a.seqs > 0) {
    seq_rows(a.offsets, 0, l.rows, b0, skip);
    seq_rows(a.offsets, a.seqs - 1, l.rows, skip, e1);
  }
  if (s == 0)
    for (int64_t i = threadIdx.x; i < b0; i += 256) a.row_seq[i] = -1;
  if (s == gridDim.x - 1)
    for (int64_t i = e1 + threadIdx.x; i < l.rows; i += 256) a.row_seq[i] = -1;
  if (a.seqs == 0) return;
  int64_t b, e;
  seq_rows(a.offsets, s, l.rows, b, e);
  int n = 0;
  for (int64_t i = b + threadIdx.x; i < e; i += 256) {
    const bool counts = l.targets[i] != l.ignore;
    a.row_seq[i] = counts ? (int32_t)s : -1;
    n += counts;
  }
  n = block_sum<256>(n, lds);
  if (threadIdx.x == 0) a.count[s] = n;
}

// Terms and gradient of one row, given its log-probability.
struct PolicyRow {
  float4 terms;  // w, policy, kl, clipped
  float dlogp;
};
__device__ __forceinline__ PolicyRow policy_row(const PolicyArgs& a, int64_t row, int s, float w,
                                                float lp) {
  PolicyRow o{{0.0f, 0.0f, 0.0f, 0.0f}, 0.0f};
  if (s < 0) return o;
  const float adv = a.adv[a.per_token ? row : s];
  const float ratio = a.old_logp ? expf(lp - a.old_logp[row]) : 1.0f;
  const float lo = 1.0f - a.clip_low, hi = 1.0f + a.clip_high;
  const float free = -adv * ratio;
  // not fminf / fmaxf: a NaN ratio stays NaN
  const float held = -adv * (ratio < lo ? lo : (ratio > hi ? hi : ratio));
  const bool clipped = held > free;
  float kl = 0.0f, dkl = 0.0f;
  if (a.ref) {
    const float gap = a.ref[row] - lp, em = expm1f(gap);
    kl = em - gap;
    dkl = -em;
  }
  o.terms = {w, clipped ? held : free, kl, clipped ? 1.0f : 0.0f};
  o.dlogp = a.weight * w * ((clipped ? 0.0f : free) + a.kl_coef * dkl);
  return o;
}

// Weight of a row of sequence s (counts of all sequences summed by the
// workgroup for the mean over tokens).
template <int THREADS>
__device__ __forceinline__ float policy_total(const PolicyArgs& a, int* lds) {
  int n = 0;
  if (a.reduction == QLORA_POLICY_TOKEN_MEAN)
    for (int64_t i = threadIdx.x; i < a.seqs; i += THREADS) n += a.count[i];
  return (float)block_sum<THREADS>(n, lds);
}
__device__ __forceinline__ float policy_weight(const PolicyArgs& a, int s, float total) {
  if (s < 0) return 0.0f;
  return a.reduction == QLORA_POLICY_TOKEN_MEAN ? 1.0f / total
                                                : 1.0f / ((float)a.seqs * (float)a.count[s]);
}

__global__ __launch_bounds__(256) void k_policy_rows(LogitsArgs l, PolicyArgs a, float* dlogp) {
  __shared__ int lds[4];
  const float total = policy_total<256>(a, lds);
  const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (row >= l.rows) return;
  const int s = a.row_seq[row];
  const PolicyRow o = policy_row(a, row, s, policy_weight(a, s, total), a.logp[row]);
  a.terms[row] = o.terms;
  if (dlogp) dlogp[row] = o.dlogp;
}

__global__ __launch_bounds__(1024) void k_policy_stats(PolicyArgs a, int64_t rows) {
  __shared__ double lds[3][16];
  double p = 0.0, k = 0.0, c = 0.0;
  for (int64_t i = threadIdx.x; i < rows; i += 1024) {
    const float4 t = a.terms[i];
    if (t.x == 0.0f) continue;   // a row without weight
    p += (double)t.x * (double)t.y;
    k += (double)t.x * (double)t.z;
    c += (double)t.x * (double)t.w;
  }
  p = block_sum<1024>(p, lds[0]);
  k = block_sum<1024>(k, lds[1]);
  c = block_sum<1024>(c, lds[2]);
  if (threadIdx.x == 0) {
    a.stats[0] = (float)(a.kl_coef == 0.0f ? p : p + (double)a.kl_coef * k);
    a.stats[1] = (float)p;
    a.stats[2] = (float)k;
    a.stats[3] = (float)c;
  }
}

hipError_t launch_logp(const LogitsArgs& l, float* logp, float* lse, RowStat* stat,
                       hipStream_t st) {
  const dim3 grid((unsigned)l.rows);
  if (l.type == QLORA_BF16)
    hipLaunchKernelGGL(k_logp<uint16_t>, grid, dim3(256), 0, st, l, logp, lse, stat);
  else hipLaunchKernelGGL(k_logp<float>, grid, dim3(256), 0, st, l, logp, lse, stat);
  return hipGetLastError();
}

hipError_t launch_dlogits(const LogitsArgs& l, const RowStat* stat, const float* lse,
                          const float* dlogp, void* dlogits, int64_t ldd, hipStream_t st) {
  const dim3 grid((unsigned)l.rows);
  if (l.type == QLORA_BF16)
    hipLaunchKernelGGL(k_dlogits<uint16_t>, grid, dim3(256), 0, st, l, stat, lse, dlogp,
                       static_cast<uint16_t*>(dlogits), ldd);
  else
    hipLaunchKernelGGL(k_dlogits<float>, grid, dim3(256), 0, st, l, stat, lse, dlogp,
                       static_cast<float*>(dlogits), ldd);
  return hipGetLastError();
}

hipError_t launch_preference(const PreferenceArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)std::max<int64_t>(a.pairs, 1);
  hipLaunchKernelGGL(k_preference, dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_policy(const LogitsArgs& l, const PolicyArgs& a, void* dlogits, int64_t ldd,
                         RowStat* stat, float* dlogp, hipStream_t st) {
  if (l.rows > 0) {
    const unsigned seqs = (unsigned)std::max<int64_t>(a.seqs, 1);
    hipLaunchKernelGGL(k_policy_count, dim3(seqs), dim3(256), 0, st, l, a);
    hipError_t e = launch_logp(l, a.logp, nullptr, stat, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_policy_rows, dim3((unsigned)((l.rows + 255) / 256)), dim3(256), 0, st, l,
                       a, dlogits ? dlogp : nullptr);
    if (dlogits) {
      e = launch_dlogits(l, stat, nullptr, dlogp, dlogits, ldd, st);
      if (e != hipSuccess) return e;
    }
  }
  hipLaunchKernelGGL(k_policy_stats, dim3(1), dim3(1024), 0, st, a, l.rows);
  return hipGetLastError();
}

}  // namespace qlora
