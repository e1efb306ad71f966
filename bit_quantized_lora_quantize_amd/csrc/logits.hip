// logits.hip -- log-probabilities of target tokens, the preference loss and
// the clipped policy loss, from a head's logits to their gradient (gfx950).
//
// Row i of the logits is softmax-distributed with inverse temperature
// `scale`.  With m its maximum and S = sum_j exp(scale (l_j - m)),
//   logp = scale (l_t - m) - log S,   lse = scale m + log S,
//   dlogits_j = scale dlogp ((j == t) - exp(scale (l_j - m) - log S)).
// The losses are functions of the logp of all tokens; see qlora.h.
//
// All kernels are bound by memory: a row is read once for its statistics and
// once more for its gradient where a token's slope needs other rows first (the
// preference loss), and once altogether where it does not (the policy loss).
// One exponential a logit and pass leaves the vector units about half busy at
// 6 TB/s.
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kInf = __builtin_huge_valf();
constexpr int kPrefThreads = 1024;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// A maximum of -inf is not subtracted: every term is then exp(-inf) = 0.
__device__ __forceinline__ float shift(float m) { return m == -kInf ? 0.0f : m; }

// exp(scale (x - m)) with k = scale * log2(e).  The difference comes first:
// logits of the type's lowest value would overflow when scaled.
__device__ __forceinline__ float term(float x, float m, float k) {
  return exp2_fast((x - m) * k);
}

// Maximum of the logits and sum of their terms against it.
struct MaxSum {
  float m, s;
};
template <int THREADS>
__device__ __forceinline__ MaxSum block_join(MaxSum v, float k, MaxSum* lds) {
  const float mw = wave_max(v.m);
  v.s = wave_sum(v.s * term(v.m, shift(mw), k));
  v.m = mw;
  if constexpr (THREADS == 64) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  constexpr int W = THREADS / 64;
  float m = lds[0].m, s = 0.0f;
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, lds[w].m);
#pragma unroll
  for (int w = 0; w < W; ++w) s += lds[w].s * term(lds[w].m, shift(m), k);
  return {m, s};
}

// A thread's part of a row's maximum and sum, in one pass: per round, kU
// vectors are loaded together, their maximum joins the running one and the
// running sum is rescaled once.  Empty threads hold m = -inf, s = 0.
template <typename T, int THREADS>
__device__ __forceinline__ MaxSum stream_row(const T* x, int vocab, float k, int lane) {
  constexpr int N = kVec<T>, kU = 32 / N;
  const RowCut<T> cut(x, vocab, lane);
  MaxSum r{-kInf, 0.0f};
  for (int v0 = lane; v0 < cut.nvec; v0 += THREADS * kU) {
    u32x4 d[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int v = v0 + i * THREADS;
      d[i] = vec_neg_inf<T>();
      if (v < cut.nvec) d[i] = load_vec(x + cut.at(v));
    }
    float f[N], m = r.m;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      unpack<T>(d[i], f);
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, f[j]);
    }
    const float z = shift(m);
    float s = r.s * term(r.m, z, k);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      unpack<T>(d[i], f);
#pragma unroll
      for (int j = 0; j < N; ++j) s += term(f[j], z, k);
    }
    r = {m, s};
  }
  if (cut.edge >= 0) {
    const float f = to_f32(x[cut.edge]), m = fmaxf(r.m, f), z = shift(m);
    r = {m, r.s * term(r.m, z, k) + term(f, z, k)};
  }
  return r;
}

// Rows of sequence s, clamped to [0, rows].
__device__ __forceinline__ void seq_rows(const int64_t* offsets, int64_t s, int64_t rows,
                                         int64_t& b, int64_t& e) {
  b = min(max(offsets[s], (int64_t)0), rows);
  e = min(max(offsets[s + 1], b), rows);
}

}  // namespace

// One workgroup per row, in one pass.  Long rows take 1024 threads: their
// loads of a whole round are in flight at once, and two workgroups a compute
// unit cover each other's reductions (8348 x 131072 BF16, a quarter ignored:
// 263 us, 6.2 TB/s; with 512 and 256 threads the whole loss takes 1 and 2 %
// longer).  FP32 maxima and sums.
template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void k_logp(LogitsArgs l, float* logp, float* lse,
                                                  RowStat* stat) {
  __shared__ MaxSum lds[16];
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
  const float k = l.scale * kLog2e, xt = to_f32(x[t]);
  const MaxSum v = block_join<THREADS>(stream_row<T, THREADS>(x, (int)l.vocab, k, threadIdx.x), k, lds);
  if (threadIdx.x == 0) {
    const float m = shift(v.m), ls = logf(v.s);
    logp[row] = (xt - m) * l.scale - ls;
    if (lse) lse[row] = m * l.scale + ls;
    if (stat) stat[row] = {m, ls};
  }
}

// Gradient of N logits of a row: -g p, and g more at the target.
struct RowGrad {
  float g, m, c, k;   // p = exp2((x - m) k - c)
  int t;
};
template <int N>
__device__ __forceinline__ void grad_terms(const RowGrad& r, int first, float* f) {
#pragma unroll
  for (int j = 0; j < N; ++j) f[j] = -r.g * exp2_fast(__builtin_fmaf(f[j] - r.m, r.k, -r.c));
  if ((uint32_t)(r.t - first) < (uint32_t)N) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] += first + j == r.t ? r.g : 0.0f;
  }
}

// A row's gradient where no logit is read, by THREADS threads: zeros, or NaN
// for a bad target.
template <typename T, int THREADS>
__device__ __forceinline__ void fill_row(T* out, int vocab, float value, int lane) {
  constexpr int N = kVec<T>;
  float f[N];
#pragma unroll
  for (int j = 0; j < N; ++j) f[j] = value;
  const u32x4 v = pack<T>(f);
  const RowCut<T> cut(out, vocab, lane);
  for (int i = lane; i < cut.nvec; i += THREADS) store_vec_once(out + cut.at(i), v);
  if (cut.edge >= 0) from_f32(value, out[cut.edge]);
}

// A row's gradient by THREADS threads, from its logits read again.
template <typename T, int THREADS>
__device__ __forceinline__ void grad_row(const T* x, T* out, int vocab, const RowGrad& q,
                                         int lane) {
  constexpr int N = kVec<T>, kU = 2;
  const RowCut<T> cut(x, vocab, lane);
  for (int v0 = lane; v0 < cut.nvec; v0 += THREADS * kU) {
    u32x4 d[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (v0 + i * THREADS < cut.nvec) d[i] = load_vec(x + cut.at(v0 + i * THREADS));
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      if (v0 + i * THREADS >= cut.nvec) continue;
      const int first = cut.at(v0 + i * THREADS);
      float f[N];
      unpack<T>(d[i], f);
      grad_terms<N>(q, first, f);
      store_vec_once(out + first, pack<T>(f));
    }
  }
  if (cut.edge >= 0) {
    float f = to_f32(x[cut.edge]);
    grad_terms<1>(q, cut.edge, &f);
    from_f32(f, out[cut.edge]);
  }
}

// One vector of a row, or one of its single elements (v past the vectors).
template <typename T>
struct GradAt {
  const T* x;
  int v, nvec;
  RowCut<T> cut;
  __device__ __forceinline__ GradAt(const LogitsArgs& l, int64_t row, int v_)
      : x(static_cast<const T*>(l.logits) + row * l.ld),
        v(v_),
        nvec(RowCut<T>(x, (int)l.vocab, 0).nvec),
        cut(x, (int)l.vocab, v_ - nvec) {}
};
// Its gradient, by one thread: q of its row but for the target t.
template <typename T>
__device__ __forceinline__ void grad_vec(const LogitsArgs& l, const GradAt<T>& at, int64_t t,
                                         RowGrad q, T* out) {
  constexpr int N = kVec<T>;
  const RowCut<T>& cut = at.cut;
  const bool none = t == l.ignore || q.g == 0.0f;
  if (none || t < 0 || t >= l.vocab) {   // zeros, or NaN for a bad target
    T e;
    from_f32(none ? 0.0f : __builtin_nanf(""), e);
    float f[N];
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = to_f32(e);
    if (at.v < at.nvec) store_vec_once(out + cut.at(at.v), pack<T>(f));
    else if (cut.edge >= 0) out[cut.edge] = e;
    return;
  }
  q.t = (int)t;
  if (at.v < at.nvec) {
    float f[N];
    unpack<T>(load_vec_once(at.x + cut.at(at.v)), f);
    grad_terms<N>(q, cut.at(at.v), f);
    store_vec_once(out + cut.at(at.v), pack<T>(f));
  } else if (cut.edge >= 0) {
    float f = to_f32(at.x[cut.edge]);
    grad_terms<1>(q, cut.edge, &f);
    from_f32(f, out[cut.edge]);
  }
}

// A row's gradient by one workgroup of 256 that takes its maximum and sum again.
template <typename T>
__device__ __forceinline__ void regrad_row(const LogitsArgs& l, int64_t row, float g, int t,
                                           T* out) {
  __shared__ MaxSum lds[4];
  const T* x = static_cast<const T*>(l.logits) + row * l.ld;
  const float k = l.scale * kLog2e;
  const MaxSum v = block_join<256>(stream_row<T, 256>(x, (int)l.vocab, k, threadIdx.x), k, lds);
  const RowGrad q{g, shift(v.m), logf(v.s) * kLog2e, k, t};
  grad_row<T, 256>(x, out, (int)l.vocab, q, threadIdx.x);
}

// From this size on an FP32 lse is off by more than 2^-18, and so is every p it
// gives; a row all at its type's lowest value would get p = 1 for every token.
// The backward then takes the row's sum again: 117 us against 84 where all rows
// of 2048 x 32000 FP32 need it, 1205 against 705 at 8348 x 131072 BF16.
constexpr float kLseHeld = 128.0f;

// One vector of one row per thread, `chunks` workgroups a row: many small
// workgroups stream best (608 us for 8348 x 131072 BF16, 6.3 TB/s).  Rounded
// once, to the logits' type.
//
// A forward pass has just read the same logits, and the last-level cache (256
// MB) still holds what it read last: row r of the launch is row last - r, and
// neither the gradient's stores nor this second and last read stay in the
// caches, where they would drive out logits yet to be read.  Against plain
// accesses: 129 to 97 us at 2048 x 32000 FP32 with a quarter of the rows
// ignored, 943 to 880 us at 8348 x 131072 BF16 (893 us first row to last).
//
// HELD: the softmax comes from stat, else from lse; compiled apart, since with the
// sum taken again in one kernel the first took 2 % longer.
template <typename T, bool HELD>
__global__ __launch_bounds__(256) void k_dlogits(LogitsArgs l, const RowStat* stat,
                                                 const float* lse, const float* dlogp, T* dlogits,
                                                 int64_t ldd, int64_t last, uint32_t chunks) {
  const uint32_t r = blockIdx.x / chunks;
  const int64_t row = last - r;
  const GradAt<T> at(l, row, (int)((blockIdx.x - r * chunks) * 256 + threadIdx.x));
  const int64_t t = l.targets[row];
  RowGrad q;
  q.k = l.scale * kLog2e;
  q.g = dlogp[row] * l.scale;
  if constexpr (HELD) {
    RowStat s = stat[row];
    // waited for with the target and the slope: loaded past their test, 922 us for 879
    asm volatile("" : "+s"(s.max), "+s"(s.logsum));
    q.m = s.max;
    q.c = s.logsum * kLog2e;
  } else {
    const float e = lse[row];
    q.m = e / l.scale;
    if (!(fabsf(e) < kLseHeld && fabsf(q.m) < kInf) && t != l.ignore && q.g != 0.0f && t >= 0 &&
        t < l.vocab) {
      // the same for the whole row: one of its workgroups takes it all, another
      // one each row (workgroup i runs on die i mod 8)
      if (blockIdx.x - r * chunks == r % chunks) regrad_row(l, row, q.g, (int)t, dlogits + row * ldd);
      return;
    }
    q.c = __builtin_fmaf(-q.m, l.scale, e) * kLog2e;   // what the quotient's rounding left
  }
  grad_vec(l, at, t, q, dlogits + row * ldd);
}

// Sums, loss and slope of one pair, half of a workgroup per sequence: the
// sequences' sums in FP64.  To every thread: the gradient of a log-probability
// of each of the two sequences, the loss, and the sequences' log-probabilities.
struct PairLoss {
  float c[2], loss;
  double s[2];
};
template <int THREADS>
__device__ __forceinline__ PairLoss pair_loss(const PreferenceArgs& a, int64_t p,
                                              double (*lds)[THREADS / 64]) {
  constexpr int kSide = THREADS / 2, W = kSide / 64;
  const int side = threadIdx.x / kSide;
  int64_t b, e;
  seq_rows(a.offsets, p + side * a.pairs, a.rows, b, e);
  double vs = 0.0, vg = 0.0, vn = 0.0;
  constexpr int U = 4;   // rows a thread loads together
  for (int64_t i0 = b + threadIdx.x % kSide; i0 < e; i0 += kSide * U) {
    float lp[U], rf[U];
    int64_t t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kSide;
      lp[u] = rf[u] = 0.0f;
      t[u] = a.ignore;
      if (i < e) {
        lp[u] = a.logp[i];
        t[u] = a.targets[i];
        if (a.ref) rf[u] = a.ref[i];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t[u] == a.ignore) continue;
      vs += (double)lp[u];
      vg += (double)lp[u] - (double)rf[u];
      vn += 1.0;
    }
  }
  vs = wave_sum(vs);
  vg = wave_sum(vg);
  vn = wave_sum(vn);
  const int wave = threadIdx.x / 64;
  if ((threadIdx.x & 63) == 0) {
    lds[0][wave] = vs;
    lds[1][wave] = vg;
    lds[2][wave] = vn;
  }
  __syncthreads();
  // every wavefront adds the W partial sums of each sequence
  double s[2], g[2], n[2];
  const int at = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s[i] = row16_sum(at < W ? lds[0][i * W + at] : 0.0);
    g[i] = row16_sum(at < W ? lds[1][i * W + at] : 0.0);
    n[i] = row16_sum(at < W ? lds[2][i * W + at] : 0.0);
  }
  if (a.length_normalize) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      n[i] = n[i] < 1.0 ? 1.0 : n[i];
      s[i] /= n[i];
      g[i] /= n[i];
    }
  }
  // the sums need 64 bits; the loss of their small difference does not
  const double h = g[0] - g[1];
  const float beta = a.beta, z = (float)((double)beta * h - (double)a.margin);
  float loss, slope;
  if (a.kind == QLORA_PREF_SIGMOID) {
    const float sm = a.smoothing, x = expf(-fabsf(z));
    const float low = log1pf(x), tail = x / (1.0f + x);   // tail = sigmoid(-|z|)
    loss = (1.0f - sm) * ((z < 0.0f ? -z : 0.0f) + low);  // softplus(-z)
    if (sm > 0.0f) loss += sm * ((z > 0.0f ? z : 0.0f) + low);
    slope = beta * (z > 0.0f ? sm - tail : tail - (1.0f - sm));
  } else if (a.kind == QLORA_PREF_HINGE) {
    loss = z < 1.0f ? 1.0f - z : (z == z ? 0.0f : z);
    slope = z < 1.0f ? -beta : (z == z ? 0.0f : z);
  } else {
    const float off = (float)(h - 0.5 / (double)beta);
    loss = off * off;
    slope = 2.0f * off;
  }
  PairLoss r{{slope * a.weight, -slope * a.weight}, loss, {s[0], s[1]}};
  if (a.length_normalize) {
    r.c[0] /= (float)n[0];
    r.c[1] /= (float)n[1];
  }
  return r;
}

// A pair's outputs, by one thread.
__device__ __forceinline__ void write_pair(const PreferenceArgs& a, int64_t p, const PairLoss& r) {
  a.loss[p] = r.loss;
  a.seq_logp[p] = (float)r.s[0];
  a.seq_logp[p + a.pairs] = (float)r.s[1];
}

// The rows before and after all sequences, [0, begin) and [end, rows).
struct Outside {
  int64_t begin, end;
};
__device__ __forceinline__ Outside outside_rows(const int64_t* offsets, int64_t seqs,
                                                int64_t rows) {
  Outside o{0, 0};
  int64_t skip;
  if (seqs > 0) {
    seq_rows(offsets, 0, rows, o.begin, skip);
    seq_rows(offsets, seqs - 1, rows, skip, o.end);
  }
  return o;
}

// One workgroup per pair: its loss, and the gradient of every log-probability
// (also of rows that do not count: their logits' gradient is 0 whatever it
// is).  The first and the last workgroup clear the rows outside.  5.6 us for
// four pairs of up to 2 x 512 rows, the latency of three dependent loads.
__global__ __launch_bounds__(kPrefThreads) void k_preference(PreferenceArgs a) {
  __shared__ double lds[3][kPrefThreads / 64];
  const int64_t p = blockIdx.x;
  if (a.dlogp) {
    const Outside o = outside_rows(a.offsets, 2 * a.pairs, a.rows);
    if (p == 0)
      for (int64_t i = threadIdx.x; i < o.begin; i += kPrefThreads) a.dlogp[i] = 0.0f;
    if (p == gridDim.x - 1)
      for (int64_t i = o.end + threadIdx.x; i < a.rows; i += kPrefThreads) a.dlogp[i] = 0.0f;
  }
  if (a.pairs == 0) return;
  const PairLoss s = pair_loss<kPrefThreads>(a, p, lds);
  if (threadIdx.x == 0) write_pair(a, p, s);
  if (!a.dlogp) return;
  constexpr int kSide = kPrefThreads / 2;
  const int side = threadIdx.x / kSide;
  int64_t b, e;
  seq_rows(a.offsets, p + side * a.pairs, a.rows, b, e);
  const float c = side ? s.c[1] : s.c[0];
  for (int64_t i = b + threadIdx.x % kSide; i < e; i += kSide) a.dlogp[i] = c;
}

// The sequence that a row lies in, -1 for none, by a full wavefront.
__device__ __forceinline__ int sequence_of(const int64_t* offsets, int64_t seqs, int64_t rows,
                                           int64_t row) {
  if (seqs == 0) return -1;   // no offsets to read
  const int lane = threadIdx.x & 63;
  int at = 0;                 // offsets at or before the row
  for (int64_t j = 0; j <= seqs; j += 64) {
    const bool before = j + lane <= seqs && offsets[j + lane] <= row;
    at += __popcll(__ballot(before));
  }
  if (at < 1 || at > seqs) return -1;
  int64_t b, e;
  seq_rows(offsets, at - 1, rows, b, e);
  return row >= b && row < e ? at - 1 : -1;
}

// Losses and gradients of a batch of few rows in one launch, once its
// log-probabilities are there: the first workgroups write a pair's loss each,
// every other one finds its row's pair, sums it again and takes one vector of
// the row per thread.
template <typename T>
__global__ __launch_bounds__(256) void k_pairs_dlogits(LogitsArgs l, PreferenceArgs a,
                                                       const RowStat* stat, T* dlogits,
                                                       int64_t ldd, uint32_t chunks) {
  __shared__ double lds[3][4];
  if ((int64_t)blockIdx.x < a.pairs) {
    const PairLoss r = pair_loss<256>(a, blockIdx.x, lds);
    if (threadIdx.x == 0) write_pair(a, blockIdx.x, r);
    return;
  }
  const uint32_t i = blockIdx.x - (uint32_t)a.pairs;
  const int64_t row = i / chunks;
  const GradAt<T> at(l, row, (int)((i - (uint32_t)row * chunks) * 256 + threadIdx.x));
  const int64_t t = l.targets[row];
  const RowStat s = stat[row];
  RowGrad q{0.0f, s.max, s.logsum * kLog2e, l.scale * kLog2e, 0};
  if (t != l.ignore) {
    const int seq = sequence_of(a.offsets, 2 * a.pairs, a.rows, row);
    if (seq >= 0) {
      const PairLoss r = pair_loss<256>(a, seq < a.pairs ? seq : seq - a.pairs, lds);
      q.g = (seq < a.pairs ? r.c[0] : r.c[1]) * l.scale;
    }
  }
  grad_vec(l, at, t, q, dlogits + row * ldd);
}

// Log-probability of one row by one wavefront.
template <typename T>
__device__ __forceinline__ void wave_logp(const LogitsArgs& l, int64_t row, float* logp,
                                          RowStat* stat) {
  const int lane = threadIdx.x & 63;
  const int64_t t = l.targets[row];
  float lp = t == l.ignore ? 0.0f : __builtin_nanf("");
  RowStat q{lp, lp};
  if (t != l.ignore && t >= 0 && t < l.vocab) {
    const T* x = static_cast<const T*>(l.logits) + row * l.ld;
    const float k = l.scale * kLog2e;
    const MaxSum v = block_join<64>(stream_row<T, 64>(x, (int)l.vocab, k, lane), k, nullptr);
    q = {shift(v.m), logf(v.s)};
    lp = (to_f32(x[t]) - q.max) * l.scale - q.logsum;
  }
  if (lane == 0) {
    logp[row] = lp;
    stat[row] = q;
  }
}

// Gradient of one row by one wavefront.
template <typename T>
__device__ __forceinline__ void wave_grad(const LogitsArgs& l, int64_t row, RowStat s, float dlogp,
                                          T* dlogits, int64_t ldd) {
  const int lane = threadIdx.x & 63;
  const int64_t t = l.targets[row];
  const float g = dlogp * l.scale;
  T* out = dlogits + row * ldd;
  const bool none = t == l.ignore || g == 0.0f;
  if (none || t < 0 || t >= l.vocab) {
    fill_row<T, 64>(out, (int)l.vocab, none ? 0.0f : __builtin_nanf(""), lane);
    return;
  }
  const RowGrad q{g, s.max, s.logsum * kLog2e, l.scale * kLog2e, (int)t};
  grad_row<T, 64>(static_cast<const T*>(l.logits) + row * l.ld, out, (int)l.vocab, q, lane);
}

// A small batch of pairs in one launch: a workgroup per pair, a wavefront per
// row.  The rows' results pass between the wavefronts through memory, at the
// barriers.
template <typename T>
__global__ __launch_bounds__(kPrefThreads) void k_preference_small(LogitsArgs l, PreferenceArgs a,
                                                                   RowStat* stat, float* logp,
                                                                   T* dlogits, int64_t ldd) {
  constexpr int W = kPrefThreads / 64;
  __shared__ double lds[3][W];
  const int64_t p = blockIdx.x;
  const int wave = threadIdx.x / 64;
  const Outside o = outside_rows(a.offsets, 2 * a.pairs, a.rows);
  if (p == 0) {
    for (int64_t row = wave; row < o.begin; row += W) {
      wave_logp<T>(l, row, logp, stat);
      if (dlogits) wave_grad<T>(l, row, RowStat{0.0f, 0.0f}, 0.0f, dlogits, ldd);
    }
  }
  if (p == gridDim.x - 1) {
    for (int64_t row = o.end + wave; row < a.rows; row += W) {
      wave_logp<T>(l, row, logp, stat);
      if (dlogits) wave_grad<T>(l, row, RowStat{0.0f, 0.0f}, 0.0f, dlogits, ldd);
    }
  }
  int64_t b[2], e[2];
  seq_rows(a.offsets, p, a.rows, b[0], e[0]);
  seq_rows(a.offsets, p + a.pairs, a.rows, b[1], e[1]);
  const int64_t first = e[0] - b[0], n = first + e[1] - b[1];
  for (int64_t i = wave; i < n; i += W)
    wave_logp<T>(l, i < first ? b[0] + i : b[1] + (i - first), logp, stat);
  __syncthreads();
  const PairLoss s = pair_loss<kPrefThreads>(a, p, lds);
  if (threadIdx.x == 0) write_pair(a, p, s);
  if (!dlogits) return;
  for (int64_t i = wave; i < n; i += W) {
    const int64_t row = i < first ? b[0] + i : b[1] + (i - first);
    wave_grad<T>(l, row, stat[row], i < first ? s.c[0] : s.c[1], dlogits, ldd);
  }
}

// One workgroup per sequence: the rows that count, and each row's sequence.
__global__ __launch_bounds__(256) void k_policy_count(LogitsArgs l, PolicyArgs a) {
  __shared__ int lds[4];
  const int64_t s = blockIdx.x;
  const Outside o = outside_rows(a.offsets, a.seqs, l.rows);
  if (s == 0)
    for (int64_t i = threadIdx.x; i < o.begin; i += 256) a.row_seq[i] = -1;
  if (s == gridDim.x - 1)
    for (int64_t i = o.end + threadIdx.x; i < l.rows; i += 256) a.row_seq[i] = -1;
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

// All rows that count, from the sequences' counts, by one workgroup.
__global__ __launch_bounds__(1024) void k_policy_total(PolicyArgs a) {
  __shared__ int lds[16];
  int n = 0;
  for (int64_t i = threadIdx.x; i < a.seqs; i += 1024) n += a.count[i];
  n = block_sum<1024>(n, lds);
  if (threadIdx.x == 0) *a.total = n;
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
  o.dlogp = a.weight * w * ((clipped ? 0.0f : free) + (a.kl_coef > 0.0f ? a.kl_coef * dkl : 0.0f));
  return o;
}

// The sequence that a row counts in (-1: in none) and its weight, by a full
// wavefront: from k_policy_count's results, or where that did not run (row_seq
// NULL) from the offsets and targets themselves.
struct Place {
  int seq;
  float w;
};
__device__ __forceinline__ Place policy_place(const LogitsArgs& l, const PolicyArgs& a,
                                              int64_t row) {
  const int lane = threadIdx.x & 63;
  const bool token_mean = a.reduction == QLORA_POLICY_TOKEN_MEAN;
  int seq, n = 0;
  if (a.row_seq) {
    seq = a.row_seq[row];
    if (seq < 0) return {-1, 0.0f};
    if (token_mean && !a.total) {
      for (int64_t i = lane; i < a.seqs; i += 64) n += a.count[i];
      n = wave_sum(n);
    } else {
      n = token_mean ? *a.total : a.count[seq];
    }
  } else {
    if (l.targets[row] == l.ignore) return {-1, 0.0f};
    seq = sequence_of(a.offsets, a.seqs, l.rows, row);
    if (seq < 0) return {-1, 0.0f};
    int64_t b, e;
    seq_rows(a.offsets, seq, l.rows, b, e);
    if (token_mean) {
      const Outside o = outside_rows(a.offsets, a.seqs, l.rows);
      b = o.begin;
      e = o.end;
    }
    for (int64_t i = b + lane; i < e; i += 64 * 8) {
      int64_t t[8];   // loaded together
#pragma unroll
      for (int u = 0; u < 8; ++u) t[u] = i + 64 * u < e ? l.targets[i + 64 * u] : l.ignore;
#pragma unroll
      for (int u = 0; u < 8; ++u) n += t[u] != l.ignore ? 1 : 0;
    }
    n = wave_sum(n);
  }
  return {seq, token_mean ? 1.0f / (float)n : 1.0f / ((float)a.seqs * (float)n)};
}

// N terms of a row to its gradient: -g p = c term, and g more at the target.
template <int N>
__device__ __forceinline__ void scale_terms(float c, float g, int t, int first, float* f) {
#pragma unroll
  for (int j = 0; j < N; ++j) f[j] *= c;
  if ((uint32_t)(t - first) < (uint32_t)N) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] += first + j == t ? g : 0.0f;
  }
}

// Loss and gradient of one row in one pass: the row's logits stay in
// registers (E of them a thread, as FP32 terms once the maximum is known),
// so they are read once and their exponentials taken once.  A longer row
// leaves L more vectors a thread in LDS, as they came; their exponentials are
// taken twice.  dlogits NULL: the loss alone, with the same bits.
//
// 15315 x 65536 BF16: 650 us, 5.9 TB/s over one read and one write (962 us as
// three passes); 8192 x 131072 BF16: 785 us (877 read twice).  Bound by memory;
// with one workgroup of the widest rows a compute unit, also by its reductions.
// The bound on registers makes the steps of 32 logits a thread spill one
// (BF16, 1024 threads) to three (FP32, 256, 512 and 1024) of them, and the FP32
// step with LDS three.
template <typename T, int THREADS, int E, int L, int MIN_WAVES>
__global__ __launch_bounds__(THREADS, MIN_WAVES) void k_policy(LogitsArgs l, PolicyArgs a,
                                                               T* dlogits, int64_t ldd) {
  constexpr int N = kVec<T>, V = E / N;
  __shared__ float lds_m[THREADS / 64], lds_s[THREADS / 64], lds_g;
  extern __shared__ u32x4 far[];                  // [L][THREADS]: each thread its own
  const int64_t row = blockIdx.x;
  const int vocab = (int)l.vocab;
  const int64_t t = l.targets[row];
  T* out = dlogits ? dlogits + row * ldd : nullptr;
  const bool lead = threadIdx.x < 64;
  if (t == l.ignore || t < 0 || t >= l.vocab) {
    const bool bad = t != l.ignore;
    const float lp = bad ? __builtin_nanf("") : 0.0f;
    if (lead) {
      const Place at = policy_place(l, a, row);
      if (threadIdx.x == 0) {
        a.logp[row] = lp;
        a.terms[row] = policy_row(a, row, at.seq, at.w, lp).terms;
        lds_g = at.seq < 0 ? 0.0f : lp;
      }
    }
    if (!out) return;
    if (bad) __syncthreads();                     // NaN only in a sequence
    fill_row<T, THREADS>(out, vocab, bad ? lds_g : 0.0f, threadIdx.x);
    return;
  }
  const T* x = static_cast<const T*>(l.logits) + row * l.ld;
  const RowCut<T> cut(x, vocab, threadIdx.x);
  const int nvec = cut.nvec;
  const float xt = to_f32(x[t]);
  u32x4 d[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * THREADS + (int)threadIdx.x;
    d[i] = vec_neg_inf<T>();
    if (v < nvec) d[i] = load_vec(x + cut.at(v));
  }
  float el = cut.edge >= 0 ? to_f32(x[cut.edge]) : -kInf;
  float e[E], m = el;
  if constexpr (L > 0) {
    u32x4 r[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int v = (V + i) * THREADS + (int)threadIdx.x;
      r[i] = vec_neg_inf<T>();
      if (v < nvec) r[i] = load_vec(x + cut.at(v));
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      if ((V + i) * THREADS >= nvec) break;       // none of the workgroup's
      far[i * THREADS + threadIdx.x] = r[i];
      float f[N];
      unpack<T>(r[i], f);
#pragma unroll
      for (int j = 0; j < N; ++j) m = fmaxf(m, f[j]);
    }
  }
  Place at{-1, 0.0f};
  if (lead) at = policy_place(l, a, row);         // while the logits arrive
#pragma unroll
  for (int i = 0; i < V; ++i) {
    unpack<T>(d[i], e + i * N);
#pragma unroll
    for (int j = 0; j < N; ++j) m = fmaxf(m, e[i * N + j]);
  }
  m = shift(block_max<THREADS>(m, lds_m));
  const float k = l.scale * kLog2e;
  float s = el = term(el, m, k);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    unpack<T>(d[i], e + i * N);
#pragma unroll
    for (int j = 0; j < N; ++j) s += e[i * N + j] = term(e[i * N + j], m, k);
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    if ((V + i) * THREADS >= nvec) break;
    float f[N];
    unpack<T>(far[i * THREADS + threadIdx.x], f);
#pragma unroll
    for (int j = 0; j < N; ++j) s += term(f[j], m, k);
  }
  s = block_sum<THREADS>(s, lds_s);
  if (lead) {
    if (threadIdx.x == 0) {
      const float lp = (xt - m) * l.scale - logf(s);
      const PolicyRow o = policy_row(a, row, at.seq, at.w, lp);
      a.logp[row] = lp;
      a.terms[row] = o.terms;
      lds_g = o.dlogp * l.scale;
    }
  }
  if (!out) return;
  __syncthreads();
  const float g = lds_g, c = -g / s;
  if (g == 0.0f) {
    fill_row<T, THREADS>(out, vocab, 0.0f, threadIdx.x);
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * THREADS + (int)threadIdx.x;
    scale_terms<N>(c, g, (int)t, cut.at(v), e + i * N);
    if (v < nvec) store_vec_once(out + cut.at(v), pack<T>(e + i * N));
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int v = (V + i) * THREADS + (int)threadIdx.x;
    if ((V + i) * THREADS >= nvec) break;
    float f[N];
    unpack<T>(far[i * THREADS + threadIdx.x], f);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = term(f[j], m, k);
    scale_terms<N>(c, g, (int)t, cut.at(v), f);
    if (v < nvec) store_vec_once(out + cut.at(v), pack<T>(f));
  }
  if (cut.edge >= 0) from_f32(el * c + (cut.edge == (int)t ? g : 0.0f), out[cut.edge]);
}

// The same where a row does not fit the registers: it is read a second time,
// from the caches as far as they reach.
template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void k_policy_long(LogitsArgs l, PolicyArgs a, T* dlogits,
                                                         int64_t ldd) {
  __shared__ MaxSum lds[THREADS / 64];
  __shared__ float lds_g;
  const int64_t row = blockIdx.x;
  const int vocab = (int)l.vocab;
  const int64_t t = l.targets[row];
  T* out = dlogits ? dlogits + row * ldd : nullptr;
  const bool lead = threadIdx.x < 64;
  const bool skip = t == l.ignore || t < 0 || t >= l.vocab;
  const T* x = static_cast<const T*>(l.logits) + row * l.ld;
  const float k = l.scale * kLog2e;
  MaxSum v{0.0f, 1.0f};
  if (!skip) v = block_join<THREADS>(stream_row<T, THREADS>(x, vocab, k, threadIdx.x), k, lds);
  const float m = shift(v.m), ls = logf(v.s);
  if (lead) {
    const Place at = policy_place(l, a, row);
    if (threadIdx.x == 0) {
      const float lp = t == l.ignore ? 0.0f
                       : skip        ? __builtin_nanf("")
                                     : (to_f32(x[t]) - m) * l.scale - ls;
      const PolicyRow o = policy_row(a, row, at.seq, at.w, lp);
      a.logp[row] = lp;
      a.terms[row] = o.terms;
      lds_g = !skip ? o.dlogp * l.scale : at.seq < 0 ? 0.0f : lp;
    }
  }
  if (!out) return;
  __syncthreads();
  const float g = lds_g;
  if (skip || g == 0.0f) {
    fill_row<T, THREADS>(out, vocab, g, threadIdx.x);
    return;
  }
  const RowGrad q{g, m, ls * kLog2e, k, (int)t};
  grad_row<T, THREADS>(x, out, vocab, q, threadIdx.x);
}

// Loss and averages from all rows' terms, by one workgroup: its loads' latency
// bounds it, 4 us at 1586 rows and 13.5 at 15315 (2 % of their call).  Many rows
// of a small vocabulary wait for it and for k_policy_count: 131072 x 500 BF16
// takes 142 us, 2^21 x 64 2.1 ms.
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
  p = wave_sum(p);
  k = wave_sum(k);
  c = wave_sum(c);
  const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
  if (lane == 0) {
    lds[0][wave] = p;
    lds[1][wave] = k;
    lds[2][wave] = c;
  }
  __syncthreads();
  if (wave) return;
  p = row16_sum(lane < 16 ? lds[0][lane] : 0.0);
  k = row16_sum(lane < 16 ? lds[1][lane] : 0.0);
  c = row16_sum(lane < 16 ? lds[2][lane] : 0.0);
  if (threadIdx.x == 0) {
    a.stats[0] = (float)(a.kl_coef == 0.0f ? p : p + (double)a.kl_coef * k);
    a.stats[1] = (float)p;
    a.stats[2] = (float)k;
    a.stats[3] = (float)c;
  }
}

template <typename T>
static void logp_by_width(const LogitsArgs& l, float* logp, float* lse, RowStat* stat,
                          hipStream_t st) {
  const dim3 grid((unsigned)l.rows);
  if (l.vocab <= 2048)
    hipLaunchKernelGGL((k_logp<T, 64>), grid, dim3(64), 0, st, l, logp, lse, stat);
  else if (l.vocab <= 16384)
    hipLaunchKernelGGL((k_logp<T, 256>), grid, dim3(256), 0, st, l, logp, lse, stat);
  else
    hipLaunchKernelGGL((k_logp<T, 1024>), grid, dim3(1024), 0, st, l, logp, lse, stat);
}

hipError_t launch_logp(const LogitsArgs& l, float* logp, float* lse, RowStat* stat,
                       hipStream_t st) {
  if (l.type == QLORA_BF16) logp_by_width<uint16_t>(l, logp, lse, stat, st);
  else logp_by_width<float>(l, logp, lse, stat, st);
  return hipGetLastError();
}

// Workgroups of 256 threads that hold a row's vectors and single elements
// (RowCut), at most: whole vectors that start at the second element leave more
// of these.
template <typename T>
static int64_t grad_chunks(const LogitsArgs& l) {
  const int64_t rest = l.vocab % kVec<T>;
  const bool shifted = sizeof(T) == 2 && ((reinterpret_cast<uintptr_t>(l.logits) >> 1 | l.ld) & 1);
  const int64_t units = l.vocab / kVec<T> + (rest || !shifted ? rest : kVec<T> - 1);
  return (units + 255) / 256;
}

template <typename T>
static void dlogits_rows(const LogitsArgs& l, const RowStat* stat, const float* lse,
                         const float* dlogp, T* dlogits, int64_t ldd, hipStream_t st) {
  const int64_t chunks = grad_chunks<T>(l);
  // a launch's threads are counted in 32 bits: at most 2^22 workgroups each
  const int64_t per = std::max<int64_t>(1, (int64_t(1) << 22) / chunks);
  for (int64_t end = l.rows; end > 0; end -= per) {
    const int64_t rows = std::min(per, end);
    const dim3 grid((unsigned)(rows * chunks));
    if (stat)
      hipLaunchKernelGGL((k_dlogits<T, true>), grid, dim3(256), 0, st, l, stat, lse, dlogp, dlogits,
                         ldd, end - 1, (uint32_t)chunks);
    else
      hipLaunchKernelGGL((k_dlogits<T, false>), grid, dim3(256), 0, st, l, stat, lse, dlogp, dlogits,
                         ldd, end - 1, (uint32_t)chunks);
  }
}

hipError_t launch_dlogits(const LogitsArgs& l, const RowStat* stat, const float* lse,
                          const float* dlogp, void* dlogits, int64_t ldd, hipStream_t st) {
  if (l.type == QLORA_BF16)
    dlogits_rows(l, stat, lse, dlogp, static_cast<uint16_t*>(dlogits), ldd, st);
  else dlogits_rows(l, stat, lse, dlogp, static_cast<float*>(dlogits), ldd, st);
  return hipGetLastError();
}

// A call on few rows is bound by its launches.  Batches of at most 32 rows and
// 2^16 logits take one, a workgroup a pair: 14 us a call against 16 with two at
// 30 x 1000, no gain any more at 60 x 1000.  The pairs' lengths are not known
// here, so the batch is bounded: one pair may hold all of it (32 pairs of 1000 x
// 1000 logits, all in one of them: 243 us against 17; spread evenly 14).
static bool small_batch(const LogitsArgs& l) {
  return l.rows <= 32 && l.rows * l.vocab <= int64_t(1) << 16;
}
// Batches of up to kFewBlocks workgroups of gradients take two, every workgroup
// summing its row's pair again: 14.5 us a call against 17.1 with three (128 x
// 32000 or 2048 x 2000 BF16, 2048 workgroups); at 3072 17 us both, at 4096 19
// to 24 against 17 to 19.  Finding a row's pair takes longer among more (256:
// 16.1 us, 1024: no gain).
constexpr int64_t kFewBlocks = 2048, kFewPairs = 256;

template <typename T>
static hipError_t preference_as(const LogitsArgs& l, const PreferenceArgs& a, RowStat* stat,
                                float* logp, T* dlogits, int64_t ldd, hipStream_t st) {
  const dim3 grid((unsigned)std::max<int64_t>(a.pairs, 1));
  if (a.pairs > 0 && small_batch(l)) {
    hipLaunchKernelGGL(k_preference_small<T>, grid, dim3(kPrefThreads), 0, st, l, a, stat, logp,
                       dlogits, ldd);
    return hipGetLastError();
  }
  const hipError_t e = launch_logp(l, logp, nullptr, stat, st);
  if (e != hipSuccess) return e;
  const int64_t chunks = grad_chunks<T>(l);
  if (l.rows * chunks <= kFewBlocks && a.pairs <= kFewPairs) {
    const int64_t blocks = a.pairs + (dlogits ? l.rows * chunks : 0);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL(k_pairs_dlogits<T>, dim3((unsigned)blocks), dim3(256), 0, st, l, a, stat,
                       dlogits, ldd, (uint32_t)chunks);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_preference, grid, dim3(kPrefThreads), 0, st, a);
  if (!dlogits) return hipGetLastError();
  return launch_dlogits(l, stat, nullptr, a.dlogp, dlogits, ldd, st);
}

hipError_t launch_preference(const LogitsArgs& l, const PreferenceArgs& a, RowStat* stat,
                             float* logp, void* dlogits, int64_t ldd, hipStream_t st) {
  if (l.type == QLORA_BF16)
    return preference_as(l, a, stat, logp, static_cast<uint16_t*>(dlogits), ldd, st);
  return preference_as(l, a, stat, logp, static_cast<float*>(dlogits), ldd, st);
}

template <typename T, int THREADS, int E, int L, int MIN_WAVES>
static void policy_held(const LogitsArgs& l, const PolicyArgs& a, T* dlogits, int64_t ldd,
                        hipStream_t st) {
  hipLaunchKernelGGL((k_policy<T, THREADS, E, L, MIN_WAVES>), dim3((unsigned)l.rows),
                     dim3(THREADS), (size_t)L * THREADS * 16, st, l, a, dlogits, ldd);
}

// The fewest threads, and logits a thread, that hold the row; steps that
// leave fewer of them idle were kept where they measured faster (us at 2^30
// bytes or less of logits): 128 threads at 3200 BF16 98 against 124, at 4000
// FP32 110 against 103; 768 at 20000 BF16 124 against 140; 48 logits at 36000
// BF16 242 against 260.
template <typename T>
static void policy_by_width(const LogitsArgs& l, const PolicyArgs& a, T* dlogits, int64_t ldd,
                            hipStream_t st) {
  constexpr int kFar = 65536 + 8 * 1024 * kVec<T>;   // with 128 KB of LDS
  const int64_t v = l.vocab;
  if constexpr (sizeof(T) == 2) {
    if (v > 2048 && v <= 4096) return policy_held<T, 128, 32, 0, 8>(l, a, dlogits, ldd, st);
  }
  if (v <= 512) policy_held<T, 64, 8, 0, 8>(l, a, dlogits, ldd, st);
  else if (v <= 2048) policy_held<T, 64, 32, 0, 6>(l, a, dlogits, ldd, st);
  else if (v <= 8192) policy_held<T, 256, 32, 0, 8>(l, a, dlogits, ldd, st);
  else if (v <= 16384) policy_held<T, 512, 32, 0, 8>(l, a, dlogits, ldd, st);
  else if (v <= 24576) policy_held<T, 768, 32, 0, 6>(l, a, dlogits, ldd, st);
  else if (v <= 32768) policy_held<T, 1024, 32, 0, 8>(l, a, dlogits, ldd, st);
  else if (v <= 49152) policy_held<T, 1024, 48, 0, 4>(l, a, dlogits, ldd, st);
  else if (v <= 65536) policy_held<T, 1024, 64, 0, 4>(l, a, dlogits, ldd, st);
  else if (v <= kFar) policy_held<T, 1024, 64, 8, 4>(l, a, dlogits, ldd, st);
  else
    hipLaunchKernelGGL((k_policy_long<T, 1024>), dim3((unsigned)l.rows), dim3(1024), 0, st, l, a,
                       dlogits, ldd);
}

// Every row needs the number of all rows that count.  Summed in each row's
// workgroup it costs a call of 8192 x 32000 BF16 92 us with 2048 sequences (277
// against 185), 18 with 512, 8 with 256; summed once, 2 to 3.
constexpr int64_t kFewCounts = 256;

hipError_t launch_policy(const LogitsArgs& l, const PolicyArgs& args, void* dlogits, int64_t ldd,
                         hipStream_t st) {
  PolicyArgs a = args;
  const bool bf16 = l.type == QLORA_BF16;
  if (l.rows > 0) {
    // in a batch of few rows a row's workgroup finds its sequence and weight
    // by itself: one launch less (20.5 to 17.3 us a call at 23 rows, no
    // difference any more at 1586)
    if (l.rows <= 1024 && a.seqs < 1024) a.row_seq = nullptr;
    if (a.row_seq)
      hipLaunchKernelGGL(k_policy_count, dim3((unsigned)std::max<int64_t>(a.seqs, 1)), dim3(256), 0,
                         st, l, a);
    if (!a.row_seq || a.reduction != QLORA_POLICY_TOKEN_MEAN || a.seqs <= kFewCounts)
      a.total = nullptr;
    if (a.total) hipLaunchKernelGGL(k_policy_total, dim3(1), dim3(1024), 0, st, a);
    if (bf16) policy_by_width(l, a, static_cast<uint16_t*>(dlogits), ldd, st);
    else policy_by_width(l, a, static_cast<float*>(dlogits), ldd, st);
  }
  hipLaunchKernelGGL(k_policy_stats, dim3(1), dim3(1024), 0, st, a, l.rows);
  return hipGetLastError();
}

}  // namespace qlora
