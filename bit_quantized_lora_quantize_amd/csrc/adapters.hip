// adapters.hip -- low-rank adapters of many requests beside one shared
// projection, forward and backward, and the token contractions that read an
// input kept in 8 bits (gfx950).
//
// Token m has the adapter a = index[m] of a bank (A [slots][r][d_in],
// B [slots][d_out][r], scale [slots]) or none:
//   forward    T = s_a X A_a^T          Y  = RN(Y0 + T B_a^T)
//   backward   U = s_a dY B_a           dX = RN(dX0 + U A_a)
//              dA_a = sum_m U^T X       dB_a = sum_m dY^T T   over a's tokens
//
// k_plan_* sort the tokens by slot (stable, so that every sum over tokens has
// one order) into tiles of up to 64 tokens of one slot; the other kernels walk
// that list, whose length only the device knows.  Two launches make a forward:
// k_shrink (FP32 partial sums over ranges of the long axis) and k_expand, which
// adds the partials, and with them the shared projection's output.  A backward
// adds k_frags (T and U as matrix operands) and k_gram (the contractions over
// tokens).  Products are BF16 on the matrix cores with FP32 sums; T and U are
// FP32 and enter them as sums of BF16 terms: two (16 bits) where the result is
// rounded to BF16, three (24 bits, all of FP32) where it is FP32.
#include "qlora_device.h"
#include "qlora_kernels.h"

namespace qlora {

namespace {

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;

// Four rows x 16 columns of 16-bit values in LDS, transposed: lane j of a group
// of 16 points at columns 4 (j % 4) .. +4 of row j / 4 and gets column j.
__device__ __forceinline__ uint2 lds_tr(const uint16_t* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)p));
}

__device__ __forceinline__ uint16_t bf16_bits(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }

// Eight elements from column `col` on, zero at and past `end`.  VEC: `row` and
// `end` allow whole 16-byte pieces.
template <bool VEC>
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t col, int64_t end) {
  if (VEC) {
    u32x4 v = {0, 0, 0, 0};
    if (col < end) v = *reinterpret_cast<const u32x4*>(row + col);
    return v;
  }
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = col + e < end ? (uint32_t)row[col + e] : 0u;
  return u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
}

// A plan of other sizes than the call's: nothing is done for it.
__device__ __forceinline__ bool plan_fits(const PlanView& p, int64_t M, int64_t slots) {
  return p.head[kPlanMagicAt] == kPlanMagic && p.head[kPlanTokens] == (int)M &&
         p.head[kPlanSlots] == (int)slots;
}

// ---------------------------------------------------------------------------
// The plan.  Tokens in spans of 1024, one wavefront a span; a span's tokens are
// ranked 64 at a time: the lanes of equal slots find each other by one ballot
// per bit of the slot.
// ---------------------------------------------------------------------------
constexpr int kSpan = 1024;

__device__ __forceinline__ int slot_of(const int32_t* index, int64_t m, int slots) {
  const int a = index[m];
  return a >= 0 && a < slots ? a : slots;
}

// Lanes of the wavefront with this lane's key (active lanes only).
__device__ __forceinline__ uint64_t same_key(int key, bool active, int bits) {
  uint64_t peers = __ballot(active);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot(active && ((key >> b) & 1));
    peers &= ((key >> b) & 1) ? set : ~set;
  }
  return peers;
}

// Exclusive sums over a workgroup of 256 threads of four counts each; `total`
// gets the sums.
__device__ __forceinline__ int4 scan4(int4 v, int4* lds, int4& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int4 s = v;
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const int4 o = {__shfl_up(s.x, off), __shfl_up(s.y, off), __shfl_up(s.z, off),
                    __shfl_up(s.w, off)};
    if (lane >= off) {
      s.x += o.x;
      s.y += o.y;
      s.z += o.z;
      s.w += o.w;
    }
  }
  if (lane == 63) lds[w] = s;
  __syncthreads();
  int4 base = {0, 0, 0, 0};
  total = base;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int4 o = lds[i];
    if (i < w) {
      base.x += o.x;
      base.y += o.y;
      base.z += o.z;
      base.w += o.w;
    }
    total.x += o.x;
    total.y += o.y;
    total.z += o.z;
    total.w += o.w;
  }
  __syncthreads();
  return int4{base.x + s.x - v.x, base.y + s.y - v.y, base.z + s.z - v.z, base.w + s.w - v.w};
}

// From the tokens of every slot (cnt[0 .. slots], the last without adapter) to
// the plan's lists; cnt becomes the first position of every slot.  tile0 and
// split0 [slots + 2] are scratch.
__device__ void plan_lists(const PlanView& p, int M, int slots, int tps, int* cnt, int* tile0,
                           int* split0, int4* red) {
  // (tokens, tiles, splits, parts) of each slot, scanned in rounds of 256
  int4 carry = {0, 0, 0, 0};
  for (int s0 = 0; s0 <= slots; s0 += 256) {
    const int s = s0 + (int)threadIdx.x;
    int4 v = {0, 0, 0, 0};
    int parts = 0;
    if (s <= slots) {
      v.x = cnt[s];
      v.y = (v.x + kPlanTile - 1) / kPlanTile;
      v.z = s < slots ? (v.y + tps - 1) / tps : 0;
      parts = v.z;
      v.w = v.z > 1 ? v.z : 0;
    }
    int4 total;
    const int4 e = scan4(v, red, total);
    if (s <= slots) {
      cnt[s] = carry.x + e.x;
      tile0[s] = carry.y + e.y;
      split0[s] = carry.z + e.z;
      if (s < slots) p.parts[s] = int2{carry.w + e.w, parts};
    }
    carry.x += total.x;
    carry.y += total.y;
    carry.z += total.z;
    carry.w += total.w;
  }
  if (threadIdx.x == 0) {
    tile0[slots + 1] = carry.y;
    split0[slots + 1] = carry.z;
  }
  __syncthreads();
  const int tiles = carry.y, with_one = tile0[slots];
  for (int t = threadIdx.x; t < tiles; t += 256) {
    int lo = 0, hi = slots;   // the last slot whose first tile is t or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (tile0[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int end = lo < slots ? cnt[lo + 1] : M;
    const int first = cnt[lo] + (t - tile0[lo]) * kPlanTile;
    p.tile[t] = int4{lo < slots ? lo : -1, first, min(kPlanTile, end - first), 0};
  }
  for (int i = threadIdx.x; i < carry.z; i += 256) {
    int lo = 0, hi = slots - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (split0[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const int j = i - split0[lo], n = split0[lo + 1] - split0[lo];
    const int first = tile0[lo] + j * tps;
    p.split[i] = int4{lo, first, min(tps, tile0[lo + 1] - first), n > 1 ? j : -1};
  }
  if (threadIdx.x == 0) {
    p.head[kPlanTiles] = with_one;
    p.head[kPlanAllTiles] = tiles;
    p.head[kPlanSplits] = carry.z;
    p.head[kPlanTokens] = M;
    p.head[kPlanSlots] = slots;
    p.head[kPlanMagicAt] = kPlanMagic;
  }
}

// Places a span's tokens: `next` (LDS, [slots + 1]) holds the next position of
// every slot.  One wavefront.
__device__ __forceinline__ void place_span(const PlanView& p, const int32_t* index, int64_t m0,
                                           int64_t M, int slots, int bits, int* next) {
  const int lane = threadIdx.x & 63;
  const int64_t end = min(M, m0 + kSpan);
  for (int64_t m = m0; m < end; m += 64) {
    const bool active = m + lane < end;
    const int key = active ? slot_of(index, m + lane, slots) : 0;
    const uint64_t peers = same_key(key, active, bits);
    const int rank = __popcll(peers & ((uint64_t(1) << lane) - 1));
    int at = 0;
    if (active && rank == 0) {         // the first lane of each slot counts for all of them
      at = next[key];
      next[key] = at + __popcll(peers);
    }
    at = __shfl(at, active ? __ffsll((unsigned long long)peers) - 1 : lane);
    if (active) p.order[at + rank] = (int)(m + lane);
  }
}

// Up to one span: everything in one workgroup.
__global__ __launch_bounds__(256) void k_plan_small(PlanView p, const int32_t* __restrict__ index,
                                                    int M, int slots, int tps, int bits) {
  __shared__ int cnt[kPlanMaxSlots + 2], tile0[kPlanMaxSlots + 2], split0[kPlanMaxSlots + 2];
  __shared__ int4 red[4];
  for (int s = threadIdx.x; s <= slots; s += 256) cnt[s] = 0;
  __syncthreads();
  for (int m = threadIdx.x; m < M; m += 256) atomicAdd(&cnt[slot_of(index, m, slots)], 1);
  __syncthreads();
  plan_lists(p, M, slots, tps, cnt, tile0, split0, red);
  __syncthreads();
  if (threadIdx.x < 64) place_span(p, index, 0, M, slots, bits, cnt);
}

// Tokens of every slot in each span.
__global__ __launch_bounds__(64) void k_plan_count(const int32_t* __restrict__ index, int64_t M,
                                                   int slots, int32_t* __restrict__ hist) {
  __shared__ int cnt[kPlanMaxSlots + 1];
  for (int s = threadIdx.x; s <= slots; s += 64) cnt[s] = 0;
  __syncthreads();
  const int64_t m0 = (int64_t)blockIdx.x * kSpan, end = min(M, m0 + kSpan);
  for (int64_t m = m0 + threadIdx.x; m < end; m += 64) atomicAdd(&cnt[slot_of(index, m, slots)], 1);
  __syncthreads();
  int32_t* h = hist + (int64_t)blockIdx.x * (slots + 1);
  for (int s = threadIdx.x; s <= slots; s += 64) h[s] = cnt[s];
}

// The lists, and in hist the first position of every span's tokens of each slot.
__global__ __launch_bounds__(256) void k_plan_lists(PlanView p, int M, int slots, int tps,
                                                    int spans, int32_t* __restrict__ hist) {
  __shared__ int cnt[kPlanMaxSlots + 2], tile0[kPlanMaxSlots + 2], split0[kPlanMaxSlots + 2];
  __shared__ int4 red[4];
  for (int s = threadIdx.x; s <= slots; s += 256) {
    int sum = 0;
    for (int b = 0; b < spans; ++b) {
      const int64_t at = (int64_t)b * (slots + 1) + s;
      const int c = hist[at];
      hist[at] = sum;
      sum += c;
    }
    cnt[s] = sum;
  }
  __syncthreads();
  plan_lists(p, M, slots, tps, cnt, tile0, split0, red);
  __syncthreads();
  for (int s = threadIdx.x; s <= slots; s += 256) p.begin[s] = cnt[s];
}

__global__ __launch_bounds__(64) void k_plan_place(PlanView p, const int32_t* __restrict__ index,
                                                   int64_t M, int slots, int bits,
                                                   const int32_t* __restrict__ hist) {
  __shared__ int next[kPlanMaxSlots + 1];
  const int32_t* h = hist + (int64_t)blockIdx.x * (slots + 1);
  for (int s = threadIdx.x; s <= slots; s += 64) next[s] = p.begin[s] + h[s];
  __syncthreads();
  place_span(p, index, (int64_t)blockIdx.x * kSpan, M, slots, bits, next);
}

// ---------------------------------------------------------------------------
// part[s][p][i] = sum over k in range s of P[token p][k] F[i][k] for the tokens
// of a tile and the factor of their slot; F is stored [r][K] (A in the forward)
// or, KN, [K][r] (B in the backward).
//
// Item = one tile and one of `splits` ranges of K.  The W wavefronts of a
// workgroup take the range's steps of 32 columns in turn, each all 64 tokens and
// all ranks: no wavefront loads what another loads, and the loop has no
// barrier.  Their sums are added through LDS at the end, in wavefront order.
// KN: a step's 32 rows of F go through LDS of the wavefront's own, which the
// transposing reads turn into operands.
// ---------------------------------------------------------------------------
template <int NB>
constexpr int shrink_waves() { return NB <= 4 ? 8 : 4; }
template <int NB, bool KN>
constexpr int shrink_lds() {
  constexpr int W = shrink_waves<NB>(), CN = NB < 4 ? NB : 4;
  constexpr int red = W * 16 * 16 * CN * 4, stage = KN ? W * 32 * (16 * NB + 8) * 2 : 0;
  return red > stage ? red : stage;
}

template <int NB, bool KN, bool VEC>
__global__ __launch_bounds__(64 * shrink_waves<NB>()) void k_shrink(ShrinkArgs a) {
  constexpr int W = shrink_waves<NB>(), CN = NB < 4 ? NB : 4;
  constexpr int LF = 16 * NB + 8;                  // staged row of F, elements
  extern __shared__ __attribute__((aligned(16))) uint8_t slds[];
  if (!plan_fits(a.plan, a.M, a.slots)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t K = a.K;
  const int r = a.r;
  const int items = a.plan.head[kPlanTiles] * a.splits;
  uint16_t* stage = reinterpret_cast<uint16_t*>(slds) + w * 32 * LF;
  float* red = reinterpret_cast<float*>(slds);

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int t = item / a.splits, s = item % a.splits;
    const int4 td = a.plan.tile[t];
    const int slot = td.x, first = td.y, count = td.z;
    const int64_t k_begin = (int64_t)s * a.kper;
    const int64_t k_end = k_begin + a.kper < K ? k_begin + a.kper : K;
    const uint16_t* xp[4];   // rows past the tile's last repeat it; their sums are not stored
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      const int row = min(16 * rb + r16, count - 1);
      xp[rb] = a.P + (int64_t)a.plan.order[first + row] * K;
    }
    const uint16_t* F = a.F + (int64_t)slot * r * K;

    f32x4 acc[4][NB];
#pragma unroll
    for (int rb = 0; rb < 4; ++rb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[rb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};

    // whole steps: loads without conditions, a step ahead
    auto load = [&](int64_t k, u32x4 (&x)[4], u32x4 (&f)[NB]) {
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) x[rb] = *reinterpret_cast<const u32x4*>(xp[rb] + k + 8 * g);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (KN) {
          const int piece = lane + 64 * nb, row = piece / (2 * NB), col = 8 * (piece % (2 * NB));
          f[nb] = *reinterpret_cast<const u32x4*>(F + (k + row) * r + (col < r ? col : 0));
        } else {
          const int i = min(16 * nb + r16, r - 1);
          f[nb] = *reinterpret_cast<const u32x4*>(F + i * K + k + 8 * g);
        }
      }
    };
    auto put_stage = [&](const u32x4 (&f)[NB]) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int piece = lane + 64 * nb, row = piece / (2 * NB), col = 8 * (piece % (2 * NB));
        *reinterpret_cast<u32x4*>(stage + row * LF + col) = f[nb];
      }
    };
    auto compute = [&](const u32x4 (&x)[4], const u32x4 (&f)[NB]) {
      if (KN) put_stage(f);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        u32x4 q = f[nb];
        if (KN) {
          const uint16_t* p = stage + (8 * g + (r16 >> 2)) * LF + 16 * nb + 4 * (r16 & 3);
          const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * LF);
          q = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
#pragma unroll
        for (int rb = 0; rb < 4; ++rb) acc[rb][nb] = mfma16(x[rb], q, acc[rb][nb]);
      }
    };
    int64_t k = k_begin + 32 * w;
    const int64_t k_whole = k_begin + (VEC ? (k_end - k_begin) / 32 * 32 : 0);
    if (k < k_whole) {
      const int64_t k_last = k + (k_whole - 1 - k) / (32 * W) * (32 * W);
      u32x4 xa[4], fa[NB], xb[4], fb[NB];
      load(k, xa, fa);
      for (; k <= k_last; k += 64 * W) {
        load(min(k + 32 * W, k_last), xb, fb);
        compute(xa, fa);
        load(min(k + 64 * W, k_last), xa, fa);
        if (k + 32 * W <= k_last) compute(xb, fb);
      }
      k = k_last + 32 * W;
    }
    // the rest: single elements, or the pieces of a last, partial step
    for (; k < k_end; k += 32 * W) {
      u32x4 x[4], f[NB];
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) x[rb] = load8<VEC>(xp[rb], k + 8 * g, k_end);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (KN) {
          const int piece = lane + 64 * nb, row = piece / (2 * NB), col = 8 * (piece % (2 * NB));
          f[nb] = k + row < k_end ? load8<VEC>(F + (k + row) * r, col, r) : u32x4{0, 0, 0, 0};
        } else {
          f[nb] = load8<VEC>(F + min(16 * nb + r16, r - 1) * K, k + 8 * g, k_end);
        }
      }
      compute(x, f);
    }

    // accumulator lane (r16, g): tokens 16 rb + 4 g + v, rank 16 nb + r16
    float* part = a.part + ((int64_t)s * a.M + first) * r;
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) {
      if (16 * rb >= count) break;
#pragma unroll
      for (int n0 = 0; n0 < NB; n0 += CN) {
        __syncthreads();   // the stage, or the last block, is no longer read
#pragma unroll
        for (int nb = 0; nb < CN; ++nb)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            red[(w * 16 + 4 * g + v) * 16 * CN + 16 * nb + r16] = acc[rb][n0 + nb][v];
        __syncthreads();
        for (int e = threadIdx.x; e < 256 * CN; e += 64 * W) {
          const int row = e / (16 * CN), i = 16 * n0 + e % (16 * CN);
          float sum = red[e];
#pragma unroll
          for (int ww = 1; ww < W; ++ww) sum += red[ww * 256 * CN + e];
          if (16 * rb + row < count && i < r) part[(int64_t)(16 * rb + row) * r + i] = sum;
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// out[token][n] = RN(in[token][n] + sum_i V[token][i] F[n][i]),
// V = scale_a * (the partial sums of k_shrink, in order), for the tokens of a
// tile and a chunk of n.  F is stored [d][r] (B in the forward) or, RN_,
// [r][d] (A in the backward).  The tile's V goes to LDS as BF16 hi + lo; a
// wavefront takes 64 columns at a time, all tokens.  F is the row operand of
// the MFMA: with its rows n = 16 (j / 4) + 4 blk + j % 4 a lane ends up with 16
// consecutive columns of one token.
// ---------------------------------------------------------------------------
template <int KS, bool RD, bool VEC>
__global__ __launch_bounds__(256) void k_expand(ExpandArgs a) {
  constexpr int LT = 32 * KS + 8;                  // LDS row of V, elements
  constexpr int LF = 72;                           // staged row of F
  extern __shared__ __attribute__((aligned(16))) uint8_t elds[];
  uint16_t* th = reinterpret_cast<uint16_t*>(elds);
  uint16_t* tl = th + 64 * LT;
  if (!plan_fits(a.plan, a.M, a.slots)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  uint16_t* stage = tl + 64 * LT + w * 32 * LF;
  const int r = a.r;
  const int64_t d = a.d;
  const bool copy = a.in != a.out;                 // tokens without an adapter are written too
  const int items = a.plan.head[copy || a.v_out ? kPlanAllTiles : kPlanTiles] * a.chunks;

  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int t = item / a.chunks, c = item % a.chunks;
    const int4 td = a.plan.tile[t];
    const int slot = td.x, first = td.y, count = td.z;
    const int nrb = (count + 15) / 16;
    if (slot >= 0) {
      __syncthreads();                             // the last item's V is no longer read
      const float sc = a.scale[slot];
      const float* part = a.part + (int64_t)first * r;
      for (int e = threadIdx.x; e < 16 * nrb * 32 * KS; e += 256) {
        const int row = e / (32 * KS), i = e % (32 * KS);
        float v = 0.0f;
        if (row < count && i < r) {
          const float* p = part + row * r + i;
          v = p[0];
          for (int s = 1; s < a.splits; ++s) v += p[(int64_t)s * a.M * r];
          v *= sc;
          if (a.v_out && c == 0) a.v_out[(int64_t)a.plan.order[first + row] * r + i] = v;
        }
        float hi, lo;
        split_bf16(v, hi, lo);
        th[row * LT + i] = (uint16_t)(__float_as_uint(hi) >> 16);
        tl[row * LT + i] = bf16_bits(lo);
      }
      __syncthreads();
    } else if (a.v_out && c == 0) {
      for (int e = threadIdx.x; e < count * r; e += 256)
        a.v_out[(int64_t)a.plan.order[first + e / r] * r + e % r] = 0.0f;
    }
    if (slot < 0 && !copy) continue;
    const uint16_t* F = a.F + (slot >= 0 ? (int64_t)slot * r * d : 0);
    int64_t tok[4];
#pragma unroll
    for (int rb = 0; rb < 4; ++rb) tok[rb] = a.plan.order[first + min(16 * rb + r16, count - 1)];
    const int64_t c_begin = (int64_t)c * a.cper;
    const int64_t c_end = c_begin + a.cper < d ? c_begin + a.cper : d;
    for (int64_t col0 = c_begin + 64 * w; col0 < c_end; col0 += 256) {
      const int64_t col = col0 + 16 * g;           // the lane's 16 columns
      u32x4 y[4][2];
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) {
        y[rb][0] = y[rb][1] = u32x4{0, 0, 0, 0};
        if (a.in && rb < nrb) {
          y[rb][0] = load8<VEC>(a.in + tok[rb] * d, col, d);
          y[rb][1] = load8<VEC>(a.in + tok[rb] * d, col + 8, d);
        }
      }
      f32x4 acc[4][4];
#pragma unroll
      for (int rb = 0; rb < 4; ++rb)
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[rb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (slot >= 0) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          u32x4 f[4];
          if (RD) {
            // rows i of F: 64 columns through LDS
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int i = 32 * ks + (lane >> 3) + 8 * u, cc = 8 * (lane & 7);
              u32x4 v = {0, 0, 0, 0};
              if (i < r) v = load8<VEC>(F + (int64_t)i * d, col0 + cc, d);
              *reinterpret_cast<u32x4*>(stage + ((lane >> 3) + 8 * u) * LF + cc) = v;
            }
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint16_t* p = stage + (8 * g + (r16 >> 2)) * LF + 16 * (r16 & 3) + 4 * b;
              const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * LF);
              f[b] = u32x4{lo.x, lo.y, hi.x, hi.y};
            }
          } else {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int64_t n = col0 + 16 * (r16 >> 2) + 4 * b + (r16 & 3);
              f[b] = load8<VEC>(F + (n < d ? n : d - 1) * r, 32 * ks + 8 * g, r);
            }
          }
#pragma unroll
          for (int rb = 0; rb < 4; ++rb) {
            if (rb < nrb) {
              const int at = (16 * rb + r16) * LT + 32 * ks + 8 * g;
              const u32x4 vh = *reinterpret_cast<const u32x4*>(th + at);
              const u32x4 vl = *reinterpret_cast<const u32x4*>(tl + at);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                acc[rb][b] = mfma16(f[b], vh, acc[rb][b]);
                acc[rb][b] = mfma16(f[b], vl, acc[rb][b]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int rb = 0; rb < 4; ++rb) {
        if (16 * rb + r16 >= count) continue;
        uint16_t* out = a.out + tok[rb] * d;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4 o;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int b = 2 * h + j / 2, v = 2 * (j & 1);
            o[j] = pack_bf16x2(bf16lo_to_f32(y[rb][h][j]) + acc[rb][b][v],
                               bf16hi_to_f32(y[rb][h][j]) + acc[rb][b][v + 1]);
          }
          const int64_t n = col + 8 * h;
          if (VEC) {
            if (n < d) *reinterpret_cast<u32x4*>(out + n) = o;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (n + e < d) out[n + e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// T and U as row operands of the contractions over tokens: per tile, BF16 term
// (hi, mid, lo: 24 bits together), 16 ranks and 32 tokens one KB in the order
// of an MFMA's lanes; zero past the tile's tokens and past the rank.  U comes
// from k_shrink's partial sums by position (or a whole U by token), T by token.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_frags(FragArgs a) {
  constexpr int L = 72;
  __shared__ __attribute__((aligned(16))) uint16_t st[3][64 * L];
  if (a.plan.head && !plan_fits(a.plan, a.M, a.slots)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int r = a.r, nb = a.nb, groups = (nb + 3) / 4;
  const int tiles = a.plan.head ? a.plan.head[kPlanTiles] : (int)((a.M + 63) / 64);
  for (int item = blockIdx.x; item < tiles * groups * 2; item += gridDim.x) {
    const int src = item & 1, grp = (item >> 1) % groups, t = (item >> 1) / groups;
    int4 td = {0, 64 * t, (int)min((int64_t)64, a.M - 64 * (int64_t)t), 0};
    if (a.plan.head) td = a.plan.tile[t];
    const int first = td.y, count = td.z, i0 = 64 * grp;
    const bool by_part = src == 1 && a.splits > 0;
    const float sc = by_part ? a.scale[td.x] : 1.0f;
    const float* v_in = src == 0 ? a.T : a.U;
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * 64; e += 256) {
      const int row = e >> 6, i = i0 + (e & 63);
      float v = 0.0f;
      if (row < count && i < r) {
        if (by_part) {
          const float* p = a.U + (int64_t)(first + row) * r + i;
          v = p[0];
          for (int s = 1; s < a.splits; ++s) v += p[(int64_t)s * a.M * r];
          v *= sc;
        } else {
          const int64_t tok = a.plan.head ? a.plan.order[first + row] : first + row;
          v = v_in[tok * r + i];
        }
      }
      float hi, rest;
      split_bf16(v, hi, rest);
      float mid, lo;
      split_bf16(rest, mid, lo);
      const int at = row * L + (e & 63);
      st[0][at] = (uint16_t)(__float_as_uint(hi) >> 16);
      st[1][at] = (uint16_t)(__float_as_uint(mid) >> 16);
      st[2][at] = bf16_bits(lo);
    }
    __syncthreads();
    uint16_t* out = src == 0 ? a.t_frags : a.u_frags;
    for (int u = w; u < 24; u += 4) {              // (term, 16 ranks, 32 tokens)
      const int term = u >> 3, b = (u >> 1) & 3, slice = u & 1;
      if (4 * grp + b >= nb) continue;
      const uint16_t* p = &st[term][(32 * slice + 8 * g + (r16 >> 2)) * L + 16 * b + 4 * (r16 & 3)];
      const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * L);
      const int64_t at = (((int64_t)t * 3 + term) * nb + 4 * grp + b) * 2 + slice;
      *reinterpret_cast<u32x4*>(out + at * 512 + lane * 8) = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  }
}

// ---------------------------------------------------------------------------
// out[i][c] = sum over the tokens of a split of V[token][i] Q[token][c]: dA
// from (U, X), dB (stored [c][i]) from (T, dY).  Item = a split (tiles of one
// slot) and 64 columns; its four wavefronts take the tiles in turn, stage 64
// tokens x 64 columns in LDS of their own (where 8-bit codes become BF16) and
// read the column operands transposed; their sums are added through LDS in
// wavefront order.  A slot's only split is its gradient; else the splits'
// results are added by k_gram_sum.
// ---------------------------------------------------------------------------
constexpr int kGL = 72;   // staged row, elements

// 64 tokens x 64 columns: BF16 as eight 16-byte pieces a lane (row 8 j + l / 8),
// codes as four (row 16 j + l / 4) with their rows' scales.
struct GramTile {
  u32x4 v[8];
  float s[4];
  uint32_t keep[4];
};

// tok: the lane's token of the tile (lane = row), -1 past its last.
template <bool PACKED, bool VEC>
__device__ __forceinline__ void gram_load(const GramSide& q, int64_t M, int64_t c0, int tok,
                                          int lane, GramTile& t) {
  if constexpr (PACKED) {
    const int64_t ldc = (q.d + 63) / 64 * 64;
    const float* sc = q.scale + c0 / 64 * M;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = __shfl(tok, 16 * j + (lane >> 2));
      t.v[j] = u32x4{0, 0, 0, 0};
      t.s[j] = 0.0f;
      t.keep[j] = 0xFFFFu;
      if (m >= 0) {
        t.v[j] = *reinterpret_cast<const u32x4*>(q.codes + m * ldc + c0 + 16 * (lane & 3));
        t.s[j] = sc[m];
        if (q.keep) {
          const int64_t col = c0 + 16 * (lane & 3);
          t.keep[j] = q.keep[m * (q.d / 32) + col / 32] >> (col & 16);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int m = __shfl(tok, 8 * j + (lane >> 3));
      t.v[j] = u32x4{0, 0, 0, 0};
      if (m >= 0) t.v[j] = load8<VEC>(q.x + m * q.d, c0 + 8 * (lane & 7), q.d);
    }
  }
}

template <bool PACKED>
__device__ __forceinline__ void gram_stage(const GramTile& t, int lane, uint16_t* st) {
  if constexpr (PACKED) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4 o[2];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const uint32_t c = t.v[j][h >> 1] >> (16 * (h & 1));
        const uint32_t b = pack_bf16x2((float)(int8_t)c * t.s[j], (float)(int8_t)(c >> 8) * t.s[j]);
        const uint32_t k = t.keep[j] >> (2 * h);
        o[h >> 2][h & 3] = b & (((k & 1) ? 0xFFFFu : 0u) | ((k & 2) ? 0xFFFF0000u : 0u));
      }
      u32x4* p = reinterpret_cast<u32x4*>(st + (16 * j + (lane >> 2)) * kGL + 16 * (lane & 3));
      p[0] = o[0];
      p[1] = o[1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<u32x4*>(st + (8 * j + (lane >> 3)) * kGL + 8 * (lane & 7)) = t.v[j];
  }
}

template <int NB, bool PACKED, bool VEC>
__device__ __forceinline__ void gram_item(const GramArgs8& a, const GramSide& q, int64_t c0,
                                          const int4& sp, uint16_t* st, f32x4 (&acc)[NB][4]) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int t_end = sp.y + sp.z;
  auto token = [&](int t) {
    if (!a.plan.head) {
      const int64_t m = 64 * (int64_t)t + lane;
      return m < a.M ? (int)m : -1;
    }
    const int4 td = a.plan.tile[t];
    return lane < td.z ? a.plan.order[td.y + lane] : -1;
  };
  GramTile cur;
  int t = sp.y + w;
  if (t < t_end) gram_load<PACKED, VEC>(q, a.M, c0, token(t), lane, cur);
  for (; t < t_end; t += 4) {
    gram_stage<PACKED>(cur, lane, st);
    if (t + 4 < t_end) gram_load<PACKED, VEC>(q, a.M, c0, token(t + 4), lane, cur);
    const uint16_t* fr = q.frags + (int64_t)t * 3 * NB * 2 * 512 + lane * 8;
#pragma unroll
    for (int slice = 0; slice < 2; ++slice) {
      u32x4 b[4];
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) {
        const uint16_t* p = st + (32 * slice + 8 * g + (r16 >> 2)) * kGL + 16 * cb + 4 * (r16 & 3);
        const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * kGL);
        b[cb] = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int term = 0; term < 3; ++term) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(fr + ((term * NB + nb) * 2 + slice) * 512);
#pragma unroll
          for (int cb = 0; cb < 4; ++cb) acc[nb][cb] = mfma16(v, b[cb], acc[nb][cb]);
        }
    }
  }
}

template <int NB, bool PACKED, bool VEC>
__global__ __launch_bounds__(256) void k_gram8(GramArgs8 a) {
  constexpr int LR = 68;                            // a reduced row, FP32
  __shared__ __attribute__((aligned(16))) uint8_t glds[4 * 64 * kGL * 2];
  static_assert(4 * 16 * LR * 4 <= 4 * 64 * kGL * 2, "reduction buffer");
  if (a.plan.head && !plan_fits(a.plan, a.M, a.slots)) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  uint16_t* st = reinterpret_cast<uint16_t*>(glds) + w * 64 * kGL;
  float* red = reinterpret_cast<float*>(glds);
  const int tiles = (int)((a.M + 63) / 64);
  const int splits = a.plan.head ? a.plan.head[kPlanSplits] : (tiles + a.tps - 1) / a.tps;
  const int ct0 = (int)((a.q[0].d + 63) / 64), ct1 = (int)((a.q[1].d + 63) / 64);
  const int64_t items = (int64_t)splits * (ct0 + ct1);
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int si = (int)(item / (ct0 + ct1));
    int ct = (int)(item % (ct0 + ct1));
    const int side = ct >= ct0 ? 1 : 0;
    if (side) ct -= ct0;
    const GramSide& q = a.q[side];
    int4 sp;
    int64_t part = -1;
    if (a.plan.head) {
      sp = a.plan.split[si];
      if (sp.w >= 0) part = a.plan.parts[sp.x].x + sp.w;
    } else {
      sp = int4{0, si * a.tps, min(a.tps, tiles - si * a.tps), 0};
      if (splits > 1) part = si;
    }
    const int64_t c0 = (int64_t)ct * 64;
    f32x4 acc[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) acc[nb][cb] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (PACKED && side == 0) gram_item<NB, true, VEC>(a, q, c0, sp, st, acc);
    else gram_item<NB, false, VEC>(a, q, c0, sp, st, acc);

    // accumulator lane (r16, g): ranks 16 nb + 4 g + v, column c0 + 16 cb + r16
    float* out = part >= 0 ? q.part + part * a.r * q.d : q.out + (int64_t)sp.x * a.r * q.d;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      __syncthreads();
#pragma unroll
      for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[(w * 16 + 4 * g + v) * LR + 16 * cb + r16] = acc[nb][cb][v];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = threadIdx.x + 256 * u;
        const int i = side ? e & 15 : e >> 6, c = side ? e >> 4 : e & 63;
        float sum = red[i * LR + c];
#pragma unroll
        for (int ww = 1; ww < 4; ++ww) sum += red[(ww * 16 + i) * LR + c];
        if (16 * nb + i < a.r && c0 + c < q.d)
          out[side ? (c0 + c) * a.r + 16 * nb + i : (16 * nb + i) * q.d + c0 + c] = sum;
      }
    }
    __syncthreads();
  }
}

// Gradients of slots with several splits (their parts added in order) and of
// slots without tokens (zeros).
__global__ __launch_bounds__(256) void k_gram_sum(GramArgs8 a, int n_parts) {
  if (a.plan.head && !plan_fits(a.plan, a.M, a.slots)) return;
  const int64_t size0 = a.r * a.q[0].d, size1 = a.r * a.q[1].d;
  const int64_t chunk = 1024;
  const int64_t ch0 = (size0 + chunk - 1) / chunk, ch1 = (size1 + chunk - 1) / chunk;
  for (int64_t item = blockIdx.x; item < a.slots * (ch0 + ch1); item += gridDim.x) {
    const int slot = (int)(item / (ch0 + ch1));
    int64_t ch = item % (ch0 + ch1);
    int2 pt = int2{0, n_parts};
    if (a.plan.head) pt = a.plan.parts[slot];
    if (pt.y == 1) continue;
    const int side = ch >= ch0 ? 1 : 0;
    if (side) ch -= ch0;
    const GramSide& q = a.q[side];
    const int64_t size = side ? size1 : size0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t e = ch * chunk + threadIdx.x + 256 * u;
      if (e >= size) continue;
      float sum = 0.0f;
      const float* p = q.part + (int64_t)pt.x * size + e;
      for (int j = 0; j < pt.y; ++j) sum = j == 0 ? p[0] : sum + p[(int64_t)j * size];
      q.out[slot * size + e] = sum;
    }
  }
}

template <typename K>
hipError_t allow_lds(K kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int NB, bool KN, bool VEC>
hipError_t launch_shrink_t(const ShrinkArgs& a, unsigned grid, hipStream_t st) {
  constexpr int lds = shrink_lds<NB, KN>();
  static const hipError_t attr = allow_lds(&k_shrink<NB, KN, VEC>, lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((k_shrink<NB, KN, VEC>), dim3(grid), dim3(64 * shrink_waves<NB>()), lds, st,
                     a);
  return hipGetLastError();
}
template <int NB>
hipError_t launch_shrink_nb(const ShrinkArgs& a, bool vec, unsigned grid, hipStream_t st) {
  if (a.kn)
    return vec ? launch_shrink_t<NB, true, true>(a, grid, st)
               : launch_shrink_t<NB, true, false>(a, grid, st);
  return vec ? launch_shrink_t<NB, false, true>(a, grid, st)
             : launch_shrink_t<NB, false, false>(a, grid, st);
}

template <int KS, bool RD, bool VEC>
hipError_t launch_expand_t(const ExpandArgs& a, unsigned grid, hipStream_t st) {
  constexpr int lds = 2 * 64 * (32 * KS + 8) * 2 + (RD ? 4 * 32 * 72 * 2 : 0);
  static const hipError_t attr = allow_lds(&k_expand<KS, RD, VEC>, lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((k_expand<KS, RD, VEC>), dim3(grid), dim3(256), lds, st, a);
  return hipGetLastError();
}
template <int KS>
hipError_t launch_expand_ks(const ExpandArgs& a, bool vec, unsigned grid, hipStream_t st) {
  if (a.rd)
    return vec ? launch_expand_t<KS, true, true>(a, grid, st)
               : launch_expand_t<KS, true, false>(a, grid, st);
  return vec ? launch_expand_t<KS, false, true>(a, grid, st)
             : launch_expand_t<KS, false, false>(a, grid, st);
}

template <int NB>
hipError_t launch_gram8_nb(const GramArgs8& a, bool vec, unsigned grid, hipStream_t st) {
  const bool packed = a.q[0].codes != nullptr;
  if (packed && vec)
    hipLaunchKernelGGL((k_gram8<NB, true, true>), dim3(grid), dim3(256), 0, st, a);
  else if (packed)
    hipLaunchKernelGGL((k_gram8<NB, true, false>), dim3(grid), dim3(256), 0, st, a);
  else if (vec)
    hipLaunchKernelGGL((k_gram8<NB, false, true>), dim3(grid), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((k_gram8<NB, false, false>), dim3(grid), dim3(256), 0, st, a);
  return hipGetLastError();
}

bool at16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
constexpr int64_t kMostGrid = 4096;

}  // namespace

hipError_t launch_gram_zero(const GramArgs8& a, hipStream_t st) {
  const int64_t chunks = (a.r * a.q[0].d + 1023) / 1024 + (a.r * a.q[1].d + 1023) / 1024;
  hipLaunchKernelGGL(k_gram_sum, dim3((unsigned)std::min<int64_t>(a.slots * chunks, 2 * kMostGrid)),
                     dim3(256), 0, st, a, 0);
  return hipGetLastError();
}

hipError_t launch_plan(const PlanView& p, const int32_t* index, int64_t M, int64_t slots,
                       hipStream_t st) {
  const int tps = plan_split_tiles(M);
  int bits = 1;
  while ((int64_t(1) << bits) <= slots) ++bits;
  if (M <= kSpan) {
    hipLaunchKernelGGL(k_plan_small, dim3(1), dim3(256), 0, st, p, index, (int)M, (int)slots, tps,
                       bits);
    return hipGetLastError();
  }
  const unsigned spans = (unsigned)((M + kSpan - 1) / kSpan);
  hipLaunchKernelGGL(k_plan_count, dim3(spans), dim3(64), 0, st, index, M, (int)slots, p.hist);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_plan_lists, dim3(1), dim3(256), 0, st, p, (int)M, (int)slots, tps,
                     (int)spans, p.hist);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_plan_place, dim3(spans), dim3(64), 0, st, p, index, M, (int)slots, bits,
                     p.hist);
  return hipGetLastError();
}

hipError_t launch_shrink(const ShrinkArgs& a0, hipStream_t st) {
  ShrinkArgs a = a0;
  a.splits = shrink_splits(a.M, a.K, &a.kper);
  const unsigned grid =
      (unsigned)std::min<int64_t>(plan_most_tiles(a.M, a.slots) * a.splits, kMostGrid);
  // whole 16-byte pieces: of the tokens' rows, and of the factor's
  const bool vec = a.K % 8 == 0 && at16(a.P) && at16(a.F) && (!a.kn || a.r % 8 == 0);
  if (a.r <= 16) return launch_shrink_nb<1>(a, vec, grid, st);
  if (a.r <= 32) return launch_shrink_nb<2>(a, vec, grid, st);
  if (a.r <= 64) return launch_shrink_nb<4>(a, vec, grid, st);
  if (a.r <= 128) return launch_shrink_nb<8>(a, vec, grid, st);
  return launch_shrink_nb<16>(a, vec, grid, st);
}

hipError_t launch_expand(const ExpandArgs& a0, hipStream_t st) {
  ExpandArgs a = a0;
  int64_t kper;
  a.splits = shrink_splits(a.M, a.K, &kper);
  // chunks of whole 256 columns, about 1024 workgroups
  const int64_t tiles = (a.M + 63) / 64, units = (a.d + 255) / 256;
  const int64_t want = std::max<int64_t>(1, std::min(units, (1024 + tiles - 1) / tiles));
  a.cper = (units + want - 1) / want * 256;
  a.chunks = (int)((a.d + a.cper - 1) / a.cper);
  const unsigned grid =
      (unsigned)std::min<int64_t>(plan_most_tiles(a.M, a.slots) * a.chunks, kMostGrid);
  const bool vec = a.d % 8 == 0 && at16(a.in) && at16(a.out) && at16(a.F) && (a.rd || a.r % 8 == 0);
  if (a.r <= 32) return launch_expand_ks<1>(a, vec, grid, st);
  if (a.r <= 64) return launch_expand_ks<2>(a, vec, grid, st);
  if (a.r <= 128) return launch_expand_ks<4>(a, vec, grid, st);
  return launch_expand_ks<8>(a, vec, grid, st);
}

hipError_t launch_gram8(const FragArgs& f0, const GramArgs8& a, hipStream_t st) {
  const int64_t tiles = a.plan.head ? plan_most_tiles(a.M, a.slots) : (a.M + 63) / 64;
  FragArgs f = f0;
  f.nb = frag_blocks(a.r);
  const int groups = (f.nb + 3) / 4;
  hipLaunchKernelGGL(k_frags, dim3((unsigned)std::min<int64_t>(tiles * groups * 2, kMostGrid)),
                     dim3(256), 0, st, f);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t splits =
      a.plan.head ? plan_most_splits(a.M, a.slots) : (tiles + a.tps - 1) / a.tps;
  const int64_t cols = (a.q[0].d + 63) / 64 + (a.q[1].d + 63) / 64;
  const unsigned grid = (unsigned)std::min<int64_t>(splits * cols, 2 * kMostGrid);
  const bool vec = a.q[1].d % 8 == 0 && at16(a.q[1].x) &&
                   (a.q[0].codes || (a.q[0].d % 8 == 0 && at16(a.q[0].x)));
  switch (f.nb) {
    case 1: e = launch_gram8_nb<1>(a, vec, grid, st); break;
    case 2: e = launch_gram8_nb<2>(a, vec, grid, st); break;
    case 4: e = launch_gram8_nb<4>(a, vec, grid, st); break;
    case 8: e = launch_gram8_nb<8>(a, vec, grid, st); break;
    default: e = launch_gram8_nb<16>(a, vec, grid, st);
  }
  if (e != hipSuccess) return e;
  // without a plan one split leaves nothing to add
  if (!a.plan.head && splits <= 1) return hipSuccess;
  const int64_t chunks = (a.r * a.q[0].d + 1023) / 1024 + (a.r * a.q[1].d + 1023) / 1024;
  hipLaunchKernelGGL(k_gram_sum, dim3((unsigned)std::min<int64_t>(a.slots * chunks, 2 * kMostGrid)),
                     dim3(256), 0, st, a, (int)splits);
  return hipGetLastError();
}

}  // namespace qlora
