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
// that list, whose length only the device knows.  k_shrink forms T or U as FP32
// partial sums over ranges of the long axis, k_finish adds those and writes them
// as matrix operands, k_expand multiplies by the other factor and adds the shared
// projection's output (for few tokens it adds the partials too: two launches make
// such a forward).  A backward adds k_gram8, the contractions over tokens, and
// k_gram_sum, which adds their splits.  Products are BF16 on the matrix cores with FP32 sums; T and U are
// FP32 and enter them as sums of BF16 terms: two (16 bits) where the result is
// rounded to BF16, three (24 bits, all of FP32) where it is FP32.
#include <type_traits>

#include "qlora_device.h"
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

__device__ __forceinline__ uint16_t bf16_bits(float v) { return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }

// Rows start at any element: vectors need not be aligned.  Where eight elements
// from `col` on would pass the row's end, the last eight of the row are loaded
// (from at8) and moved down (past8 elements dropped at the front, zeros behind),
// so that no lane waits for single elements; rows of fewer than eight take those
// (few8).
__device__ __forceinline__ int64_t at8(int64_t col, int64_t end) { return col < end - 8 ? col : end - 8; }
__device__ __forceinline__ u32x4 past8(u32x4 v, int64_t drop) {
  const int s = (int)(drop < 8 ? drop : 8);
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = s & 4 ? (j < 2 ? v[j + 2] : 0u) : v[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = s & 2 ? (j < 3 ? o[j + 1] : 0u) : o[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = s & 1 ? (o[j] >> 16) | (j < 3 ? o[j + 1] << 16 : 0u) : o[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = s & 8 ? 0u : o[j];
  return o;
}
__device__ __forceinline__ u32x4 few8(const uint16_t* row, int64_t col, int64_t end) {
  u32x4 o = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t x = row[col + e < end ? col + e : end - 1];
    o[e >> 1] |= col + e < end ? x << (16 * (e & 1)) : 0u;
  }
  return o;
}
// Eight elements from column `col` on, zero at and past `end`.
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int64_t col, int64_t end) {
  if (end < 8) return few8(row, col, end);
  return past8(load_vec(row + at8(col, end)), col - at8(col, end));
}
__device__ __forceinline__ u32x4 only_if(bool ok, u32x4 v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = ok ? v[j] : 0u;
  return v;
}

// Ranks past 64 are worked on in groups of 64, items of their own: the groups of
// one item are eight workgroups apart, so that they run on one XCD and share what
// they read in its L2.  (All 128 ranks in one workgroup left one wavefront a SIMD.)
__device__ __forceinline__ int64_t ranked(int64_t item, int groups, int64_t items, int& group) {
  const int64_t block = item / (8 * groups), rest = item % (8 * groups);
  const int64_t left = items - 8 * block, width = left < 8 ? left : 8;
  group = (int)(rest / width);
  return 8 * block + rest % width;
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
    const int end = cnt[lo + 1];
    p.split_first[i] = cnt[lo] + 64 * j * tps;
    p.split[i] = int4{lo, first, min(64 * tps, end - cnt[lo] - 64 * j * tps), n > 1 ? j : -1};
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
    // eight spans' counts at a time: the loop is bound by the latency of its loads
    int sum = 0;
    for (int b0 = 0; b0 < spans; b0 += 8) {
      int32_t* h = hist + (int64_t)b0 * (slots + 1) + s;
      int c[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) c[b] = b0 + b < spans ? h[(int64_t)b * (slots + 1)] : 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (b0 + b < spans) h[(int64_t)b * (slots + 1)] = sum;
        sum += c[b];
      }
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
// Item = one tile and one of `splits` ranges of K.  The four wavefronts of a
// workgroup take the range's steps in turn, each all 64 tokens and all ranks:
// no wavefront loads what another loads, and the loop has no barrier.  A step's
// loads are 16 a wavefront and not a step ahead: two workgroups a compute unit
// hide more than a second set of registers does (16384 x 4096, rank 64: 55 us; a
// step ahead, with one workgroup, a third more; read at 5.7 TB/s it would be 24).
// The sums
// are added through LDS at the end, in wavefront order.  KN: a step's rows
// of F go through LDS of the wavefront's own, which the transposing reads turn
// into operands.
// ---------------------------------------------------------------------------
constexpr int kShrinkWaves = 4;
constexpr int kShrinkSlices = 2;   // K slices of 32 a step: whole lines of a row
template <int NB, bool KN>
constexpr int shrink_lds() {
  constexpr int CN = NB < 4 ? NB : 4;
  constexpr int red = kShrinkWaves * 16 * 16 * CN * 4;
  constexpr int stage = KN ? kShrinkWaves * 32 * kShrinkSlices * (16 * NB + 8) * 2 : 0;
  return red > stage ? red : stage;
}

// V's row of a position as k_expand's operand: BF16 hi, then lo, of rp ranks.
__device__ __forceinline__ void put_vrow(uint16_t* vrows, int64_t pos, int i, int rp, float v) {
  float hi, lo;
  split_bf16(v, hi, lo);
  uint16_t* row = vrows + pos * 2 * rp;
  row[i] = (uint16_t)(__float_as_uint(hi) >> 16);
  row[rp + i] = bf16_bits(lo);
}

// One item with RB blocks of 16 tokens.  FAST: K of eight or
// more and, KN, rows of F that are whole 16-byte pieces.
template <int NB, bool KN, bool FAST, int RB>
__device__ __forceinline__ void shrink_item(const ShrinkArgs& a, const int4& td, int s, int i0, uint8_t* lds) {
  constexpr int W = kShrinkWaves, CN = NB < 4 ? NB : 4, SK = kShrinkSlices;
  constexpr int LF = 16 * NB + 8;                  // staged row of F, elements
  constexpr int STEP = 32 * SK;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t K = a.K;
  const int r = a.r;
  uint16_t* stage = reinterpret_cast<uint16_t*>(lds) + w * STEP * LF;
  float* red = reinterpret_cast<float*>(lds);
  const int slot = td.x, first = td.y, count = td.z;
  const int64_t k_begin = (int64_t)s * a.kper;
  const int64_t k_end = k_begin + a.kper < K ? k_begin + a.kper : K;
  const uint16_t* F = a.F + (int64_t)slot * r * K;
  const uint16_t* xp[RB];   // rows past the tile's last repeat it; their sums are not stored
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int row = min(16 * rb + r16, count - 1);
    const int64_t tok = a.plan.head ? a.plan.order[first + row] : first + row;
    xp[rb] = a.P + tok * K;
  }

  f32x4 acc[RB][NB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) acc[rb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};

  // whole steps: loads without conditions (F's first: their addresses wait for
  // nothing)
  auto load = [&](int64_t k, const int (&off)[SK], int rows, u32x4 (&x)[SK][RB], u32x4 (&f)[SK * NB]) {
#pragma unroll
    for (int u = 0; u < SK * NB; ++u) {
      if (KN) {
        const int piece = lane + 64 * u, row = min(piece / (2 * NB), rows), col = i0 + 8 * (piece % (2 * NB));
        f[u] = load_vec(F + (k + row) * r + (col < r ? col : 0));
      } else {
        const int i = min(i0 + 16 * (u / SK) + r16, r - 1);
        f[u] = load_vec(F + i * K + k + off[u % SK]);
      }
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int sl = 0; sl < SK; ++sl) x[sl][rb] = load_vec(xp[rb] + k + off[sl]);
  };
  int off[SK];                                     // the lane's columns of a step
#pragma unroll
  for (int sl = 0; sl < SK; ++sl) off[sl] = 32 * sl + 8 * g;
  auto compute = [&](const u32x4 (&x)[SK][RB], const u32x4 (&f)[SK * NB]) {
    if (KN) {
#pragma unroll
      for (int u = 0; u < SK * NB; ++u) {
        const int piece = lane + 64 * u, row = piece / (2 * NB), col = 8 * (piece % (2 * NB));
        *reinterpret_cast<u32x4*>(stage + row * LF + col) = f[u];
      }
    }
#pragma unroll
    for (int sl = 0; sl < SK; ++sl)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        u32x4 q = f[nb * SK + sl];
        if (KN) {
          const uint16_t* p = stage + (32 * sl + 8 * g + (r16 >> 2)) * LF + 16 * nb + 4 * (r16 & 3);
          const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * LF);
          q = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) acc[rb][nb] = mfma16(x[sl][rb], q, acc[rb][nb]);
      }
  };
  int64_t k = k_begin + STEP * w;
  const int64_t k_whole = shrink_whole_end(k_begin, k_end, K, r, KN && !FAST, STEP);
  if (k < k_whole) {
    const int64_t k_last = k + (k_whole - 1 - k) / (STEP * W) * (STEP * W);
    u32x4 x[SK][RB], f[SK * NB];
    for (; k <= k_last; k += STEP * W) {
      load(k, off, STEP - 1, x, f);
      __builtin_amdgcn_sched_barrier(0);           // all of a step's loads before its products
      compute(x, f);
    }
    k = k_last + STEP * W;
  }
  // what is left: a partial step, or one and a whole one that the rule keeps out
  for (; k < k_end; k += STEP * W) {
    u32x4 x[SK][RB], f[SK * NB];
    if constexpr (FAST) {
      // K ends it (the ranges before the last are whole steps)
      int end_off[SK];
#pragma unroll
      for (int sl = 0; sl < SK; ++sl) end_off[sl] = (int)(at8(k + off[sl], k_end) - k);
      load(k, end_off, (int)(k_end - 1 - k), x, f);
#pragma unroll
      for (int sl = 0; sl < SK; ++sl) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) x[sl][rb] = past8(x[sl][rb], off[sl] - end_off[sl]);
        if (!KN) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) f[nb * SK + sl] = past8(f[nb * SK + sl], off[sl] - end_off[sl]);
        }
      }
      if (KN) {
#pragma unroll
        for (int u = 0; u < SK * NB; ++u) f[u] = only_if(k + (lane + 64 * u) / (2 * NB) < k_end, f[u]);
      }
    } else {
#pragma unroll
      for (int sl = 0; sl < SK; ++sl)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) x[sl][rb] = load8(xp[rb], k + off[sl], k_end);
#pragma unroll
      for (int u = 0; u < SK * NB; ++u) {
        if (KN) {
          const int piece = lane + 64 * u, row = piece / (2 * NB), col = i0 + 8 * (piece % (2 * NB));
          const int64_t at = k + row < k_end ? k + row : k_end - 1;
          f[u] = only_if(k + row < k_end, load8(F + at * r, col, r));
        } else {
          f[u] = load8(F + min(i0 + 16 * (u / SK) + r16, r - 1) * K, k + off[u % SK], k_end);
        }
      }
    }
    compute(x, f);
  }

  // accumulator lane (r16, g): tokens 16 rb + 4 g + v, rank 16 nb + r16
  float* part = a.part + ((int64_t)s * a.M + first) * r;
  const float sc = a.vrows ? a.scale[slot] : 0.0f;
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    if (16 * rb >= count) break;
#pragma unroll
    for (int n0 = 0; n0 < NB; n0 += CN) {
      lds_barrier();   // the stage, or the last block, is no longer read
#pragma unroll
      for (int nb = 0; nb < CN; ++nb)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[(w * 16 + 4 * g + v) * 16 * CN + 16 * nb + r16] = acc[rb][n0 + nb][v];
      lds_barrier();
#pragma unroll
      for (int e0 = 0; e0 < 256 * CN; e0 += 64 * W) {
        const int e = e0 + threadIdx.x;
        if (256 * CN % (64 * W) != 0 && e >= 256 * CN) break;
        const int row = e / (16 * CN), i = i0 + 16 * n0 + e % (16 * CN);
        float sum = red[e];
#pragma unroll
        for (int ww = 1; ww < W; ++ww) sum += red[ww * 256 * CN + e];
        if (16 * rb + row >= count) continue;
        if (a.vrows) {
          const int pos = first + 16 * rb + row;
          const float v = i < r ? sum * sc : 0.0f;
          put_vrow(a.vrows, pos, i, a.rp, v);
          if (NB == 1) put_vrow(a.vrows, pos, i + 16, 32, 0.0f);
          if (a.v_out && i < r) a.v_out[(int64_t)a.plan.order[pos] * r + i] = v;
        } else if (i < r) {
          part[(16 * rb + row) * r + i] = sum;
        }
      }
    }
  }
  lds_barrier();
}

template <int NB, bool KN, bool FAST>
__global__ __launch_bounds__(64 * kShrinkWaves, 2) void k_shrink(ShrinkArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t slds[];
  int4 td = {0, 0, 0, 0};
  const int t0 = min((int)(blockIdx.x / a.groups) / a.splits, a.most - 1);
  int tiles = (int)((a.M + 63) / 64);
  if (a.plan.head) {
    // the grid has no more workgroups than the list room for items
    td = a.plan.tile[t0];
    if (!plan_fits(a.plan, a.M, a.slots)) return;
    tiles = a.plan.head[kPlanTiles];
  }
  const int items = tiles * a.splits;
  for (int it = blockIdx.x; it < items * a.groups; it += gridDim.x) {
    int group;
    const int item = (int)ranked(it, a.groups, items, group);
    const int t = item / a.splits, s = item % a.splits;
    if (!a.plan.head) td = int4{0, 64 * t, (int)min((int64_t)64, a.M - 64 * (int64_t)t), 0};
    else if (t != t0) td = a.plan.tile[t];
    // few tokens: no registers and loads for blocks of tokens that are not there
    if (td.z <= 16) shrink_item<NB, KN, FAST, 1>(a, td, s, 64 * group, slds);
    else shrink_item<NB, KN, FAST, 4>(a, td, s, 64 * group, slds);
  }
}

// The sums of k_shrink's partial results, in order: up to Q pieces of N ranks
// part + at[] on, `stride` between the at most SM splits.  Every load is
// issued before the first sum.
template <int SM, int Q, int N>
__device__ __forceinline__ void sum_parts(const float* part, const int (&at)[Q], const bool (&on)[Q],
                                          int splits, int64_t stride, float (&v)[Q][N]) {
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  auto get = [&](const float* p, float* f) {
    if constexpr (N == 4) {
      const vec x = *reinterpret_cast<const vec*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = x[j];
    } else {
      f[0] = *p;
    }
  };
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int j = 0; j < N; ++j) v[q][j] = 0.0f;
  float x[SM][Q][N];
#pragma unroll
  for (int s = 0; s < SM; ++s)
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (s < splits && on[q]) get(part + s * stride + at[q], x[s][q]);
#pragma unroll
  for (int s = 0; s < SM; ++s)
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (s < splits && on[q]) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[q][j] = s == 0 ? x[s][q][j] : v[q][j] + x[s][q][j];
      }
}

// ---------------------------------------------------------------------------
// out[token][n] = RN(in[token][n] + sum_i V[token][i] F[n][i]),
// V of k_shrink or k_finish as BF16 hi + lo.  F is stored [d][r] (B in the
// forward) or, RD, [r][d] (A in the backward).  Item = a few tiles of one slot
// and 256 columns (fewer at ranks past 64), whose part of F stays in LDS: a wavefront takes 16 tokens of a
// tile at a time, 512 bytes of each row, and loads the next tile's while it works
// on this one, without a barrier.  Neighbouring items are the neighbouring
// columns of the same tokens, so that what the chip works on at a time is whole
// rows.  F is the row operand of the MFMA: with its rows in the order of
// unit_column a lane ends up with twice eight consecutive columns of a token; LDS
// of the wavefront's own turns them so that its loads and stores are whole
// 128-byte lines (64 bytes of 16 rows an instruction took 164 us for the rows of
// 16384 x 11008 alone, lines 138; the whole kernel takes 160, 158 without staging F).
//
// Items of up to 16 tokens (decoding) have nothing to reuse F for: there each
// wavefront takes 64 columns and reads F from memory.
// ---------------------------------------------------------------------------
// Columns of an item: as many as leave LDS for two or three workgroups.
template <int KS>
constexpr int expand_cols() { return KS <= 2 ? 256 : (KS == 4 ? 128 : 64); }
constexpr int kTurn = 68;   // a row of 64 sums in the wavefront's LDS, FP32

// The column that row j of MFMA block b (0..3) stands for in a unit of 64.
__device__ __forceinline__ int unit_column(int j, int b) {
  return 32 * (b >> 1) + 8 * (j >> 2) + 4 * (b & 1) + (j & 3);
}

// F's part in LDS: rows n of 32 KS + 8 ranks, or RD rows i of its columns + 8; zero
// past r and past d.
template <int KS, bool RD>
constexpr int expand_ld() { return RD ? expand_cols<KS>() + 8 : 32 * KS + 8; }
template <int KS, bool RD>
constexpr int expand_lds() { return (RD ? 32 * KS : expand_cols<KS>()) * expand_ld<KS, RD>() * 2; }
constexpr int kTurnBytes = 4 * 16 * kTurn * 4;

// Block b's operand of unit u, ranks 32 ks .. +32.
template <int KS, bool RD>
__device__ __forceinline__ u32x4 expand_f(const uint16_t* fl, int u, int b, int ks, int lane) {
  constexpr int L = expand_ld<KS, RD>();
  const int r16 = lane & 15, g = lane >> 4;
  if (RD) {
    const uint16_t* p = fl + (32 * ks + 8 * g + (r16 >> 2)) * L + 64 * u + unit_column(4 * (r16 & 3), b);
    const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * L);
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  }
  return *reinterpret_cast<const u32x4*>(fl + (64 * u + unit_column(r16, b)) * L + 32 * ks + 8 * g);
}

// Eight results: y + s.
__device__ __forceinline__ u32x4 expand_result(u32x4 y, const f32x4& s0, const f32x4& s1) {
  u32x4 o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x4& s = j < 2 ? s0 : s1;
    o[j] = pack_bf16x2(bf16lo_to_f32(y[j]) + s[2 * (j & 1)], bf16hi_to_f32(y[j]) + s[2 * (j & 1) + 1]);
  }
  return o;
}
__device__ __forceinline__ void store8(uint16_t* row, int64_t col, int64_t end, u32x4 o) {
  if (col + 8 <= end) {
    store_vec(row + col, o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < end) row[col + e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
  }
}

// V of the lane's operand (ranks 32 ks + 8 g .. +8 of the token at `pos`) as hi
// and lo: read, or SUMS, from k_shrink's partial results (r a multiple of 4).
// `save`: also to the caller, by token.
template <int KS, bool SUMS>
__device__ __forceinline__ void expand_v(const ExpandArgs& a, int pos, int ks, float sc, bool save,
                                         u32x4& vh, u32x4& vl) {
  const int g = (threadIdx.x & 63) >> 4, i = 32 * ks + 8 * g;
  if constexpr (!SUMS) {
    const uint16_t* v = a.vrows + (int64_t)pos * 64 * KS + i;
    vh = *reinterpret_cast<const u32x4*>(v);
    vl = *reinterpret_cast<const u32x4*>(v + 32 * KS);
  } else {
    const int r = a.r;
    const int at[2] = {pos * r + (i < r ? i : 0), pos * r + (i + 4 < r ? i + 4 : 0)};
    const bool on[2] = {i < r, i + 4 < r};
    float v[2][4];
    sum_parts<kShrinkSplits, 2, 4>(a.part, at, on, a.splits, a.M * r, v);
    float* out = save ? a.v_out + (int64_t)a.plan.order[pos] * r + i : nullptr;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[q][j] = on[q] ? v[q][j] * sc : 0.0f;
        if (save && on[q]) out[4 * q + j] = v[q][j];
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = v[j >> 1][2 * (j & 1)], y = v[j >> 1][2 * (j & 1) + 1];
      vh[j] = pack_bf16x2(x, y);
      vl[j] = pack_bf16x2(x - bf16lo_to_f32(vh[j]), y - bf16hi_to_f32(vh[j]));
    }
  }
}

template <int KS, bool RD, bool R8, bool DEEP, bool SUMS>
__device__ __forceinline__ void expand_many(const ExpandArgs& a, int slot, int first, int tokens,
                                            int64_t c0, uint8_t* lds) {
  constexpr int L = expand_ld<KS, RD>(), COLS = expand_cols<KS>(), U = COLS / 64;
  uint16_t* fl = reinterpret_cast<uint16_t*>(lds + kTurnBytes);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* turn = reinterpret_cast<float*>(lds) + w * 16 * kTurn;
  const int r16 = lane & 15, g = lane >> 4, l8 = lane >> 3, c8 = 8 * (lane & 7);
  const int r = a.r, tiles = (tokens + 63) / 64;
  const int64_t d = a.d;
  const bool whole = c0 + COLS <= d;
  const uint16_t* F = a.F + (int64_t)slot * r * d;

  // Of a tile's 16 tokens: as an operand's column lane r16's, of its rows in
  // memory the lane's two, l8 and 8 + l8 (past the last token: that one again).
  struct Rows {
    u32x4 y[U][2], v[KS][2];
    int64_t at[2];
  };
  auto place = [&](int j, int row) { return first + min(64 * j + 16 * w + row, tokens - 1); };
  auto token = [&](int j, int (&tok)[2]) {
    tok[0] = a.plan.order[place(j, l8)];
    tok[1] = a.plan.order[place(j, 8 + l8)];
  };
  const float sc = SUMS ? a.scale[slot] : 1.0f;
  auto load_v = [&](int j, Rows& t) {
    const bool save = SUMS && a.v_out && c0 == 0 && 64 * j + 16 * w + r16 < tokens;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      expand_v<KS, SUMS>(a, place(j, r16), ks, sc, save, t.v[ks][0], t.v[ks][1]);
  };
  auto load_y = [&](const int (&tok)[2], Rows& t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t.at[h] = tok[h] * d + c0 + c8;
      if (!a.in) continue;
#pragma unroll
      for (int u = 0; u < U; ++u)
        t.y[u][h] = d >= 8 ? load_vec(a.in + tok[h] * d + at8(c0 + 64 * u + c8, d)) : few8(a.in + tok[h] * d, c8, d);
    }
  };
  auto work = [&](int j, Rows& t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c0 + 64 * u >= d) break;
      f32x4 acc[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const u32x4 f = expand_f<KS, RD>(fl, u, b, ks, lane);
          acc[b] = mfma16(f, t.v[ks][0], acc[b]);
          acc[b] = mfma16(f, t.v[ks][1], acc[b]);
        }
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<f32x4*>(turn + r16 * kTurn + unit_column(4 * g, b)) = acc[b];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* s = turn + (8 * h + l8) * kTurn + c8;
        const int64_t col = c0 + 64 * u + c8;
        u32x4 y = {0, 0, 0, 0};
        if (a.in) y = whole || d < 8 ? t.y[u][h] : past8(t.y[u][h], col - at8(col, d));
        const u32x4 o = expand_result(y, *reinterpret_cast<const f32x4*>(s),
                                      *reinterpret_cast<const f32x4*>(s + 4));
        if (64 * j + 16 * w + 8 * h + l8 >= tokens) continue;
        if (whole) store_vec(a.out + t.at[h] + 64 * u, o);
        else store8(a.out + t.at[h] - c0 - c8, col, d, o);
      }
    }
  };

  Rows ta;
  const bool mine = 16 * w < tokens;               // a first tile of few tokens leaves wavefronts out
  int next[2];
  if (mine) {
    token(0, next);
    load_y(next, ta);                              // in flight while F is staged
    if (!SUMS) load_v(0, ta);
    if (DEEP) token(1, next);
  }
  lds_barrier();                                   // the last item's F is no longer read
  if (RD) {
    constexpr int P = COLS / 8;
#pragma unroll 4
    for (int e = threadIdx.x; e < 32 * KS * P; e += 256) {
      const int i = e / P, cc = 8 * (e % P);
      const uint16_t* row = F + (int64_t)(i < r ? i : 0) * d;
      const u32x4 v = only_if(i < r, whole ? load_vec(row + c0 + cc) : load8(row, c0 + cc, d));
      *reinterpret_cast<u32x4*>(fl + i * L + cc) = v;
    }
  } else {
    constexpr int P = 4 * KS;
#pragma unroll 4
    for (int e = threadIdx.x; e < COLS * P; e += 256) {
      const int n = e / P, i = 8 * (e % P);
      const bool ok = c0 + n < d && i < r;
      const uint16_t* row = F + (c0 + n < d ? c0 + n : 0) * r;
      const u32x4 v = only_if(ok, R8 ? load_vec(row + (i < r ? i : 0)) : load8(row, i, r));
      *reinterpret_cast<u32x4*>(fl + n * L + i) = v;
    }
  }
  lds_barrier();
  if (!mine) return;
  if constexpr (!DEEP) {
    if (SUMS) load_v(0, ta);
    work(0, ta);
  } else {
    Rows tb;
    for (int j = 0; j < tiles; j += 2) {
      if (j + 1 < tiles) {
        load_v(j + 1, tb);
        load_y(next, tb);
        token(j + 2, next);
      }
      work(j, ta);
      if (j + 1 >= tiles) break;
      if (j + 2 < tiles) {
        load_v(j + 2, ta);
        load_y(next, ta);
        token(j + 3, next);
      }
      work(j + 1, tb);
    }
  }
}

// Up to 16 tokens: wavefront w takes columns 64 w .. of the item's.
template <int KS, bool RD, bool R8, bool SUMS>
__device__ __forceinline__ void expand_few(const ExpandArgs& a, int slot, int first, int tokens,
                                           int64_t c0, uint8_t* lds) {
  constexpr int LF = 72;                           // staged row of F
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int r = a.r;
  const int64_t d = a.d, col0 = c0 + 64 * w;
  if (RD) lds_barrier();                           // another item's F is no longer read
  if (64 * w >= expand_cols<KS>() || col0 >= d) return;
  const bool whole = col0 + 64 <= d;
  uint16_t* stage = reinterpret_cast<uint16_t*>(lds) + w * 32 * LF;
  const uint16_t* F = a.F + (int64_t)slot * r * d;
  f32x4 acc[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 f[KS][4];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (RD) {
        const int i = 32 * ks + (lane >> 3) + 8 * u;
        const int64_t col = col0 + 8 * (lane & 7);
        const uint16_t* row = F + (int64_t)(i < r ? i : 0) * d;
        f[ks][u] = only_if(i < r, whole ? load_vec(row + col) : load8(row, col, d));
      } else {
        const int64_t n = col0 + unit_column(r16, u);
        const uint16_t* row = F + (n < d ? n : 0) * r;
        const int i = 32 * ks + 8 * g;
        if (R8) f[ks][u] = only_if(n < d && i < r, load_vec(row + (i < r ? i : 0)));
        else f[ks][u] = only_if(n < d, load8(row, i, r));
      }
    }
  const int pos = first + min(r16, tokens - 1);
  const int64_t tok = a.plan.order[pos];
  const float sc = SUMS ? a.scale[slot] : 1.0f;
  const bool save = SUMS && a.v_out && col0 == 0 && r16 < tokens;
  u32x4 y[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = col0 + 32 * h + 8 * g;
    y[h] = u32x4{0, 0, 0, 0};
    if (a.in) y[h] = whole ? load_vec(a.in + tok * d + col) : load8(a.in + tok * d, col, d);
  }
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    u32x4 vh, vl;
    expand_v<KS, SUMS>(a, pos, ks, sc, save, vh, vl);
    if (RD) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *reinterpret_cast<u32x4*>(stage + ((lane >> 3) + 8 * u) * LF + 8 * (lane & 7)) = f[ks][u];
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      u32x4 q = f[ks][b];
      if (RD) {
        const uint16_t* p = stage + (8 * g + (r16 >> 2)) * LF + unit_column(4 * (r16 & 3), b);
        const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * LF);
        q = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
      acc[b] = mfma16(q, vh, acc[b]);
      acc[b] = mfma16(q, vl, acc[b]);
    }
  }
  if (r16 >= tokens) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) 
    store8(a.out + tok * d, col0 + 32 * h + 8 * g, d, expand_result(y[h], acc[2 * h], acc[2 * h + 1]));
}

// Tokens without an adapter: their rows' columns copied, T zero.
__device__ __forceinline__ void expand_none(const ExpandArgs& a, const int4& td, int64_t c0, int cols) {
  const int64_t n = min((int64_t)cols, a.d - c0);
  const int vecs = (int)((n + 7) / 8);
  if (a.in != a.out) {
    for (int e = threadIdx.x; e < td.z * vecs; e += 256) {
      const int64_t at = (int64_t)a.plan.order[td.y + e / vecs] * a.d + c0;
      const int64_t col = 8 * (int64_t)(e % vecs);
      store8(a.out + at, col, n, a.in ? load8(a.in + at, col, n) : u32x4{0, 0, 0, 0});
    }
  }
  if (a.v_out && c0 == 0)
    for (int e = threadIdx.x; e < td.z * a.r; e += 256)
      a.v_out[(int64_t)a.plan.order[td.y + e / a.r] * a.r + e % a.r] = 0.0f;
}

// DEEP: items of several tiles, from the list of splits; else single tiles.
template <int KS, bool RD, bool R8, bool DEEP, bool SUMS>
__global__ __launch_bounds__(256, KS > 4 ? 1 : (DEEP || KS > 2 ? 2 : 3)) void k_expand(ExpandArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t elds[];
  // the grid has no more workgroups than the lists room for items
  const int g0 = min((int)blockIdx.x / a.chunks / a.subs, a.most - 1);
  int4 rec = DEEP ? a.plan.split[g0] : a.plan.tile[g0];
  int first = DEEP ? a.plan.split_first[g0] : rec.y;
  if (!plan_fits(a.plan, a.M, a.slots)) return;
  const int tiles = a.plan.head[kPlanTiles];
  const int with_one = (DEEP ? a.plan.head[kPlanSplits] * a.subs : tiles) * a.chunks;
  // tokens without an adapter only where something is written for them
  const int none = a.in != a.out || a.v_out ? (a.plan.head[kPlanAllTiles] - tiles) * a.chunks : 0;
  for (int item = blockIdx.x; item < with_one + none; item += gridDim.x) {
    if (item >= with_one) {
      expand_none(a, a.plan.tile[tiles + (item - with_one) / a.chunks],
                  (int64_t)((item - with_one) % a.chunks) * expand_cols<KS>(), expand_cols<KS>());
      continue;
    }
    const int64_t c0 = (int64_t)(item % a.chunks) * expand_cols<KS>();
    const int group = item / a.chunks;
    if (item != (int)blockIdx.x) {
      rec = DEEP ? a.plan.split[group / a.subs] : a.plan.tile[group];
      first = DEEP ? a.plan.split_first[group / a.subs] : rec.y;
    }
    const int skip = DEEP ? group % a.subs * a.tpi * 64 : 0;
    const int tokens = DEEP ? min(rec.z - skip, a.tpi * 64) : rec.z;
    if (tokens <= 0) continue;
    if (tokens <= 16) expand_few<KS, RD, R8, SUMS>(a, rec.x, first + skip, tokens, c0, elds);
    else expand_many<KS, RD, R8, DEEP, SUMS>(a, rec.x, first + skip, tokens, c0, elds);
  }
}

// ---------------------------------------------------------------------------
// What k_shrink's partial sums become: V = scale_a * (their sum, in order) as
// k_expand's rows (vrows), by token (v_out), and as a row operand of the
// contractions over tokens (u_frags); the caller's T as such an operand
// (t_frags).
//
// Row operands: per tile, BF16 term (hi, mid, lo: 24 bits together), 16 ranks
// and 32 tokens one KB in the order of an MFMA's lanes; zero past the tile's
// tokens and past the rank.
// ---------------------------------------------------------------------------
template <int SM>
__global__ __launch_bounds__(256) void k_finish(FinishVArgs a) {
  constexpr int L = 72;
  __shared__ __attribute__((aligned(16))) uint16_t st[3][32 * L];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int r = a.r, nb = a.nb, groups = (nb + 3) / 4, sides = a.t_frags ? 2 : 1;
  const int per_tile = 2 * groups * sides;         // item = 32 tokens of a tile, 64 ranks, side
  int4 td = {0, 0, 0, 0};
  int tiles = (int)((a.M + 63) / 64);
  if (a.plan.head) {
    td = a.plan.tile[min((int)blockIdx.x / per_tile, a.most - 1)];
    if (!plan_fits(a.plan, a.M, a.slots)) return;
    tiles = a.plan.head[kPlanTiles];
  }
  for (int item = blockIdx.x; item < tiles * per_tile; item += gridDim.x) {
    const int t = item / per_tile, sub = item % per_tile;
    const int slice = sub & 1, grp = (sub >> 1) % groups;
    const bool is_t = (sub >> 1) / groups == 1;
    if (!a.plan.head) td = int4{0, 64 * t, (int)min((int64_t)64, a.M - 64 * (int64_t)t), 0};
    else if (item != (int)blockIdx.x) td = a.plan.tile[t];
    const int first = td.y + 32 * slice, count = min(32, td.z - 32 * slice), i0 = 64 * grp;
    uint16_t* frags = is_t ? a.t_frags : a.u_frags;
    if (count <= 0 && !frags) continue;
    const float sc = !is_t && a.scale ? a.scale[td.x] : a.one_scale;
    const int64_t stride = a.M * r;
    const int cols = min(64, max(16 * nb, a.vrows && !is_t ? a.rp : 0) - i0);
    const int rows = frags ? 32 : (count + 15) / 16 * 16;
    lds_barrier();
    auto fill = [&](auto ranks) {
      constexpr int N = decltype(ranks)::value, Q = 2, PR = 64 / N;
#pragma unroll 1
      for (int e0 = threadIdx.x; e0 < rows * PR; e0 += 256 * Q) {
        float v[Q][N];
        bool on[Q];
        int at[Q];
        int64_t tok[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int e = e0 + 256 * q, row = e / PR, i = i0 + N * (e % PR);
          on[q] = row < count && i < r;
          at[q] = on[q] ? row * r + i : 0;
          tok[q] = 0;
          if (on[q] && (is_t || a.v_out)) tok[q] = a.plan.head ? a.plan.order[first + row] : first + row;
        }
        if (!is_t) {
          sum_parts<SM, Q, N>(a.V + (int64_t)first * r, at, on, a.splits, stride, v);
        } else {
#pragma unroll
          for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int j = 0; j < N; ++j)
              v[q][j] = on[q] ? a.T[tok[q] * r + i0 + N * ((e0 + 256 * q) % PR) + j] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int e = e0 + 256 * q, row = e / PR, i = N * (e % PR);
          if (row >= rows || i >= cols) continue;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float x = on[q] ? (is_t ? v[q][j] : v[q][j] * sc) : 0.0f;
            if (!is_t && on[q] && a.v_out) a.v_out[tok[q] * r + i0 + i + j] = x;
            float hi, rest, mid, lo;
            split_bf16(x, hi, rest);
            split_bf16(rest, mid, lo);
            st[0][row * L + i + j] = (uint16_t)(__float_as_uint(hi) >> 16);
            st[1][row * L + i + j] = (uint16_t)(__float_as_uint(mid) >> 16);
            st[2][row * L + i + j] = bf16_bits(lo);
          }
        }
      }
    };
    if (r % 4 == 0) fill(std::integral_constant<int, 4>{});
    else fill(std::integral_constant<int, 1>{});
    lds_barrier();
    if (frags) {
      for (int u = w; u < 12; u += 4) {            // (term, 16 ranks)
        const int term = u >> 2, b = u & 3;
        if (4 * grp + b >= nb) continue;
        const uint16_t* p = &st[term][(8 * g + (r16 >> 2)) * L + 16 * b + 4 * (r16 & 3)];
        const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * L);
        const int64_t at = (((int64_t)t * 3 + term) * nb + 4 * grp + b) * 2 + slice;
        *reinterpret_cast<u32x4*>(frags + at * 512 + lane * 8) = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
    }
    if (!is_t && a.vrows) {
      // the lo of a pair is what the mid of three is
      const int pieces = min(64, a.rp - i0) / 8;
      for (int e = threadIdx.x; e < count * 2 * pieces; e += 256) {
        const int row = e / (2 * pieces), h = e / pieces & 1, i = 8 * (e % pieces);
        *reinterpret_cast<u32x4*>(a.vrows + (int64_t)(first + row) * 2 * a.rp + h * a.rp + i0 + i) =
            *reinterpret_cast<const u32x4*>(&st[h][row * L + i]);
      }
    }
  }
  // gradients of slots without tokens
  if (!a.zero_a) return;
  const int64_t na = (int64_t)r * a.d_a, n = na + (int64_t)r * a.d_b;
  const int64_t chunk = 4096;
  const int64_t per_slot = (n + chunk - 1) / chunk;
  for (int64_t item = blockIdx.x; item < a.slots * per_slot; item += gridDim.x) {
    const int slot = (int)(item / per_slot);
    if (a.plan.parts[slot].y != 0) continue;
    for (int64_t e = item % per_slot * chunk + threadIdx.x; e < min(n, (item % per_slot + 1) * chunk); e += 256) {
      if (e < na) a.zero_a[slot * na + e] = 0.0f;
      else a.zero_b[slot * (n - na) + e - na] = 0.0f;
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
// results are added by k_gram_sum.  A split of one tile has nothing to add: there
// each wavefront takes a column tile (141 tokens of 11 slots, 10880 to 5184
// features, 20 ranks: 22 us against 28 with three of four wavefronts idle).
// ---------------------------------------------------------------------------
constexpr int kGL = 72;   // staged row, elements

// 64 tokens x 64 columns: BF16 as eight 16-byte pieces a lane (row 8 j + l / 8),
// codes as four (row 16 j + l / 4) with their rows' scales.  As loaded: rows past
// the split's last repeat it, pieces past the row's end are its last eight.
struct GramTile {
  u32x4 v[8];
  float s[4];
  uint32_t keep[4];
};

// tok: the lane's token of the tile (lane = row).  NARROW: rows of fewer than
// eight (their code costs the others registers).
template <bool PACKED, bool NARROW>
__device__ __forceinline__ void gram_load(const GramSide& q, int64_t M, int64_t c0, int tok,
                                          int lane, GramTile& t) {
  if constexpr (PACKED) {
    const int64_t ldc = (q.d + 63) / 64 * 64;
    const uint8_t* codes = q.codes + c0 + 16 * (lane & 3);
    const float* sc = q.scale + c0 / 64 * M;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = __shfl(tok, 16 * j + (lane >> 2));
      t.v[j] = *reinterpret_cast<const u32x4*>(codes + row * ldc);
      t.s[j] = sc[row];
      if (q.keep) t.keep[j] = q.keep[row * (q.d / 32) + (c0 + 16 * (lane & 3)) / 32];
    }
  } else if (!NARROW || q.d >= 8) {
    const uint16_t* x = q.x + at8(c0 + 8 * (lane & 7), q.d);
#pragma unroll
    for (int j = 0; j < 8; ++j) t.v[j] = load_vec(x + __shfl(tok, 8 * j + (lane >> 3)) * q.d);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      t.v[j] = few8(q.x + __shfl(tok, 8 * j + (lane >> 3)) * q.d, c0 + 8 * (lane & 7), q.d);
  }
}

// rows: the tile's tokens; those behind are zeros.
template <bool PACKED, bool NARROW>
__device__ __forceinline__ void gram_stage(const GramSide& q, int64_t c0, int rows, GramTile& t,
                                           int lane, uint16_t* st) {
  if constexpr (PACKED) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t keep = q.keep ? t.keep[j] >> (16 * (lane & 1)) : 0xFFFFu;
      keep = 16 * j + (lane >> 2) < rows ? keep : 0u;
      u32x4 o[2];
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const uint32_t c = t.v[j][h >> 1] >> (16 * (h & 1));
        const uint32_t b = pack_bf16x2((float)(int8_t)c * t.s[j], (float)(int8_t)(c >> 8) * t.s[j]);
        const uint32_t k = keep >> (2 * h);
        o[h >> 2][h & 3] = b & (((k & 1) ? 0xFFFFu : 0u) | ((k & 2) ? 0xFFFF0000u : 0u));
      }
      u32x4* p = reinterpret_cast<u32x4*>(st + (16 * j + (lane >> 2)) * kGL + 16 * (lane & 3));
      p[0] = o[0];
      p[1] = o[1];
    }
  } else {
    if (c0 + 64 > q.d && (!NARROW || q.d >= 8)) {
      const int64_t col = c0 + 8 * (lane & 7);
#pragma unroll
      for (int j = 0; j < 8; ++j) t.v[j] = past8(t.v[j], col - at8(col, q.d));
    }
    if (rows < 64) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t.v[j] = only_if(8 * j + (lane >> 3) < rows, t.v[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<u32x4*>(st + (8 * j + (lane >> 3)) * kGL + 8 * (lane & 7)) = t.v[j];
  }
}

// A wavefront's part of a split: tiles w, w + 4, ...  sp: {slot, first tile,
// tokens, }, `first` the split's first position.
// AHEAD: the operands of both halves of a tile before the next tile's rows.  Loads
// return in order, so behind those the second half's wait for memory (4096
// tokens, 4096 to 4096 features, 64 ranks, 4 slots: 39.4 us, ahead 33.5, although
// 22 registers spill then); at 64 ranks the kernel for codes, which spills 5
// without it, has no registers left (6385 tokens, 4736 to 2605 features, 50 ranks
// 44 us, ahead 52).
template <int NB, bool PACKED, bool NARROW, bool AHEAD>
__device__ __forceinline__ void gram_item(const GramArgs8& a, const GramSide& q, int64_t c0,
                                          const int4& sp, int first, int w, int group,
                                          uint16_t* st, f32x4 (&acc)[NB][4]) {
  const int lane = threadIdx.x & 63;
  const int r16 = lane & 15, g = lane >> 4;
  const int tiles = (sp.z + 63) / 64;
  if (w >= tiles) return;
  auto token = [&](int j) {
    const int at = first + min(64 * j + lane, sp.z - 1);
    return a.plan.head ? a.plan.order[at] : at;
  };
  // the group's blocks of 16 ranks, three terms, of 32 tokens
  auto load_v = [&](const uint16_t* fr, int slice, u32x4 (&v)[NB][3]) {
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int term = 0; term < 3; ++term)
        v[n][term] = *reinterpret_cast<const u32x4*>(fr + ((term * a.nb + NB * group + n) * 2 + slice) * 512);
  };
  int next = token(w);
  GramTile cur;
  gram_load<PACKED, NARROW>(q, a.M, c0, next, lane, cur);
  next = token(w + 4);
  for (int j = w; j < tiles; j += 4) {
    // in the order of their use
    const uint16_t* fr = q.frags + (int64_t)(sp.y + j) * 3 * a.nb * 2 * 512 + lane * 8;
    u32x4 v[1 + AHEAD][NB][3];
    load_v(fr, 0, v[0]);
    gram_stage<PACKED, NARROW>(q, c0, sp.z - 64 * j, cur, lane, st);
    if (AHEAD) load_v(fr, 1, v[AHEAD]);
    if (j + 4 < tiles) {
      gram_load<PACKED, NARROW>(q, a.M, c0, next, lane, cur);
      next = token(j + 8);
    }
#pragma unroll
    for (int slice = 0; slice < 2; ++slice) {
      if (!AHEAD && slice == 1) load_v(fr, 1, v[0]);
      u32x4 b[4];
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) {
        const uint16_t* p = st + (32 * slice + 8 * g + (r16 >> 2)) * kGL + 16 * cb + 4 * (r16 & 3);
        const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * kGL);
        b[cb] = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
          for (int cb = 0; cb < 4; ++cb) acc[n][cb] = mfma16(v[AHEAD * slice][n][term], b[cb], acc[n][cb]);
    }
  }
}

template <int NB, bool PACKED, bool NARROW>
__global__ __launch_bounds__(256, 2) void k_gram8(GramArgs8 a) {
  constexpr int LR = 68;                            // a reduced row, FP32
  constexpr bool AHEAD = NB < 4 || !PACKED;
  __shared__ __attribute__((aligned(16))) uint8_t glds[4 * 64 * kGL * 2];
  static_assert(4 * 16 * LR * 4 <= 4 * 64 * kGL * 2, "reduction buffer");
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  uint16_t* st = reinterpret_cast<uint16_t*>(glds) + w * 64 * kGL;
  float* red = reinterpret_cast<float*>(glds);
  const int tiles = (int)((a.M + 63) / 64);
  const int ct0 = (int)((a.q[0].d + 63) / 64), ct1 = (int)((a.q[1].d + 63) / 64);
  const int ct01 = ct0 + ct1;
  int splits = (tiles + a.tps - 1) / a.tps;
  int4 sp = {0, 0, 0, 0};
  int first = 0, s_at = 0;
  if (a.plan.head) {
    // (in bounds whatever the plan holds: the grid stops at its room)
    const int s0 = (int)min((int64_t)blockIdx.x / a.groups / ct01, (int64_t)a.most - 1);
    s_at = s0;
    sp = a.plan.split[s0];
    first = a.plan.split_first[s0];
    if (!plan_fits(a.plan, a.M, a.slots)) return;
    splits = a.plan.head[kPlanSplits];
  }
  const int64_t items = (int64_t)splits * ct01;
  for (int64_t it = blockIdx.x; it < items * a.groups; it += gridDim.x) {
    int group;
    const int64_t item = ranked(it, a.groups, items, group);
    const int si = (int)(item / ct01);
    int ct = (int)(item % ct01);
    const int side = ct >= ct0 ? 1 : 0;
    if (side) ct -= ct0;
    const GramSide& q = a.q[side];
    int64_t part = -1;
    if (a.plan.head) {
      if (si != s_at) {
        s_at = si;
        sp = a.plan.split[si];
        first = a.plan.split_first[si];
      }
      if (sp.w >= 0) part = a.plan.parts[sp.x].x + sp.w;
    } else {
      first = 64 * si * a.tps;
      sp = int4{0, si * a.tps, (int)min((int64_t)64 * a.tps, a.M - first), 0};
      if (splits > 1) part = si;
    }
    // one tile: each wavefront a column tile of its own, and nothing to add
    const bool alone = sp.z <= 64;
    if (alone) {
      if (ct & 3) continue;
      ct += w;
    }
    const int64_t c0 = (int64_t)ct * 64;
    f32x4 acc[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) acc[nb][cb] = f32x4{0.f, 0.f, 0.f, 0.f};
    float* out = part >= 0 ? q.part + part * a.r * q.d : q.out + (int64_t)sp.x * a.r * q.d;
    if (!alone || c0 < q.d) {
      if (PACKED && side == 0) gram_item<NB, true, NARROW, AHEAD>(a, q, c0, sp, first, alone ? 0 : w, group, st, acc);
      else gram_item<NB, false, NARROW, AHEAD>(a, q, c0, sp, first, alone ? 0 : w, group, st, acc);
    }
    if (alone) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int cb = 0; cb < 4; ++cb)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int64_t c = c0 + 16 * cb + r16;
            const int rank = 16 * NB * group + 16 * nb + 4 * g + v;
            if (rank < a.r && c < q.d) out[side ? c * a.r + rank : rank * q.d + c] = acc[nb][cb][v];
          }
      continue;
    }

    // accumulator lane (r16, g): ranks 16 nb + 4 g + v of the group, column c0 + 16 cb + r16
    const int i0 = 16 * NB * group;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      lds_barrier();
#pragma unroll
      for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[(w * 16 + 4 * g + v) * LR + 16 * cb + r16] = acc[nb][cb][v];
      lds_barrier();
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = threadIdx.x + 256 * u;
        const int i = side ? e & 15 : e >> 6, c = side ? e >> 4 : e & 63;
        float sum = red[i * LR + c];
#pragma unroll
        for (int ww = 1; ww < 4; ++ww) sum += red[(ww * 16 + i) * LR + c];
        const int rank = i0 + 16 * nb + i;
        if (rank < a.r && c0 + c < q.d) out[side ? (c0 + c) * a.r + rank : rank * q.d + c0 + c] = sum;
      }
    }
    lds_barrier();
  }
}

// Gradients of slots with several splits: their parts added in order (none:
// zeros).
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
    if (pt.y == 1 || (a.plan.head && pt.y == 0)) continue;
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

constexpr int64_t kMostGrid = 4096;

template <typename K>
hipError_t allow_lds(K kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int NB, bool KN, bool FAST>
hipError_t launch_shrink_t(const ShrinkArgs& a, unsigned grid, hipStream_t st) {
  constexpr int lds = shrink_lds<NB, KN>();
  static const hipError_t attr = allow_lds(&k_shrink<NB, KN, FAST>, lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((k_shrink<NB, KN, FAST>), dim3(grid), dim3(64 * kShrinkWaves), lds, st, a);
  return hipGetLastError();
}
template <int NB>
hipError_t launch_shrink_nb(const ShrinkArgs& a, unsigned grid, hipStream_t st) {
  const bool fast = a.K >= 8 && (!a.kn || a.r % 8 == 0);
  if (a.kn) return fast ? launch_shrink_t<NB, true, true>(a, grid, st)
                        : launch_shrink_t<NB, true, false>(a, grid, st);
  return fast ? launch_shrink_t<NB, false, true>(a, grid, st)
              : launch_shrink_t<NB, false, false>(a, grid, st);
}

template <int KS, bool RD, bool R8, bool DEEP, bool SUMS>
hipError_t launch_expand_t(const ExpandArgs& a, unsigned grid, hipStream_t st) {
  constexpr int few = RD ? 4 * 32 * 72 * 2 : 0, many = kTurnBytes + expand_lds<KS, RD>();
  constexpr int lds = many > few ? many : few;
  static const hipError_t attr = allow_lds(&k_expand<KS, RD, R8, DEEP, SUMS>, lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((k_expand<KS, RD, R8, DEEP, SUMS>), dim3(grid), dim3(256), lds, st, a);
  return hipGetLastError();
}
template <int KS, bool RD, bool R8>
hipError_t launch_expand_mode(const ExpandArgs& a, unsigned grid, hipStream_t st) {
  // (expand_sums: the forward of few tokens and ranks)
  if constexpr (!RD && KS <= 2)
    if (a.part) return launch_expand_t<KS, RD, R8, false, true>(a, grid, st);
  return a.tpi > 1 ? launch_expand_t<KS, RD, R8, true, false>(a, grid, st)
                   : launch_expand_t<KS, RD, R8, false, false>(a, grid, st);
}
template <int KS>
hipError_t launch_expand_ks(const ExpandArgs& a, unsigned grid, hipStream_t st) {
  if (a.rd) return launch_expand_mode<KS, true, true>(a, grid, st);
  return a.r % 8 == 0 ? launch_expand_mode<KS, false, true>(a, grid, st)
                      : launch_expand_mode<KS, false, false>(a, grid, st);
}

template <int NB>
hipError_t launch_gram8_nb(GramArgs8 a, hipStream_t st) {
  const int64_t tiles = (a.M + 63) / 64;
  a.most = (int)(a.plan.head ? plan_most_splits(a.M, a.slots) : (tiles + a.tps - 1) / a.tps);
  const int64_t cols = (a.q[0].d + 63) / 64 + (a.q[1].d + 63) / 64;
  a.nb = frag_blocks(a.r);
  a.groups = a.nb / NB;
  const unsigned grid = (unsigned)std::min<int64_t>(a.most * cols * a.groups, 2 * kMostGrid);
  auto run = [&](auto narrow) {
    constexpr bool NARROW = decltype(narrow)::value;
    if (a.q[0].codes) hipLaunchKernelGGL((k_gram8<NB, true, NARROW>), dim3(grid), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_gram8<NB, false, NARROW>), dim3(grid), dim3(256), 0, st, a);
  };
  if (std::min(a.q[0].d, a.q[1].d) < 8) run(std::true_type{});
  else run(std::false_type{});
  return hipGetLastError();
}


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
  if (a.splits > 1) a.vrows = nullptr;             // k_finish forms V
  const int64_t tiles = a.plan.head ? plan_most_tiles(a.M, a.slots) : (a.M + 63) / 64;
  a.groups = std::max(1, frag_blocks(a.r) / 4);
  a.rp = (int)vrow_ranks(a.r);
  a.most = (int)tiles;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles * a.splits * a.groups, kMostGrid);
  if (a.r <= 16) return launch_shrink_nb<1>(a, grid, st);
  if (a.r <= 32) return launch_shrink_nb<2>(a, grid, st);
  return launch_shrink_nb<4>(a, grid, st);
}

hipError_t launch_expand(const ExpandArgs& a0, hipStream_t st) {
  ExpandArgs a = a0;
  const int64_t cols = a.r <= 64 ? expand_cols<2>() : (a.r <= 128 ? expand_cols<4>() : expand_cols<8>());
  a.chunks = (int)((a.d + cols - 1) / cols);
  // more tiles an item where there are enough items
  const int64_t tiles = (a.M + kPlanTile - 1) / kPlanTile;
  a.tpi = (int)std::max<int64_t>(1, std::min<int64_t>(8, tiles * a.chunks / 1024));
  if (a.part) a.tpi = 1;
  const bool deep = a.tpi > 1;
  a.subs = deep ? (plan_split_tiles(a.M) + a.tpi - 1) / a.tpi : 1;
  a.most = (int)(deep ? plan_most_splits(a.M, a.slots) : plan_most_tiles(a.M, a.slots));
  const int64_t most = (int64_t)a.most * a.subs + (deep ? (a.M + 63) / 64 : 0);
  const unsigned grid = (unsigned)std::min<int64_t>(most * a.chunks, kMostGrid);
  if (a.r <= 32) return launch_expand_ks<1>(a, grid, st);
  if (a.r <= 64) return launch_expand_ks<2>(a, grid, st);
  if (a.r <= 128) return launch_expand_ks<4>(a, grid, st);
  return launch_expand_ks<8>(a, grid, st);
}

hipError_t launch_finish_v(const FinishVArgs& f0, hipStream_t st) {
  FinishVArgs f = f0;
  f.nb = frag_blocks(f.r);
  const int64_t tiles = f.plan.head ? plan_most_tiles(f.M, f.slots) : (f.M + 63) / 64;
  f.most = (int)tiles;
  if (f.rp == 0) f.rp = (int)vrow_ranks(f.r);
  int64_t items = tiles * 2 * ((f.nb + 3) / 4) * (f.t_frags ? 2 : 1);
  if (f.zero_a) items = std::max<int64_t>(items, std::min<int64_t>(f.slots * ((f.r * (f.d_a + f.d_b) + 4095) / 4096), 1024));
  const dim3 grid((unsigned)std::min<int64_t>(items, kMostGrid));
  if (f.splits <= 4) hipLaunchKernelGGL(k_finish<4>, grid, dim3(256), 0, st, f);
  else hipLaunchKernelGGL(k_finish<kShrinkSplits>, grid, dim3(256), 0, st, f);
  return hipGetLastError();
}

hipError_t launch_gram8(const GramArgs8& a, hipStream_t st) {
  const int64_t tiles = (a.M + 63) / 64;
  hipError_t e = hipSuccess;
  const int64_t splits = (tiles + a.tps - 1) / std::max(a.tps, 1);
  switch (frag_blocks(a.r)) {
    case 1: e = launch_gram8_nb<1>(a, st); break;
    case 2: e = launch_gram8_nb<2>(a, st); break;
    default: e = launch_gram8_nb<4>(a, st);
  }
  if (e != hipSuccess) return e;
  // with one split a slot at most nothing is left to add
  if (a.plan.head ? a.M <= int64_t(kPlanTile) * plan_split_tiles(a.M) : splits <= 1)
    return hipSuccess;
  const int64_t chunks = (a.r * a.q[0].d + 1023) / 1024 + (a.r * a.q[1].d + 1023) / 1024;
  hipLaunchKernelGGL(k_gram_sum, dim3((unsigned)std::min<int64_t>(a.slots * chunks, 2 * kMostGrid)),
                     dim3(256), 0, st, a, (int)splits);
  return hipGetLastError();
}

}  // namespace qlora
