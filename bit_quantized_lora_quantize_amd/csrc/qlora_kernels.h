// qlora_kernels.h -- launch interfaces between the host library (api.cpp) and
// the HIP kernels of libqlora.  Internal; not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qlora.h"

namespace qlora {

// Event pair around the next weight-kernel launch: only in the timing build
// (QLORA_TIMING_HOOK, libqlora_timed.so) that benchmarks use to time single
// kernels; the library itself keeps no state and these are empty.
#ifdef QLORA_TIMING_HOOK
void weight_kernel_begin(hipStream_t st);
void weight_kernel_end(hipStream_t st);
#else
inline void weight_kernel_begin(hipStream_t) {}
inline void weight_kernel_end(hipStream_t) {}
#endif

// ----------------------------------------------------------- quantization
constexpr int kLutSize = 129;     // buckets floor(64 x) + 64 for x in [-1, 1]
constexpr int64_t kTreeLds = 4096; // top tree levels done in one workgroup

// Nearest-level decision table for x in [-1, 1]: bucket b covers
// [(b-64)/64, (b-63)/64) and idx = base[b] + (x >= thr[b]).
struct IndexLut {
  float thr[kLutSize];
  uint8_t base[kLutSize];
};

struct QuantWorkspace {
  float* absmax;  // [n1]
  double* part;   // [Gp] group sums, Gp = next power of two >= G
};

hipError_t launch_quantize(const float* W, int64_t n, uint8_t* codes, uint8_t* scale_codes,
                           float* scale2, float* mean, const QuantWorkspace& ws,
                           const IndexLut& lut, hipStream_t st);
// The top of the mean's tree: part[0..Gp) (Gp a power of two) summed by the
// stride-halving tree, mean = FP32(sum / n1).
void launch_mean_tree(double* part, int64_t Gp, int64_t n1, float* mean, hipStream_t st);
// Workgroups for `work` items at `per_block` per workgroup, in [1, max_blocks].
int grid_for(int64_t work, int per_block, int max_blocks);

// General block sizes: first-level blocks of `block` elements (a power of
// two, 32..4096), second-level groups of `group` scales (a power of two,
// 16..1024), any n >= 1 (short last block and group).  Workspace: absmax
// FP32 [n1], part FP64 [power of two >= ceil(n1 / group)].
struct BlockedQuant {
  const float* W;
  int64_t n, block, group;
  uint8_t* codes;
  uint8_t* scale_codes;
  float* scale2;
  float* mean;
  float* absmax;
  double* part;
};
hipError_t launch_quantize_blocked(const BlockedQuant& q, const IndexLut& lut, hipStream_t st);
hipError_t launch_dequant_blocked(const uint8_t* codes, const uint8_t* scale_codes,
                                  const float* scale2, const float* mean, int64_t n,
                                  int64_t block, int64_t group, uint16_t* out, hipStream_t st);
hipError_t launch_dequant(const uint8_t* codes, const uint8_t* scale_codes, const float* scale2,
                          const float* mean, int64_t n, uint16_t* out, hipStream_t st);

// ------------------------------------------------------------- rank-r work
constexpr int kMaxGroup = 8;
// Index of the problem of a grouped launch that workgroup (or task) x
// belongs to: the number of problems i >= 1 with begin(i) <= x, begin
// nondecreasing.  All the begins are read at once (independent loads of
// the kernel arguments), not one after another.
template <typename Begin>
__device__ __forceinline__ int group_index(int count, int x, Begin begin) {
  int di = 0;
#pragma unroll
  for (int i = 1; i < kMaxGroup; ++i) {
    const int b = begin(i);
    di += (i < count && x >= b) ? 1 : 0;
  }
  return di;
}

// Quantize / dequantize of up to kMaxGroup tensors per launch (one list),
// each with the arithmetic of a single call.  Encode workgroups: Gp per
// tensor from enc_begin; second-level workgroups from scale_begin;
// dequantize workgroups: wgs per tensor from begin.
struct QuantItem {
  const float* W;
  int64_t n1, G, Gp;
  int64_t len;            // tree length left for the last launch (<= kTreeLds)
  uint8_t* codes;
  uint8_t* scale_codes;
  float* scale2;
  float* mean;
  float* absmax;          // workspace [n1]
  double* part;           // workspace [Gp]
  int enc_begin, scale_begin;
};
struct QuantList {
  QuantItem d[kMaxGroup];
  int count;
  int enc_wgs, scale_wgs;
};
// One QuantItem of a tensor of n weights (its len and begins are set by
// launch_quantize_list).
QuantItem quant_item(const float* W, int64_t n, uint8_t* codes, uint8_t* scale_codes,
                     float* scale2, float* mean, const QuantWorkspace& ws);
hipError_t launch_quantize_list(QuantList& a, const IndexLut& lut, hipStream_t st);

struct DequantItem {
  const uint8_t* codes;
  const uint8_t* scale_codes;
  const float* scale2;
  const float* mean;
  int64_t n1;
  uint16_t* out;
  int wgs, begin;
};
struct DequantList {
  DequantItem d[kMaxGroup];
  int count;
  int wgs;
};
hipError_t launch_dequant_list(DequantList& a, hipStream_t st);

// Small-M rank-r product (M <= 16), up to kMaxGroup problems per launch, as
// kRankSmallSplits partial sums over consecutive quarters of K:
//   part[s][m][n] = sum_{k in quarter s} P[m][k] Q[n][k],
// P [M][K] BF16, Q [N][ldq] BF16, part FP32 [kRankSmallSplits][M][N].
// v = scale * (((part[0] + part[1]) + part[2]) + part[3]) is formed by the
// consumer (weight-streaming epilogue or launch_rank_finish) in that order,
// so every path gets the same bits.  One 4-wavefront workgroup per
// 16-column block, problem and quarter; wavefronts take consecutive parts
// of the quarter and add their sums in wavefront order.  The first
// workgroup of a problem also clears zero[0 .. zero_count) (split-K counters
// of the following weight-streaming launch).
constexpr int kRankSmallSplits = 4;
struct RankSmallDesc {
  const uint16_t* P;
  const uint16_t* Q;
  int64_t K, ldq, N;
  float* part;
  uint32_t* zero;
  int64_t zero_count;
  int wg_begin;     // first workgroup of this problem (set by the launcher)
};
struct RankSmallArgs {
  RankSmallDesc d[kMaxGroup];
  int count;
  int64_t M;
};
hipError_t launch_rank_small(const RankSmallArgs& a, hipStream_t st);

// Large-M rank-r product in one pass, no partials:
//   v[m][n] = scale * sum_k P[m][k] Q[n][k],  P [M][K], Q [N][ldq], N <= 256.
// Outputs, each optional (NULL skips): out FP32 [M][N]; hl BF16 [M][2 rp],
// hi | lo split of v with zeros for n in [N, rp) (rp a multiple of 32,
// rp >= N); ht / lt the transposed hi / lo BF16 copies, element (n, m) at
// frag_index(n, m, ldt), with zeros for m in [M, ldt) and n in [N, round_up(N,
// 32)) (ldt a multiple of 16, >= M; round_up(N, 32) * ldt elements).
// Fragment order of the transposed rank-r copies (the token contraction's
// MFMA row operand): 32-row x 16-token chunks of 1 KB, chunk (i / 32, k / 16)
// at chunk index (i / 32) * (ldt / 16) + k / 16, and inside a chunk the
// 16-byte piece of lane (i % 32) + 32 ((k / 8) % 2) holding tokens k & ~7 ..
// +8, so a wavefront reads one chunk with one contiguous 1 KB load.
__host__ __device__ inline int64_t frag_index(int64_t i, int64_t k, int64_t ldt) {
  return (((i >> 5) * (ldt >> 4) + (k >> 4)) * 64 + (i & 31) + 32 * ((k >> 3) & 1)) * 8 + (k & 7);
}

struct RankRowsArgs {
  const uint16_t* P;
  const uint16_t* Q;
  int64_t M, N, K, ldq;
  float scale;
  float* out;
  uint16_t* hl;
  int64_t rp;
  uint16_t* ht;
  uint16_t* lt;
  int64_t ldt;
  // optional keep bits of P (row-major words, bit k % 32 of word
  // [m * K / 32 + k / 32]; K a multiple of 32): P elements with bit 0 count as
  // zero.  Only launch_rank_split (k_rank_part) takes them.
  const uint32_t* pmask = nullptr;
  // Q given as stored [K][ldq] (element (n, k) at Q[k * ldq + n]) instead of
  // [N][ldq]: only launch_rank_split takes it, with N, ldq and K multiples
  // of 8, P, Q 16-byte aligned and no keep bits.
  bool q_kn = false;
};
hipError_t launch_rank_rows(const RankRowsArgs& a, hipStream_t st);
// The same product (same outputs) through K-split partials part
// [rank_k_splits(M, K)][M][N] FP32 and k_rank_finish (splits added in order);
// K or ldq not a multiple of 8, or unaligned P / Q, take launch_rank_rows.
// extra (optional): one more finish problem with the same M, run in the same
// finish launch.
struct FinishDesc;
hipError_t launch_rank_split(const RankRowsArgs& a, float* part, hipStream_t st,
                             const FinishDesc* extra = nullptr);
// K splits of launch_rank_split: about 512 workgroups of 64 rows; each split
// a multiple of 128 columns.  *kper receives the split length.
#ifndef QLORA_RANK_TARGET_WGS
#define QLORA_RANK_TARGET_WGS 512
#endif
inline int rank_k_splits(int64_t M, int64_t K, int64_t* kper) {
  const int64_t rb = (M + 63) / 64;
  const int64_t maxs = (K + 127) / 128;
  int64_t ks = (QLORA_RANK_TARGET_WGS + rb - 1) / rb;
  ks = ks < 1 ? 1 : (ks > maxs ? maxs : ks);
  int64_t per = ((K + ks - 1) / ks + 127) / 128 * 128;
  if (per < 128) per = 128;
  *kper = per;
  return (int)((K + per - 1) / per);
}

// Finish of split partials: v[m][n] = scale * sum_s part[s][m][n] (s
// ascending).  out (optional) = v, FP32 [M][N]; ht/lt (optional) = the
// transposed hi/lo BF16 pair of v in fragment order (as for RankRowsArgs).
// Up to kMaxGroup independent problems per launch.
struct FinishDesc {
  const float* part;
  float* out;
  uint16_t* ht;
  uint16_t* lt;
  int64_t M, N, ldt;
  float scale;
  int splits;
  int wg_begin;
  uint16_t* hl;   // optional row-major split: hl[m][n] = hi, hl[m][rp + n] = lo, zero for n in [N, rp)
  int64_t rp;
};
struct FinishArgs {
  FinishDesc d[kMaxGroup];
  int count;
};
hipError_t launch_rank_finish(const FinishArgs& a, hipStream_t st);
// Single-problem convenience form.
hipError_t launch_rank_finish(const float* part, int splits, int64_t M, int64_t N, float scale,
                              float* out, uint16_t* ht, uint16_t* lt, int64_t ldt,
                              uint16_t* hl, int64_t rp, hipStream_t st);

// The same finish for many rows (one workgroup per 16 rows x 64 columns,
// coalesced partial reads and transposed writes through LDS); identical
// outputs.  The list form runs up to kMaxGroup problems with the same M in
// one launch.
hipError_t launch_rank_finish_rows(const float* part, int splits, int64_t M, int64_t N,
                                   float scale, float* out, uint16_t* ht, uint16_t* lt,
                                   int64_t ldt, uint16_t* hl, int64_t rp, hipStream_t st);
hipError_t launch_rank_finish_rows(const FinishDesc* d, int count, hipStream_t st);

// Transpose of a BF16 matrix in[rows][cols] into out[cols][ldo]:
// out[c][i] = in[i][c] for i < rows, and 0 for i in [rows, ldo).
hipError_t launch_transpose_bf16(const uint16_t* in, int64_t rows, int64_t cols, uint16_t* out,
                                 int64_t ldo, hipStream_t st);

// Token contractions out = P^T Q over the M tokens: part[s][i][c] = sum
// over tokens m in split s of P[m][i] * Q[m][c], then out = sum_s part[s]
// (s ascending), out[c][i] if transposed else out[i][c].  P is given
// transposed as a hi + lo BF16 pair in fragment order (frag_index, ldp >= M
// a multiple of 16, round_up(R, 32) rows, zero-padded); Q BF16 [M][N]
// (16-byte aligned); R <= 256; m_per_split a multiple of 128.  Up to two
// problems with the same M, R and ldp run in one contraction launch and one
// finish launch.
struct GramProblem {
  const uint16_t* Pt_hi;
  const uint16_t* Pt_lo;
  const uint16_t* Q;
  int64_t N, m_per_split;
  int splits;
  float* part;   // [splits][R][N]
  float* out;
  bool transposed;
  // optional keep bits of Q (row-major words [M][N / 32], N a multiple of
  // 32): Q elements with bit 0 count as zero
  const uint32_t* qmask = nullptr;
};
hipError_t launch_grams(const GramProblem* p, int count, int64_t ldp, int64_t M, int64_t R,
                        hipStream_t st);

// ------------------------------------------------- optimizer step
// Tensors are handled in batches of up to kOptBatch per launch (descriptors
// passed by value), so a step over many small adapter tensors costs a few
// launches rather than a few per tensor.
constexpr int kOptBatch = 32;
constexpr int64_t kOptMaxElems = int64_t(1) << 32;  // per tensor
constexpr int kAdamwChunk = 1024;                   // elements per workgroup

// acc[0] += sum over tensors t (in order) of the FP64 sum of grads[t][i]^2
// (groups of 256 by the stride-halving tree, then the tree over the group
// sums padded to a power of two).  part: FP64, sum over t of that power of
// two (sumsq_part_len); sums: FP64 [count].  grads and n are host arrays.
int64_t sumsq_part_len(int64_t n);
hipError_t launch_sumsq(const float* const* grads, const int64_t* n, int count, double* acc,
                        double* part, double* sums, hipStream_t st);
struct AdamwDesc {
  float* param;       // FP32 master [n]
  uint16_t* p16;      // optional BF16 copy [n]
  const float* grad;  // [n]
  float* m;           // first moment [n]
  float* v;           // second moment [n]
  int64_t n;
};
struct AdamwScalars {
  float lr, lrwd, b1, ob1, b2, ob2, bc1, bc2, eps, max_norm;
};
// One AdamW step over `count` tensors (host array of descriptors, n > 0);
// sumsq (device, may be NULL: no clipping) gives the clip coefficient.
hipError_t launch_adamw(const AdamwDesc* d, int count, const AdamwScalars& h,
                        const double* sumsq, hipStream_t st);

// ------------------------------------------------- LoRA dropout mask
// Xm = X with the dropped elements cleared (may be NULL) and the keep bits
// keep[k * ldw + m / 32] (may be NULL); d even, X rows 4-byte aligned.
struct DropoutArgs {
  const uint16_t* X;
  uint16_t* Xm;
  uint32_t* keep;
  int64_t M, d, ldw;      // ldw = ceil(M / 32)
  uint32_t thr;           // keep when the generator word >= thr
  uint32_t key_lo, key_hi, off_lo, off_hi;
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st);
// The same mask as keep bits only, in two layouts (either may be NULL):
// keep [d][ldw] (bit m % 32 of word [k][m / 32], as launch_dropout) and
// rbits [M][d / 32] (bit k % 32 of word [m][k / 32]), d a multiple of 32.
// X and Xm are not used.
hipError_t launch_dropout_bits(const DropoutArgs& a, uint32_t* rbits, hipStream_t st);

// ------------------------------------------------- LoRA merge
// out[n][k] = RN_fp32(Wh[n][k] + scale * sum_i B[n][i] A[i][k]) (FP64
// evaluation), Wh the restored BF16 weight of the quantized state.
struct MergeArgs {
  const uint8_t* codes;
  const uint8_t* scodes;
  const float* scale2;
  const float* mean;
  const uint16_t* A;      // [r][d_in]
  const uint16_t* B;      // [d_out][r]
  float* out;             // [d_out][d_in]
  int64_t d_out, d_in, r;
  float scale;
};
hipError_t launch_merge(const MergeArgs& a, hipStream_t st);

// ------------------------------------------------- small-M forward (GEMV)
// Y[m][n] = RNE_bf16( sum_k X[m][k] Wh[n][k] + sum_i T[m][i] B[n][i] ),
// T = t_scale * XA A^T, for m < M <= 16, up to kMaxGroup layers per launch.
//
// Work.  A weight unit is one 64-row tile of one layer's weight times one
// 256-wide K super-step; a layer's units are listed tile by tile,
// super-step by super-step.  A T task forms one partial of T over a chunk
// of tchunk_ss super-steps for 16 ranks: tpart[c][m][i] = sum over the
// chunk's columns k of XA[m][k] A[i][k]; a layer has ceil(r / 16) x tchunks
// of them.  Each layer's work is one list: its T tasks first, each counted
// as tcost units, then its weight units (toff = n_tasks x tcost onwards).
//
// The weight-streaming launch gives layer i a block of wgs_i workgroups
// (wg_begin ..), the blocks sized in proportion to the layers' work so that
// the launch has kGemvWgs workgroups, four on every compute unit, each with
// about the same work.  Workgroup j of a layer takes the contiguous range
// gemv_unit_begin(j) .. gemv_unit_begin(j + 1) of the layer's list (uq or
// uq + 1 units, the first urem workgroups one more): the T tasks that start
// in it, then its weight units, writing one FP32 partial per tile it
// touches into slot j - gemv_wg_of(toff + first unit of the tile) of that
// tile (part[slot][m][n], at most kGemvMaxSlots slots per tile).
//
// The finish launch (one workgroup per 64 output columns) adds a tile's
// slots in order, forms T = t_scale * (((tpart[0] + tpart[1]) + ...) in
// chunk order, adds the LoRA term, rounds Y and, from the workgroup of the
// first columns, writes T_save.  The backward's recompute of T runs the same
// T tasks (launch_gemv_tasks) and k_rank_finish adds the same partials in
// the same order: both get the same bits.
#ifndef QLORA_GEMV_WGS
#define QLORA_GEMV_WGS 1024
#endif
constexpr int kGemvRows = 64;                       // rows per tile (16 per wavefront)
constexpr int kGemvWgs = QLORA_GEMV_WGS;            // workgroups of one launch
constexpr int kGemvMaxSlots = 16;                   // partials per tile, at most
constexpr int kGemvMaxChunks = 16;                  // T chunks per layer, at most
struct GemvDesc {
  const uint8_t* codes;
  const uint8_t* scodes;
  const float* scale2;
  const float* mean;
  const uint16_t* X;      // [M][d_in], 16-byte aligned: the base product's input
  const uint16_t* XA;     // LoRA branch input [M][d_in] (X, or X with dropped
                          // elements cleared), 16-byte aligned
  const uint16_t* A;      // [r][d_in], 16-byte aligned
  const uint16_t* B;      // [d_out][r]
  float* T_save;          // T FP32 [M][r] or NULL
  uint16_t* Y;            // [M][d_out]
  float* part;            // [kGemvMaxSlots][M][d_out]
  float* tpart;           // [tchunks][M][r]
  int64_t d_out, d_in, r;
  float t_scale;
  int tiles;              // 64-row tiles
  int nss;                // 256-wide super-steps of K
  int units;              // weight units: tiles * nss
  int tchunks;            // T chunks
  int tchunk_ss;          // super-steps per T chunk
  int n_tasks;            // T tasks: ceil(r / 16) * tchunks
  int tcost;              // units a T task counts for
  int toff;               // n_tasks * tcost
  int task_begin;         // first T task of this layer (T tasks alone)
  int wgs;                // workgroups of this layer in the streaming launch
  int wg_begin;           // its first workgroup there
  int uq, urem;           // (toff + units) / wgs and (toff + units) % wgs
  int fin_begin;          // first finish workgroup of this layer
};
struct GemvArgs {
  GemvDesc d[kMaxGroup];
  int count;
  int M;
  int wgs;                // workgroups of the weight-streaming launch
  int tasks;              // workgroups of a T-tasks-alone launch
  int fin_wgs;            // workgroups of the finish launch
  bool vec_b;             // every B 16-byte aligned with r % 8 == 0
};
// First unit of workgroup j of a list split over workgroups with
// q = units / wgs, rem = units % wgs (the first rem get one unit more), and
// the workgroup of unit u.  Lists hold fewer than 2^31 units.
__host__ __device__ inline int gemv_unit_begin(int j, int q, int rem) {
  return j * q + (j < rem ? j : rem);
}
__host__ __device__ inline int gemv_wg_of(int u, int q, int rem) {
  const int big = rem * (q + 1);
  return u < big ? (int)((unsigned)u / (unsigned)(q + 1))
                 : rem + (int)((unsigned)(u - big) / (unsigned)q);
}
// LDS of the weight-streaming launch: a ring of kGemvRing staged X
// super-steps of 16 rows x 512 bytes (rows past M zero), which also holds a
// T task's reduction buffer.
#ifndef QLORA_GEMV_RING
#define QLORA_GEMV_RING 4
#endif
constexpr int kGemvRing = QLORA_GEMV_RING;
inline int64_t gemv_lds_bytes(int64_t M) {
  (void)M;
  return (int64_t)kGemvRing * 16 * 512;
}
hipError_t launch_gemv(const GemvArgs& a, hipStream_t st);
// The T tasks of `a` alone (one workgroup per task; no weight streaming).
hipError_t launch_gemv_tasks(const GemvArgs& a, hipStream_t st);

// ------------------------------------------------- large-M fused GEMM
// Forward: Y = RNE_bf16(X Wh^T + [T_hi T_lo] [B B]^T), dequant tiles in LDS.
// Backward: dX = RNE_bf16(dY Wh + [U_hi U_lo] [A A]), W tiles written
// transposed into LDS.
struct GemmArgs {
  const uint8_t* codes;
  const uint8_t* scodes;
  const float* scale2;
  const float* mean;
  const uint16_t* act;    // X [M][d_in] (forward) or dY [M][d_out] (backward)
  const uint16_t* ext;    // T or U split into BF16 terms: [M][2*RP], hi | lo, RP = r rounded up to 32
  const uint16_t* lw;     // B [d_out][r] (forward) or A [r][d_in] (backward)
  uint16_t* out;          // Y [M][d_out] or dX [M][d_in]
  int64_t M, d_out, d_in, r;
  // backward with LoRA dropout: keep bit of (m, c) is bit m % 32 of
  // keep[c * keep_ld + m / 32]; the LoRA term of dX is cleared where it is 0
  const uint32_t* keep;
  int64_t keep_ld;
};
hipError_t launch_gemm_fwd(const GemmArgs& a, hipStream_t st);
hipError_t launch_gemm_bwd(const GemmArgs& a, hipStream_t st);

// ------------------------------------------------- input gradient, few tokens
constexpr int kDxSplits = 8;   // at most
// Ranges of the outputs that k_dx_few sums apart, for about 1024 items.
inline int dx_few_splits(int64_t M, int64_t d_out, int64_t d_in, int64_t* nper) {
  const int64_t items = std::max<int64_t>(1, (M + 63) / 64 * (d_in / 64));
  int64_t s = std::min<int64_t>((1024 + items - 1) / items, (d_out + 127) / 128);
  s = std::max<int64_t>(1, std::min<int64_t>(s, kDxSplits));
  *nper = ((d_out + s - 1) / s + 127) / 128 * 128;
  return (int)((d_out + *nper - 1) / *nper);
}
// Whether it takes the place of the fused GEMM: while the GEMM has up to 64 tiles
// of 256 x 256 (whole backward, rank 16, this and the GEMM: 4096 -> 4096, 32 tiles
// 78 us and 118, 48 tiles 103 and 125, 64 tiles 113 and 126, 80 tiles 143 and 129,
// 128 tiles 205 and 133; 64 tiles of 1024 -> 4096 121 and 137, of 4096 -> 11008 257
// and 279, 80 of these 331 and 282), and for rows of dY that are no whole 16-byte
// pieces, which the GEMM loads by element (2048 tokens 4096 -> 4099 396 and 667, 8192
// tokens 1388 and 1424, 8192 tokens -> 4100 819 and 1240).
inline bool dx_few(int64_t M, int64_t d_out, int64_t d_in) {
  return d_out % 8 != 0 || (M + 255) / 256 * ((d_in + 255) / 256) <= 64;
}
struct DxFewArgs {
  const uint8_t* codes;
  const uint8_t* scodes;
  const float* scale2;
  const float* mean;
  const uint16_t* dY;      // [M][d_out]
  const uint16_t* u_hl;    // [M][2 rp] BF16 hi | lo of U
  const uint16_t* A;       // [r][d_in]
  uint16_t* dX;            // [M][d_in]
  float* part;             // [splits][M][d_in]
  int64_t M, d_out, d_in, r, rp;
  const uint32_t* keep;    // as GemmArgs
  int64_t keep_ld;
  int64_t nper;            // nper, splits: set by launch_dx_few
  int splits;
};
hipError_t launch_dx_few(const DxFewArgs& a, hipStream_t st);

// ------------------------------------------------- norms
// Element types are QLORA_BF16 / QLORA_F32; the operations are stated at
// qlora_norm_fwd and qlora_norm_bwd.
struct NormFwdArgs {
  const void* x;
  const void* r;      // residual or NULL
  const void* gamma;
  const void* beta;   // or NULL
  void* h;            // X + R, written when r is given
  void* y;
  float* mean;        // or NULL
  float* rstd;        // or NULL
  int64_t rows, d;
  float eps;
  int kind, type, w_type;
};
hipError_t launch_norm_fwd(const NormFwdArgs& a, hipStream_t st);

struct NormBwdArgs {
  const void* dy;
  const void* h;
  const void* dh;     // or NULL
  const void* gamma;
  const float* mean;  // NULL for RMS
  const float* rstd;
  void* dx;
  float* dgamma;      // or NULL
  float* dbeta;       // or NULL
  float* part;        // [norm_parts(rows, d)][2][d] partial weight gradients
  int64_t rows, d;
  int kind, type, w_type;
};
// Row groups whose weight gradients are summed apart (rows >= 1).
int norm_parts(int64_t rows, int64_t d);
hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t st);

// ------------------------------------------------- losses on logits
struct LogitsArgs {
  const void* logits;
  const int64_t* targets;
  int64_t rows, vocab, ld;
  int64_t ignore;
  int type;
  float scale;
};
// What a gradient needs of a row's softmax: p = exp(scale * (l - max) - logsum).
struct RowStat {
  float max, logsum;
};
// logp (and lse, stat: either may be NULL) of every row.
hipError_t launch_logp(const LogitsArgs& l, float* logp, float* lse, RowStat* stat,
                       hipStream_t st);
// dlogits from per-row coefficients; the softmax comes from stat, or from
// lse where stat is NULL.
hipError_t launch_dlogits(const LogitsArgs& l, const RowStat* stat, const float* lse,
                          const float* dlogp, void* dlogits, int64_t ldd, hipStream_t st);

struct PreferenceArgs {
  const int64_t* targets;
  const int64_t* offsets;  // [2 pairs + 1]
  const float* logp;
  const float* ref;        // or NULL
  int64_t rows, pairs, ignore;
  int kind, length_normalize;
  float beta, smoothing, margin, weight;
  float* seq_logp;         // [2 pairs]
  float* loss;             // [pairs]
  float* dlogp;            // [rows], or NULL for the loss alone
};
// a.logp is logp; dlogits NULL: the loss alone (a.dlogp is then not used).
// rows >= 0; without rows only the losses are written.
hipError_t launch_preference(const LogitsArgs& l, const PreferenceArgs& a, RowStat* stat,
                             float* logp, void* dlogits, int64_t ldd, hipStream_t st);

struct PolicyArgs {
  const int64_t* offsets;  // [seqs + 1]
  const float* adv;
  const float* old_logp;   // or NULL
  const float* ref;        // or NULL
  int64_t seqs;
  int reduction, per_token;
  float clip_low, clip_high, kl_coef, weight;
  float* logp;
  float* stats;            // [4]
  int32_t* count;          // [seqs] rows of each sequence that count
  int32_t* total;          // [1] their sum
  int32_t* row_seq;        // [rows] sequence of each row, -1 without one
  float4* terms;           // [rows] w, policy, kl, clipped
};
// dlogits NULL: the loss alone.
hipError_t launch_policy(const LogitsArgs& l, const PolicyArgs& a, void* dlogits, int64_t ldd,
                         hipStream_t st);

// ------------------------------------------------- activations in 8 bits
// codes [M][round_up(d, 64)], scale [ceil(d / 64)][M].
hipError_t launch_pack8(int type, const void* X, int64_t M, int64_t d, uint8_t* codes,
                        float* scale, hipStream_t st);
hipError_t launch_unpack8(const uint8_t* codes, const float* scale, int64_t M, int64_t d, int type,
                          void* X, hipStream_t st);

// ------------------------------------------------- adapters of many requests
// The plan of a batch: its tokens sorted by slot, those without adapter last,
// in tiles of up to kPlanTile tokens of one slot.
constexpr int kPlanTile = 64;
constexpr int kPlanMaxSlots = 2048;
constexpr int kPlanMagic = 0x51504C4E;
// head[]: tiles of tokens with an adapter, tiles of all, splits, M, slots
constexpr int kPlanTiles = 0, kPlanAllTiles = 1, kPlanSplits = 2, kPlanTokens = 3, kPlanSlots = 4,
              kPlanMagicAt = 5, kPlanHead = 16;
struct PlanView {
  int32_t* head;   // [kPlanHead]; NULL (contractions only): one slot, every token, in order
  int32_t* order;  // [M] token at each position
  int32_t* begin;  // [slots + 1] first position of each slot (batches of several spans)
  int4* tile;      // {slot (-1: none), first position, tokens, 0}: one load
  int4* split;     // {slot, first tile, tokens, number among its slot's splits (-1: the only one)}
  int32_t* split_first;   // their first positions
  int2* parts;     // [slots] {its splits' first partial result, its splits}
  int32_t* hist;   // scratch of the plan's own kernels
};
// Tiles of a token split of the weight gradients: 8 to 16 (four splits of one
// slot where that gives them), more where one slot would have 64 splits and more.
// Half as many (2048 tokens, 4096 x 4096, rank 64) took 22 us instead of 18 and
// 10 instead of 6 to add the parts.
inline int plan_split_tiles(int64_t M) {
  const int64_t tiles = (M + kPlanTile - 1) / kPlanTile;
  const int64_t four = std::min<int64_t>(16, std::max<int64_t>(8, (tiles + 3) / 4));
  return (int)std::max<int64_t>(four, (tiles + 63) / 64);
}
// Bounds of what the device counts.
inline int64_t plan_most_tiles(int64_t M, int64_t slots) {
  return std::min<int64_t>(M, M / kPlanTile + slots + 1);
}
inline int64_t plan_most_splits(int64_t M, int64_t slots) {
  return std::min<int64_t>(M, M / (int64_t(kPlanTile) * plan_split_tiles(M)) + slots);
}
// Splits of slots that have two or more: such a slot with n tokens has at most
// twice n / (tokens of a split).
inline int64_t plan_most_parts(int64_t M) {
  return 2 * M / (int64_t(kPlanTile) * plan_split_tiles(M));
}
hipError_t launch_plan(const PlanView& p, const int32_t* index, int64_t M, int64_t slots,
                       hipStream_t st);

// Ranges of the long axis K that k_shrink sums apart, for about 1024 items: two
// workgroups a compute unit, several times over, so that one's start and end
// overlap another's loads.  16384 tokens: K 4096, rank 64 in four ranges 55 us (and
// 9 to add them), in two 63 (8), in one 82; K 11008, rank 16 in four 80, in two 102.
constexpr int kShrinkSplits = 8;   // at most
inline int shrink_splits(int64_t M, int64_t K, int64_t* kper) {
  const int64_t tiles = std::max<int64_t>(1, (M + kPlanTile - 1) / kPlanTile);
  int64_t s = std::min<int64_t>((1024 + tiles - 1) / tiles, (K + 255) / 256);
  s = std::max<int64_t>(1, std::min<int64_t>(s, kShrinkSplits));
  *kper = ((K + s - 1) / s + 255) / 256 * 256;
  return (int)((K + *kper - 1) / *kper);
}
// Where the steps of a range [k_begin, k_end) of K end that k_shrink loads
// without conditions.  Rows of F stored [K][r] are taken in pieces of eight: where
// those do not end with the row (r % 8 != 0), the last piece of row k ends at
// element k r + round_up(r, 8), up to seven rows on (r = 1), and has to end within
// K r: that keeps the last (round_up(r, 8) - 1) / r rows of F out, in whichever
// range they lie.
__host__ __device__ inline int64_t shrink_whole_end(int64_t k_begin, int64_t k_end, int64_t K, int r,
                                                    bool kn, int step) {
  const int64_t last = K - (kn ? ((r + 7) / 8 * 8 - 1) / r : 0), end = k_end < last ? k_end : last;
  return k_begin + (end > k_begin ? end - k_begin : 0) / step * step;
}
// Ranks of a row of V in k_expand's operand (hi, then lo).
inline int64_t vrow_ranks(int64_t r) { return r <= 32 ? 32 : (r <= 64 ? 64 : (r <= 128 ? 128 : 256)); }
struct ShrinkArgs {
  PlanView plan;
  int64_t M, slots, K, kper;
  int r;
  int splits, groups, rp, most;   // and kper: set by launch_shrink
  bool kn;              // F as [K][r] (else [r][K])
  const uint16_t* P;    // [M][K]
  const uint16_t* F;    // [slots] of them
  float* part;          // [splits][M][r], by position
  // with one split, instead of part:
  const float* scale;   // [slots]
  uint16_t* vrows;      // [M][2 vrow_ranks(r)] by position, or NULL (part)
  float* v_out;         // [M][r] by token, or NULL
};
hipError_t launch_shrink(const ShrinkArgs& a, hipStream_t st);

struct FinishVArgs {
  PlanView plan;
  int64_t M, slots;
  int r, nb, most;         // nb, most: set by launch_finish_v
  int rp;                  // ranks of a row of vrows; 0: vrow_ranks(r)
  int splits;              // of the partial sums
  const float* scale;      // [slots]; NULL: one_scale
  float one_scale;
  const float* V;          // [splits][M][r] partial sums, by position
  const float* T;          // [M][r] by token, with t_frags
  uint16_t* vrows;         // outputs, each or NULL
  float* v_out;
  uint16_t* u_frags;       // V's
  uint16_t* t_frags;       // T's
  // with a plan: gradients of the slots without tokens, to be cleared, or NULL
  float* zero_a;           // [slots][r d_a]
  float* zero_b;           // [slots][r d_b]
  int64_t d_a, d_b;
};
hipError_t launch_finish_v(const FinishVArgs& a, hipStream_t st);
// Blocks of 16 ranks in the operands of the contractions.
inline int frag_blocks(int64_t r) {
  return r <= 16 ? 1 : (r <= 32 ? 2 : (r <= 64 ? 4 : (r <= 128 ? 8 : 16)));
}
// Elements of one side's operands for `tiles` tiles.
inline int64_t frag_elems(int64_t tiles, int64_t r) { return tiles * 3 * frag_blocks(r) * 1024; }

struct ExpandArgs {
  PlanView plan;
  int64_t M, slots, d;
  int r, chunks, subs, tpi, most;   // all but r set by launch_expand
  bool rd;                 // F as [r][d] (else [d][r])
  const uint16_t* vrows;   // [M][2 vrow_ranks(r)] by position, or
  const float* part;       // (expand_sums) k_shrink's partial sums,
  int splits;              // so many, with
  const float* scale;      // [slots]
  const uint16_t* F;       // [slots] of them
  const uint16_t* in;      // [M][d], NULL: zeros; may be out
  uint16_t* out;
  float* v_out;            // [M][r] or NULL: V (from partial sums), zeros without an adapter
};
// Whether the forward's expansion adds the partial sums itself, in every
// workgroup again, rather than have k_finish do it once in a launch of its own:
// one token 9 us in two kernels and 12 in three, 64 decoding 15 and 16.5, 1531
// tokens (4096 -> 1003, rank 20) 20 and 24.5.
inline bool expand_sums(int64_t M, int64_t r) { return M <= 2048 && r <= 64 && r % 4 == 0; }
hipError_t launch_expand(const ExpandArgs& a, hipStream_t st);

struct GramSide {
  const uint16_t* x;       // BF16 [M][d], or
  const uint8_t* codes;    // 8-bit codes [M][round_up(d, 64)] (side 0 only) with
  const float* scale;      // their scales [ceil(d / 64)][M] and
  const uint32_t* keep;    // keep words [M][d / 32] or NULL
  const uint16_t* frags;   // U's or T's
  float* out;              // [slots][r][d], side 1 [slots][d][r]
  float* part;             // partial results, [][r][d] or [][d][r]
  int64_t d;
};
struct GramArgs8 {
  PlanView plan;
  int64_t M, slots, r;
  int tps;                 // tiles a split
  int most, nb, groups;    // set by launch_gram8
  GramSide q[2];           // dA from (U, X), dB from (T, dY)
};
hipError_t launch_gram8(const GramArgs8& a, hipStream_t st);
// Zeros in both outputs.
hipError_t launch_gram_zero(const GramArgs8& a, hipStream_t st);

// ------------------------------------------------- host-side checks
// qlora_linear_fwd's argument checks for a workspace of ws_bytes bytes (not
// dereferenced): QLORA_ERR_WORKSPACE when the call needs more.
int linear_fwd_check(const qlora_nf4_t* q, const uint16_t* X, int64_t M, const uint16_t* A,
                     const uint16_t* B, int64_t r, uint16_t* Y, float* T_save, size_t ws_bytes);

}  // namespace qlora
