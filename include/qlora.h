/*
 * qlora.h -- C ABI of libqlora: the frozen-base NF4 LoRA linear layer on an
 * AMD CDNA4 (gfx950) GPU.
 *
 * Sources of the operations (the pages):
 *   [QP]  "第 04 篇：QLoRA 原理" (jupiter-lab.pages.dev, QLoRA principles)
 *   [CP]  "QLoRA" concept page (compassingai.com), sections
 *         "NF4 量化機制詳解" (NF4 steps) and "雙重量化" (double quantization).
 *
 * Conventions for every entry point
 *   - Every array argument is a DEVICE pointer to caller-owned memory.  The
 *     library allocates nothing, frees nothing and keeps no state between
 *     calls (the one exception is the fixed device array that
 *     qlora_linear_fwd_noalloc works in); it never synchronizes.  Work is
 *     enqueued on `stream` (a
 *     hipStream_t; NULL means the null stream) and the call returns at once.
 *   - All matrices are dense row-major (logits and their gradients: rows of
 *     stride ld).  BF16 values are passed as their
 *     uint16_t bit patterns.
 *   - Arguments are checked on the host before anything is enqueued; on any
 *     error the call returns a negative qlora_status and enqueues nothing.
 *     A failing kernel launch returns QLORA_ERR_HIP (work enqueued before it
 *     on the same call may have run).  Non-finite inputs are a precondition
 *     violation and are not detected, except where an entry point says
 *     otherwise.
 *   - Pointers marked (16B) must be 16-byte aligned.
 *   - Calls that share a workspace buffer must be ordered (same stream or
 *     explicit events); calls on different buffers may overlap freely.
 */
#ifndef QLORA_H
#define QLORA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  QLORA_OK = 0,
  QLORA_ERR_NULL = -1,       /* a required pointer is NULL                  */
  QLORA_ERR_SHAPE = -2,      /* a size is out of its documented range        */
  QLORA_ERR_ALIGN = -3,      /* a (16B) pointer is not 16-byte aligned       */
  QLORA_ERR_WORKSPACE = -4,  /* workspace smaller than qlora_workspace_bytes */
  QLORA_ERR_HIP = -5,        /* the HIP runtime reported an error            */
  QLORA_ERR_SCRATCH = -6     /* the call needs more than the library's fixed
                                device scratch (qlora_linear_fwd_noalloc)    */
} qlora_status;

/* Block sizes fixed by the method: 64 weights share one first-level scale
 * ([QP §3.4], [CP, NF4 量化機制詳解] step 1), 256 first-level scales share one
 * second-level FP32 scale ([QP §5.2], [CP, 雙重量化]). */
#define QLORA_BLOCK 64
#define QLORA_GROUP 256

/*
 * NF4 + double-quantized weight W[d_out, d_in] ([QP §2.1, §5.2, §6.1]).
 * n = d_out*d_in weights, flattened row-major; n1 = n/64 blocks;
 * G = ceil(n1/256) groups.  Requires d_in % 64 == 0 (no block straddles a
 * row), d_out >= 1.
 *   codes        uint8[n/2] (16B)  4-bit level indices, two per byte; element
 *                                  2j in the low nibble of byte j [QP §2.1].
 *   scale_codes  uint8[n1]         OCP FP8 E4M3FN codes of the centred block
 *                                  scales, (absmax_b - mean) / scale2[b/256].
 *   scale2       float[G]          second-level scales: the group's largest
 *                                  |absmax - mean| divided by 448.
 *   scale_mean   float[1]          mean of all n1 block absmax values.
 * The restored weight of element e in block b is
 *   RNE_bf16(codebook[idx_e] * (fp8(scale_codes[b]) * scale2[b/256] + mean))
 * with every FP32 operation rounded separately (no fused multiply-add), and
 * codebook = the 16 NF4 levels printed in [QP §4.3].
 */
typedef struct {
  int64_t d_out;
  int64_t d_in;
  uint8_t *codes;
  uint8_t *scale_codes;
  float *scale2;
  float *scale_mean;
} qlora_nf4_t;

/* Byte sizes of the four buffers of an NF4 weight (host only, no GPU use).
 * Returns QLORA_ERR_SHAPE for d_out < 1, d_in < 64 or d_in % 64 != 0, and
 * QLORA_ERR_NULL when an output pointer is NULL. */
int qlora_nf4_sizes(int64_t d_out, int64_t d_in, size_t *codes_bytes,
                    size_t *scale_codes_bytes, size_t *scale2_bytes,
                    size_t *scale_mean_bytes);

/* Operations for qlora_workspace_bytes. */
#define QLORA_OP_QUANTIZE 0
#define QLORA_OP_FWD 1
#define QLORA_OP_BWD 2
#define QLORA_OP_FWD_DROPOUT 3
#define QLORA_OP_BWD_DROPOUT 4
#define QLORA_OP_BWD_PACKED 5          /* qlora_linear_bwd_packed */
#define QLORA_OP_BWD_PACKED_DROPOUT 6  /* the same with dropout   */

/* Device workspace (bytes) that one call of `op` needs for these sizes
 * (M and r are ignored for QLORA_OP_QUANTIZE).  Host only.  Returns 0 for
 * sizes the call would reject. */
size_t qlora_workspace_bytes(int op, int64_t d_out, int64_t d_in, int64_t M,
                             int64_t r);

/*
 * Quantize W (FP32 [d_out, d_in], (16B)) into `q` ([QP §3.4, §4.3, §5.2];
 * [CP, NF4 量化機制詳解; 雙重量化]):
 *   1. absmax a_b of each 64-element block;
 *   2. x = w / a_b (IEEE FP32 division); a zero block gives x = 0;
 *   3. index of the nearest NF4 level, ties to the lower index;
 *   4. two indices per byte;
 *   5. mean of the a_b (FP64 sum in a fixed stride-halving tree: pairs
 *      (j, j+128), (j, j+64), ... within each group of 256, then the same
 *      tree over the group sums padded with zeros to a power of two; the
 *      FP64 quotient by n1 is rounded to FP32);
 *   6. per group: scale2 = max |a_b - mean| / 448 and FP8 E4M3FN codes of
 *      (a_b - mean) / scale2, round to nearest even, saturating at 448;
 *      a group whose scale2 is 0 stores code 0.
 * Deterministic: repeated calls give identical bytes.
 * q->codes (16B), q->scale_codes, q->scale2, q->scale_mean are outputs.
 * workspace (16B) >= qlora_workspace_bytes(QLORA_OP_QUANTIZE, ...).
 */
int qlora_quantize_nf4(const float *W, const qlora_nf4_t *q, void *workspace,
                       size_t workspace_bytes, void *stream);

/*
 * Double dequantization ([QP §2.3, §6.1]): W_bf16[d_out, d_in] (16B) gets the
 * restored weights of `q` as BF16 bit patterns, bit-exact with the formula
 * under qlora_nf4_t.  Needs no workspace.
 */
int qlora_dequant_bf16(const qlora_nf4_t *q, uint16_t *W_bf16, void *stream);

/*
 * LoRA merge into the base ([QP §12.3]; restored weight as in
 * qlora_dequant_bf16): the merged weight
 *     Wm[n][k] = RN_fp32( Wh[n][k] + s * sum_i B[n][i] A[i][k] ),
 * s = lora_alpha / r (FP32), with the right-hand side evaluated in FP64
 * (rank index ascending, every product and sum rounded on its own) and
 * rounded once to FP32.  When q_out is not NULL the merged weight is then
 * quantized into q_out exactly as qlora_quantize_nf4 would (the second
 * rounding that the merge into a 4-bit base implies).
 *   q        quantized base (input)
 *   A        BF16 [r, d_in]  (16B)    1 <= r <= 256
 *   B        BF16 [d_out, r]          any alignment
 *   W_merged FP32 [d_out, d_in] (16B) output
 *   q_out    NULL, or a quantized state of the same shape (output; may not
 *            alias q or W_merged)
 * workspace (16B) >= qlora_workspace_bytes(QLORA_OP_QUANTIZE, d_out, d_in,
 * 0, 0) when q_out is given (unused otherwise).  Deterministic.
 */
int qlora_merge_nf4(const qlora_nf4_t *q, const uint16_t *A, const uint16_t *B,
                    int64_t r, float lora_alpha, float *W_merged,
                    const qlora_nf4_t *q_out, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * Forward of the LoRA linear layer on the frozen NF4 base
 * ([QP §1.2, §2.2, §2.3, §6.3]; column-vector form y = W x + (alpha/r) B A x,
 * written here for token rows):
 *     Y = X Wh^T + s (X A^T) B^T,      s = lora_alpha / r (FP32),
 * where Wh is the restored BF16 weight.  Products take BF16 inputs and
 * accumulate in FP32; Y is rounded once to BF16.  The rank-r intermediate
 * T = s X A^T is formed in FP32 and enters the second product as the sum of
 * two BF16 terms (hi + lo), so it carries about 16 significant bits.  T is
 * deliberately not a BF16 tensor: one BF16 rounding of T (and of U in the
 * backward) would spend most of the 2e-3 relative error allowed for dA and
 * dB, so it is saved and handed to the backward as FP32.
 *   X       BF16 [M, d_in]  (16B)        M >= 0 tokens (M = 0: no work)
 *   A       BF16 [r, d_in]  (16B)        1 <= r <= 256
 *   B       BF16 [d_out, r]              any alignment
 *   Y       BF16 [M, d_out] (16B)        output
 *   T_save  FP32 [M, r]     (16B) or NULL: receives T for the backward.
 * workspace (16B) >= qlora_workspace_bytes(QLORA_OP_FWD, d_out, d_in, M, r).
 * Sizes per call: d_out <= 2^21, d_in <= 2^21 and M <= 2^21 tokens (the
 * kernels' device byte offsets are 32-bit within a tile or split), else
 * QLORA_ERR_SHAPE; the same holds for the backward.
 * M <= 16 runs a weight-streaming kernel (HBM-bound); larger M runs the
 * fused dequant-GEMM on the matrix cores.  No full BF16 copy of W is made.
 */
int qlora_linear_fwd(const qlora_nf4_t *q, const uint16_t *X, int64_t M,
                     const uint16_t *A, const uint16_t *B, int64_t r,
                     float lora_alpha, uint16_t *Y, float *T_save,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward of the same layer for the upstream gradient dY ([QP §2.4, §6.4,
 * §6.5]; [CP, 推論與訓練的精度關係]): gradients reach X, A and B; the frozen
 * base takes part in dX but gets no gradient of its own.
 *     U  = s dY B                 (FP32, [M, r])
 *     dX = dY Wh + U A            (BF16 out, FP32 accumulation)
 *     dA = U^T X                  (FP32 [r, d_in])
 *     dB = s dY^T (X A^T) = dY^T T (FP32 [d_out, r])
 * U and T enter the products as hi + lo BF16 pairs as in the forward.
 *   X, A, B, r, lora_alpha as in qlora_linear_fwd; dY BF16 [M, d_out] (16B).
 *   T_saved FP32 [M, r] (16B) from qlora_linear_fwd, or NULL to recompute.
 *   dX      BF16 [M, d_in] (16B) or NULL to skip the input gradient.
 *   dA      FP32 [r, d_in] (16B), dB FP32 [d_out, r] (16B): overwritten
 *           (M = 0 writes zeros).
 * workspace (16B) >= qlora_workspace_bytes(QLORA_OP_BWD, d_out, d_in, M, r).
 * dA and dB are reduced over tokens in a fixed order: results are
 * deterministic.
 */
int qlora_linear_bwd(const qlora_nf4_t *q, const uint16_t *X,
                     const uint16_t *dY, int64_t M, const uint16_t *A,
                     const uint16_t *B, int64_t r, float lora_alpha,
                     const float *T_saved, uint16_t *dX, float *dA, float *dB,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * qlora_linear_fwd without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  The workspace comes from a fixed device
 * array inside the library, QLORA_STATIC_SCRATCH_BYTES bytes on each GPU the
 * library runs on, held until the process ends; the call itself allocates
 * nothing.  Same arguments, checks, kernels and results (bit for bit) as
 * qlora_linear_fwd.  A call whose workspace (qlora_workspace_bytes(
 * QLORA_OP_FWD, ...)) exceeds the array returns QLORA_ERR_SCRATCH and
 * enqueues nothing; every projection shape of the LLaMA-7B and -65B layers
 * fits at r <= 64 for any M up to 40000 tokens.  Every call on one GPU
 * shares that GPU's array:
 * calls that may overlap on one GPU (other streams, unordered host threads)
 * race and must not be issued.  Nothing in the array needs to start at zero.
 */
#define QLORA_STATIC_SCRATCH_BYTES (32u << 20)
int qlora_linear_fwd_noalloc(const qlora_nf4_t *q, const uint16_t *X, int64_t M,
                             const uint16_t *A, const uint16_t *B, int64_t r,
                             float lora_alpha, uint16_t *Y, float *T_save,
                             void *stream);

/*
 * Forward of up to QLORA_MAX_GROUP layers that share the token count M, in
 * one pass: the same operation as qlora_linear_fwd for every item (each with
 * its own weight, LoRA factors, outputs and workspace sized by
 * qlora_workspace_bytes(QLORA_OP_FWD, ...)).  For M <= 16 all items run in
 * one weight-streaming launch (which also forms every T) and one finish
 * launch, so the projections of a decoder layer stream their packed weights
 * back to back; the K split of each weight is chosen over the whole group,
 * so an item's Y may differ from a single call's by FP32 summation order
 * (T does not).  For larger M the items run one after another.  Items must
 * not share outputs or workspace.
 * Returns the first failing item's status (nothing enqueued on argument
 * errors).
 */
#define QLORA_MAX_GROUP 8
typedef struct {
  qlora_nf4_t w;
  const uint16_t *X;
  const uint16_t *A;
  const uint16_t *B;
  int64_t r;
  float lora_alpha;
  uint16_t *Y;
  float *T_save;
  void *workspace;
  size_t workspace_bytes;
} qlora_fwd_item;

int qlora_linear_fwd_many(int count, const qlora_fwd_item *items, int64_t M,
                          void *stream);

/*
 * Quantize (dequantize) up to QLORA_MAX_GROUP tensors in one call: the same
 * operation as qlora_quantize_nf4 (qlora_dequant_bf16) for every item, with
 * the same results bit for bit, in two launches (one) for the whole list
 * when no tensor has more than 2^20 first-level blocks, so the projections
 * of a layer pay the launch and call overhead once.  Each item has its own
 * input, output and (quantize) workspace sized by
 * qlora_workspace_bytes(QLORA_OP_QUANTIZE, ...); items must not share any
 * of them.  Returns the first failing item's status (nothing enqueued on
 * argument errors) or QLORA_ERR_SHAPE when count is not in
 * 1 .. QLORA_MAX_GROUP.
 */
typedef struct {
  const float *W;           /* FP32 [q.d_out, q.d_in] (16B) */
  qlora_nf4_t q;            /* output state */
  void *workspace;          /* (16B) */
  size_t workspace_bytes;
} qlora_quant_item;

int qlora_quantize_nf4_many(int count, const qlora_quant_item *items, void *stream);

typedef struct {
  qlora_nf4_t q;            /* input state */
  uint16_t *W_bf16;         /* BF16 [q.d_out, q.d_in] (16B) output */
} qlora_dequant_item;

int qlora_dequant_bf16_many(int count, const qlora_dequant_item *items, void *stream);

/*
 * General block sizes ([QP §5.5]: the first-level block size B1 trades
 * scale metadata, about 8 / B1 bits per weight after double quantization,
 * against error; the second-level group size B2 makes the same trade for
 * the scales).  The same quantization as qlora_quantize_nf4 over a flat
 * array of n >= 1 values with
 *   block  B1: a power of two, 32 <= B1 <= 4096 (the layer format uses 64),
 *   group  B2: a power of two, 16 <= B2 <= 1024 (the layer format uses 256),
 * and no divisibility requirement: a short last block takes the absmax of
 * the elements it has, a short last group likewise.  With n1 = ceil(n/B1)
 * and G = ceil(n1/B2):
 *   codes        uint8[ceil(n/2)] (16B); for odd n the high nibble of the
 *                last byte is 0.
 *   scale_codes  uint8[n1];  scale2 float[G];  scale_mean float[1].
 * With B1 = 64, B2 = 256 and n % 64 == 0 the bytes equal those of
 * qlora_quantize_nf4 for the same values.  n <= 2^40.
 */
typedef struct {
  int64_t n;
  int64_t block;
  int64_t group;
  uint8_t *codes;
  uint8_t *scale_codes;
  float *scale2;
  float *scale_mean;
} qlora_nf4_blocked_t;

/* Buffer sizes of the blocked format (host only); QLORA_ERR_SHAPE for an
 * unsupported n, block or group. */
int qlora_nf4_blocked_sizes(int64_t n, int64_t block, int64_t group,
                            size_t *codes_bytes, size_t *scale_codes_bytes,
                            size_t *scale2_bytes);

/* Workspace of qlora_quantize_nf4_blocked (host only); 0 when unsupported. */
size_t qlora_quantize_blocked_workspace_bytes(int64_t n, int64_t block,
                                              int64_t group);

/* Quantize W (FP32 [n], (16B)) into q.  workspace (16B) >=
 * qlora_quantize_blocked_workspace_bytes(n, block, group). */
int qlora_quantize_nf4_blocked(const float *W, const qlora_nf4_blocked_t *q,
                               void *workspace, size_t workspace_bytes,
                               void *stream);

/* Double dequantization of q to BF16 [n] (16B). */
int qlora_dequant_bf16_blocked(const qlora_nf4_blocked_t *q, uint16_t *W_bf16,
                               void *stream);

/*
 * LoRA dropout in training mode ([QP §6.3]: the LoRA branch takes D(x)
 * instead of x, the base branch x; inference has no dropout):
 *     D(X) = keep * X / (1 - p),
 * keep drawn per element of X [M, d_in] from a counter-based generator, so
 * the backward regenerates the forward's mask from the same parameters:
 * element (m, k) takes output word m % 4 of Philox4x32-10 (Salmon, Moraes,
 * Dror, Shaw, SC'11) at counter (k, floor(m / 4), offset_lo, offset_hi)
 * under key (seed_lo, seed_hi), and is kept when that word is at least
 * floor(p * 2^32).  Use a new offset (or seed) for every layer and step.
 */
typedef struct {
  float p;          /* drop probability, 0 <= p < 1 (else QLORA_ERR_SHAPE) */
  uint64_t seed;    /* generator key                                       */
  uint64_t offset;  /* counter words 2 and 3                               */
  /* Optional saved mask of a layer call with M > 16 tokens (ignored for
   * M <= 16 and by qlora_dropout_mask), device memory (16B):
   *   keep_rows  [M, d_in / 32] words: bit (k % 32) of word [m][k / 32]
   *   keep_cols  [d_in, ceil(M / 32)] words: bit (m % 32) of word [k][m / 32]
   * (bits of rows m >= M are 0).  When both are non-NULL,
   * qlora_linear_fwd_dropout writes them, and qlora_linear_bwd_dropout reads
   * them instead of regenerating the mask, so the generator runs once per
   * training step; they must then hold the mask of the same M, d_in, p,
   * seed and offset.  NULL: nothing written, the backward regenerates. */
  uint32_t *keep_rows;
  uint32_t *keep_cols;
} qlora_dropout_t;

/*
 * The mask alone: X_kept = X with the dropped elements set to +0 (kept ones
 * unchanged; the 1 / (1 - p) is not applied) and, if keep_bits is not NULL,
 * keep_bits[k * ceil(M/32) + m/32] bit (m % 32) = keep of element (m, k)
 * (bits of rows m >= M are 0).
 *   X, X_kept  BF16 [M, d] (16B), d % 8 == 0, d <= 2^21, M <= 2^21;
 *   X_kept or keep_bits may be NULL (not both; X may be NULL without X_kept).
 */
int qlora_dropout_mask(const uint16_t *X, int64_t M, int64_t d,
                       const qlora_dropout_t *drop, uint16_t *X_kept,
                       uint32_t *keep_bits, void *stream);

/*
 * qlora_linear_fwd with LoRA dropout:
 *     Y = X Wh^T + s (D(X) A^T) B^T,   T = s D(X) A^T (saved in T_save).
 * The kernels form keep * X (exact) and fold 1 / (1 - p) into the scale:
 * s' = FP32(FP32(lora_alpha / r) / FP32(1 - p)).  With p = 0 the results
 * equal qlora_linear_fwd's bit for bit.  Same arguments and limits as
 * qlora_linear_fwd, plus `drop` (host pointer, not NULL); workspace (16B) >=
 * qlora_workspace_bytes(QLORA_OP_FWD_DROPOUT, d_out, d_in, M, r).
 */
int qlora_linear_fwd_dropout(const qlora_nf4_t *q, const uint16_t *X,
                             int64_t M, const uint16_t *A, const uint16_t *B,
                             int64_t r, float lora_alpha,
                             const qlora_dropout_t *drop, uint16_t *Y,
                             float *T_save, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * Backward of qlora_linear_fwd_dropout for the same X and `drop` (the mask
 * is regenerated, or read from drop->keep_rows / keep_cols when both are
 * given and M > 16):
 *     U  = s dY B
 *     dX = dY Wh + keep * (U A) / (1 - p)
 *     dA = U^T D(X),   dB = dY^T T   with T = s D(X) A^T.
 * Arguments and limits as qlora_linear_bwd, plus `drop`; T_saved (if given)
 * must come from qlora_linear_fwd_dropout with the same `drop`; workspace
 * (16B) >= qlora_workspace_bytes(QLORA_OP_BWD_DROPOUT, d_out, d_in, M, r).
 * With p = 0 the results equal qlora_linear_bwd's bit for bit.
 */
int qlora_linear_bwd_dropout(const qlora_nf4_t *q, const uint16_t *X,
                             const uint16_t *dY, int64_t M, const uint16_t *A,
                             const uint16_t *B, int64_t r, float lora_alpha,
                             const qlora_dropout_t *drop, const float *T_saved,
                             uint16_t *dX, float *dA, float *dB,
                             void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * Optimizer step on the LoRA factors ([QP §7.3]: AdamW with one first and
 * one second moment per trainable parameter, 32-bit; [QP §10.2]: optional
 * clipping by the global gradient norm).  Only A and B train.
 *
 * Tensors are processed in batches of up to 32 per kernel launch, so a step
 * over many small adapter tensors costs a few launches.  One tensor of the
 * step (all arrays device memory, any 4-byte alignment; 16-byte aligned
 * arrays, 8-byte for the BF16 copy, take wider accesses, same results):
 */
typedef struct {
  float *param;          /* FP32 master values [n], updated in place        */
  uint16_t *param_bf16;  /* BF16 copy [n] written after the step (RNE), or  */
                         /* NULL                                            */
  const float *grad;     /* FP32 gradient [n]                               */
  float *m;              /* first moment [n], updated in place              */
  float *v;              /* second moment [n], updated in place             */
  int64_t n;             /* element count, 0 <= n <= 2^32                   */
} qlora_adamw_param;

/*
 * acc[0] += sum over the listed tensors (in list order, FP64) of the sum of
 * their squared gradients, each taken in groups of 256 by the stride-halving
 * tree (pairs (j, j+128), (j, j+64), ..., (j, j+1)) and then by the same tree
 * over the group sums padded with zeros to a power of two.  acc is one FP64
 * device value the caller zeroes before the first call of a step; several
 * calls accumulate in call order.  workspace (16B-aligned device memory)
 * >= qlora_sumsq_workspace_bytes(count, params) for the same list (about
 * 8 bytes per 128 elements plus 8 per tensor; 0 for an invalid list).
 * QLORA_ERR_SHAPE for count < 0 or n outside [0, 2^32]; QLORA_ERR_NULL for
 * a missing acc, workspace or gradient (n > 0); QLORA_ERR_ALIGN,
 * QLORA_ERR_WORKSPACE.
 */
int qlora_grad_sumsq(int count, const qlora_adamw_param *params, double *acc,
                     void *workspace, size_t workspace_bytes, void *stream);
size_t qlora_sumsq_workspace_bytes(int count, const qlora_adamw_param *params);

/*
 * AdamW with decoupled weight decay, step number `step` >= 1 (bias
 * corrections bc_i = 1 - beta_i^step, evaluated in FP64 on the host and
 * rounded to FP32).  With grad_sumsq (device FP64 from qlora_grad_sumsq) the
 * gradients are first scaled by c = min(1, max_grad_norm / (norm + 1e-6)),
 * norm = FP32(sqrt(sumsq)); with NULL, c = 1.  Per element, FP32, each
 * operation rounded on its own in this order:
 *   g = g * c;   p = p - (lr * wd) * p;
 *   m = b1 * m + (1 - b1) * g;   v = b2 * v + (1 - b2) * (g * g);
 *   p = p - lr * ((m / bc1) / (sqrt(v / bc2) + eps));   p_bf16 = RNE_bf16(p).
 * The square root is correctly rounded.  Tensors with n = 0 are skipped.
 * QLORA_ERR_SHAPE for step < 1, count < 0, n outside [0, 2^32] or beta
 * outside [0, 1); QLORA_ERR_NULL for a missing array (n > 0).
 */
int qlora_adamw_step(int count, const qlora_adamw_param *params, float lr,
                     float beta1, float beta2, float eps, float weight_decay,
                     int64_t step, const double *grad_sumsq,
                     float max_grad_norm, void *stream);

/*
 * The operators around the linear layers of a fine-tuning step: the norm in
 * front of the projections, and the losses on the head's logits.
 *
 * Element types of their arrays.  Arrays of these entry points need the
 * alignment of their element type only (rows of odd length start anywhere);
 * 16-byte aligned rows are fastest.  The norms' results do not depend on the
 * alignment.  Sums over a row of BF16 logits start at its first 4-byte
 * boundary, so that log-probabilities, losses and gradients may differ in
 * their rounding between rows at even and at odd elements.  Infinities and
 * NaN in their inputs are allowed and propagate as IEEE arithmetic has it
 * (a logit of -inf is a token that cannot be drawn).
 */
#define QLORA_BF16 0
#define QLORA_F32 1

/*
 * Norm over the last axis, with the residual addition in front of it:
 *     H = RN(X + R)                    (R given; else H = X)
 *     LAYER:  Y = (H - mean) * rstd * gamma + beta,  mean = sum(H) / d,
 *             rstd = 1 / sqrt(sum((H - mean)^2) / d + eps)
 *     RMS:    Y = H * rstd * gamma,    rstd = 1 / sqrt(sum(H^2) / d + eps)
 * Sums and statistics are FP32 (the variance from the centred values); H is
 * rounded to its type first and the norm is that of the rounded H, so the
 * backward, which reads H, sees the same values.  Y is rounded once.
 *   kind    QLORA_NORM_LAYER or QLORA_NORM_RMS
 *   X, R    [M, d] of `type`; R NULL for no residual.  0 <= M <= 2^21,
 *           1 <= d <= 2^21.
 *   gamma   [d] of `w_type`; beta [d] of `w_type` or NULL (RMS: NULL, else
 *           QLORA_ERR_SHAPE)
 *   eps     finite, >= 0
 *   H       [M, d] output, needed with R (may be X or R); NULL without (else
 *           QLORA_ERR_SHAPE)
 *   Y       [M, d] output (may be X when R is NULL)
 *   mean    FP32 [M] or NULL (not written for RMS); rstd FP32 [M] or NULL:
 *           saved for the backward
 */
#define QLORA_NORM_LAYER 0
#define QLORA_NORM_RMS 1
int qlora_norm_fwd(int kind, int type, const void *X, const void *R, int64_t M,
                   int64_t d, int w_type, const void *gamma, const void *beta,
                   float eps, void *H, void *Y, float *mean, float *rstd,
                   void *stream);

/*
 * Backward of qlora_norm_fwd: with n = (H - mean) * rstd and u = dY * gamma,
 *     dX = (u - sum(u) / d - n * sum(u * n) / d) * rstd + dH
 *     dgamma = sum over rows of dY * n,   dbeta = sum over rows of dY
 * (RMS: mean = 0 and no sum(u) term).  dH is the gradient that reaches H past
 * the norm (the residual stream); dX is the gradient of X and of R.
 *   dY, H   [M, d] of `type` (H: the forward's H, or its X without residual)
 *   dH      [M, d] of `type` or NULL
 *   mean    FP32 [M] (LAYER), rstd FP32 [M]: from the forward
 *   dX      [M, d] output of `type` (may be dY or dH)
 *   dgamma  FP32 [d] or NULL, dbeta FP32 [d] or NULL (RMS: NULL, else
 *           QLORA_ERR_SHAPE): overwritten (M = 0 writes zeros).  With both
 *           NULL (frozen norm) no workspace is used.
 * workspace (16B) >= qlora_norm_workspace_bytes(M, d) when dgamma or dbeta
 * is given.  Sums over rows are taken in a fixed order: deterministic.
 */
int qlora_norm_bwd(int kind, int type, const void *dY, const void *H,
                   const void *dH, int64_t M, int64_t d, int w_type,
                   const void *gamma, const float *mean, const float *rstd,
                   void *dX, float *dgamma, float *dbeta, void *workspace,
                   size_t workspace_bytes, void *stream);
/* Host only; 0 for sizes the call would reject. */
size_t qlora_norm_workspace_bytes(int64_t M, int64_t d);

/*
 * Logits of a batch of tokens and the tokens they are judged by.  Row i's
 * distribution is softmax(scale * logits[i]); a row whose target is
 * ignore_index does not count (its log-probability is 0, its gradient row is
 * 0, its logits are not read).  Any other target outside [0, vocab) gives a
 * NaN log-probability, and nothing is read for it; what that does to the
 * gradients is said at each entry point.
 *   logits  [rows, ld] of `type`, vocab <= ld <= 2^32 (columns vocab .. ld - 1
 *           are neither read nor written).  0 <= rows <= 2^21,
 *           1 <= vocab <= 2^24.
 *   scale   > 0, at most 2^126 (1 / temperature)
 */
typedef struct {
  const void *logits;
  const int64_t *targets;  /* [rows] */
  int64_t rows, vocab, ld;
  int64_t ignore_index;
  int type;                /* QLORA_BF16 or QLORA_F32 */
  float scale;
} qlora_logits_t;

/*
 * Log-probability of each row's target, and the log of the row's summed
 * exponentials:
 *     lse = log(sum_j exp(scale * l_j)),   logp = scale * l_target - lse.
 * Taken from the row's maximum on, sums in FP32.
 *   logp, lse  FP32 [rows] outputs, lse NULL when no backward follows; both
 *              0 in rows that do not count.
 */
int qlora_token_logp(const qlora_logits_t *l, float *logp, float *lse,
                     void *stream);

/*
 * Gradient of the logits for upstream gradients of the log-probabilities:
 *     dlogits[i][j] = scale * dlogp[i] * ((j == target_i) - p_ij),
 *     p_ij = exp(scale * l_ij - lse_i).
 * Rows that do not count and rows with dlogp = 0 are written as zeros without
 * being read.  p carries the rounding of the FP32 lse, 2^-18 at most: a row
 * whose lse is 128 or more in size (or no number) has its sum taken again.
 *   lse         FP32 [rows]: qlora_token_logp's, on the same logits and scale
 *   dlogp       FP32 [rows]; dlogits [rows, ldd] output of l->type,
 *               vocab <= ldd <= 2^32; may be the logits' own buffer (ldd = ld).
 * A row with a target outside the vocabulary gets NaN, with dlogp = 0 zeros.
 */
int qlora_token_logp_bwd(const qlora_logits_t *l, const float *lse,
                         const float *dlogp, void *dlogits, int64_t ldd,
                         void *stream);

/*
 * Preference loss over pairs of answers, from the logits to their gradient.
 * Sequence i is the rows offsets[i] .. offsets[i + 1] - 1; sequences 0 ..
 * pairs - 1 are the preferred answers and pairs .. 2 pairs - 1, in the same
 * order, the others.  With s_i = sum of logp over the sequence's rows that
 * count, and g_i = sum of (logp - ref_logp) over them (ref_logp NULL: g_i =
 * s_i), each divided by the number of such rows when length_normalize is set
 * (an empty sequence gives 0):
 *     h = g_p - g_(pairs + p),   z = beta * h - margin
 *     SIGMOID  loss_p = (1 - e) softplus(-z) + e softplus(z), e = label_smoothing
 *     HINGE    loss_p = max(0, 1 - z)
 *     SQUARED  loss_p = (h - 1 / (2 beta))^2
 * and dlogits is the gradient of weight * sum_p loss_p.  (On one frozen base,
 * ref_logp is qlora_token_logp on the logits of the same layers without
 * their adapter.)  Sums over a sequence are FP64.
 *   l          the logits of all sequences
 *   offsets    int64 [2 pairs + 1], nondecreasing, in [0, rows] (device
 *              memory: values outside are clamped to that range); rows that
 *              no sequence holds get zero gradients, also for a target outside
 *              the vocabulary; in a sequence such a target makes its pair's
 *              loss NaN, and the gradient of both answers' rows that count.
 *              0 <= pairs <= 2^20
 *   ref_logp   FP32 [rows] or NULL
 *   logp       FP32 [rows] output; seq_logp FP32 [2 pairs] output (s_i);
 *   loss       FP32 [pairs] output
 *   dlogits    [rows, ldd] output of l->type, as in qlora_token_logp_bwd, or
 *              NULL for the loss alone
 * QLORA_ERR_SHAPE for beta not finite and > 0, label_smoothing outside
 * [0, 1) or with another kind than SIGMOID, margin or weight not finite, a
 * margin with SQUARED.  workspace (16B) >=
 * qlora_preference_workspace_bytes(rows).  Deterministic.
 */
#define QLORA_PREF_SIGMOID 0
#define QLORA_PREF_HINGE 1
#define QLORA_PREF_SQUARED 2
typedef struct {
  int kind;
  int length_normalize;
  float beta, label_smoothing, margin, weight;
} qlora_preference_t;

int qlora_preference_loss(const qlora_logits_t *l, const int64_t *offsets,
                          int64_t pairs, const float *ref_logp,
                          const qlora_preference_t *par, float *logp,
                          float *seq_logp, float *loss, void *dlogits,
                          int64_t ldd, void *workspace, size_t workspace_bytes,
                          void *stream);
/* Host only; 0 for rows outside the documented range. */
size_t qlora_preference_workspace_bytes(int64_t rows);

/*
 * Clipped policy loss with a KL term, from the logits to their gradient.
 * For every row t that counts and lies in a sequence s (rows offsets[s] ..
 * offsets[s + 1] - 1), with a its advantage:
 *     ratio = exp(logp - old_logp)          (old_logp NULL: 1, on-policy)
 *     policy = max(-a ratio, -a clamp(ratio, 1 - clip_low, 1 + clip_high))
 *     kl     = exp(ref_logp - logp) - (ref_logp - logp) - 1  (ref NULL: 0)
 *     loss   = sum over t of w_t (policy_t + kl_coef kl_t)
 *     TOKEN_MEAN     w_t = 1 / (number of such rows)
 *     SEQUENCE_MEAN  w_t = 1 / (sequences * number of such rows of s)
 * dlogits is the gradient of weight * loss; where the clipped branch is the
 * larger one the policy term has no gradient, at equality the unclipped
 * branch's counts.  The gradient comes from the same pass over the logits
 * as the loss: rows of up to 131072 BF16 or 98304 FP32 logits are read once.
 *   offsets     int64 [sequences + 1] as in qlora_preference_loss, but that a
 *               target outside the vocabulary makes its own row's gradient NaN
 *               alone (and the loss where there is old_logp or a KL term).
 *               0 <= sequences <= 2^21
 *   advantages  FP32 [rows] with per_token, else FP32 [sequences]
 *   old_logp, ref_logp  FP32 [rows] or NULL (ref_logp NULL needs kl_coef 0,
 *               else QLORA_ERR_NULL)
 *   logp        FP32 [rows] output
 *   stats       FP32 [4] output: loss, sum w policy, sum w kl, sum w [the
 *               clipped branch is the larger one]
 *   dlogits     [rows, ldd] output of l->type, as in qlora_token_logp_bwd, or
 *               NULL for the loss alone
 * QLORA_ERR_SHAPE for clip_low outside [0, 1], clip_high or kl_coef not
 * finite or < 0, weight not finite.  workspace (16B) >=
 * qlora_policy_workspace_bytes(rows, sequences).  Deterministic.
 */
#define QLORA_POLICY_TOKEN_MEAN 0
#define QLORA_POLICY_SEQUENCE_MEAN 1
typedef struct {
  int reduction;
  int per_token;
  float clip_low, clip_high, kl_coef, weight;
} qlora_policy_t;

int qlora_policy_loss(const qlora_logits_t *l, const int64_t *offsets,
                      int64_t sequences, const float *advantages,
                      const float *old_logp, const float *ref_logp,
                      const qlora_policy_t *par, float *logp, float *stats,
                      void *dlogits, int64_t ldd, void *workspace,
                      size_t workspace_bytes, void *stream);
/* Host only; 0 for sizes outside the documented range. */
size_t qlora_policy_workspace_bytes(int64_t rows, int64_t sequences);

/*
 * Activations in 8 bits: what a training step keeps of a layer's input for the
 * backward, at 1 + 1/16 bytes a value.  Blocks of 64 values of a row (the last
 * one shorter where d % 64 != 0) share an FP32 scale:
 *     a = max |x| over the block,  scale = RN(a / 127)
 *     code = the integer nearest to 127 x / a, ties to even (exactly decided)
 *     restored x = RN(RN_fp32(code * scale)), rounded to its type
 * (the scale stops where 127 times it is FP32's largest value).  Blocks with
 * a < 2^-119 restore as zeros.  A block that holds an infinity or a
 * NaN restores as NaN in all its elements.  Deterministic.
 *   codes  int8 [M, round_up(d, 64)] (16B); columns d .. are written as 0
 *   scale  FP32 [ceil(d / 64), M]: block by block, so that the scales of
 *          neighbouring tokens lie together
 * 0 <= M <= 2^21, 1 <= d <= 2^21.  X [M, d] of `type` (QLORA_BF16, QLORA_F32)
 * needs the alignment of its element type only; 16-byte aligned rows are
 * fastest.
 */
typedef struct {
  int64_t M, d;
  uint8_t *codes;
  float *scale;
} qlora_packed_t;

/* Byte sizes of the two buffers (host only). */
int qlora_pack8_sizes(int64_t M, int64_t d, size_t *codes_bytes, size_t *scale_bytes);
int qlora_pack8(int type, const void *X, const qlora_packed_t *p, void *stream);
int qlora_unpack8(const qlora_packed_t *p, int type, void *X, void *stream);

/*
 * qlora_linear_bwd from an input kept in 8 bits: X is the BF16 matrix that
 * qlora_unpack8 restores from X8, which is never written out.  dA and dB take
 * U and T with 24 bits, where qlora_linear_bwd takes 16.
 *   X8       M tokens of d_in values; T_saved is required (the forward's T).
 *   drop     NULL, or the forward's LoRA dropout: as qlora_linear_bwd_dropout
 *            (saved mask or regenerated; T_saved from that forward).
 * Other arguments and limits as qlora_linear_bwd; workspace (16B) >=
 * qlora_workspace_bytes(QLORA_OP_BWD_PACKED, ...), with drop
 * QLORA_OP_BWD_PACKED_DROPOUT.
 */
int qlora_linear_bwd_packed(const qlora_nf4_t *q, const qlora_packed_t *X8,
                            const uint16_t *dY, int64_t M, const uint16_t *A,
                            const uint16_t *B, int64_t r, float lora_alpha,
                            const qlora_dropout_t *drop, const float *T_saved,
                            uint16_t *dX, float *dA, float *dB, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * Low-rank adapters of many requests beside one shared projection: a bank of
 * `slots` adapters of one rank (lower ranks padded with zeros), each token with
 * the adapter of its own request or with none.
 *   A      BF16 [slots, r, d_in]
 *   B      BF16 [slots, d_out, r]
 *   scale  FP32 [slots] device memory: lora_alpha / r of each
 * 1 <= slots <= 2048, 1 <= r <= 256, 1 <= d_in, d_out <= 2^21.  Arrays of these
 * entry points need the alignment of their element type only (the plan and the
 * workspace: 16 bytes); 16-byte aligned rows (widths and, in B, a rank that are
 * multiples of 8) are fastest.  Infinities and NaN of a token stay with that
 * token in Y, T and dX and reach its own slot's dA and dB; a slot's stay with
 * its tokens.  An infinity (and a T or U past BF16's range) can come out of the
 * second products as a NaN: T and U enter them as sums of BF16 terms.
 */
typedef struct {
  int64_t slots, r, d_in, d_out;
  const uint16_t *A;
  const uint16_t *B;
  const float *scale;
} qlora_adapters_t;

/*
 * The plan of a batch, made once for all of its projections and both
 * directions: its tokens sorted by slot.
 *   index  int32 [M] device memory: each token's slot; a value outside
 *          [0, slots) means no adapter.  0 <= M <= 2^21.
 *   plan   (16B) device memory of qlora_adapters_plan_bytes(M, slots) bytes
 *          (host only; 0 for sizes the call would reject), an output that the
 *          calls below read.  They write nothing where the plan they get was
 *          made for another M or number of slots.
 */
size_t qlora_adapters_plan_bytes(int64_t M, int64_t slots);
int qlora_adapters_plan(const int32_t *index, int64_t M, int64_t slots, void *plan,
                        size_t plan_bytes, void *stream);

/*
 * Forward: for token m with the adapter a,
 *     T[m] = scale_a X[m] A_a^T,    Y[m] = RN(Y0[m] + T[m] B_a^T),
 * without one T[m] = 0 and Y[m] = Y0[m].  Y0 is the shared projection's output
 * (a qlora_linear_fwd with lora_alpha = 0, or any other).  Products take BF16
 * inputs and accumulate in FP32; T enters the second as a hi + lo BF16 pair.
 *   X       BF16 [M, d_in] (rows of tokens without an adapter are not read)
 *   Y0      BF16 [M, d_out] or NULL (zeros)
 *   Y       BF16 [M, d_out] output, may be Y0
 *   T_save  FP32 [M, r] or NULL: for the backward
 * workspace (16B) >= qlora_adapters_workspace_bytes(0, bank, M).  Deterministic;
 * a token's results do not depend on the other tokens' values and places.  M
 * decides in how many ranges the sums over d_in are taken: in a batch of another
 * size the last bits can differ.
 */
int qlora_adapters_fwd(const qlora_adapters_t *bank, const void *plan, size_t plan_bytes,
                       const uint16_t *X, int64_t M, const uint16_t *Y0, uint16_t *Y,
                       float *T_save, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward of qlora_adapters_fwd for the upstream gradient dY:
 *     U[m] = scale_a dY[m] B_a,        dX[m] = RN(dX0[m] + U[m] A_a)
 *     dA_a = sum of U[m]^T X[m],       dB_a = sum of dY[m]^T T[m]
 * over the tokens m of slot a; dX[m] = dX0[m] for a token without an adapter,
 * zeros in dA and dB for a slot without tokens.  U enters dX as a hi + lo BF16
 * pair, U and T enter dA and dB with 24 bits.
 *   X, X8    the forward's X: BF16 [M, d_in], or kept in 8 bits (M tokens of
 *            d_in values, restored to BF16); exactly one, the other NULL
 *   T        FP32 [M, r]: the forward's T_save
 *   dY       BF16 [M, d_out]
 *   dX0      BF16 [M, d_in] or NULL (zeros): the shared projection's gradient
 *   dX       BF16 [M, d_in] output, may be dX0 (not X or dY); NULL to skip
 *   dA       FP32 [slots, r, d_in], dB FP32 [slots, d_out, r]: overwritten
 *            (M = 0 writes zeros)
 * workspace (16B) >= qlora_adapters_workspace_bytes(1, bank, M).  Sums over
 * tokens have a fixed order: deterministic (M decides the ranges of the sums over
 * d_out, as in the forward).
 */
int qlora_adapters_bwd(const qlora_adapters_t *bank, const void *plan, size_t plan_bytes,
                       const uint16_t *X, const qlora_packed_t *X8, const float *T,
                       const uint16_t *dY, int64_t M, const uint16_t *dX0, uint16_t *dX,
                       float *dA, float *dB, void *workspace, size_t workspace_bytes,
                       void *stream);
/* Host only; 0 for sizes the calls would reject. */
size_t qlora_adapters_workspace_bytes(int backward, const qlora_adapters_t *bank, int64_t M);

/* Static English text for a qlora_status value. */
const char *qlora_status_string(int status);

/* ABI version: (major << 16) | minor. */
int qlora_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_H */
