// api_train.cpp -- host side of the entry points around the linear layers:
// norms, token log-probabilities, the preference loss and the policy loss.
// Argument checks, workspace carving and launch order; the operations are
// stated in include/qlora.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_util.h"
#include "qlora.h"
#include "qlora_kernels.h"

using namespace qlora;

namespace {

constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxSequences = int64_t(1) << 21;
constexpr float kMaxScale = 0x1p126f;   // scale * log2(e) stays finite

bool type_ok(int t) { return t == QLORA_BF16 || t == QLORA_F32; }

// Aligned to an element of `type`.
bool elem_aligned(const void* p, int type) {
  return (reinterpret_cast<uintptr_t>(p) & (type == QLORA_F32 ? 3u : 1u)) == 0;
}
template <class T>
bool aligned_as(const T* p) {
  return (reinterpret_cast<uintptr_t>(p) & (sizeof(T) - 1)) == 0;
}

// Shape, type and scale of a logits batch; its pointers are checked apart
// (an empty batch needs none).
int check_logits_shape(const qlora_logits_t* l) {
  if (!l) return QLORA_ERR_NULL;
  if (l->rows < 0 || l->rows > kMaxTokens || l->vocab < 1 || l->vocab > kMaxVocab ||
      l->ld < l->vocab || l->ld > (int64_t(1) << 32) || !type_ok(l->type))
    return QLORA_ERR_SHAPE;
  if (!(l->scale > 0.0f && l->scale <= kMaxScale)) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

int check_logits_arrays(const qlora_logits_t* l) {
  if (!l->logits || !l->targets) return QLORA_ERR_NULL;
  if (!elem_aligned(l->logits, l->type) || !aligned_as(l->targets)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

// The gradient's buffer: its own, or the logits' with the same rows.
int check_dlogits(const qlora_logits_t* l, const void* dlogits, int64_t ldd) {
  if (ldd < l->vocab || ldd > (int64_t(1) << 32)) return QLORA_ERR_SHAPE;
  if (dlogits == l->logits && ldd != l->ld) return QLORA_ERR_SHAPE;
  if (!elem_aligned(dlogits, l->type)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

LogitsArgs logits_args(const qlora_logits_t* l) {
  return LogitsArgs{l->logits, l->targets,      l->rows, l->vocab,
                    l->ld,     l->ignore_index, l->type, l->scale};
}

struct PreferencePlan {
  RowStat* stat;
  float* dlogp;
  size_t bytes;
};
PreferencePlan plan_preference(int64_t rows, void* ws) {
  PreferencePlan p{};
  Carver c(ws);
  p.stat = c.take<RowStat>(rows);
  p.dlogp = c.take<float>(rows);
  p.bytes = c.off + 256;
  return p;
}

struct PolicyPlan {
  int32_t* count;
  int32_t* total;
  int32_t* row_seq;
  float4* terms;
  size_t bytes;
};
PolicyPlan plan_policy(int64_t rows, int64_t seqs, void* ws) {
  PolicyPlan p{};
  Carver c(ws);
  p.count = c.take<int32_t>(seqs);
  p.total = c.take<int32_t>(1);
  p.row_seq = c.take<int32_t>(rows);
  p.terms = c.take<float4>(rows);
  p.bytes = c.off + 256;
  return p;
}

}  // namespace

extern "C" {

int qlora_norm_fwd(int kind, int type, const void* X, const void* R, int64_t M, int64_t d,
                   int w_type, const void* gamma, const void* beta, float eps, void* H, void* Y,
                   float* mean, float* rstd, void* stream) {
  if ((kind != QLORA_NORM_LAYER && kind != QLORA_NORM_RMS) || !type_ok(type) || !type_ok(w_type))
    return QLORA_ERR_SHAPE;
  if (M < 0 || M > kMaxTokens || d < 1 || d > kMaxLinearDim) return QLORA_ERR_SHAPE;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return QLORA_ERR_SHAPE;
  if (kind == QLORA_NORM_RMS && beta) return QLORA_ERR_SHAPE;
  if (H && !R) return QLORA_ERR_SHAPE;   // it would stay unwritten
  if (M == 0) return QLORA_OK;
  if (!X || !gamma || !Y || (R && !H)) return QLORA_ERR_NULL;
  if (!elem_aligned(X, type) || !elem_aligned(R, type) || !elem_aligned(H, type) ||
      !elem_aligned(Y, type) || !elem_aligned(gamma, w_type) || !elem_aligned(beta, w_type) ||
      !aligned_as(mean) || !aligned_as(rstd))
    return QLORA_ERR_ALIGN;
  const NormFwdArgs a{X, R, gamma, beta, H, Y, mean, rstd, M, d, eps, kind, type, w_type};
  return hip_status(launch_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t qlora_norm_workspace_bytes(int64_t M, int64_t d) {
  if (M < 0 || M > kMaxTokens || d < 1 || d > kMaxLinearDim) return 0;
  Carver c(nullptr);
  c.take<float>(M > 0 ? 2 * d * norm_parts(M, d) : 0);
  return c.off + 256;
}

int qlora_norm_bwd(int kind, int type, const void* dY, const void* H, const void* dH, int64_t M,
                   int64_t d, int w_type, const void* gamma, const float* mean, const float* rstd,
                   void* dX, float* dgamma, float* dbeta, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if ((kind != QLORA_NORM_LAYER && kind != QLORA_NORM_RMS) || !type_ok(type) || !type_ok(w_type))
    return QLORA_ERR_SHAPE;
  if (M < 0 || M > kMaxTokens || d < 1 || d > kMaxLinearDim) return QLORA_ERR_SHAPE;
  if (kind == QLORA_NORM_RMS && dbeta) return QLORA_ERR_SHAPE;
  const bool weights = dgamma || dbeta;
  if (M == 0 && !weights) return QLORA_OK;
  if (M > 0 && (!dY || !H || !gamma || !rstd || !dX || (kind == QLORA_NORM_LAYER && !mean)))
    return QLORA_ERR_NULL;
  if (weights && !workspace) return QLORA_ERR_NULL;
  if (!elem_aligned(dY, type) || !elem_aligned(H, type) || !elem_aligned(dH, type) ||
      !elem_aligned(dX, type) || !elem_aligned(gamma, w_type) || !aligned_as(mean) ||
      !aligned_as(rstd) || !aligned_as(dgamma) || !aligned_as(dbeta) ||
      (weights && !aligned16(workspace)))
    return QLORA_ERR_ALIGN;
  if (weights && workspace_bytes < qlora_norm_workspace_bytes(M, d)) return QLORA_ERR_WORKSPACE;
  Carver c(weights ? workspace : nullptr);
  float* part = c.take<float>(1);
  const NormBwdArgs a{dY, H,      dH,    gamma, kind == QLORA_NORM_LAYER ? mean : nullptr, rstd,
                      dX, dgamma, dbeta, part,  M,                                         d,
                      kind, type, w_type};
  return hip_status(launch_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

int qlora_token_logp(const qlora_logits_t* l, float* logp, float* lse, void* stream) {
  int s = check_logits_shape(l);
  if (s) return s;
  if (l->rows == 0) return QLORA_OK;
  s = check_logits_arrays(l);
  if (s) return s;
  if (!logp) return QLORA_ERR_NULL;
  if (!aligned_as(logp) || !aligned_as(lse)) return QLORA_ERR_ALIGN;
  return hip_status(launch_logp(logits_args(l), logp, lse, nullptr,
                                static_cast<hipStream_t>(stream)));
}

int qlora_token_logp_bwd(const qlora_logits_t* l, const float* lse, const float* dlogp,
                         void* dlogits, int64_t ldd, void* stream) {
  int s = check_logits_shape(l);
  if (s) return s;
  if (l->rows == 0) return QLORA_OK;
  s = check_logits_arrays(l);
  if (s) return s;
  if (!lse || !dlogp || !dlogits) return QLORA_ERR_NULL;
  if (!aligned_as(lse) || !aligned_as(dlogp)) return QLORA_ERR_ALIGN;
  s = check_dlogits(l, dlogits, ldd);
  if (s) return s;
  return hip_status(launch_dlogits(logits_args(l), nullptr, lse, dlogp, dlogits, ldd,
                                   static_cast<hipStream_t>(stream)));
}

size_t qlora_preference_workspace_bytes(int64_t rows) {
  if (rows < 0 || rows > kMaxTokens) return 0;
  return plan_preference(rows, nullptr).bytes;
}

int qlora_preference_loss(const qlora_logits_t* l, const int64_t* offsets, int64_t pairs,
                          const float* ref_logp, const qlora_preference_t* par, float* logp,
                          float* seq_logp, float* loss, void* dlogits, int64_t ldd,
                          void* workspace, size_t workspace_bytes, void* stream) {
  int s = check_logits_shape(l);
  if (s) return s;
  if (!par) return QLORA_ERR_NULL;
  const bool sigmoid = par->kind == QLORA_PREF_SIGMOID, squared = par->kind == QLORA_PREF_SQUARED;
  if (!sigmoid && !squared && par->kind != QLORA_PREF_HINGE) return QLORA_ERR_SHAPE;
  if (pairs < 0 || pairs > kMaxSequences / 2) return QLORA_ERR_SHAPE;
  if (!(par->beta > 0.0f) || !std::isfinite(par->beta) || !std::isfinite(par->margin) ||
      !std::isfinite(par->weight) || (squared && par->margin != 0.0f))
    return QLORA_ERR_SHAPE;
  if (!(par->label_smoothing >= 0.0f && par->label_smoothing < 1.0f) ||
      (!sigmoid && par->label_smoothing != 0.0f))
    return QLORA_ERR_SHAPE;
  if (l->rows == 0 && pairs == 0) return QLORA_OK;
  if (l->rows > 0) {
    s = check_logits_arrays(l);
    if (s) return s;
    if (!logp || !workspace) return QLORA_ERR_NULL;
    if (dlogits) {
      s = check_dlogits(l, dlogits, ldd);
      if (s) return s;
    }
  }
  if (pairs > 0 && (!offsets || !seq_logp || !loss)) return QLORA_ERR_NULL;
  if (!aligned_as(offsets) || !aligned_as(ref_logp) || !aligned_as(logp) ||
      !aligned_as(seq_logp) || !aligned_as(loss) || !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  const PreferencePlan p = plan_preference(l->rows, workspace);
  if (l->rows > 0 && workspace_bytes < p.bytes) return QLORA_ERR_WORKSPACE;
  const bool grad = dlogits && l->rows > 0;
  const PreferenceArgs a{l->targets, offsets,   logp,  ref_logp,  l->rows,
                         pairs,      l->ignore_index,  par->kind, par->length_normalize,
                         par->beta,  par->label_smoothing, par->margin, par->weight,
                         seq_logp,   loss,      grad ? p.dlogp : nullptr};
  return hip_status(launch_preference(logits_args(l), a, p.stat, logp, grad ? dlogits : nullptr,
                                      ldd, static_cast<hipStream_t>(stream)));
}

size_t qlora_policy_workspace_bytes(int64_t rows, int64_t sequences) {
  if (rows < 0 || rows > kMaxTokens || sequences < 0 || sequences > kMaxSequences) return 0;
  return plan_policy(rows, sequences, nullptr).bytes;
}

int qlora_policy_loss(const qlora_logits_t* l, const int64_t* offsets, int64_t sequences,
                      const float* advantages, const float* old_logp, const float* ref_logp,
                      const qlora_policy_t* par, float* logp, float* stats, void* dlogits,
                      int64_t ldd, void* workspace, size_t workspace_bytes, void* stream) {
  int s = check_logits_shape(l);
  if (s) return s;
  if (!par) return QLORA_ERR_NULL;
  if (par->reduction != QLORA_POLICY_TOKEN_MEAN && par->reduction != QLORA_POLICY_SEQUENCE_MEAN)
    return QLORA_ERR_SHAPE;
  if (sequences < 0 || sequences > kMaxSequences) return QLORA_ERR_SHAPE;
  if (!(par->clip_low >= 0.0f && par->clip_low <= 1.0f) || !(par->clip_high >= 0.0f) ||
      !std::isfinite(par->clip_high) || !(par->kl_coef >= 0.0f) || !std::isfinite(par->kl_coef) ||
      !std::isfinite(par->weight))
    return QLORA_ERR_SHAPE;
  if (!stats || (!ref_logp && par->kl_coef > 0.0f)) return QLORA_ERR_NULL;
  if (l->rows > 0) {
    s = check_logits_arrays(l);
    if (s) return s;
    if (!logp || !workspace || (sequences > 0 && (!offsets || !advantages)))
      return QLORA_ERR_NULL;
    if (dlogits) {
      s = check_dlogits(l, dlogits, ldd);
      if (s) return s;
    }
  }
  if (!aligned_as(offsets) || !aligned_as(advantages) || !aligned_as(old_logp) ||
      !aligned_as(ref_logp) || !aligned_as(logp) || !aligned_as(stats) || !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  const PolicyPlan p = plan_policy(l->rows, sequences, workspace);
  if (l->rows > 0 && workspace_bytes < p.bytes) return QLORA_ERR_WORKSPACE;
  const PolicyArgs a{offsets,        advantages,     old_logp,       ref_logp,
                     sequences,      par->reduction, par->per_token, par->clip_low,
                     par->clip_high, par->kl_coef,   par->weight,    logp,
                     stats,          p.count,        p.total,        p.row_seq,
                     p.terms};
  return hip_status(launch_policy(logits_args(l), a, dlogits, ldd,
                                  static_cast<hipStream_t>(stream)));
}

}  // extern "C"
