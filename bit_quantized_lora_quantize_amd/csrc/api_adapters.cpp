// api_adapters.cpp -- host side of the 8-bit activation checkpoints and of the
// adapters of many requests.  Argument checks, workspace carving and launch
// order; the operations are stated in include/qlora.h.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_util.h"
#include "qlora.h"
#include "qlora_kernels.h"

using namespace qlora;

namespace {

constexpr int64_t kMaxRank = 256;

bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Plan {
  PlanView v;
  size_t bytes;
};
Plan plan_view(int64_t M, int64_t slots, const void* base) {
  Plan p{};
  Carver c(const_cast<void*>(base));
  p.v.head = c.take<int32_t>(kPlanHead);
  p.v.order = c.take<int32_t>(M);
  p.v.begin = c.take<int32_t>(slots + 1);
  p.v.tile = c.take<int4>(plan_most_tiles(M, slots));
  p.v.split = c.take<int4>(plan_most_splits(M, slots));
  p.v.split_first = c.take<int32_t>(plan_most_splits(M, slots));
  p.v.parts = c.take<int2>(slots);
  p.v.hist = c.take<int32_t>(M > 1024 ? cdiv(M, 1024) * (slots + 1) : 0);
  p.bytes = c.off + 256;
  return p;
}
bool plan_ok(int64_t M, int64_t slots) {
  return M >= 0 && M <= kMaxTokens && slots >= 1 && slots <= kPlanMaxSlots;
}

bool bank_ok(const qlora_adapters_t* b) {
  return b->slots >= 1 && b->slots <= kPlanMaxSlots && b->r >= 1 && b->r <= kMaxRank &&
         b->d_in >= 1 && b->d_in <= kMaxLinearDim && b->d_out >= 1 && b->d_out <= kMaxLinearDim;
}

struct AdaptersPlan {
  float* part;        // [splits][M][r]
  uint16_t* vrows;    // [M][2 vrow_ranks(r)]
  uint16_t* t_frags;  // backward
  uint16_t* u_frags;
  float* da_part;     // [parts][r][d_in]
  float* db_part;     // [parts][d_out][r]
  size_t bytes;
};
AdaptersPlan plan_adapters(bool backward, const qlora_adapters_t* b, int64_t M, void* ws) {
  AdaptersPlan p{};
  Carver c(ws);
  int64_t kper;
  p.part = c.take<float>(shrink_splits(M, backward ? b->d_out : b->d_in, &kper) * M * b->r);
  p.vrows = c.take<uint16_t>(M * 2 * vrow_ranks(b->r));
  if (backward) {
    const int64_t tiles = plan_most_tiles(M, b->slots);
    p.t_frags = c.take<uint16_t>(frag_elems(tiles, b->r));
    p.u_frags = c.take<uint16_t>(frag_elems(tiles, b->r));
    p.da_part = c.take<float>(plan_most_parts(M) * b->r * b->d_in);
    p.db_part = c.take<float>(plan_most_parts(M) * b->r * b->d_out);
  }
  p.bytes = c.off + 256;
  return p;
}

// What both directions refuse, pointers of an empty batch aside.
int check_bank(const qlora_adapters_t* b, int64_t M) {
  if (!b) return QLORA_ERR_NULL;
  if (!bank_ok(b) || M < 0 || M > kMaxTokens) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}
int check_bank_arrays(const qlora_adapters_t* b, const void* plan, size_t plan_bytes, int64_t M) {
  if (!b->A || !b->B || !b->scale || !plan) return QLORA_ERR_NULL;
  if (!aligned2(b->A) || !aligned2(b->B) || !aligned4(b->scale) || !aligned16(plan))
    return QLORA_ERR_ALIGN;
  if (plan_bytes < plan_view(M, b->slots, nullptr).bytes) return QLORA_ERR_WORKSPACE;
  return QLORA_OK;
}

}  // namespace

extern "C" {

int qlora_pack8_sizes(int64_t M, int64_t d, size_t* codes_bytes, size_t* scale_bytes) {
  if (!codes_bytes || !scale_bytes) return QLORA_ERR_NULL;
  if (M < 0 || M > kMaxTokens || d < 1 || d > kMaxLinearDim) return QLORA_ERR_SHAPE;
  *codes_bytes = size_t(M * round_up(d, 64));
  *scale_bytes = size_t(M * cdiv(d, 64)) * sizeof(float);
  return QLORA_OK;
}

int qlora_pack8(int type, const void* X, const qlora_packed_t* p, void* stream) {
  if (!p) return QLORA_ERR_NULL;
  if ((type != QLORA_BF16 && type != QLORA_F32) || p->M < 0 || p->M > kMaxTokens || p->d < 1 ||
      p->d > kMaxLinearDim)
    return QLORA_ERR_SHAPE;
  if (p->M == 0) return QLORA_OK;
  if (!X || !p->codes || !p->scale) return QLORA_ERR_NULL;
  if (!(type == QLORA_F32 ? aligned4(X) : aligned2(X)) || !aligned16(p->codes) ||
      !aligned4(p->scale))
    return QLORA_ERR_ALIGN;
  return hip_status(launch_pack8(type, X, p->M, p->d, p->codes, p->scale,
                                 static_cast<hipStream_t>(stream)));
}

int qlora_unpack8(const qlora_packed_t* p, int type, void* X, void* stream) {
  if (!p) return QLORA_ERR_NULL;
  if ((type != QLORA_BF16 && type != QLORA_F32) || p->M < 0 || p->M > kMaxTokens || p->d < 1 ||
      p->d > kMaxLinearDim)
    return QLORA_ERR_SHAPE;
  if (p->M == 0) return QLORA_OK;
  if (!X || !p->codes || !p->scale) return QLORA_ERR_NULL;
  if (!(type == QLORA_F32 ? aligned4(X) : aligned2(X)) || !aligned16(p->codes) ||
      !aligned4(p->scale))
    return QLORA_ERR_ALIGN;
  return hip_status(launch_unpack8(p->codes, p->scale, p->M, p->d, type, X,
                                   static_cast<hipStream_t>(stream)));
}

size_t qlora_adapters_plan_bytes(int64_t M, int64_t slots) {
  return plan_ok(M, slots) ? plan_view(M, slots, nullptr).bytes : 0;
}

int qlora_adapters_plan(const int32_t* index, int64_t M, int64_t slots, void* plan,
                        size_t plan_bytes, void* stream) {
  if (!plan_ok(M, slots)) return QLORA_ERR_SHAPE;
  if (!plan || (M > 0 && !index)) return QLORA_ERR_NULL;
  if (!aligned4(index) || !aligned16(plan)) return QLORA_ERR_ALIGN;
  const Plan p = plan_view(M, slots, plan);
  if (plan_bytes < p.bytes) return QLORA_ERR_WORKSPACE;
  return hip_status(launch_plan(p.v, index, M, slots, static_cast<hipStream_t>(stream)));
}

size_t qlora_adapters_workspace_bytes(int backward, const qlora_adapters_t* bank, int64_t M) {
  if (check_bank(bank, M)) return 0;
  return plan_adapters(backward != 0, bank, M, nullptr).bytes;
}

int qlora_adapters_fwd(const qlora_adapters_t* bank, const void* plan, size_t plan_bytes,
                       const uint16_t* X, int64_t M, const uint16_t* Y0, uint16_t* Y,
                       float* T_save, void* workspace, size_t workspace_bytes, void* stream) {
  int s = check_bank(bank, M);
  if (s) return s;
  if (M == 0) return QLORA_OK;
  s = check_bank_arrays(bank, plan, plan_bytes, M);
  if (s) return s;
  if (!X || !Y || !workspace) return QLORA_ERR_NULL;
  if (!aligned2(X) || !aligned2(Y0) || !aligned2(Y) || !aligned4(T_save) || !aligned16(workspace))
    return QLORA_ERR_ALIGN;
  const AdaptersPlan w = plan_adapters(false, bank, M, workspace);
  if (workspace_bytes < w.bytes) return QLORA_ERR_WORKSPACE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const PlanView v = plan_view(M, bank->slots, plan).v;
  ShrinkArgs sa{};
  sa.plan = v;
  sa.M = M;
  sa.slots = bank->slots;
  sa.K = bank->d_in;
  sa.r = (int)bank->r;
  sa.P = X;
  sa.F = bank->A;
  sa.part = w.part;
  sa.scale = bank->scale;
  sa.vrows = w.vrows;
  sa.v_out = T_save;
  s = hip_status(launch_shrink(sa, st));
  if (s) return s;
  int64_t kper;
  const int splits = shrink_splits(M, bank->d_in, &kper);
  const bool sums = splits > 1 && expand_sums(M, bank->r);
  if (splits > 1 && !sums) {
    FinishVArgs fa{};
    fa.plan = v;
    fa.M = M;
    fa.slots = bank->slots;
    fa.r = (int)bank->r;
    fa.splits = splits;
    fa.scale = bank->scale;
    fa.V = w.part;
    fa.vrows = w.vrows;
    fa.v_out = T_save;
    s = hip_status(launch_finish_v(fa, st));
    if (s) return s;
  }
  ExpandArgs ea{};
  ea.plan = v;
  ea.M = M;
  ea.slots = bank->slots;
  ea.d = bank->d_out;
  ea.r = (int)bank->r;
  ea.vrows = w.vrows;
  ea.part = sums ? w.part : nullptr;
  ea.splits = splits;
  ea.scale = bank->scale;
  ea.F = bank->B;
  ea.in = Y0;
  ea.out = Y;
  ea.v_out = T_save;
  return hip_status(launch_expand(ea, st));
}

int qlora_adapters_bwd(const qlora_adapters_t* bank, const void* plan, size_t plan_bytes,
                       const uint16_t* X, const qlora_packed_t* X8, const float* T,
                       const uint16_t* dY, int64_t M, const uint16_t* dX0, uint16_t* dX, float* dA,
                       float* dB, void* workspace, size_t workspace_bytes, void* stream) {
  int s = check_bank(bank, M);
  if (s) return s;
  if (X8 && (X8->M != M || X8->d != bank->d_in)) return QLORA_ERR_SHAPE;
  if ((X && X8) || (dX0 && !dX)) return QLORA_ERR_SHAPE;
  if (!dA || !dB) return QLORA_ERR_NULL;
  if (!aligned4(dA) || !aligned4(dB)) return QLORA_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  GramArgs8 ga{};
  ga.M = M;
  ga.slots = bank->slots;
  ga.r = bank->r;
  ga.q[0].out = dA;
  ga.q[0].d = bank->d_in;
  ga.q[1].out = dB;
  ga.q[1].d = bank->d_out;
  if (M == 0) return hip_status(launch_gram_zero(ga, st));
  s = check_bank_arrays(bank, plan, plan_bytes, M);
  if (s) return s;
  if ((!X && !X8) || !T || !dY || !workspace) return QLORA_ERR_NULL;
  if (X8 && (!X8->codes || !X8->scale)) return QLORA_ERR_NULL;
  if (!aligned2(X) || !aligned2(dY) || !aligned2(dX0) || !aligned2(dX) || !aligned4(T) ||
      !aligned16(workspace) || (X8 && (!aligned16(X8->codes) || !aligned4(X8->scale))))
    return QLORA_ERR_ALIGN;
  if (dX && (dX == dY || dX == X)) return QLORA_ERR_SHAPE;   // both are read after it is written
  const AdaptersPlan w = plan_adapters(true, bank, M, workspace);
  if (workspace_bytes < w.bytes) return QLORA_ERR_WORKSPACE;
  const PlanView v = plan_view(M, bank->slots, plan).v;
  ShrinkArgs sa{};
  sa.plan = v;
  sa.M = M;
  sa.slots = bank->slots;
  sa.K = bank->d_out;
  sa.r = (int)bank->r;
  sa.kn = true;
  sa.P = dY;
  sa.F = bank->B;
  sa.part = w.part;
  s = hip_status(launch_shrink(sa, st));
  if (s) return s;
  FinishVArgs fa{};
  fa.plan = v;
  fa.M = M;
  fa.slots = bank->slots;
  fa.r = (int)bank->r;
  int64_t kper;
  fa.splits = shrink_splits(M, bank->d_out, &kper);
  fa.scale = bank->scale;
  fa.V = w.part;
  fa.T = T;
  fa.vrows = dX ? w.vrows : nullptr;
  fa.u_frags = w.u_frags;
  fa.t_frags = w.t_frags;
  fa.zero_a = dA;
  fa.zero_b = dB;
  fa.d_a = bank->d_in;
  fa.d_b = bank->d_out;
  s = hip_status(launch_finish_v(fa, st));
  if (s) return s;
  if (dX) {
    ExpandArgs ea{};
    ea.plan = v;
    ea.M = M;
    ea.slots = bank->slots;
    ea.d = bank->d_in;
    ea.r = (int)bank->r;
    ea.rd = true;
    ea.vrows = w.vrows;
    ea.F = bank->A;
    ea.in = dX0;
    ea.out = dX;
    s = hip_status(launch_expand(ea, st));
    if (s) return s;
  }
  ga.plan = v;
  ga.tps = plan_split_tiles(M);
  ga.q[0].x = X;
  if (X8) {
    ga.q[0].codes = X8->codes;
    ga.q[0].scale = X8->scale;
  }
  ga.q[0].frags = w.u_frags;
  ga.q[0].part = w.da_part;
  ga.q[1].x = dY;
  ga.q[1].frags = w.t_frags;
  ga.q[1].part = w.db_part;
  return hip_status(launch_gram8(ga, st));
}

}  // extern "C"
