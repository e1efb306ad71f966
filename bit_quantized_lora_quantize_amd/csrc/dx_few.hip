// dx_few.hip -- the NF4 LoRA layer's input gradient where the fused GEMM's tiles
// of 256 x 256 leave most of the GPU idle (gfx950):
//   dX = dY Wh + keep * (U A)
// U as BF16 hi | lo rows, Wh restored as everywhere (RNE_bf16 of level * scale),
// FP32 sums, one rounding.
//
// Item = 64 tokens, one block column of 64 inputs and a range of outputs n; the
// ranges' FP32 sums are added by k_dx_sum, in order.  The four wavefronts of a
// workgroup take 32 rows of W in turn: a lane restores half a block (32 weights)
// into LDS of the wavefront's own, whose transposing reads are the column
// operand of v_mfma_f32_16x16x32_bf16; dY comes straight from memory as the row
// operand, a step ahead.  The first range also adds U A, ahead of its weights so
// that dropped positions can be cleared between the two.  Bound by latency and,
// from about 64 tokens on, by the restore, which every 64 tokens repeat.
#include "qlora_device.h"
#include "qlora_kernels.h"
#include "row_ops.h"

namespace qlora {

namespace {

constexpr int kLd = 72;   // staged row of 64 weights
constexpr int kLr = 68;   // a reduced row of 64 sums, FP32

// What a lane needs of a step: half a block's codes and its scale, and dY.
template <int RB>
struct Step {
  u32x4 codes;
  uint32_t sc;
  float s2;
  u32x4 y[RB];
};

template <int RB>
__device__ __forceinline__ void dx_item(const DxFewArgs& a, int64_t m0, int64_t kb, int s,
                                        uint8_t* lds) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4, row = lane >> 1, half = lane & 1;
  uint16_t* st = reinterpret_cast<uint16_t*>(lds) + w * 32 * kLd;
  float* red = reinterpret_cast<float*>(lds);
  const int64_t nb = a.d_in / kBlock, c0 = kb * kBlock;
  const int64_t n_begin = (int64_t)s * a.nper;
  const int64_t n_end = n_begin + a.nper < a.d_out ? n_begin + a.nper : a.d_out;
  const float mean = a.mean[0];
  int64_t tok[RB];   // rows past the last token repeat it; their sums are not stored
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int64_t m = m0 + 16 * rb + r16;
    tok[rb] = m < a.M ? m : a.M - 1;
  }
  f32x4 acc[RB][4];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) acc[rb][cb] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto products = [&](const u32x4 (&y)[RB]) {
    u32x4 b[4];
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) {
      const uint16_t* p = st + (8 * g + (r16 >> 2)) * kLd + 16 * cb + 4 * (r16 & 3);
      const uint2 lo = lds_tr(p), hi = lds_tr(p + 4 * kLd);
      b[cb] = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int cb = 0; cb < 4; ++cb) acc[rb][cb] = mfma16(y[rb], b[cb], acc[rb][cb]);
  };

  if (s == 0) {
    // [U_hi | U_lo] [A; A], 32 ranks a step
    const int steps = 2 * (int)a.rp / 32;
    for (int e = w; e < steps; e += 4) {
      const int64_t i = (32 * e + row) % a.rp;
      u32x4* to = reinterpret_cast<u32x4*>(st + row * kLd + 32 * half);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4 v = {0, 0, 0, 0};
        if (i < a.r) v = load_vec(a.A + i * a.d_in + c0 + 32 * half + 8 * j);
        to[j] = v;
      }
      u32x4 y[RB];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
        y[rb] = *reinterpret_cast<const u32x4*>(a.u_hl + tok[rb] * 2 * a.rp + 32 * e + 8 * g);
      products(y);
    }
    if (a.keep) {
      // accumulator lane (r16, g): tokens 16 rb + 4 g + v, input c0 + 16 cb + r16
#pragma unroll
      for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const int64_t m = m0 + 16 * rb;
          const uint32_t k = m < a.M ? a.keep[(c0 + 16 * cb + r16) * a.keep_ld + m / 32] >> (m % 32) : 0u;
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[rb][cb][v] = (k >> (4 * g + v)) & 1u ? acc[rb][cb][v] : 0.0f;
        }
    }
  }

  auto load = [&](int64_t n0, Step<RB>& t) {
    // a row past the range has scale 0
    const int64_t n = n0 + row < n_end ? n0 + row : n_end - 1;
    t.codes = *reinterpret_cast<const u32x4*>(a.codes + (n * a.d_in + c0) / 2 + 16 * half);
    t.sc = a.scodes[n * nb + kb];
    t.s2 = a.scale2[(n * nb + kb) / kGroup];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const uint16_t* p = a.dY + tok[rb] * a.d_out;
      const int64_t at = n0 + 8 * g;
      if (n0 + 32 <= n_end) {                      // the same for the whole wavefront
        t.y[rb] = load_vec(p + at);
      } else {
        u32x4 v = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = p[at + e < n_end ? at + e : n_end - 1];
          v[e >> 1] |= (at + e < n_end ? x : 0u) << (16 * (e & 1));
        }
        t.y[rb] = v;
      }
    }
  };
  auto step = [&](int64_t n0, const Step<RB>& t) {
    const bool in = n0 + row < n_end;
    const Nf4Table tab = nf4_table(restored_scale(t.sc, in ? t.s2 : 0.0f, in ? mean : 0.0f));
    u32x4* to = reinterpret_cast<u32x4*>(st + row * kLd + 32 * half);
#pragma unroll
    for (int j = 0; j < 4; ++j) to[j] = nf4_dequant8(t.codes[j], tab);
    products(t.y);
  };
  int64_t n = n_begin + 32 * w;
  if (n < n_end) {
    Step<RB> ta, tb;
    load(n, ta);
    for (; n < n_end; n += 256) {
      if (n + 128 < n_end) load(n + 128, tb);
      step(n, ta);
      if (n + 128 >= n_end) break;
      if (n + 256 < n_end) load(n + 256, ta);
      step(n + 128, tb);
    }
  }

  // the wavefronts' sums, added in their order
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    if (m0 + 16 * rb >= a.M) break;
    lds_barrier();
#pragma unroll
    for (int cb = 0; cb < 4; ++cb)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[(w * 16 + 4 * g + v) * kLr + 16 * cb + r16] = acc[rb][cb][v];
    lds_barrier();
    const int i = threadIdx.x >> 4, c = 4 * (threadIdx.x & 15);
    f32x4 sum = *reinterpret_cast<const f32x4*>(red + i * kLr + c);
#pragma unroll
    for (int ww = 1; ww < 4; ++ww) sum += *reinterpret_cast<const f32x4*>(red + (ww * 16 + i) * kLr + c);
    const int64_t m = m0 + 16 * rb + i;
    if (m >= a.M) continue;
    const int64_t at = m * a.d_in + c0 + c;
    if (a.part) {
      *reinterpret_cast<f32x4*>(a.part + (int64_t)s * a.M * a.d_in + at) = sum;
    } else {
      *reinterpret_cast<uint2*>(a.dX + at) = make_uint2(pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3]));
    }
  }
  lds_barrier();
}

__global__ __launch_bounds__(256) void k_dx_few(DxFewArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * 32 * kLd * 2];
  static_assert(4 * 16 * kLr * 4 <= 4 * 32 * kLd * 2, "reduction buffer");
  const int64_t mts = (a.M + 63) / 64, kbs = a.d_in / kBlock;
  const int64_t items = mts * kbs * a.splits;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    // the tokens' tiles run fastest: they share the weights
    const int64_t m0 = item % mts * 64, rest = item / mts;
    const int64_t kb = rest % kbs;
    const int s = (int)(rest / kbs);
    if (a.M - m0 <= 16) dx_item<1>(a, m0, kb, s, lds);
    else dx_item<4>(a, m0, kb, s, lds);
  }
}

// dX = RN(the ranges' sums, in order), eight values a thread.
__global__ __launch_bounds__(256) void k_dx_sum(const float* __restrict__ part, int splits,
                                                int64_t count, uint16_t* __restrict__ dX) {
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; e < count;
       e += (int64_t)gridDim.x * 2048) {
    f32x4 x[kDxSplits][2];
#pragma unroll
    for (int s = 0; s < kDxSplits; ++s)
      if (s < splits) {
        x[s][0] = *reinterpret_cast<const f32x4*>(part + s * count + e);
        x[s][1] = *reinterpret_cast<const f32x4*>(part + s * count + e + 4);
      }
    f32x4 lo = x[0][0], hi = x[0][1];
#pragma unroll
    for (int s = 1; s < kDxSplits; ++s)
      if (s < splits) {
        lo += x[s][0];
        hi += x[s][1];
      }
    *reinterpret_cast<u32x4*>(dX + e) = u32x4{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                                             pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
  }
}

}  // namespace

hipError_t launch_dx_few(const DxFewArgs& a0, hipStream_t st) {
  DxFewArgs a = a0;
  a.splits = dx_few_splits(a.M, a.d_out, a.d_in, &a.nper);
  float* part = a.part;
  if (a.splits == 1) a.part = nullptr;
  const int64_t items = (a.M + 63) / 64 * (a.d_in / kBlock) * a.splits;
  hipLaunchKernelGGL(k_dx_few, dim3((unsigned)std::min<int64_t>(items, 8192)), dim3(256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t count = a.M * a.d_in;
  hipLaunchKernelGGL(k_dx_sum, dim3((unsigned)std::min<int64_t>((count + 2047) / 2048, 4096)), dim3(256),
                     0, st, part, a.splits, count, a.dX);
  return hipGetLastError();
}

}  // namespace qlora
