// C ABI of the experts of a mixture-of-experts layer for a few tokens:
// argument checks and launch.
#include <algorithm>

#include "experts.hpp"
#include "host.hpp"

namespace mxg {
namespace {

constexpr int64_t EXP_MAX_DIM = 1 << 17;   // activation offsets stay below 2^31

int64_t up16(int64_t n) { return cdiv(n, 16) * 16; }

// The weight format of an operand format, its unit of K and its scales.
struct ExpertsFormat {
  int wf;
  int64_t unit;
  bool scales;
};
bool experts_format(int fmt, ExpertsFormat &f) {
  switch (fmt) {
    case MXG_INT8: f = {WF_INT8, 16, true}; return true;
    case MXG_BF16: f = {WF_BF16, 8, false}; return true;
    case MXG_MXFP8_E4M3: f = {WF_E4M3, 32, true}; return true;
    case MXG_MXFP8_E5M2: f = {WF_E5M2, 32, true}; return true;
    case MXG_MXFP4_E2M1: f = {WF_E2M1, 32, true}; return true;
    case MXG_FP8_E4M3_BLOCK: f = {WF_BLOCK, 128, true}; return true;
    default: return false;
  }
}

// Workspace: h's two planes, the count of live experts, their records, the pairs.
struct ExpertsSpace {
  int64_t live, rec, pair, bytes;
};
ExpertsSpace experts_space(int64_t T, int topk, int64_t F) {
  ExpertsSpace s;
  s.live = up16(4 * T * topk * F);
  s.rec = s.live + 16;
  s.pair = s.rec + T * topk * (int64_t)sizeof(ExpertRec);
  s.bytes = s.pair + T * topk * (int64_t)sizeof(ExpertPair);
  return s;
}

template <int FMAX>
void launch_experts(int wf, const ExpertsArgs &a, unsigned up, unsigned down, hipStream_t stream) {
  auto go = [&](auto fc) {
    constexpr int WF = decltype(fc)::value;
    hipLaunchKernelGGL((experts_up_kernel<WF, FMAX>), dim3(up), dim3(64 * UP_WAVES), 0, stream, a);
    hipLaunchKernelGGL((experts_down_kernel<WF, FMAX>), dim3(down), dim3(64 * DOWN_WAVES), down_lds_bytes(a.T), stream, a);
  };
  switch (wf) {
    case WF_INT8: go(std::integral_constant<int, WF_INT8>{}); break;
    case WF_BF16: go(std::integral_constant<int, WF_BF16>{}); break;
    case WF_E4M3: go(std::integral_constant<int, WF_E4M3>{}); break;
    case WF_E5M2: go(std::integral_constant<int, WF_E5M2>{}); break;
    case WF_E2M1: go(std::integral_constant<int, WF_E2M1>{}); break;
    default: go(std::integral_constant<int, WF_BLOCK>{}); break;
  }
}

}  // namespace

int experts_init() {
  hipFuncAttributes attr;
  return hipFuncGetAttributes(&attr, (const void *)experts_up_kernel<WF_INT8, 1>) == hipSuccess ? MXG_OK : MXG_ERR_HIP;
}

}  // namespace mxg

using namespace mxg;

extern "C" int64_t moe_experts_workspace_bytes(int64_t T, int topk, int64_t F) {
  if (T < 0 || T > EXP_MAX_T || topk < 1 || topk > EXP_MAX_TOPK || F < 0 || F > EXP_MAX_DIM) return -1;
  return experts_space(T, topk, F).bytes;
}

extern "C" int moe_experts_validate(int fmt, const void *x, const int32_t *ids, const float *weights, const void *w1,
                                    const void *s1, const void *w2, const void *s2, const void *residual,
                                    const void *out, int64_t T, int64_t E, int topk, int64_t D, int64_t F,
                                    int activation, const void *workspace, int64_t workspace_bytes) {
  ExpertsFormat f;
  if (!experts_format(fmt, f)) return MXG_ERR_INVALID_ARG;
  if ((activation < MXG_ACT_NONE || activation > MXG_ACT_SILU) && activation != MXG_ACT_SWIGLU) return MXG_ERR_INVALID_ARG;
  if (T < 0 || E < 1 || topk < 1 || D < 0 || F < 0) return MXG_ERR_INVALID_ARG;
  if (T > EXP_MAX_T || E > EXP_MAX_E || topk > EXP_MAX_TOPK || D > EXP_MAX_DIM || F > EXP_MAX_DIM) return MXG_ERR_UNSUPPORTED;
  if (D % f.unit != 0 || F % f.unit != 0) return MXG_ERR_UNSUPPORTED;
  if (T == 0 || D == 0) return MXG_OK;
  if (!out || !ids || !weights || !workspace) return MXG_ERR_INVALID_ARG;
  if (workspace_bytes < experts_space(T, topk, F).bytes) return MXG_ERR_INVALID_ARG;
  if (F > 0 && (!x || !w1 || !w2 || (f.scales && (!s1 || !s2)))) return MXG_ERR_INVALID_ARG;
  // INT8 and block scales are FP32; E8M0 scales are bytes
  const uintptr_t sa = f.wf == WF_INT8 || f.wf == WF_BLOCK ? 4 : 1;
  if (!aligned(out, 16) || !aligned(residual, 16) || !aligned(x, 16) || !aligned(w1, 16) || !aligned(w2, 16) ||
      !aligned(workspace, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(s1, sa) || !aligned(s2, sa))
    return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

extern "C" int moe_experts(int fmt, const void *x, const int32_t *ids, const float *weights, const void *w1,
                           const void *s1, const void *w2, const void *s2, const void *residual, void *out, int64_t T,
                           int64_t E, int topk, int64_t D, int64_t F, int activation, void *workspace,
                           int64_t workspace_bytes, hipStream_t stream) {
  const int v = moe_experts_validate(fmt, x, ids, weights, w1, s1, w2, s2, residual, out, T, E, topk, D, F, activation,
                                     workspace, workspace_bytes);
  if (v != MXG_OK || T == 0 || D == 0) return v;
  ExpertsFormat f;
  experts_format(fmt, f);
  const ExpertsSpace sp = experts_space(T, topk, F);
  uint8_t *ws = (uint8_t *)workspace;
  ExpertsArgs a = {};
  a.x = (const uint16_t *)x;
  a.ids = ids;
  a.w = weights;
  a.w1 = (const uint8_t *)w1;
  a.w2 = (const uint8_t *)w2;
  a.s1 = s1;
  a.s2 = s2;
  a.residual = (const uint16_t *)residual;
  a.out = (uint16_t *)out;
  a.h = (uint16_t *)ws;
  a.live = (int32_t *)(ws + sp.live);
  a.rec = (ExpertRec *)(ws + sp.rec);
  a.pair = (ExpertPair *)(ws + sp.pair);
  a.D = D;
  a.F = F;
  a.N1 = activation == MXG_ACT_SWIGLU ? 2 * F : F;
  a.T = (int)T;
  a.E = (int)E;
  a.topk = topk;
  a.act = activation;
  a.tiles = (int)cdiv(a.N1, 16 * UP_FN);
  const int64_t most = std::min<int64_t>(E, T * topk);   // live experts at most
  // Parts of K per expert, so that few experts give every wave work.  F = 0:
  // none, and neither weights nor scales (which may be null) are touched.
  a.parts = F == 0 ? 0 : (int)std::max<int64_t>(1, std::min<int64_t>(DOWN_WAVES, cdiv(2 * DOWN_WAVES, most)));
  const unsigned up = (unsigned)(1 + most * a.tiles), down = (unsigned)cdiv(D, 16 * DOWN_FN);
  if (T <= 16) launch_experts<1>(f.wf, a, up, down, stream);
  else launch_experts<4>(f.wf, a, up, down, stream);
  return launch_status();
}
