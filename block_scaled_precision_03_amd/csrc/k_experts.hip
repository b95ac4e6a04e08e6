// C ABI of the experts of a mixture-of-experts layer for a few tokens:
// argument checks and launch.
#include <algorithm>
#include <cmath>

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
  int private_t;
  int64_t (*row_bytes)(int64_t);
};
bool experts_format(int fmt, ExpertsFormat &f) {
  switch (fmt) {
    case MXG_INT8: f = {WF_INT8, 16, true, WeightFormat<WF_INT8>::PRIVATE_T, WeightFormat<WF_INT8>::row_bytes}; return true;
    case MXG_BF16: f = {WF_BF16, 8, false, WeightFormat<WF_BF16>::PRIVATE_T, WeightFormat<WF_BF16>::row_bytes}; return true;
    case MXG_MXFP8_E4M3: f = {WF_E4M3, 32, true, WeightFormat<WF_E4M3>::PRIVATE_T, WeightFormat<WF_E4M3>::row_bytes}; return true;
    case MXG_MXFP8_E5M2: f = {WF_E5M2, 32, true, WeightFormat<WF_E5M2>::PRIVATE_T, WeightFormat<WF_E5M2>::row_bytes}; return true;
    case MXG_MXFP4_E2M1: f = {WF_E2M1, 32, true, WeightFormat<WF_E2M1>::PRIVATE_T, WeightFormat<WF_E2M1>::row_bytes}; return true;
    case MXG_FP8_E4M3_BLOCK: f = {WF_BLOCK, 128, true, WeightFormat<WF_BLOCK>::PRIVATE_T, WeightFormat<WF_BLOCK>::row_bytes}; return true;
    default: return false;
  }
}

// Workspace: h's two planes, the counts, the records, the pairs, the splits' sums.
struct ExpertsSpace {
  int64_t count, rec, pair, part, bytes;
};
ExpertsSpace experts_space(int64_t T, int topk, int64_t F) {
  const int64_t P = T * topk;
  ExpertsSpace s;
  s.count = up16(4 * P * F);
  s.rec = s.count + 16 + 4 * EXP_SPLIT_BLOCKS;
  s.pair = s.rec + P * (int64_t)sizeof(ExpertRec);
  s.part = up16(s.pair + P * (int64_t)sizeof(ExpertPair));
  s.bytes = s.part + 4 * T * 64 * EXP_SPLIT_BLOCKS;
  return s;
}

template <int WF, int ROWS, int TM>
void launch_pair(const ExpertsArgs &a, unsigned up, unsigned down, hipStream_t stream) {
  hipLaunchKernelGGL((experts_up_kernel<WF, ROWS>), dim3(up), dim3(64 * EXP_WAVES), 0, stream, a);
  hipLaunchKernelGGL((experts_down_kernel<WF, ROWS, TM>), dim3(down), dim3(64 * EXP_WAVES), 0, stream, a);
}

template <int WF>
void launch_experts(const ExpertsArgs &a, unsigned up, unsigned down, hipStream_t stream) {
  constexpr int FEW = WeightFormat<WF>::PRIVATE_T;
  if (a.T <= FEW) launch_pair<WF, 0, FEW>(a, up, down, stream);
  else if (a.T <= 16 && a.rows == 8) launch_pair<WF, 8, 16>(a, up, down, stream);
  else if (a.T <= 16) launch_pair<WF, 16, 16>(a, up, down, stream);
  else if (a.rows == 8) launch_pair<WF, 8, EXP_MAX_T>(a, up, down, stream);
  else launch_pair<WF, 16, EXP_MAX_T>(a, up, down, stream);
}

}  // namespace

int experts_init() {
  hipFuncAttributes attr;
  return hipFuncGetAttributes(&attr, (const void *)experts_up_kernel<WF_INT8, 0>) == hipSuccess ? MXG_OK : MXG_ERR_HIP;
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
  // INT8 and block scales are FP32; E8M0 scales are read in aligned words
  const uintptr_t sa = f.wf == WF_INT8 || f.wf == WF_BLOCK ? 4 : 16;
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
  a.count = (int32_t *)(ws + sp.count);
  a.arrived = a.count + 4;
  a.rec = (ExpertRec *)(ws + sp.rec);
  a.pair = (ExpertPair *)(ws + sp.pair);
  a.part = (float *)(ws + sp.part);
  a.D = D;
  a.F = F;
  a.N1 = activation == MXG_ACT_SWIGLU ? 2 * F : F;
  a.T = (int)T;
  a.E = (int)E;
  a.topk = topk;
  a.act = activation;
  const bool few = T <= f.private_t;
  const int64_t P = T * topk, live = std::min<int64_t>(E, P);
  // One or two tokens: 16 rows of W1 per workgroup with K split over the waves
  // where 64 rows would leave compute units idle or K is long enough for
  // four times as many starts, each of which reads the choice (P slots); else 64
  // rows.  Fitted to 189 calls with both timed, weights cold: 0.2 % over the faster
  // one on average, at most 9 %.  Both sides, 16 and 64 rows, in us of the call (here and
  // below: copies of the weights in turn, none of them cached): MXFP8, 1 token, 8 of
  // 7168 x 2304 95.7, 112; 4 of 1024 x 512 INT8 10.1, 11.4; 2 of 2048 x 8192 INT8 33.2, 30.1;
  // 2 tokens, 16 of 2048 x 768 INT8 29.6, 27.8.
  const int64_t up_units = cdiv(f.row_bytes(D), 128);
  a.split_k = few && (4 * live * cdiv(a.N1, 64) < 3 * cu_count() || 2 * up_units >= 32 + 3 * P);
  a.up_tiles = (int)cdiv(a.N1, a.split_k ? 16 : 64);
  a.down_tiles = (int)cdiv(D, few ? 16 : 64);
  // Few columns leave compute units idle: the list of the records' units is
  // split over several workgroups (at most EXP_SPLIT_BLOCKS in all, which bounds
  // their sums).  A split costs its share of the last workgroup's additions, about
  // 0.2 + 0.006 T us, and saves units: 0.8 us each, shared, and a quarter private
  // (the call, in us: 37 tokens, 24 experts of 2080 x 1440 MXFP8, 1, 8 and 15
  // splits: 224, 82, 77; 64 tokens, 8 of 4096 x 4096 block FP8, 1 and 8: 252, 117; 16
  // tokens, 64 of 7168 x 2304 INT8, 1, 2 and 4: 860, 596, 501; a short list, 1 token, 4
  // of 1024 x 512 INT8, 1 and 2: 10.2, 10.7).
  const double units = (double)live * (double)cdiv(f.row_bytes(F), 128) / (few ? EXP_WAVES : 1);
  const double best = std::sqrt(units * 0.8 / (0.2 + 0.006 * (double)T));
  a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(EXP_SPLIT_BLOCKS / a.down_tiles, (int64_t)best));
  if (few && units < 24.0) a.splits = 1;
  // Up to 5 tokens per expert that has any: records of 8, whose smaller
  // stages leave room for more of them in flight; else 16 (an expert of more
  // tokens than that is read again).  Both sides, 8 and 16, in us of the call: 16 tokens,
  // 2 per expert, 64 of 7168 x 2304 INT8 494, 498; 37 tokens, 7 per expert, 24 of 2080
  // x 1440 MXFP8 83, 77; 64 tokens, 16 per expert, 8 of 4096 x 4096 block FP8 147, 116.
  a.rows = P <= 5 * live ? 8 : EXP_ROWS;
  // records: experts with tokens, and one more per `rows` tokens of an expert
  const int64_t most = live + (P - live) / a.rows;
  // F = 0: no tiles, no list; neither weights nor scales (which may be null) are touched
  const unsigned up = (unsigned)(1 + most * a.up_tiles), down = (unsigned)(a.down_tiles * a.splits);
  switch (f.wf) {
    case WF_INT8: launch_experts<WF_INT8>(a, up, down, stream); break;
    case WF_BF16: launch_experts<WF_BF16>(a, up, down, stream); break;
    case WF_E4M3: launch_experts<WF_E4M3>(a, up, down, stream); break;
    case WF_E5M2: launch_experts<WF_E5M2>(a, up, down, stream); break;
    case WF_E2M1: launch_experts<WF_E2M1>(a, up, down, stream); break;
    default: launch_experts<WF_BLOCK>(a, up, down, stream); break;
  }
  return launch_status();
}
