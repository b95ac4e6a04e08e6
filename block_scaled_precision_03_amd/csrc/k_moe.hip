// C ABI of the mixture-of-experts operators around the grouped GEMMs:
// argument checks, kernel choice from static shapes, launch.
#include <algorithm>
#include <type_traits>

#include "host.hpp"
#include "moe.hpp"

namespace mxg {
int moe_init() {
  hipFuncAttributes attr;
  return hipFuncGetAttributes(&attr, (const void *)route_place_kernel) == hipSuccess ? MXG_OK : MXG_ERR_HIP;
}
}  // namespace mxg

using namespace mxg;

static_assert(MOE_SOFTMAX == MXG_MOE_SOFTMAX && MOE_SIGMOID == MXG_MOE_SIGMOID && MOE_GROUP_MAX == MXG_MOE_GROUP_MAX &&
                  MOE_GROUP_TOP2 == MXG_MOE_GROUP_TOP2,
              "router codes");

namespace {

constexpr int64_t ROUTE_MAX_T = 1 << 24;       // a block's counts stay within 16 bits
constexpr int MAX_SLOTS = 64;                  // topk of quantize and combine
constexpr int64_t QUANT_MAX_K = 131056;

// Blocks of the router and tokens of each (a multiple of 64).
int64_t route_tpb(int64_t T) { return ROUTE_TG * cdiv(cdiv(T, ROUTE_TG), ROUTE_MAX_BLOCKS); }
int64_t route_blocks(int64_t T) { return cdiv(T, route_tpb(T)); }
int64_t padded_e(int64_t E) { return (E + 7) / 8 * 8; }

// Common checks of the router and its gradient.
int check_route(int dtype, int64_t T, int64_t E, int topk, int score) {
  if (dtype != MXG_BF16 && dtype != MXG_F32) return MXG_ERR_INVALID_ARG;
  if (score != MXG_MOE_SOFTMAX && score != MXG_MOE_SIGMOID) return MXG_ERR_INVALID_ARG;
  if (T < 0 || E < 0 || topk < 0) return MXG_ERR_INVALID_ARG;
  if (E < 1 || E > MOE_MAX_E || topk < 1 || topk > MOE_MAX_TOPK || topk > E) return MXG_ERR_UNSUPPORTED;
  if (T > ROUTE_MAX_T) return MXG_ERR_UNSUPPORTED;
  return MXG_OK;
}

// The lanes of a token (16, or 64 where 16 do not hold its experts or
// choices) and the experts of a lane.
struct RouteShape {
  int lpt, vpt, lpg, per;
};

bool fit_shape(int lpt, int E, int n_group, int topk, RouteShape &r) {
  int slots = 1;
  while (slots < n_group) slots *= 2;
  if (slots > lpt || topk > lpt) return false;
  r.lpt = lpt;
  r.lpg = lpt / slots;
  r.per = (int)cdiv(E / n_group, r.lpg);
  r.vpt = r.per <= 4 ? 4 : (r.per <= 8 ? 8 : (r.per <= 16 ? 16 : 32));
  return r.per <= (lpt == 16 ? 16 : 32);
}

typedef void (*route_fn)(RouteArgs);

template <class IN, bool MAPS, bool ONE>
route_fn pick_route(const RouteShape &s) {
  if (s.lpt == 16)
    return s.vpt == 4 ? route_kernel<IN, 16, 4, MAPS, ONE>
                      : (s.vpt == 8 ? route_kernel<IN, 16, 8, MAPS, ONE> : route_kernel<IN, 16, 16, MAPS, ONE>);
  if (s.vpt == 4) return route_kernel<IN, 64, 4, MAPS, ONE>;
  if (s.vpt == 8) return route_kernel<IN, 64, 8, MAPS, ONE>;
  return s.vpt == 16 ? route_kernel<IN, 64, 16, MAPS, ONE> : route_kernel<IN, 64, 32, MAPS, ONE>;
}

template <class IN>
route_fn pick_route(const RouteShape &s, bool maps, bool one) {
  if (!maps) return pick_route<IN, false, false>(s);
  return one ? pick_route<IN, true, true>(s) : pick_route<IN, true, false>(s);
}

}  // namespace

extern "C" int64_t moe_route_workspace_bytes(int64_t T, int64_t E) {
  if (T < 0 || T > ROUTE_MAX_T || E < 1 || E > MOE_MAX_E) return -1;
  if (T <= ROUTE_TG) return 0;
  return route_blocks(T) * padded_e(E) * 2;
}

extern "C" int moe_route(int dtype, const void *logits, const float *bias, int32_t *ids, float *weights, int64_t T,
                         int64_t E, int topk, int score, int n_group, int topk_group, int group_score,
                         int renormalize, float scale, int64_t *m_sizes, int32_t *row_of, int32_t *slot_of,
                         void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  const int v = check_route(dtype, T, E, topk, score);
  if (v != MXG_OK) return v;
  if (group_score != MXG_MOE_GROUP_MAX && group_score != MXG_MOE_GROUP_TOP2) return MXG_ERR_INVALID_ARG;
  if (n_group < 1 || n_group > 64 || E % n_group != 0 || topk_group < 1 || topk_group > n_group)
    return MXG_ERR_UNSUPPORTED;
  const bool maps = m_sizes != nullptr;
  if ((row_of != nullptr) != maps || (slot_of != nullptr) != maps) {
    // with no token the two row maps have no entry
    if (T != 0) return MXG_ERR_INVALID_ARG;
  }
  if (maps && !aligned(m_sizes, 8)) return MXG_ERR_MISALIGNED;
  if (T == 0) {
    if (!maps) return MXG_OK;
    hipLaunchKernelGGL(moe_zero_sizes_kernel, dim3(1), dim3(256), 0, stream, m_sizes, (int)E);
    return launch_status();
  }
  if (!logits || !ids || !weights) return MXG_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(row_of, 4) || !aligned(slot_of, 4))
    return MXG_ERR_MISALIGNED;
  const bool one = T <= ROUTE_TG;
  if (maps && !one) {
    if (!workspace || workspace_bytes < moe_route_workspace_bytes(T, E)) return MXG_ERR_INVALID_ARG;
    if (!aligned(workspace, 16)) return MXG_ERR_MISALIGNED;
  }
  RouteArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.T = T;
  a.E = (int)E;
  a.topk = topk;
  a.score = score;
  a.n_group = n_group;
  a.topk_group = topk_group;
  a.group_score = group_score;
  a.renorm = renormalize != 0;
  a.scale = scale;
  a.m_sizes = m_sizes;
  a.row_of = row_of;
  a.slot_of = slot_of;
  a.counts = (uint16_t *)workspace;
  a.Ep = (int)padded_e(E);
  a.tpb = route_tpb(T);
  a.nblk = (int)route_blocks(T);
  // A whole wave per token where there are few tokens (the shortest chain),
  // else four tokens per wave.
  RouteShape s;
  const bool fits = T > 16 ? (fit_shape(16, a.E, n_group, topk, s) || fit_shape(64, a.E, n_group, topk, s))
                           : fit_shape(64, a.E, n_group, topk, s);
  if (!fits) return MXG_ERR_UNSUPPORTED;
  a.lpg = s.lpg;
  a.per = s.per;
  // A block of the choice: the tokens of a row of counts (64 wherever they
  // give every compute unit a row), 32 of them where that leaves half of the
  // compute units idle (256 experts, 8 chosen: a block of 64 tokens takes 13.2
  // us, one of 32 takes 8.2), and 16 without maps; up to 16 waves, so that its
  // tokens run at once.
  a.halves = maps && !one && a.tpb == ROUTE_TG && 2 * a.nblk <= cu_count();
  a.tpc = !maps ? 16 : a.halves ? ROUTE_TG / 2 : a.tpb;
  const unsigned blocks = (unsigned)(!maps ? cdiv(T, 16) : a.halves ? 2 * a.nblk : a.nblk);
  const int64_t per_block = std::min<int64_t>(std::min<int64_t>(T, ROUTE_TG), a.tpc);
  const int threads = (int)std::min<int64_t>(1024, std::max<int64_t>(256, cdiv(per_block * s.lpt, 64) * 64));
  route_fn fn = dtype == MXG_BF16 ? pick_route<uint16_t>(s, maps, one) : pick_route<float>(s, maps, one);
  hipLaunchKernelGGL(fn, dim3(blocks), dim3((unsigned)threads), 0, stream, a);
  if (maps && !one) hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)a.nblk), dim3(a.nblk > 32 ? 1024 : 256), 0, stream, a);
  return launch_status();
}

extern "C" int moe_route_backward(int dtype, const void *logits, const int32_t *ids, const float *grad, void *dlogits,
                                  int64_t T, int64_t E, int topk, int score, int renormalize, float scale,
                                  hipStream_t stream) {
  const int v = check_route(dtype, T, E, topk, score);
  if (v != MXG_OK) return v;
  if (T == 0) return MXG_OK;
  if (!logits || !ids || !grad || !dlogits) return MXG_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(dlogits, 16) || !aligned(ids, 4) || !aligned(grad, 4)) return MXG_ERR_MISALIGNED;
  const bool four = E <= 256 && topk <= 16;      // 16 lanes per token, four tokens per wave
  const int lpt = four ? 16 : 64, per = (int)cdiv(E, lpt);
  RouteGradArgs a = {logits, ids, grad, dlogits, T, (int)E, topk, score, renormalize != 0, scale, per};
  auto go = [&](auto in) {
    typedef decltype(in) IN;
    void (*fn)(RouteGradArgs) = four ? (per <= 4   ? route_backward_kernel<IN, 16, 4>
                                        : per <= 8 ? route_backward_kernel<IN, 16, 8>
                                                   : route_backward_kernel<IN, 16, 16>)
                                     : (per <= 4   ? route_backward_kernel<IN, 64, 4>
                                        : per <= 8 ? route_backward_kernel<IN, 64, 8>
                                                   : route_backward_kernel<IN, 64, 16>);
    hipLaunchKernelGGL(fn, dim3((unsigned)cdiv(T, 256 / lpt)), dim3(256), 0, stream, a);
  };
  if (dtype == MXG_BF16) go((uint16_t)0);
  else go(0.0f);
  return launch_status();
}

extern "C" int mxgemm_quantize_int8(int dtype, const void *x, void *codes, float *scales, int64_t T, int64_t K,
                                    const int32_t *row_of, int topk, hipStream_t stream) {
  if ((dtype != MXG_BF16 && dtype != MXG_F32) || T < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (topk < 1 || topk > MAX_SLOTS || K % 16 != 0 || K > QUANT_MAX_K || T >= MAX_DIM || T * topk >= MAX_DIM)
    return MXG_ERR_UNSUPPORTED;
  if (row_of == nullptr && topk != 1) return MXG_ERR_INVALID_ARG;
  if (T == 0 || K == 0) return MXG_OK;
  if (!x || !codes || !scales) return MXG_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(row_of, 4)) return MXG_ERR_MISALIGNED;
  QuantArgs a = {x, (int8_t *)codes, scales, T, K, row_of, topk};
  // A wave per row up to 4096 values (four pieces of 16 per lane), else a
  // workgroup per row, in registers up to 16384 values.
  auto go = [&](auto in) {
    typedef decltype(in) IN;
    void (*fn)(QuantArgs) = K <= 1024    ? quant_int8_kernel<IN, 64, 1, false>
                            : K <= 4096  ? quant_int8_kernel<IN, 64, 4, false>
                            : K <= 8192  ? quant_int8_kernel<IN, 256, 2, false>
                            : K <= 16384 ? quant_int8_kernel<IN, 256, 4, false>
                                         : quant_int8_kernel<IN, 256, 4, true>;
    hipLaunchKernelGGL(fn, flat_grid(K <= 4096 ? cdiv(T, 4) : T), dim3(256), 0, stream, a);
  };
  if (dtype == MXG_BF16) go((uint16_t)0);
  else go(0.0f);
  return launch_status();
}

namespace {
int check_combine(const void *y, const float *w, const int32_t *row_of, int64_t T, int topk, int64_t N, int64_t rows) {
  if (T < 0 || N < 0 || rows < 0) return MXG_ERR_INVALID_ARG;
  if (topk < 1 || topk > MAX_SLOTS || T >= MAX_DIM || N >= MAX_DIM || rows >= MAX_DIM || T * topk >= MAX_DIM)
    return MXG_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return MXG_OK;
  if (!w || !row_of || (!y && rows > 0)) return MXG_ERR_INVALID_ARG;
  if (!aligned(y, 16) || !aligned(w, 4) || !aligned(row_of, 4)) return MXG_ERR_MISALIGNED;
  return MXG_OK;
}
}  // namespace

extern "C" int moe_combine(const void *y, const float *w, const int32_t *row_of, void *out, int64_t T, int topk,
                           int64_t N, int64_t rows, hipStream_t stream) {
  const int v = check_combine(y, w, row_of, T, topk, N, rows);
  if (v != MXG_OK || T == 0 || N == 0) return v;
  if (!out) return MXG_ERR_INVALID_ARG;
  if (!aligned(out, 16)) return MXG_ERR_MISALIGNED;
  CombineArgs a = {(const uint16_t *)y, w, row_of, (uint16_t *)out, T, N, rows, topk};
  const bool vec = N % 8 == 0;
  const dim3 grid((unsigned)cdiv(N, vec ? 2048 : 256), (unsigned)std::min<int64_t>(T, 65535), (unsigned)cdiv(T, 65535));
  hipLaunchKernelGGL(vec ? combine_kernel<8> : combine_kernel<1>, grid, dim3(256), 0, stream, a);
  return launch_status();
}

extern "C" int moe_combine_backward(const void *dout, const void *y, const float *w, const int32_t *row_of, void *dy,
                                    float *dw, int64_t T, int topk, int64_t N, int64_t rows, hipStream_t stream) {
  const int v = check_combine(y, w, row_of, T, topk, N, rows);
  if (v != MXG_OK || T == 0) return v;
  if (!dw) return MXG_ERR_INVALID_ARG;
  if (N == 0) {
    // empty sums
    if (!aligned(dw, 4)) return MXG_ERR_MISALIGNED;
    hipLaunchKernelGGL(fill_f32_kernel, dim3((unsigned)cdiv(T * topk, 256)), dim3(256), 0, stream, dw, T * topk, 0.0f);
    return launch_status();
  }
  if (!dout || (!dy && rows > 0)) return MXG_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !aligned(dy, 16) || !aligned(dw, 4)) return MXG_ERR_MISALIGNED;
  CombineGradArgs a = {(const uint16_t *)dout, (const uint16_t *)y, w, row_of, (uint16_t *)dy, dw, T, N, rows, topk};
  const bool vec = N % 8 == 0;
  const unsigned threads = (unsigned)std::min<int64_t>(256, cdiv(cdiv(N, vec ? 8 : 1), 64) * 64);
  hipLaunchKernelGGL(vec ? combine_backward_kernel<8> : combine_backward_kernel<1>, flat_grid(T), dim3(threads), 0,
                     stream, a);
  return launch_status();
}
