// C ABI of the 8-bit integer GEMM, dense and grouped: argument checks,
// kernel choice from static shapes, launch.
#include <algorithm>
#include <cmath>

#include "host.hpp"
#include "int8.hpp"

namespace mxg {
namespace {

// 128 * 128 * K must stay below 2^31.
constexpr int64_t INT8_MAX_K = 131056;

int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (M >= MAX_DIM || N >= MAX_DIM || K % 16 != 0 || K > INT8_MAX_K) return MXG_ERR_UNSUPPORTED;
  return MXG_OK;
}

// Kernel of a product of G groups with at most M rows in all, from upper
// bounds of the tile counts (MXG_GROUPED_*).
int int8_variant(int G, int64_t M, int64_t N, int64_t K) {
  if (G < 1 || M <= 0 || N <= 0 || K <= 0) return MXG_GROUPED_STREAM64;
  const double cus = cu_count(), nst = (double)cdiv(K, 128);
  const double t64 = 0.8 * (double)(cdiv(M, 64) + G - 1) * (double)cdiv(N, 64) * nst / (2 * cus);
  const double t128 = std::max(1.6 * (double)(cdiv(M, 128) + G - 1) * (double)cdiv(N, 128) * nst / (2 * cus), 1.1 * nst);
  const double td = std::ceil((double)(cdiv(M, DBM) + G - 1) * (double)cdiv(N, DBN) / cus) * (1.4 * nst + 10.0);
  if (t64 <= t128 && t64 <= td) return MXG_GROUPED_STREAM64;
  return t128 <= td ? MXG_GROUPED_STREAM128 : MXG_GROUPED_TILED;
}

int launch(Int8Args &a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0 || a.No == 0) return MXG_OK;
  if (a.K == 0) {
    const int64_t blocks = cdiv(a.M * a.No, 256);
    if (blocks > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(int8_fill_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
    return launch_status();
  }
  const int v = int8_variant(a.G, a.M, a.N, a.K);
  const bool tiled = v == MXG_GROUPED_TILED;
  const int BT = tiled ? DBM : (v == MXG_GROUPED_STREAM64 ? 64 : 128);
  a.tiles_n = (int)cdiv(a.N, BT);
  const int64_t tiles = (cdiv(a.M, BT) + a.G - 1) * a.tiles_n;
  if (tiles > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
  if (tiled) {
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, cu_count());
    void (*fn)(Int8Args) = a.act == ACT_SWIGLU      ? int8_tiled_kernel<ACT_SWIGLU>
                           : a.act == ACT_RELU      ? int8_tiled_kernel<ACT_RELU>
                           : a.act == ACT_GELU_TANH ? int8_tiled_kernel<ACT_GELU_TANH>
                           : a.act == ACT_SILU      ? int8_tiled_kernel<ACT_SILU>
                                                    : int8_tiled_kernel<ACT_NONE>;
    hipLaunchKernelGGL(fn, dim3(grid), dim3(DNW8 * 64), 0, stream, a);
  } else {
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, 2ll * cu_count());
    if (BT == 64)
      hipLaunchKernelGGL((int8_stream_kernel<64, 64, 2>), dim3(grid), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((int8_stream_kernel<128, 128, 1>), dim3(grid), dim3(256), 0, stream, a);
  }
  return launch_status();
}

}  // namespace

int int8_validate(int fmtA, int fmtB, int layout, const void *A, const void *sA, const void *B, const void *sB,
                  const void *D, int64_t M, int64_t N, int64_t K) {
  if (layout != MXG_NT && layout != MXG_NN && layout != MXG_TN) return MXG_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (fmtA != MXG_INT8 || fmtB != MXG_INT8 || layout != MXG_NT) return MXG_ERR_UNSUPPORTED;
  const int v = check_sizes(M, N, K);
  if (v != MXG_OK) return v;
  if (M == 0 || N == 0) return MXG_OK;
  if (!D) return MXG_ERR_INVALID_ARG;
  if (!aligned(D, 16)) return MXG_ERR_MISALIGNED;
  if (K == 0) return MXG_OK;
  if (!A || !B || !sA || !sB) return MXG_ERR_INVALID_ARG;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, 4) || !aligned(sB, 4)) return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

int int8_dense_variant(int64_t M, int64_t N, int64_t K) {
  switch (int8_variant(1, M, N, K)) {
    case MXG_GROUPED_STREAM64: return MXG_DENSE_TILE64;
    case MXG_GROUPED_STREAM128: return MXG_DENSE_TILE128;
    case MXG_GROUPED_ROWS: return MXG_DENSE_ROWS;
    default: return MXG_DENSE_TILE256;
  }
}

int int8_run(const void *A, const void *sA, const void *B, const void *sB, void *D, int64_t M, int64_t N,
             int64_t K, const void *bias, int act, hipStream_t stream) {
  Int8Args a = {};
  a.A = (const uint8_t *)A;
  a.B = (const uint8_t *)B;
  a.sA = (const float *)sA;
  a.sB = (const float *)sB;
  a.bias = (const uint16_t *)bias;
  a.D = (uint16_t *)D;
  a.M = M;
  a.N = N;
  a.K = K;
  a.No = act == MXG_ACT_SWIGLU ? N / 2 : N;
  a.G = 1;
  a.act = act;
  return launch(a, stream);
}

int int8_init() {
  hipFuncAttributes attr;
  return hipFuncGetAttributes(&attr, (const void *)int8_tiled_kernel<ACT_NONE>) == hipSuccess ? MXG_OK : MXG_ERR_HIP;
}

}  // namespace mxg

using namespace mxg;

static_assert(ACT_SWIGLU == MXG_ACT_SWIGLU, "activation codes");

extern "C" int grouped_int8_gemm_validate(int G, const int64_t *m_sizes, const void *XQ, const float *x_scale,
                                          const void *WQ, const float *w_scale, const void *D, int64_t totM,
                                          int64_t N, int64_t K, int activation) {
  if (G < 1 || G > MXG_GROUPED_MAX_G) return MXG_ERR_UNSUPPORTED;
  if ((activation < MXG_ACT_NONE || activation > MXG_ACT_SILU) && activation != MXG_ACT_SWIGLU)
    return MXG_ERR_INVALID_ARG;
  const int v = check_sizes(totM, N, K);
  if (v != MXG_OK) return v;
  if (!m_sizes) return MXG_ERR_INVALID_ARG;
  if (activation == MXG_ACT_SWIGLU && N % 2 != 0) return MXG_ERR_UNSUPPORTED;
  if (totM == 0 || N == 0) return MXG_OK;
  if (!D) return MXG_ERR_INVALID_ARG;
  if (!aligned(D, 16) || !aligned(m_sizes, 8)) return MXG_ERR_MISALIGNED;
  if (K == 0) return MXG_OK;
  if (!XQ || !x_scale || !WQ || !w_scale) return MXG_ERR_INVALID_ARG;
  if (!aligned(XQ, 16) || !aligned(WQ, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4))
    return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

extern "C" int grouped_int8_gemm_variant(int G, int64_t totM, int64_t N, int64_t K) {
  return int8_variant(G, totM, N, K);
}

extern "C" int grouped_int8_gemm_run(int G, const int64_t *m_sizes, const void *XQ, const float *x_scale,
                                     const void *WQ, const float *w_scale, void *D, int64_t totM, int64_t N,
                                     int64_t K, int activation, hipStream_t stream) {
  const int v = grouped_int8_gemm_validate(G, m_sizes, XQ, x_scale, WQ, w_scale, D, totM, N, K, activation);
  if (v != MXG_OK) return v;
  Int8Args a = {};
  a.A = (const uint8_t *)XQ;
  a.B = (const uint8_t *)WQ;
  a.sA = x_scale;
  a.sB = w_scale;
  a.m_sizes = m_sizes;
  a.D = (uint16_t *)D;
  a.M = totM;
  a.N = N;
  a.K = K;
  a.No = activation == MXG_ACT_SWIGLU ? N / 2 : N;
  a.G = G;
  a.act = activation;
  return launch(a, stream);
}
