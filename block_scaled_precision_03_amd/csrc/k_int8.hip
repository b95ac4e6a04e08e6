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

// The kernels: streaming through registers in 16 x 16 or 32 x 32 tiles,
// through LDS in 64 x 64 or 128 x 128 tiles, 256 x 256 tiles.
enum Kernel { ROWS16, ROWS32, STREAM64, STREAM128, TILED };

// Row tiles of b rows that a call can have at most: n groups that own rows
// take n + (M - n) / b, which grows with n.
int64_t max_row_tiles(int G, int64_t M, int b) {
  const int64_t n = std::min<int64_t>(G, M);
  return n + (M - n) / b;
}

// Estimated microseconds of each kernel, from static shapes alone (m_sizes
// stays on the device).  The rows are taken to fall on the groups at random:
// `live` of them own rows, and each of those fills half of its last row tile
// but at least one tile.  The constants are fitted to 170 dense calls of 1 ..
// 16384 rows and 706 grouped ones of 2 .. 1024 groups and 1 .. 16384 rows (N 256
// .. 28672, K 256 .. 14336), all kernels timed on each.  There the choice takes 1 % more than the fastest kernel on
// average, over 14 % more in 1 of 100 calls and at most 29 %; on 420 more calls,
// drawn afterwards, 1.4 %, over 14 % more in 11 and at most 42 %.  Both sides
// where the choice turns, in us: 3 x 3829 x 3984 5.9 in ROWS16, 14.4 in STREAM64; 65 x
// 12000 x 4096 55 and 17; 200 x 2000 x 400 5.3 in ROWS32, 5.9 in STREAM64; 777 x
// 5002 x 4112 84 and 49, 38 in STREAM128; 2049 x 8000 x 2064 68 in STREAM128, 58
// in TILED; 6449 x 1003 x 1040 22 and 28; 64 groups, 128 rows x 1536 x 4096 58 in
// ROWS16, 64 in STREAM64, 109 in TILED; 256 groups, 256 rows x 4096 x 7168 808,
// 738 and 1021; 8 groups, 1024 rows x 4608 x 7168 83 in STREAM128, 103 in TILED,
// 2048 rows 120 and 105.
Kernel choose(int G, int64_t M, int64_t N, int64_t K) {
  if (G < 1 || M <= 0 || N <= 0 || K <= 0) return STREAM64;
  const double cus = cu_count(), nst = (double)cdiv(K, 128);
  const double live = G == 1 ? 1.0 : G * (1.0 - std::pow(1.0 - 1.0 / G, (double)M));
  auto tiles = [&](int b) {
    return (G == 1 ? (double)cdiv(M, b) : std::max(live, (double)M / b + 0.5 * live)) * (double)cdiv(N, b);
  };
  // weights, activations and output once, at the rate of each kernel (TB/s)
  const double bytes = live * (double)N * (double)K + (double)M * (double)K + 2.0 * (double)M * (double)N;
  auto mem = [&](double rate) { return bytes / (rate * 1e6); };
  double t[5];
  // ROWS: a compute unit's 31 (25) bytes per ns of operands, tiles of full rows
  auto rows = [&](int b, double t0, double rate, double per_tile, double m) {
    const double n = tiles(b), ops = (std::min((double)b, (double)M / live) + b) * (double)K;
    return t0 + std::max(std::max(1.0, n / cus) * ops / rate, m) + per_tile * n / cus;
  };
  t[ROWS16] = rows(16, 2.71, 30.7e3, 0.432, mem(5.52));
  t[ROWS32] = rows(32, 3.15, 24.9e3, 0.788, mem(4.07));
  // STREAM: two workgroups per compute unit, a K step's time in a round of tiles
  auto stream = [&](int b, double t0, double alone, double shared, double per_tile, double m) {
    const double n = tiles(b), step = n <= cus ? alone : shared * std::ceil(n / (2 * cus));
    return t0 + std::max(nst * step, m) + per_tile * n / (2 * cus);
  };
  t[STREAM64] = stream(64, 3.63, 0.401, 0.536, 1.10, mem(7.19));
  t[STREAM128] = stream(128, 4.26, 0.81, 1.21, 1.39, mem(6.70));
  const double nt = tiles(DBM);
  t[TILED] = 5.03 + std::max(std::ceil(nt / cus) * (nst * (nt <= cus ? 1.44 : 1.57) + 4.22), mem(3.82));
  return (Kernel)(std::min_element(t, t + 5) - t);
}

int int8_variant(int G, int64_t M, int64_t N, int64_t K) {
  switch (choose(G, M, N, K)) {
    case STREAM64: return MXG_GROUPED_STREAM64;
    case STREAM128: return MXG_GROUPED_STREAM128;
    case TILED: return MXG_GROUPED_TILED;
    default: return MXG_GROUPED_ROWS;
  }
}

template <bool RES>
void (*pick_tiled(int act))(Int8Args) {
  return act == ACT_SWIGLU      ? int8_tiled_kernel<ACT_SWIGLU, RES>
         : act == ACT_RELU      ? int8_tiled_kernel<ACT_RELU, RES>
         : act == ACT_GELU_TANH ? int8_tiled_kernel<ACT_GELU_TANH, RES>
         : act == ACT_SILU      ? int8_tiled_kernel<ACT_SILU, RES>
                                : int8_tiled_kernel<ACT_NONE, RES>;
}

int launch(Int8Args &a, hipStream_t stream) {
  if (a.M == 0 || a.N == 0 || a.No == 0) return MXG_OK;
  if (a.K == 0) {
    const int64_t blocks = cdiv(a.M * a.No, 256);
    if (blocks > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
    hipLaunchKernelGGL(int8_fill_kernel, flat_grid(blocks), dim3(256), 0, stream, a);
    return launch_status();
  }
  const Kernel k = choose(a.G, a.M, a.N, a.K);
  const int BT = k == ROWS16 ? 16 : k == ROWS32 ? 32 : k == STREAM64 ? 64 : k == STREAM128 ? 128 : DBM;
  a.tiles_n = (int)cdiv(a.N, BT);
  const int64_t tiles = max_row_tiles(a.G, a.M, BT) * a.tiles_n;
  if (tiles > 0x7FFFFFF0) return MXG_ERR_UNSUPPORTED;
  void (*fn)(Int8Args);
  int64_t grid = 0;
  int threads = 256;
  const bool res = a.R != nullptr || a.Z != nullptr;
  switch (k) {
    case ROWS16:
      fn = res ? int8_rows_kernel<1, 1, 4, 4, true> : int8_rows_kernel<1, 1, 4, 4>;
      grid = (tiles + 7) / 8 * 8;          // eight bands (XCDs) of equal length
      break;
    case ROWS32:
      fn = res ? int8_rows_kernel<2, 2, 8, 2, true> : int8_rows_kernel<2, 2, 8, 2>;
      grid = (tiles + 7) / 8 * 8;
      threads = 512;
      break;
    case STREAM64:
      fn = res ? int8_stream_kernel<64, 64, 1, 4, true> : int8_stream_kernel<64, 64, 1, 4>;
      grid = std::min<int64_t>(tiles, 2ll * cu_count());
      break;
    case STREAM128:
      fn = res ? int8_stream_kernel<128, 128, 1, 2, true> : int8_stream_kernel<128, 128, 1, 2>;
      grid = std::min<int64_t>(tiles, 2ll * cu_count());
      break;
    default:
      fn = res ? pick_tiled<true>(a.act) : pick_tiled<false>(a.act);
      grid = std::min<int64_t>(tiles, cu_count());
      threads = DNW8 * 64;
  }
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3((unsigned)threads), 0, stream, a);
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
             int64_t K, const void *bias, int act, const void *residual, void *z, hipStream_t stream) {
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
  a.R = (const uint16_t *)residual;
  a.Z = (uint16_t *)z;
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
