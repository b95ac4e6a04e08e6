// C ABI of the gfx950 block-scaled GEMM library: argument validation, tile
// and grid selection from static shapes, and kernel launch.  The host never
// reads device memory; every call enqueues one kernel on the caller's
// stream (the tensor-wise quantizer four, see mxgemm_quantize_tensor; a
// grouped GEMM on 256 x 256 tiles two when the last round of its tiles
// goes to the streaming kernel) or returns an error before enqueueing
// anything.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <algorithm>
#include <cmath>
#include <map>
#include <mutex>
#include <stdio.h>
#include <tuple>

#include "../../include/mxgemm.h"
#include "host.hpp"
#include "kernels.hpp"
#include "preshuffle.hpp"
#include "quant.hpp"
#include "diag.hpp"

using namespace mxg;

namespace {

struct FmtInfo {
  bool ok;
  bool mx;      // E8M0 block scales (else one FP32 per tensor)
  int elem;     // F_E4M3 / F_E5M2 / F_E2M1
};

FmtInfo fmt_info(int f) {
  switch (f) {
    case MXG_MXFP8_E4M3: return {true, true, F_E4M3};
    case MXG_MXFP8_E5M2: return {true, true, F_E5M2};
    case MXG_MXFP4_E2M1: return {true, true, F_E2M1};
    case MXG_FP8_E4M3_TENSOR: return {true, false, F_E4M3};
    case MXG_FP8_E5M2_TENSOR: return {true, false, F_E5M2};
    default: return {false, false, 0};
  }
}

// Largest operand extents the 32-bit in-kernel offsets support.
constexpr int64_t MAX_ROW_BYTES = 1ll << 22;   // bytes of K per row (256 rows < 2^30)
constexpr int64_t MAX_T_BYTES = 0x7FFFFFF0ll;   // a transposed operand, whole
constexpr int64_t MAX_RES_COLS = 1 << 22;      // residual epilogue: 256 rows < 2^31 bytes
constexpr int64_t MAX_PSB_BYTES = (1ll << 32) - (1ll << 16);   // a preshuffled B, whole

// The persistent grouped kernels run GS_OCC workgroups per compute unit (74
// KiB of LDS each with the group table: 64 x 64 tiles with two 128-K steps
// per ring stage, 128 x 128 tiles with one; two ring slots), so that one
// workgroup's wait-barrier-compute chain overlaps the other's.
constexpr int GS_OCC = 2;

// The 256 x 256 grouped kernel leaves a partial last round of tiles to the
// streaming kernel when those tiles' pieces (128 x 64, or 64 x 64 when they
// fit one round) take at most this many rounds of it (grouped_split_end).
// That kernel runs with two 128-K steps per ring stage (99 KiB of LDS), one
// workgroup per compute unit: half the waits and barriers per K step of the
// one-step ring, whose two workgroups per unit took no less time per piece.
constexpr int GROUPED_TAIL_ROUNDS = 2;

}  // namespace

// Kernel choice for a dense call from its static shapes: the persistent
// 256 x 256 kernel, or (NT only) 64 x 64 tiles with one workgroup each when
// the output has too few 256 x 256 tiles to occupy the compute units.
// Estimated times, fitted to both kernels on MI355X (MXFP8, preshuffled B,
// M x N from 256 x 256 to 4096 x 4096, K from 256 to 8192): the persistent
// kernel ~6 us + 1.3 us per 128-K step per round of one tile per compute
// unit; 64 x 64 tiles ~3 us + 0.72 us per step per round (their fragments
// come straight from memory, three steps ahead, so a step costs a fraction
// of a load's latency).  Over that sweep the choice is the faster kernel
// everywhere but at 2048 x 2048 x 256 (2.7 us slower).
extern "C" int mxgemm_dense_variant(int fmtA, int fmtB, int layout, int64_t M, int64_t N, int64_t K) {
  if (fmtA == MXG_INT8 && fmtB == MXG_INT8) return int8_dense_variant(M, N, K);
  if (layout != MXG_NT || M <= 0 || N <= 0 || K <= 0) return MXG_DENSE_TILE256;
  const double cus = cu_count(), nst = (double)(K / 128);
  const double t256 = 6.0 + std::ceil((double)(cdiv(M, DBM) * cdiv(N, DBN)) / cus) * 1.3 * nst;
  const double t64 = 3.0 + std::ceil((double)(cdiv(M, SBM) * cdiv(N, SBN)) / cus) * 0.72 * nst;
  return t64 < t256 ? MXG_DENSE_TILE64 : MXG_DENSE_TILE256;
}

extern "C" const char *mxgemm_status_string(int s) {
  switch (s) {
    case MXG_OK: return "ok";
    case MXG_ERR_INVALID_ARG: return "invalid argument";
    case MXG_ERR_UNSUPPORTED: return "unsupported format, layout or shape";
    case MXG_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case MXG_ERR_HIP: return "HIP runtime error";
    case MXG_ERR_IO: return "tune cache file could not be read or written, or is malformed";
    default: return "unknown status";
  }
}

namespace {
// A kernel of each file that mxgemm_run_residual alone may launch from.
int residual_kernels_init() {
  const dense_fn fns[] = {pick_residual_mx_a4(F_E4M3, false, FUSE_RES), pick_residual_mx_a5(F_E4M3, false, FUSE_RES),
                          pick_residual_tw_a4(F_E4M3, false, FUSE_RES), pick_residual_tw_a5(F_E4M3, false, FUSE_RES),
                          pick_residual_fp4(false, FUSE_RES), pick_rows(F_E4M3, F_E4M3, true, false, 0),
                          pick_small(F_E4M3, F_E4M3, true, false, FUSE_RES)};
  hipFuncAttributes attr;
  for (const dense_fn fn : fns)
    if (hipFuncGetAttributes(&attr, (const void *)fn) != hipSuccess) return MXG_ERR_HIP;
  return MXG_OK;
}
}  // namespace

extern "C" int mxgemm_init(void) {
  // Touch the device so the code object is loaded before any graph capture.
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MXG_ERR_HIP;
  hipFuncAttributes attr;
  if (hipFuncGetAttributes(&attr, (const void *)pick_dense_mx_a4(F_E4M3, MXG_NT, false, false)) != hipSuccess)
    return MXG_ERR_HIP;
  (void)cu_count();
  int v = int8_init();
  if (v == MXG_OK) v = moe_init();
  if (v == MXG_OK) v = experts_init();
  if (v == MXG_OK) v = residual_init();
  return v == MXG_OK ? residual_kernels_init() : v;
}

extern "C" int mxgemm_validate(int fmtA, int fmtB, int layout, const void *A, const void *sA,
                    const void *B, const void *sB, const void *D, int64_t M, int64_t N,
                    int64_t K) {
  const bool psb = (fmtB & MXG_PRESHUFFLED) != 0;
  const FmtInfo fa = fmt_info(fmtA), fb = fmt_info(fmtB & ~MXG_PRESHUFFLED);
  const bool ia = fmtA == MXG_INT8, ib = (fmtB & ~MXG_PRESHUFFLED) == MXG_INT8;
  if ((!fa.ok && !ia) || (!fb.ok && !ib)) return MXG_ERR_INVALID_ARG;
  if (ia || ib) return int8_validate(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K);
  if (layout != MXG_NT && layout != MXG_NN && layout != MXG_TN) return MXG_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (M >= MAX_DIM || N >= MAX_DIM) return MXG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MXG_OK;
  if (!D) return MXG_ERR_INVALID_ARG;
  if (!aligned(D, 16)) return MXG_ERR_MISALIGNED;
  if (K == 0) return MXG_OK;
  if (!A || !B || !sA || !sB) return MXG_ERR_INVALID_ARG;
  if (fa.mx != fb.mx) return MXG_ERR_UNSUPPORTED;
  if ((fa.elem == F_E2M1) != (fb.elem == F_E2M1)) return MXG_ERR_UNSUPPORTED;
  const bool fp4 = fa.elem == F_E2M1;
  // A transposed packed E2M1 operand holds two columns per byte: its
  // contiguous dimension must fill whole 16-byte pieces.
  if (fp4 && layout == MXG_TN && M % 32 != 0) return MXG_ERR_UNSUPPORTED;
  if (fp4 && layout != MXG_NT && N % 32 != 0) return MXG_ERR_UNSUPPORTED;
  if (psb && layout != MXG_NT) return MXG_ERR_UNSUPPORTED;
  if (K % (fp4 ? 256 : 128) != 0) return MXG_ERR_UNSUPPORTED;
  const int64_t kb = fp4 ? K / 2 : K;
  if (kb > MAX_ROW_BYTES) return MXG_ERR_UNSUPPORTED;
  // A transposed operand is addressed from a tile's first column through
  // all K rows with one 32-bit range-checked offset.
  if (layout == MXG_TN && (M % 16 != 0 || M * K >= MAX_T_BYTES)) return MXG_ERR_UNSUPPORTED;
  if ((layout == MXG_TN || layout == MXG_NN) && (N % 16 != 0 || N * K >= MAX_T_BYTES))
    return MXG_ERR_UNSUPPORTED;
  if (fa.mx && (M * (K / 32) >= (1ll << 31) || cdiv(N, 64) * 64 * (K / 32) >= (1ll << 31)))
    return MXG_ERR_UNSUPPORTED;
  // A preshuffled B is addressed from its start with one 32-bit offset per
  // DMA (column group, K step and lane); it must stay below 2^32.
  if (psb && mxgemm_preshuffle_b_bytes(fmtB & ~MXG_PRESHUFFLED, N, K) > MAX_PSB_BYTES)
    return MXG_ERR_UNSUPPORTED;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(sA, fa.mx ? 16 : 4) || !aligned(sB, fb.mx ? 16 : 4))
    return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

// Kernel choice of the residual epilogue, every kernel by one kind of
// estimate from static shapes: the tiles of ROWS_TILES (rows.hpp), the 64 x 64 kernel
// (small.hpp) and the 256 x 256 one with its epilogue between two tiles.  Fitted to
// 1488 calls of 1 .. 16000 rows (N 96 .. 16000, K 256 .. 14336, MXFP8 and MXFP4, plain
// and preshuffled B, no activation and GELU, cold weights), every kernel timed on each
// (the tiles of up to 32 rows not above 64, 128 and 1024 rows): 0.6 % over the fastest on
// average, over 14 % in 13 of them, at most 34 %; fitted to two thirds of them, 0.6 %
// on the others, over 14 % in 1 of 496.  Both sides where the choice turns, in us (best
// of ROWS_TILES; 64 x 64; 256 x 256): MXFP8 233 x 5186 x 2432 22.8, 40.7, 41.5; 731 x
// 1472 x 512 12.4, 12.8, 20.8; 794 x 2496 x 7680 54, 135, 109; 1517 x 2304 x 768 25.9, 31.7,
// 25.3; MXFP4, preshuffled, 1991 x 1408 x 768 17.5, 12.3, 19.7; 541 x 4800 x 2304 26.3, 26.4,
// 29.0; 2384 x 2944 x 1280 48, 33, 24.
namespace {
enum : int { RES_TILE64 = ROWS_TILE_COUNT, RES_TILE256 };     // 0 .. ROWS_TILE_COUNT - 1: ROWS_TILES
int residual_kernel(int fmtA, int fmtB, int layout, int64_t M, int64_t N, int64_t K) {
  if (layout != MXG_NT || M <= 0 || N <= 0 || K < 128) return RES_TILE256;
  const bool psb = (fmtB & MXG_PRESHUFFLED) != 0, fp4 = fmtA == MXG_MXFP4_E2M1;
  const double cus = cu_count(), nst = (double)(K / 128), kb = fp4 ? 0.5 * K : (double)K;
  const double bytes = (double)N * kb + (double)M * kb + 4.0 * (double)M * (double)N;
  // ROWS_TILES: start; a tile's own time; a compute unit's operand bytes and all memory's per us
  struct Model { double t0, tile, rate, mem; };
  const Model model[2][ROWS_TILE_COUNT] = {
      {{2.25, 1.20, 44.0e3, 4.29e6}, {1.39, 2.52, 58.6e3, 3.77e6}, {1.61, 2.31, 51.6e3, 3.59e6}, {1.40, 3.19, 49.2e3, 3.01e6}, {0.23, 5.17, 47.9e3, 3.06e6}},
      {{2.15, 1.43, 46.0e3, 4.83e6}, {1.40, 2.57, 61.8e3, 3.96e6}, {1.57, 2.54, 58.7e3, 4.00e6}, {1.41, 3.37, 54.3e3, 3.33e6}, {0.0, 5.59, 52.6e3, 2.63e6}}};
  // the others: start; a K step's time in a round of tiles; a tile's (a round's) own time
  const double t64[2][2][3] = {{{3.58, 0.95, 1.73}, {3.63, 0.592, 1.07}}, {{3.34, 0.623, 1.73}, {3.60, 0.379, 1.21}}};
  const double t256[2][2][3] = {{{3.51, 1.70, 13.62}, {2.45, 0.77, 14.86}}, {{0.65, 1.29, 18.82}, {0.0, 0.78, 17.92}}};
  const double *s = t64[psb][fp4], *b = t256[psb][fp4], n64 = (double)(cdiv(M, SBM) * cdiv(N, SBN));
  double least = b[0] + std::ceil((double)(cdiv(M, DBM) * cdiv(N, DBN)) / cus) * (b[1] * nst + b[2]);
  int best = RES_TILE256;
  auto take = [&](int kernel, double us) {
    if (us < least) {
      least = us;
      best = kernel;
    }
  };
  take(RES_TILE64, s[0] + std::ceil(n64 / cus) * s[1] * nst + s[2] * n64 / cus);
  for (int i = 0; i < ROWS_TILE_COUNT; ++i) {
    const RowsTile &t = ROWS_TILES[i];
    const Model &m = model[psb][i];
    const int64_t tm = cdiv(M, t.rows);
    const double n = (double)(tm * cdiv(N, t.cols)), ops = (std::min((double)t.rows, (double)M / tm) + t.cols) * kb;
    // tiles per compute unit: whole rounds where one fills it
    const double load = t.per_cu > 1 ? std::max(1.0, n / cus) : std::ceil(n / cus);
    take(i, m.t0 + std::max(load * (m.tile + ops / m.rate), bytes / m.mem));
  }
  return best;
}
}  // namespace

extern "C" int mxgemm_residual_variant(int fmtA, int fmtB, int layout, int64_t M, int64_t N, int64_t K) {
  if (fmtA == MXG_INT8) return mxgemm_dense_variant(fmtA, fmtB, layout, M, N, K);
  const int k = residual_kernel(fmtA, fmtB, layout, M, N, K);
  return k == RES_TILE256 ? MXG_DENSE_TILE256 : k == RES_TILE64 ? MXG_DENSE_TILE64 : MXG_DENSE_ROWS;
}

namespace {
// Kernel selection for the dense path (the instantiations live in the k_*.hip
// translation units).
dense_fn pick_dense(int ea, int eb, bool mx, int layout, bool psb, int fuse) {
  if (fuse == FUSE_RES || fuse == FUSE_RES_ACT) {
    if (layout != MXG_NT) return nullptr;
    if (ea == F_E2M1 || eb == F_E2M1) return ea == eb && mx ? pick_residual_fp4(psb, fuse) : nullptr;
    if (ea == F_E4M3) return mx ? pick_residual_mx_a4(eb, psb, fuse) : pick_residual_tw_a4(eb, psb, fuse);
    if (ea == F_E5M2) return mx ? pick_residual_mx_a5(eb, psb, fuse) : pick_residual_tw_a5(eb, psb, fuse);
    return nullptr;
  }
  if (ea == F_E2M1 || eb == F_E2M1)
    return (ea == F_E2M1 && eb == F_E2M1 && mx) ? pick_dense_fp4(layout, psb, fuse) : nullptr;
  if (ea == F_E4M3) return mx ? pick_dense_mx_a4(eb, layout, psb, fuse) : pick_dense_tw_a4(eb, layout, psb, fuse);
  if (ea == F_E5M2) return mx ? pick_dense_mx_a5(eb, layout, psb, fuse) : pick_dense_tw_a5(eb, layout, psb, fuse);
  return nullptr;
}

__global__ void zero_bf16_kernel(uint16_t *D, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) D[i] = 0;
}

// K == 0 with the fused epilogue: D[m, n] = act(0 + bias[n]) + R[m, n].
__global__ void bias_act_fill_kernel(uint16_t *D, int64_t M, int64_t N, const uint16_t *bias, int act,
                                     const uint16_t *R, uint16_t *Z) {
  const int64_t i = flat_block() * 256 + threadIdx.x;
  if (i >= M * N) return;
  const float z = bias ? __uint_as_float((uint32_t)bias[i % N] << 16) : 0.0f;
  float v = activate(act, z);
  if (R) v += __uint_as_float((uint32_t)R[i] << 16);
  if (Z) Z[i] = (uint16_t)pack_bf16x2(z, 0.0f);
  D[i] = (uint16_t)pack_bf16x2(v, 0.0f);
}

int run_dense(int fmtA, int fmtB, int layout, const void *A, const void *sA, const void *B, const void *sB,
              void *D, int64_t M, int64_t N, int64_t K, const void *bias, int act, const void *residual, void *z,
              bool res, hipStream_t stream) {
  if (fmtA == MXG_INT8) return int8_run(A, sA, B, sB, D, M, N, K, bias, act, residual, z, stream);
  const int fuse = residual != nullptr || z != nullptr        ? (act != MXG_ACT_NONE ? FUSE_RES_ACT : FUSE_RES)
                   : bias != nullptr || act != MXG_ACT_NONE ? FUSE_ACT
                                                            : FUSE_NONE;
  if (M == 0 || N == 0) return MXG_OK;
  if (K == 0) {
    const int64_t n = M * N;
    if (fuse != FUSE_NONE)
      hipLaunchKernelGGL(bias_act_fill_kernel, flat_grid(cdiv(n, 256)), dim3(256), 0, stream, (uint16_t *)D, M, N,
                         (const uint16_t *)bias, act, (const uint16_t *)residual, (uint16_t *)z);
    else
      hipLaunchKernelGGL(zero_bf16_kernel, dim3((unsigned)cdiv(n, 256)), dim3(256), 0, stream,
                         (uint16_t *)D, n);
    return launch_status();
  }
  const bool psb = (fmtB & MXG_PRESHUFFLED) != 0;
  const FmtInfo fa = fmt_info(fmtA), fb = fmt_info(fmtB & ~MXG_PRESHUFFLED);
  const int tile = res ? residual_kernel(fmtA, fmtB, layout, M, N, K)
                   : mxgemm_dense_variant(fmtA, fmtB, layout, M, N, K) == MXG_DENSE_TILE64 ? RES_TILE64
                                                                                        : RES_TILE256;
  const bool rows = tile < ROWS_TILE_COUNT, small = tile == RES_TILE64;
  dense_fn fn = rows    ? pick_rows(fa.elem, fb.elem, fa.mx, psb, tile)
                : small ? pick_small(fa.elem, fb.elem, fa.mx, psb, fuse)
                        : pick_dense(fa.elem, fb.elem, fa.mx, layout, psb, fuse);
  if (!fn) return MXG_ERR_UNSUPPORTED;
  const bool fp4 = fa.elem == F_E2M1;
  DenseArgs a = {};
  a.A = (const uint8_t *)A;
  a.B = (const uint8_t *)B;
  a.sA = sA;
  a.sB = sB;
  a.D = (uint16_t *)D;
  a.M = M;
  a.N = N;
  a.K = K;
  a.a_bytes = fp4 ? M * K / 2 : M * K;
  a.b_bytes = psb ? mxgemm_preshuffle_b_bytes(fmtB & ~MXG_PRESHUFFLED, N, K) : (fp4 ? N * K / 2 : N * K);
  a.sa_bytes = fa.mx ? M * (K / 32) : 4;
  a.sb_bytes = fb.mx ? (psb ? mxgemm_preshuffle_scales_bytes(N, K) : N * (K / 32)) : 4;
  a.tiles_m = (int)cdiv(M, rows ? ROWS_TILES[tile].rows : small ? SBM : DBM);
  a.tiles_n = (int)cdiv(N, rows ? ROWS_TILES[tile].cols : small ? SBN : DBN);
  a.bias = (const uint16_t *)bias;
  a.act = act;
  a.R = (const uint16_t *)residual;
  a.Z = (uint16_t *)z;
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  if (tiles > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
  if (rows) {
    hipLaunchKernelGGL(fn, dim3((unsigned)tiles), dim3((unsigned)(64 * ROWS_TILES[tile].waves)), 0, stream, a);
    return launch_status();
  }
  if (small) {
    // one workgroup of four waves per 64 x 64 tile
    hipLaunchKernelGGL(fn, dim3((unsigned)tiles), dim3(256), 0, stream, a);
    return launch_status();
  }
  // Persistent grid: one workgroup per compute unit, each walking its tiles.
  const int64_t blocks = tiles < cu_count() ? tiles : cu_count();
  hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(DNW8 * 64), 0, stream, a);
  return launch_status();
}
}  // namespace

extern "C" int mxgemm_run(int fmtA, int fmtB, int layout, const void *A, const void *sA, const void *B,
               const void *sB, void *D, int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const int v = mxgemm_validate(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K);
  if (v != MXG_OK) return v;
  return run_dense(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K, nullptr, MXG_ACT_NONE, nullptr, nullptr, false, stream);
}

extern "C" int mxgemm_validate_fused(int fmtA, int fmtB, int layout, const void *A, const void *sA,
                                     const void *B, const void *sB, const void *D, int64_t M, int64_t N,
                                     int64_t K, const void *bias, int activation) {
  // SwiGLU is built for the integer GEMM alone
  const bool swiglu = activation == MXG_ACT_SWIGLU && fmtA == MXG_INT8;
  if ((activation < MXG_ACT_NONE || activation > MXG_ACT_SILU) && !swiglu) return MXG_ERR_INVALID_ARG;
  const int v = mxgemm_validate(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K);
  if (v != MXG_OK) return v;
  if (bias == nullptr && activation == MXG_ACT_NONE) return MXG_OK;
  if (layout != MXG_NT) return MXG_ERR_UNSUPPORTED;
  if (swiglu && N % 2 != 0) return MXG_ERR_UNSUPPORTED;
  if (bias != nullptr) {
    // the bias is staged by 4-byte DMAs of column pairs
    if (N % 2 != 0) return MXG_ERR_UNSUPPORTED;
    if (!aligned(bias, 4)) return MXG_ERR_MISALIGNED;
  }
  return MXG_OK;
}

extern "C" int mxgemm_run_fused(int fmtA, int fmtB, int layout, const void *A, const void *sA, const void *B,
                                const void *sB, void *D, int64_t M, int64_t N, int64_t K, const void *bias,
                                int activation, hipStream_t stream) {
  const int v = mxgemm_validate_fused(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K, bias, activation);
  if (v != MXG_OK) return v;
  return run_dense(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K, bias, activation, nullptr, nullptr, false, stream);
}

extern "C" int mxgemm_validate_residual(int fmtA, int fmtB, int layout, const void *A, const void *sA, const void *B,
                                        const void *sB, const void *D, int64_t M, int64_t N, int64_t K, const void *bias,
                                        int activation, const void *residual, const void *z) {
  const int v = mxgemm_validate_fused(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K, bias, activation);
  if (v != MXG_OK) return v;
  if (residual == nullptr && z == nullptr) return MXG_OK;
  if (layout != MXG_NT) return MXG_ERR_UNSUPPORTED;
  // the residual kernels address a tile's rows with one 32-bit offset
  if (N > MAX_RES_COLS) return MXG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MXG_OK;
  if (z != nullptr && (z == D || z == residual)) return MXG_ERR_INVALID_ARG;
  if (!aligned(residual, 16) || !aligned(z, 16)) return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

extern "C" int mxgemm_run_residual(int fmtA, int fmtB, int layout, const void *A, const void *sA, const void *B,
                                   const void *sB, void *D, int64_t M, int64_t N, int64_t K, const void *bias,
                                   int activation, const void *residual, void *z, hipStream_t stream) {
  const int v = mxgemm_validate_residual(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K, bias, activation, residual, z);
  if (v != MXG_OK) return v;
  return run_dense(fmtA, fmtB, layout, A, sA, B, sB, D, M, N, K, bias, activation, residual, z, true, stream);
}

extern "C" int grouped_fp8_gemm_validate(int G, const int64_t *m_sizes, const void *XQ, const float *x_scale,
                              const void *WQ, const float *w_scale, const void *D, int64_t totM,
                              int64_t N, int64_t K, int b_preshuffled) {
  (void)b_preshuffled;
  if (G < 1 || G > MXG_GROUPED_MAX_G) return MXG_ERR_UNSUPPORTED;
  if (totM < 0 || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (!m_sizes) return MXG_ERR_INVALID_ARG;
  if (N % 128 != 0 || K % 128 != 0) return MXG_ERR_UNSUPPORTED;
  if (totM >= MAX_DIM || N >= MAX_DIM || K > MAX_ROW_BYTES) return MXG_ERR_UNSUPPORTED;
  if (totM * (K / 128) * 4 >= (1ll << 31)) return MXG_ERR_UNSUPPORTED;
  if (totM == 0 || N == 0) return MXG_OK;
  if (!D) return MXG_ERR_INVALID_ARG;
  if (!aligned(D, 16) || !aligned(m_sizes, 8)) return MXG_ERR_MISALIGNED;
  if (K == 0) return MXG_OK;
  if (!XQ || !x_scale || !WQ || !w_scale) return MXG_ERR_INVALID_ARG;
  if (!aligned(XQ, 16) || !aligned(WQ, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4))
    return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

namespace {
__global__ void grouped_zero_kernel(const int64_t *m_sizes, int G, uint16_t *D, int64_t totM,
                                    int64_t N) {
  // K == 0: every row that belongs to a group becomes zero.
  int64_t covered = 0;
  for (int g = 0; g < G; ++g) {
    int64_t s = m_sizes[g];
    const int64_t room = totM - covered;
    covered += s < 0 ? 0 : (s > room ? room : s);
  }
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < covered * N) D[i] = 0;
}
}  // namespace

namespace {
// One grouped GEMM with the given kernel (arguments already validated).
int launch_grouped(int variant, int G, const int64_t *m_sizes, const void *XQ, const float *x_scale,
                   const void *WQ, const float *w_scale, void *D, int64_t totM, int64_t N, int64_t K,
                   int b_preshuffled, hipStream_t stream) {
  if (totM == 0 || N == 0) return MXG_OK;
  if (K == 0) {
    hipLaunchKernelGGL(grouped_zero_kernel, dim3((unsigned)cdiv(totM * N, 256)), dim3(256), 0,
                       stream, m_sizes, G, (uint16_t *)D, totM, N);
    return launch_status();
  }
  GroupedArgs a = {};
  a.m_sizes = m_sizes;
  a.XQ = (const uint8_t *)XQ;
  a.WQ = (const uint8_t *)WQ;
  a.xs = x_scale;
  a.ws = w_scale;
  a.D = (uint16_t *)D;
  a.totM = totM;
  a.N = N;
  a.K = K;
  a.G = G;
  // streaming tiles: 64 x 64 or 128 x 128 (N % 128 == 0)
  const int BM = variant == MXG_GROUPED_STREAM64 ? 64 : 128;
  const int BN = variant == MXG_GROUPED_STREAM64 ? 64 : 128;
  a.tiles_n = (int)(N / BN);
  const int64_t blocks = (cdiv(totM, BM) + G - 1) * a.tiles_n;
  if (blocks > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
  // persistent kernels: GS_OCC workgroups per compute unit (fewer if fewer tiles)
  const unsigned P = (unsigned)std::min<int64_t>(blocks, (int64_t)GS_OCC * cu_count());
  const bool pre = b_preshuffled != 0;
  if (variant == MXG_GROUPED_STREAM64 || variant == MXG_GROUPED_STREAM128) {
    hipLaunchKernelGGL(pick_grouped_stream(BM, pre), dim3(P), dim3(256), 0, stream, a);
  } else {
    // matrix-core regime: the dense pipeline with groupwise scales, 256 x
    // 256 tiles, one persistent workgroup per compute unit
    DenseArgs d = {};
    d.A = (const uint8_t *)XQ;
    d.B = (const uint8_t *)WQ;
    d.sA = x_scale;
    d.sB = w_scale;
    d.D = (uint16_t *)D;
    d.M = totM;
    d.N = N;
    d.K = K;
    d.a_bytes = totM * K;
    d.b_bytes = (int64_t)G * N * K;
    d.sa_bytes = totM * (K / 128) * 4;
    d.sb_bytes = (int64_t)G * (N / 128) * (K / 128) * 4;
    d.tiles_n = (int)cdiv(N, DBN);
    d.tiles_m = (int)(cdiv(totM, DBM) + G - 1);      // upper bound; the kernel counts them
    d.m_sizes = m_sizes;
    d.G = G;
    const int64_t tiles = (int64_t)d.tiles_m * d.tiles_n;
    if (tiles > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, cu_count());
    // With at most `grid` tiles there is one round and no tail to split off.
    const bool tail = tiles > (int64_t)grid;
    const unsigned tail_grid = (unsigned)cu_count();
    d.tail_grid = (int)tail_grid;
    d.tail_rounds = tail ? GROUPED_TAIL_ROUNDS : 0;
    hipLaunchKernelGGL(pick_grouped_dense(pre), dim3(grid), dim3(DNW8 * 64), 0, stream, d);
    if (tail) {
      a.tiles_n = (int)(N / 64);
      a.tiles_nb = d.tiles_n;
      a.main_grid = (int)grid;
      a.tail_rounds = GROUPED_TAIL_ROUNDS;
      hipLaunchKernelGGL(pick_grouped_tail(pre), dim3(tail_grid), dim3(256), 0, stream, a);
    }
  }
  return launch_status();
}
}  // namespace

extern "C" int grouped_fp8_gemm_run(int G, const int64_t *m_sizes, const void *XQ, const float *x_scale,
                         const void *WQ, const float *w_scale, void *D, int64_t totM, int64_t N,
                         int64_t K, int b_preshuffled, hipStream_t stream) {
  const int v = grouped_fp8_gemm_validate(G, m_sizes, XQ, x_scale, WQ, w_scale, D, totM, N, K,
                                          b_preshuffled);
  if (v != MXG_OK) return v;
  return launch_grouped(grouped_fp8_gemm_variant(G, totM, N, K, b_preshuffled), G, m_sizes, XQ, x_scale,
                        WQ, w_scale, D, totM, N, K, b_preshuffled, stream);
}

namespace {
// Static tile table of the grouped GEMM, keyed as "Add FlyDSL grouped
// groupwise FP8 GEMM for ROCm" (Tile selection) keys its autotuned winners:
// (nextPow2(totM), N, K, b_preshuffled), here for G = 8 (the pages' G).
// Each entry is the fastest of the three kernels measured on MI355X at
// totM = 2^log2m with the benchmark's kind of m_sizes (one empty group,
// uneven cuts), by the sum of its warm time (the same weights every call)
// and its cold time (weight copies totalling more than the 256 MB
// last-level cache rotated between calls: a layer whose weights are not
// cached); the times after each entry are warm / cold us of the 64 x 64
// streaming, 128 x 128 streaming and 256 x 256 dense-pipeline kernels, in
// that order.
struct GroupedTile {
  int32_t N, K;
  int8_t log2m, pre, variant;
};
const GroupedTile GROUPED_TILES[] = {
    {1280, 8192, 7, 0, 0},   //   26.8 /  34.6    49.7 /  60.6    91.1 /  93.0 us
    {1280, 8192, 7, 1, 0},   //   26.3 /  33.9    49.9 /  57.5    91.3 /  93.4 us
    {1280, 8192, 8, 0, 0},   //   27.5 /  36.9    50.4 /  61.5    93.2 /  97.1 us
    {1280, 8192, 8, 1, 0},   //   26.7 /  34.9    50.2 /  57.9    93.1 /  96.2 us
    {1280, 8192, 9, 0, 0},   //   33.3 /  36.4    51.5 /  62.0   109.9 / 114.4 us
    {1280, 8192, 9, 1, 0},   //   32.4 /  35.1    51.3 /  58.5   110.2 / 113.5 us
    {1280, 8192, 10, 0, 0},   //   34.6 /  42.6    52.4 /  62.4   115.2 / 120.2 us
    {1280, 8192, 10, 1, 0},   //   34.3 /  41.1    52.4 /  59.8   115.3 / 120.5 us
    {1280, 8192, 11, 0, 2},   //   56.5 /  71.9    56.4 /  64.2   108.4 / 112.0 us
    {1280, 8192, 11, 1, 2},   //   53.5 /  65.7    52.8 /  59.4   107.6 / 111.9 us
    {1280, 8192, 12, 0, 2},   //  100.0 / 108.4    75.0 /  79.2   114.6 / 117.0 us
    {1280, 8192, 12, 1, 2},   //   92.1 / 100.1    66.0 /  72.5   112.3 / 116.1 us
    {1280, 8192, 13, 0, 1},   //  203.3 / 214.5   124.5 / 138.4   115.6 / 116.6 us
    {1280, 8192, 13, 1, 1},   //  187.7 / 203.4   120.2 / 130.3   111.6 / 114.6 us
    {1280, 8192, 14, 0, 1},   //  389.7 / 381.1   218.9 / 223.0   219.3 / 220.3 us
    {1280, 8192, 14, 1, 2},   //  380.6 / 370.0   215.5 / 219.8   219.7 / 220.0 us
    {2048, 7168, 7, 0, 0},   //   25.5 /  33.9    44.8 /  55.2    80.4 /  86.0 us
    {2048, 7168, 7, 1, 0},   //   25.2 /  31.4    44.5 /  52.8    81.7 /  83.3 us
    {2048, 7168, 8, 0, 0},   //   25.9 /  34.7    45.5 /  55.8    83.1 /  90.6 us
    {2048, 7168, 8, 1, 0},   //   25.7 /  32.2    44.8 /  53.3    84.6 /  87.6 us
    {2048, 7168, 9, 0, 0},   //   31.7 /  38.6    48.4 /  56.7   101.3 / 108.8 us
    {2048, 7168, 9, 1, 0},   //   30.5 /  36.3    46.7 /  54.2   101.1 / 106.0 us
    {2048, 7168, 10, 0, 2},   //   49.9 /  64.9    49.0 /  57.5   109.1 / 117.2 us
    {2048, 7168, 10, 1, 2},   //   48.0 /  60.9    47.3 /  54.1   108.8 / 114.0 us
    {2048, 7168, 11, 0, 2},   //   75.3 /  93.1    66.4 /  73.5   100.7 / 106.5 us
    {2048, 7168, 11, 1, 2},   //   68.6 /  84.8    59.0 /  67.0    97.2 / 102.8 us
    {2048, 7168, 12, 0, 2},   //  133.6 / 149.6   102.0 / 115.4   112.8 / 114.9 us
    {2048, 7168, 12, 1, 2},   //  116.6 / 137.1    98.2 / 108.8   108.1 / 111.2 us
    {2048, 7168, 13, 0, 1},   //  270.3 / 284.3   162.0 / 181.0   154.4 / 155.7 us
    {2048, 7168, 13, 1, 1},   //  255.6 / 271.4   158.3 / 172.2   152.8 / 153.7 us
    {2048, 7168, 14, 0, 1},   //  523.3 / 527.4   291.3 / 303.3   272.4 / 273.0 us
    {2048, 7168, 14, 1, 1},   //  515.6 / 515.6   283.2 / 292.5   268.5 / 270.2 us
    {4096, 4096, 7, 0, 0},   //   22.0 /  30.9    30.8 /  38.4    54.6 /  55.7 us
    {4096, 4096, 7, 1, 0},   //   22.0 /  25.5    29.1 /  33.7    52.3 /  54.1 us
    {4096, 4096, 8, 0, 0},   //   22.3 /  31.4    31.3 /  38.2    55.8 /  58.4 us
    {4096, 4096, 8, 1, 0},   //   22.2 /  27.1    29.2 /  34.0    53.8 /  56.7 us
    {4096, 4096, 9, 0, 2},   //   37.5 /  44.5    33.2 /  40.0    74.9 /  77.1 us
    {4096, 4096, 9, 1, 2},   //   35.6 /  41.8    31.6 /  35.6    72.1 /  74.9 us
    {4096, 4096, 10, 0, 2},   //   47.5 /  62.2    43.3 /  48.8    83.1 /  84.6 us
    {4096, 4096, 10, 1, 2},   //   43.8 /  56.8    39.4 /  45.1    80.0 /  83.8 us
    {4096, 4096, 11, 0, 2},   //   78.4 /  96.1    67.0 /  75.1    76.4 /  77.5 us
    {4096, 4096, 11, 1, 2},   //   72.8 /  85.6    61.8 /  67.5    72.1 /  73.3 us
    {4096, 4096, 12, 0, 2},   //  156.7 / 162.5    98.6 / 107.3   133.3 / 132.2 us
    {4096, 4096, 12, 1, 2},   //  130.3 / 149.3    91.4 / 100.4   129.3 / 130.4 us
    {4096, 4096, 13, 0, 1},   //  304.7 / 315.8   178.5 / 189.2   178.2 / 180.7 us
    {4096, 4096, 13, 1, 2},   //  286.9 / 301.5   170.8 / 187.2   177.7 / 180.6 us
    {4096, 4096, 14, 0, 1},   //  590.2 / 599.0   344.6 / 351.9   304.9 / 317.6 us
    {4096, 4096, 14, 1, 1},   //  567.7 / 587.2   334.6 / 344.7   302.0 / 316.1 us
    {7168, 2304, 7, 0, 2},   //   25.0 /  30.3    25.6 /  28.0    37.7 /  40.0 us
    {7168, 2304, 7, 1, 2},   //   24.6 /  29.5    23.9 /  26.7    36.4 /  38.9 us
    {7168, 2304, 8, 0, 2},   //   24.9 /  30.0    24.9 /  28.5    39.8 /  41.6 us
    {7168, 2304, 8, 1, 2},   //   25.0 /  29.6    24.3 /  27.6    38.2 /  40.3 us
    {7168, 2304, 9, 0, 2},   //   34.2 /  40.5    30.2 /  32.4    57.2 /  59.6 us
    {7168, 2304, 9, 1, 2},   //   33.1 /  38.9    27.2 /  31.5    56.0 /  58.3 us
    {7168, 2304, 10, 0, 2},   //   48.5 /  62.0    42.3 /  50.7    68.0 /  69.5 us
    {7168, 2304, 10, 1, 2},   //   45.6 /  55.6    38.8 /  47.5    65.3 /  67.7 us
    {7168, 2304, 11, 0, 2},   //   89.2 /  98.0    63.1 /  67.2    98.6 /  98.3 us
    {7168, 2304, 11, 1, 2},   //   79.6 /  89.9    56.8 /  62.5    96.1 /  96.7 us
    {7168, 2304, 12, 0, 2},   //  172.5 / 169.4    98.5 / 104.4   120.3 / 120.7 us
    {7168, 2304, 12, 1, 2},   //  144.5 / 161.2    93.1 / 100.4   118.1 / 119.8 us
    {7168, 2304, 13, 0, 1},   //  319.2 / 321.7   187.3 / 194.5   168.2 / 171.4 us
    {7168, 2304, 13, 1, 1},   //  294.3 / 317.1   184.9 / 191.4   167.8 / 171.1 us
    {7168, 2304, 14, 0, 1},   //  622.5 / 618.1   365.4 / 370.1   299.2 / 305.3 us
    {7168, 2304, 14, 1, 1},   //  611.1 / 615.0   360.3 / 365.7   299.5 / 303.7 us
};

int grouped_table_variant(int G, int64_t totM, int64_t N, int64_t K, int pre) {
  if (G != 8 || totM <= 0) return -1;
  int log2m = 0;
  while ((1ll << log2m) < totM) ++log2m;          // nextPow2(totM) = 2^log2m
  for (const GroupedTile &t : GROUPED_TILES)
    if (t.N == N && t.K == K && t.log2m == log2m && t.pre == (pre != 0)) return t.variant;
  return -1;
}
}  // namespace

// Kernel choice from the static shapes (the host never reads m_sizes): the
// static table above when it lists the shape, else the estimated time of
// each kernel from upper bounds of the tile counts.
//  - persistent, 64 x 64 or 128 x 128 tiles (weight streaming): ~0.8 or
//    ~1.6 us per 128-K tile step per workgroup, GS_OCC workgroups per
//    compute unit walking all tile steps evenly (the 128 x 128 kernel at
//    least ~1.1 us per K step: a tile's time when its workgroup has the
//    compute unit to itself);
//  - persistent 256 x 256 tiles on the dense pipeline (matrix-core regime):
//    one tile per compute unit per round, ~1.67 us per 128-K step plus
//    ~20 us per round (pipeline start, epilogue); a partial last round that
//    goes to the streaming kernel (grouped_split_end) ~0.55 us per 128-K
//    step plus ~5 us per round of its pieces (one per compute unit);
// each at least the weights' bytes at ~5 TB/s.  The constants are fitted to
// the table's warm-plus-cold times; at 58 of its 64 points the estimate
// picks the table's kernel, and at the other 6 one within 12% of it.
namespace {
// Autotuned winners of the grouped GEMM, keyed as "Add FlyDSL grouped
// groupwise FP8 GEMM for ROCm" (Tile selection) keys its persisted cache:
// (nextPow2(totM), N, K, b_preshuffled), here with G as well, since the tile
// count depends on it.  Filled by grouped_fp8_gemm_autotune or a cache file;
// consulted before the static table.
typedef std::tuple<int, int, int64_t, int64_t, int> TuneKey;   // G, log2 nextPow2(totM), N, K, preshuffled
std::mutex tune_mutex;
std::map<TuneKey, int> tune_cache;

int ceil_log2(int64_t x) {
  int l = 0;
  while ((1ll << l) < x) ++l;
  return l;
}

TuneKey tune_key(int G, int64_t totM, int64_t N, int64_t K, int pre) {
  return TuneKey(G, ceil_log2(totM), N, K, pre != 0 ? 1 : 0);
}

bool valid_variant(int v) {
  return v == MXG_GROUPED_STREAM64 || v == MXG_GROUPED_TILED || v == MXG_GROUPED_STREAM128;
}
}  // namespace

namespace {
int grouped_model_variant(int G, int64_t totM, int64_t N, int64_t kbytes);
}  // namespace

extern "C" int grouped_fp8_gemm_variant(int G, int64_t totM, int64_t N, int64_t K, int b_preshuffled) {
  if (G < 1 || totM <= 0 || N <= 0 || K <= 0) return MXG_GROUPED_STREAM64;
  {
    std::lock_guard<std::mutex> lock(tune_mutex);
    const auto it = tune_cache.find(tune_key(G, totM, N, K, b_preshuffled));
    if (it != tune_cache.end()) return it->second;
  }
  const int listed = grouped_table_variant(G, totM, N, K, b_preshuffled);
  if (listed >= 0) return listed;
  return grouped_model_variant(G, totM, N, K);
}

namespace {
// The cost model of the grouped kernel choice (see above), for K given in
// bytes per row (FP8: K; BF16: 2K): every kernel's step is one 128-byte K
// chunk, and the weights stream G N kbytes bytes.
int grouped_model_variant(int G, int64_t totM, int64_t N, int64_t kbytes) {
  const int64_t K = kbytes;
  const double cus = cu_count(), nst = (double)(K / 128);
  const double wbytes = (double)G * (double)N * (double)K;
  const double wmin = wbytes / 5.0e6;
  const double slots = (double)GS_OCC * cus;
  const double t64 = std::max(0.8 * (double)(cdiv(totM, 64) + G - 1) * (double)(N / 64) * nst / slots, wmin);
  const double t128 = std::max(std::max(1.6 * (double)(cdiv(totM, 128) + G - 1) * (double)(N / 128) * nst / slots,
                                        1.1 * nst), wmin);
  const double tiles_d = (double)(cdiv(totM, DBM) + G - 1) * (double)cdiv(N, DBN);
  const double round_d = 1.67 * nst + 20.0;
  const double full = std::floor(tiles_d / cus), r = tiles_d - full * cus;
  double t_d = full * round_d;
  if (r > 0) {
    const double pieces = (16.0 * r <= cus ? 16.0 : 8.0) * r;   // grouped_tail_pieces
    const double pr = std::ceil(pieces / cus);                   // streaming rounds of them
    t_d += (full >= 1 && pr <= GROUPED_TAIL_ROUNDS) ? pr * (0.55 * nst + 5.0) : round_d;
  }
  t_d = std::max(t_d, wmin);
  if (t64 <= t128 && t64 <= t_d) return MXG_GROUPED_STREAM64;
  return t128 <= t_d ? MXG_GROUPED_STREAM128 : MXG_GROUPED_TILED;
}
}  // namespace

extern "C" int grouped_fp8_gemm_autotune(int G, const int64_t *m_sizes, const void *XQ, const float *x_scale,
                                         const void *WQ, const float *w_scale, void *D, int64_t totM,
                                         int64_t N, int64_t K, int b_preshuffled, int reps, int *variant_out,
                                         float *us_out, hipStream_t stream) {
  const int v = grouped_fp8_gemm_validate(G, m_sizes, XQ, x_scale, WQ, w_scale, D, totM, N, K,
                                          b_preshuffled);
  if (v != MXG_OK) return v;
  if (reps < 1 || reps > 1000) return MXG_ERR_INVALID_ARG;
  if (totM == 0 || N == 0 || K == 0) return MXG_ERR_INVALID_ARG;   // nothing to time
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(stream, &cap) != hipSuccess) return MXG_ERR_HIP;
  if (cap != hipStreamCaptureStatusNone) return MXG_ERR_INVALID_ARG;   // it waits on events
  const int variants[3] = {MXG_GROUPED_STREAM64, MXG_GROUPED_STREAM128, MXG_GROUPED_TILED};
  float us[3] = {0.f, 0.f, 0.f};
  hipEvent_t e0, e1;
  if (hipEventCreate(&e0) != hipSuccess) return MXG_ERR_HIP;
  if (hipEventCreate(&e1) != hipSuccess) {
    (void)hipEventDestroy(e0);
    return MXG_ERR_HIP;
  }
  int rc = MXG_OK;
  for (int i = 0; i < 3 && rc == MXG_OK; ++i) {
    // one untimed launch, then reps timed ones back to back
    rc = launch_grouped(variants[i], G, m_sizes, XQ, x_scale, WQ, w_scale, D, totM, N, K, b_preshuffled, stream);
    if (rc != MXG_OK) break;
    if (hipEventRecord(e0, stream) != hipSuccess) { rc = MXG_ERR_HIP; break; }
    for (int r = 0; r < reps && rc == MXG_OK; ++r)
      rc = launch_grouped(variants[i], G, m_sizes, XQ, x_scale, WQ, w_scale, D, totM, N, K, b_preshuffled, stream);
    if (rc != MXG_OK) break;
    float ms = 0.f;
    if (hipEventRecord(e1, stream) != hipSuccess || hipEventSynchronize(e1) != hipSuccess ||
        hipEventElapsedTime(&ms, e0, e1) != hipSuccess) {
      rc = MXG_ERR_HIP;
      break;
    }
    us[i] = ms * 1000.f / (float)reps;
  }
  (void)hipEventDestroy(e0);
  (void)hipEventDestroy(e1);
  if (rc != MXG_OK) return rc;
  int best = 0;
  for (int i = 1; i < 3; ++i)
    if (us[i] < us[best]) best = i;
  {
    std::lock_guard<std::mutex> lock(tune_mutex);
    tune_cache[tune_key(G, totM, N, K, b_preshuffled)] = variants[best];
  }
  if (variant_out) *variant_out = variants[best];
  if (us_out)
    for (int i = 0; i < 3; ++i) us_out[variants[i]] = us[i];
  return MXG_OK;
}

extern "C" int mxgemm_tune_cache_save(const char *path) {
  if (!path) return MXG_ERR_INVALID_ARG;
  FILE *f = fopen(path, "w");
  if (!f) return MXG_ERR_IO;
  bool ok = fprintf(f, "# grouped G log2(nextPow2(totM)) N K b_preshuffled variant\n") > 0;
  {
    std::lock_guard<std::mutex> lock(tune_mutex);
    for (const auto &kv : tune_cache)
      ok = ok && fprintf(f, "grouped %d %d %lld %lld %d %d\n", std::get<0>(kv.first), std::get<1>(kv.first),
                         (long long)std::get<2>(kv.first), (long long)std::get<3>(kv.first),
                         std::get<4>(kv.first), kv.second) > 0;
  }
  ok = (fclose(f) == 0) && ok;
  return ok ? MXG_OK : MXG_ERR_IO;
}

extern "C" int mxgemm_tune_cache_load(const char *path) {
  if (!path) return MXG_ERR_INVALID_ARG;
  FILE *f = fopen(path, "r");
  if (!f) return MXG_ERR_IO;
  std::map<TuneKey, int> entries;
  char line[256];
  bool ok = true;
  while (ok && fgets(line, sizeof line, f)) {
    if (line[0] == '#' || line[0] == '\n') continue;
    int G = 0, l2 = 0, pre = 0, var = 0;
    long long N = 0, K = 0;
    char tail = 0;
    const int n = sscanf(line, "grouped %d %d %lld %lld %d %d %c", &G, &l2, &N, &K, &pre, &var, &tail);
    ok = n == 6 && G >= 1 && G <= MXG_GROUPED_MAX_G && l2 >= 0 && l2 < 48 && N > 0 && K > 0 &&
         (pre == 0 || pre == 1) && valid_variant(var);
    if (ok) entries[TuneKey(G, l2, (int64_t)N, (int64_t)K, pre)] = var;
  }
  ok = ok && !ferror(f);
  fclose(f);
  if (!ok) return MXG_ERR_IO;
  std::lock_guard<std::mutex> lock(tune_mutex);
  for (const auto &kv : entries) tune_cache[kv.first] = kv.second;
  return MXG_OK;
}

extern "C" int mxgemm_tune_cache_clear(void) {
  std::lock_guard<std::mutex> lock(tune_mutex);
  tune_cache.clear();
  return MXG_OK;
}

extern "C" int64_t mxgemm_tune_cache_size(void) {
  std::lock_guard<std::mutex> lock(tune_mutex);
  return (int64_t)tune_cache.size();
}

extern "C" int64_t mxgemm_preshuffle_b_bytes(int fmtB, int64_t N, int64_t K) {
  const FmtInfo f = fmt_info(fmtB & ~MXG_PRESHUFFLED);
  if (!f.ok || N < 0 || K < 0 || K % 128 != 0) return -1;
  // Whole 256-row tiles (four column groups each), so that a dense tile on
  // the last columns finds all its column groups inside the buffer.
  const int64_t ncg = cdiv(N, 256) * 4, nks = K / 128;
  return ncg * nks * (f.elem == F_E2M1 ? 4096 : 8192);
}

extern "C" int mxgemm_preshuffle_b(int fmtB, int layout, const void *B, void *B_out, int64_t N, int64_t K,
                        hipStream_t stream) {
  const FmtInfo f = fmt_info(fmtB & ~MXG_PRESHUFFLED);
  if (!f.ok || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (layout != MXG_NT && layout != MXG_NN && layout != MXG_TN) return MXG_ERR_INVALID_ARG;
  const bool fp4 = f.elem == F_E2M1;
  const bool tb = layout != MXG_NT;   // B stored [K, N]
  if (K % (fp4 ? 256 : 128) != 0) return MXG_ERR_UNSUPPORTED;
  if (fp4 && tb) return MXG_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return MXG_OK;
  if (!B || !B_out) return MXG_ERR_INVALID_ARG;
  if (!aligned(B, 16) || !aligned(B_out, 16)) return MXG_ERR_MISALIGNED;
  const int64_t chunks = mxgemm_preshuffle_b_bytes(fmtB, N, K) / 16;
  const unsigned grid = (unsigned)cdiv(chunks, 256);
  if (fp4)
    hipLaunchKernelGGL((preshuffle_b_kernel<true, false>), dim3(grid), dim3(256), 0, stream,
                       (const uint8_t *)B, (uint8_t *)B_out, N, K, chunks);
  else if (tb)
    hipLaunchKernelGGL((preshuffle_b_kernel<false, true>), dim3(grid), dim3(256), 0, stream,
                       (const uint8_t *)B, (uint8_t *)B_out, N, K, chunks);
  else
    hipLaunchKernelGGL((preshuffle_b_kernel<false, false>), dim3(grid), dim3(256), 0, stream,
                       (const uint8_t *)B, (uint8_t *)B_out, N, K, chunks);
  return launch_status();
}

extern "C" int64_t mxgemm_preshuffle_scales_bytes(int64_t rows, int64_t K) {
  if (rows < 0 || K < 0 || K % 32 != 0) return -1;
  return cdiv(rows, 64) * cdiv(K, 512) * 1024;
}

extern "C" int mxgemm_preshuffle_scales(const void *s, void *s_out, int64_t rows, int64_t K,
                             hipStream_t stream) {
  if (rows < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (K % 32 != 0) return MXG_ERR_UNSUPPORTED;
  if (rows == 0 || K == 0) return MXG_OK;
  if (!s || !s_out) return MXG_ERR_INVALID_ARG;
  if (!aligned(s, 4) || !aligned(s_out, 16)) return MXG_ERR_MISALIGNED;
  const int64_t words = mxgemm_preshuffle_scales_bytes(rows, K) / 4;
  hipLaunchKernelGGL(preshuffle_scales_kernel, dim3((unsigned)cdiv(words, 256)), dim3(256), 0,
                     stream, (const uint8_t *)s, (uint32_t *)s_out, rows, K, words);
  return launch_status();
}

extern "C" int grouped_fp8_preshuffle_b(int G, const void *WQ, void *WQ_out, int64_t N, int64_t K,
                             hipStream_t stream) {
  if (G < 1 || G > MXG_GROUPED_MAX_G || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (N % 128 != 0 || K % 128 != 0) return MXG_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return MXG_OK;
  if (!WQ || !WQ_out) return MXG_ERR_INVALID_ARG;
  if (!aligned(WQ, 16) || !aligned(WQ_out, 16)) return MXG_ERR_MISALIGNED;
  // Each group's [N, K] block maps to a same-size preshuffled block; the
  // whole [G*N, K] stack is one B operand whose 16-row tiles never straddle
  // two groups (N % 16 == 0).
  const int64_t chunks = (int64_t)G * N * K / 16;
  hipLaunchKernelGGL((preshuffle_b_kernel<false, false>), dim3((unsigned)cdiv(chunks, 256)),
                     dim3(256), 0, stream, (const uint8_t *)WQ, (uint8_t *)WQ_out,
                     (int64_t)G * N, K, chunks);
  return launch_status();
}


extern "C" int grouped_bf16_gemm_validate(int G, const int64_t *m_sizes, const void *X, const void *W,
                                          const void *D, int64_t totM, int64_t N, int64_t K,
                                          int b_preshuffled) {
  (void)b_preshuffled;
  if (G < 1 || G > MXG_GROUPED_MAX_G) return MXG_ERR_UNSUPPORTED;
  if (totM < 0 || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (!m_sizes) return MXG_ERR_INVALID_ARG;
  if (N % 64 != 0 || K % 64 != 0) return MXG_ERR_UNSUPPORTED;
  if (totM >= MAX_DIM || N >= MAX_DIM || 2 * K > MAX_ROW_BYTES) return MXG_ERR_UNSUPPORTED;
  if (totM == 0 || N == 0) return MXG_OK;
  if (!D) return MXG_ERR_INVALID_ARG;
  if (!aligned(D, 16) || !aligned(m_sizes, 8)) return MXG_ERR_MISALIGNED;
  if (K == 0) return MXG_OK;
  if (!X || !W) return MXG_ERR_INVALID_ARG;
  if (!aligned(X, 16) || !aligned(W, 16)) return MXG_ERR_MISALIGNED;
  return MXG_OK;
}

extern "C" int grouped_bf16_gemm_run(int G, const int64_t *m_sizes, const void *X, const void *W, void *D,
                                     int64_t totM, int64_t N, int64_t K, int b_preshuffled,
                                     hipStream_t stream) {
  const int v = grouped_bf16_gemm_validate(G, m_sizes, X, W, D, totM, N, K, b_preshuffled);
  if (v != MXG_OK) return v;
  if (totM == 0 || N == 0) return MXG_OK;
  if (K == 0) {
    hipLaunchKernelGGL(grouped_zero_kernel, dim3((unsigned)cdiv(totM * N, 256)), dim3(256), 0,
                       stream, m_sizes, G, (uint16_t *)D, totM, N);
    return launch_status();
  }
  const int variant = grouped_bf16_gemm_variant(G, totM, N, K);
  const bool pre = b_preshuffled != 0;
  GroupedArgs a = {};
  a.m_sizes = m_sizes;
  a.XQ = (const uint8_t *)X;
  a.WQ = (const uint8_t *)W;
  a.D = (uint16_t *)D;
  a.totM = totM;
  a.N = N;
  a.K = K;
  a.G = G;
  if (variant != MXG_GROUPED_TILED) {
    // 64 x 64 or 128 x 128 tiles (128 x 64 when N is an odd multiple of 64)
    const int BM = variant == MXG_GROUPED_STREAM64 ? 64 : 128;
    const int BN = BM == 128 && N % 128 == 0 ? 128 : 64;
    a.tiles_n = (int)(N / BN);
    const int64_t blocks = (cdiv(totM, BM) + G - 1) * a.tiles_n;
    if (blocks > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
    const unsigned P = (unsigned)std::min<int64_t>(blocks, (int64_t)GS_OCC * cu_count());
    hipLaunchKernelGGL(pick_grouped_stream_bf16(BM, BN, pre), dim3(P), dim3(256), 0, stream, a);
    return launch_status();
  }
  // 256 x 256 tiles on the dense pipeline, one persistent workgroup per
  // compute unit, every group's rows cut into 256-row tiles; a partial last
  // round goes to the streaming kernel in pieces (grouped_split_end)
  DenseArgs d = {};
  d.A = (const uint8_t *)X;
  d.B = (const uint8_t *)W;
  d.D = (uint16_t *)D;
  d.M = totM;
  d.N = N;
  d.K = K;
  d.a_bytes = totM * K * 2;
  d.b_bytes = (int64_t)G * N * K * 2;
  d.tiles_n = (int)cdiv(N, DBN);
  d.tiles_m = (int)(cdiv(totM, DBM) + G - 1);      // upper bound; the kernel counts them
  d.m_sizes = m_sizes;
  d.G = G;
  const int64_t tiles = (int64_t)d.tiles_m * d.tiles_n;
  if (tiles > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, cu_count());
  const bool tail = tiles > (int64_t)grid;
  const unsigned tail_grid = (unsigned)cu_count();
  d.tail_grid = (int)tail_grid;
  d.tail_rounds = tail ? GROUPED_TAIL_ROUNDS : 0;
  hipLaunchKernelGGL(pick_grouped_bf16(pre), dim3(grid), dim3(DNW8 * 64), 0, stream, d);
  if (tail) {
    a.tiles_n = (int)(N / 64);
    a.tiles_nb = d.tiles_n;
    a.main_grid = (int)grid;
    a.tail_rounds = GROUPED_TAIL_ROUNDS;
    hipLaunchKernelGGL(pick_grouped_tail_bf16(pre), dim3(tail_grid), dim3(256), 0, stream, a);
  }
  return launch_status();
}

extern "C" int grouped_bf16_gemm_variant(int G, int64_t totM, int64_t N, int64_t K) {
  if (G < 1 || totM <= 0 || N <= 0 || K <= 0) return MXG_GROUPED_STREAM64;
  return grouped_model_variant(G, totM, N, 2 * K);
}

extern "C" int grouped_bf16_preshuffle_b(int G, const void *W, void *W_out, int64_t N, int64_t K,
                                         hipStream_t stream) {
  if (G < 1 || G > MXG_GROUPED_MAX_G || N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (N % 64 != 0 || K % 64 != 0) return MXG_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return MXG_OK;
  if (!W || !W_out) return MXG_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(W_out, 16)) return MXG_ERR_MISALIGNED;
  // The byte permutation of the 8-bit weights applied to each group's
  // [N, 2K] bytes: the layout is defined on 128-byte K chunks of 64-row
  // column groups, which is what the BF16 kernel reads.
  const int64_t chunks = (int64_t)G * N * (2 * K) / 16;
  hipLaunchKernelGGL((preshuffle_b_kernel<false, false>), dim3((unsigned)cdiv(chunks, 256)),
                     dim3(256), 0, stream, (const uint8_t *)W, (uint8_t *)W_out,
                     (int64_t)G * N, 2 * K, chunks);
  return launch_status();
}

extern "C" int mxgemm_mfma_ceiling(int fmt, int64_t iters, void *clk, hipStream_t stream) {
  const FmtInfo f = fmt_info(fmt);
  if (!f.ok || iters < 0 || !clk) return MXG_ERR_INVALID_ARG;
  if (!aligned(clk, 8)) return MXG_ERR_MISALIGNED;
  const unsigned grid = (unsigned)cu_count();
  if (f.elem == F_E2M1)
    hipLaunchKernelGGL((mfma_ceiling_kernel<F_E2M1>), dim3(grid), dim3(512), 0, stream, iters, (uint64_t *)clk);
  else
    hipLaunchKernelGGL((mfma_ceiling_kernel<F_E4M3>), dim3(grid), dim3(512), 0, stream, iters, (uint64_t *)clk);
  return launch_status();
}

extern "C" int mxgemm_quantize_mx(int fmt, const float *x, void *codes, void *scales, int64_t rows, int64_t K,
                                  hipStream_t stream) {
  const FmtInfo f = fmt_info(fmt);
  if (!f.ok || !f.mx || rows < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (K % 32 != 0) return MXG_ERR_UNSUPPORTED;
  if (rows == 0 || K == 0) return MXG_OK;
  if (!x || !codes || !scales) return MXG_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16)) return MXG_ERR_MISALIGNED;
  const int64_t n8 = rows * K / 8;
  const int64_t blocks = cdiv(n8, 256);
  if (rows >= MAX_DIM || K > MAX_ROW_BYTES || blocks > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
  const float *xf = x;
  uint8_t *c = (uint8_t *)codes, *s = (uint8_t *)scales;
  if (f.elem == F_E4M3)
    hipLaunchKernelGGL((quant_mx_kernel<F_E4M3>), dim3((unsigned)blocks), dim3(256), 0, stream, xf, c, s, n8);
  else if (f.elem == F_E5M2)
    hipLaunchKernelGGL((quant_mx_kernel<F_E5M2>), dim3((unsigned)blocks), dim3(256), 0, stream, xf, c, s, n8);
  else
    hipLaunchKernelGGL((quant_mx_kernel<F_E2M1>), dim3((unsigned)blocks), dim3(256), 0, stream, xf, c, s, n8);
  return launch_status();
}

extern "C" int mxgemm_quantize_tensor(int fmt, const float *x, void *codes, float *scale, int64_t n,
                                      hipStream_t stream) {
  const FmtInfo f = fmt_info(fmt);
  if (!f.ok || f.mx || n < 0 || !scale) return MXG_ERR_INVALID_ARG;
  if (n % 8 != 0) return MXG_ERR_UNSUPPORTED;
  if (n > 0 && (!x || !codes)) return MXG_ERR_INVALID_ARG;
  if ((n > 0 && (!aligned(x, 16) || !aligned(codes, 16))) || !aligned(scale, 4)) return MXG_ERR_MISALIGNED;
  const int64_t n8 = n / 8;
  const int64_t blocks = cdiv(n8, 256);
  if (blocks > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
  uint32_t *word = (uint32_t *)scale;
  uint8_t *c = (uint8_t *)codes;
  hipLaunchKernelGGL(tensor_amax_clear_kernel, dim3(1), dim3(64), 0, stream, word);
  if (n8 > 0) {
    const unsigned amax_blocks = (unsigned)std::min<int64_t>(blocks, (int64_t)8 * cu_count());
    hipLaunchKernelGGL(tensor_amax_kernel, dim3(amax_blocks), dim3(256), 0, stream, x, n8, word);
    if (f.elem == F_E4M3)
      hipLaunchKernelGGL((tensor_quant_kernel<F_E4M3>), dim3((unsigned)blocks), dim3(256), 0, stream, x, c,
                         (const uint32_t *)word, n8);
    else
      hipLaunchKernelGGL((tensor_quant_kernel<F_E5M2>), dim3((unsigned)blocks), dim3(256), 0, stream, x, c,
                         (const uint32_t *)word, n8);
  }
  if (f.elem == F_E4M3) hipLaunchKernelGGL((tensor_scale_kernel<F_E4M3>), dim3(1), dim3(64), 0, stream, word);
  else hipLaunchKernelGGL((tensor_scale_kernel<F_E5M2>), dim3(1), dim3(64), 0, stream, word);
  return launch_status();
}

static_assert(QG_MAX == MXG_GROUPED_MAX_G, "group table of the activation quantizer");
static_assert(ACT_NONE == MXG_ACT_NONE && ACT_RELU == MXG_ACT_RELU && ACT_GELU_TANH == MXG_ACT_GELU_TANH &&
                  ACT_SILU == MXG_ACT_SILU,
              "activation codes");

extern "C" int grouped_fp8_quantize_act(int G, const int64_t *m_sizes, const float *x, void *codes,
                                        float *x_scale, int64_t totM, int64_t K, hipStream_t stream) {
  if (G < 1 || G > MXG_GROUPED_MAX_G) return MXG_ERR_UNSUPPORTED;
  if (totM < 0 || K < 0 || !m_sizes) return MXG_ERR_INVALID_ARG;
  if (K % 128 != 0) return MXG_ERR_UNSUPPORTED;
  if (totM >= MAX_DIM || K > MAX_ROW_BYTES || totM * (K / 128) * 4 >= (1ll << 31)) return MXG_ERR_UNSUPPORTED;
  if (totM == 0 || K == 0) return MXG_OK;
  if (!x || !codes || !x_scale) return MXG_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(x_scale, 4) || !aligned(m_sizes, 8))
    return MXG_ERR_MISALIGNED;
  const int64_t nblk = totM * (K / 128);
  const unsigned grid = (unsigned)std::min<int64_t>(cdiv(nblk, 16), 8ll * cu_count());
  hipLaunchKernelGGL(quant_group_act_kernel, dim3(grid), dim3(256), 0, stream, m_sizes, G, x,
                     (uint8_t *)codes, x_scale, totM, K);
  return launch_status();
}

extern "C" int grouped_fp8_quantize_weight(int G, const float *w, void *codes, float *w_scale, int64_t N, int64_t K,
                                           hipStream_t stream) {
  if (G < 1 || G > MXG_GROUPED_MAX_G) return MXG_ERR_UNSUPPORTED;
  if (N < 0 || K < 0) return MXG_ERR_INVALID_ARG;
  if (N % 128 != 0 || K % 128 != 0) return MXG_ERR_UNSUPPORTED;
  if (N >= MAX_DIM || K > MAX_ROW_BYTES) return MXG_ERR_UNSUPPORTED;
  if (N == 0 || K == 0) return MXG_OK;
  if (!w || !codes || !w_scale) return MXG_ERR_INVALID_ARG;
  if (!aligned(w, 16) || !aligned(codes, 4) || !aligned(w_scale, 4)) return MXG_ERR_MISALIGNED;
  const int64_t blocks = (int64_t)G * (N / 128) * (K / 128);
  if (blocks > 0x7FFFFFFF) return MXG_ERR_UNSUPPORTED;
  hipLaunchKernelGGL(quant_group_weight_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, w, (uint8_t *)codes,
                     w_scale, N, K);
  return launch_status();
}
