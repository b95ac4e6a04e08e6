// Dense NT GEMM for few rows, MX and tensor-wise formats, with the residual
// epilogue (mxgemm_run_residual): BM = 16 FM rows x BN = 16 FN columns per
// workgroup of W waves that split K between them, step st of 128 K to wave st %
// W.  Operands go from memory straight to registers in the scaled matrix-core
// instruction's order, U steps ahead, through range-checked loads (rows past M
// or N read zeros); nothing is shared between waves but the final sum, in
// LDS, in a fixed order.  A weight is read once, so this is a stream of B
// wherever M is small; the 64 x 64 tiles of small.hpp leave most compute units
// idle there and walk all of K in every wave.
#pragma once
#include "small.hpp"

namespace mxg {

constexpr int ROWS_WAVES = 8;

template <int FA, int FB, int SMODE, bool PSB, int FM, int FN, int U>
__global__ __launch_bounds__(64 * ROWS_WAVES) void dense_rows_kernel(DenseArgs p) {
  constexpr bool FP4 = FA == F_E2M1, MX = SMODE == SM_MX;
  constexpr int W = ROWS_WAVES, BM = 16 * FM, BN = 16 * FN;
  __shared__ v4f part[W][FM * FN][64];
  const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tn = (int)blockIdx.x / p.tiles_m, tm = (int)blockIdx.x - tn * p.tiles_m;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int64_t KB = FP4 ? p.K / 2 : p.K, sk = p.K / 32;
  const int nst = (int)(p.K / 128);
  constexpr int PS = FP4 ? 64 : 128;               // bytes per K step and row

  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + m0 * KB, clamp_records(p.a_bytes - m0 * KB));
  // preshuffled B: column groups of 64 rows, 16 of them (a subtile) in each
  // 1 KiB (FP8: 2 KiB) piece of a K step; the tile is inside one group
  constexpr int CG = FP4 ? 4096 : 8192;
  const int64_t bbase = PSB ? n0 / 64 * nst * CG + (n0 % 64) / 16 * (CG / 4) : n0 * KB;
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B + bbase, clamp_records(p.b_bytes - bbase));
  __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.A, 0), rsb = make_rsrc(p.A, 0);
  if constexpr (MX) {
    rsa = make_rsrc((const uint8_t *)p.sA + m0 * sk, clamp_records(p.sa_bytes - m0 * sk));
    const int64_t sbb = PSB ? n0 / 64 * ((p.K + 511) / 512) * 1024 + (n0 % 64) / 16 * 256 : n0 * sk;
    rsb = make_rsrc((const uint8_t *)p.sB + sbb, clamp_records(p.sb_bytes - sbb));
  }
  auto load16 = [&](__amdgpu_buffer_rsrc_t r, uint32_t o) {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, (int)o, 0, 0));
  };
  auto frag = [&](__amdgpu_buffer_rsrc_t r, uint32_t o, uint32_t second) -> v8i {
    const v4i lo = load16(r, o);
    if constexpr (FP4) return __builtin_shufflevector(lo, lo, 0, 1, 2, 3, -1, -1, -1, -1);
    const v4i hi = load16(r, o + second);
    return (v8i){lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  };

  v8i fa[U][FM], fb[U][FN];
  uint32_t sa[U][FM], sb[U][FN];
  auto load = [&](int s, int st) {
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      if constexpr (PSB) fb[s][b] = frag(rb, (uint32_t)(st * CG + b * (CG / 4) + lane * 16), 1024u);
      else fb[s][b] = frag(rb, (uint32_t)((16 * b + i16) * KB + (int64_t)st * PS + 16 * q), 64u);
      if constexpr (MX)
        sb[s][b] = buf_load_u32(rsb, PSB ? (uint32_t)((st >> 2) * 1024 + b * 256 + lane * 4)
                                         : (uint32_t)((16 * b + i16) * sk + 4 * st));
    }
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      fa[s][a] = frag(ra, (uint32_t)((16 * a + i16) * KB + (int64_t)st * PS + 16 * q), 64u);
      if constexpr (MX) sa[s][a] = buf_load_u32(rsa, (uint32_t)((16 * a + i16) * sk + 4 * st));
    }
  };
  v4f acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = (v4f){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < U; ++s)
    if (w + s * W < nst) load(s, w + s * W);
  for (int st = w; st < nst; st += U * W) {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int k = st + s * W;
      if (k < nst) {
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
          for (int b = 0; b < FN; ++b) {
            // lane (i, q) uses 32-K block q of its row; preshuffled words hold
            // four K steps of that block
            const int ea = MX ? (int)(sa[s][a] >> (8 * q)) : E8M0_ONE_X4;
            const int eb = MX ? (int)(sb[s][b] >> (8 * (PSB ? k & 3 : q))) : E8M0_ONE_X4;
            acc[a][b] = mfma_scaled<FB, FA>(fb[s][b], fa[s][a], acc[a][b], eb, ea);
          }
        if (k + U * W < nst) load(s, k + U * W);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) part[w][a * FN + b][lane] = acc[a][b];
  __syncthreads();
  float alpha = 1.0f;
  if constexpr (SMODE == SM_TENSOR) alpha = *(const float *)p.sA * *(const float *)p.sB;
  for (int f = w; f < FM * FN; f += W) {
    const int64_t r = m0 + 16 * (f / FN) + i16, col = n0 + 16 * (f % FN) + 4 * q;
    if (r >= p.M || col >= p.N) continue;
    const int64_t o = r * p.N + col, room = p.N - col;
    const bool wide = (p.N & 3) == 0;
    v4f near = {0.f, 0.f, 0.f, 0.f}, bias = {0.f, 0.f, 0.f, 0.f};
    if (p.R) near = load_bf16x4(p.R + o, room, wide);
    if (p.bias) bias = load_bf16x4(p.bias + col, room, false);
    v4f v = part[0][f][lane];
#pragma unroll
    for (int k = 1; k < W; ++k) v += part[k][f][lane];
    if constexpr (SMODE == SM_TENSOR) v = v * alpha;
    v += bias;
    if (p.Z) store_bf16x4(p.Z + o, v, room, wide);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = activate_select(p.act, v[k]);
    store_bf16x4(p.D + o, v + near, room, wide);
  }
}

}  // namespace mxg
