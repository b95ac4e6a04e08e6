// Dense NT GEMM for few rows or columns (or few tiles), MX and tensor-wise formats, with the
// residual epilogue (mxgemm_run_residual): AR rows x 16 FN columns per workgroup
// of W waves that split K between them; their sums meet in LDS in a fixed order.
// The 64 x 64 tiles of small.hpp leave most compute units idle there and walk
// all of K in every wave.
//
// Operands and scales come by DMA through a ring of U stages in LDS per wave:
// a DMA of 1 KiB takes eight rows' 128-byte lines whole, where loads in the
// matrix instruction's order take sixteen rows' halves, which a compute unit's
// cache path serves at a fraction of the rate (1 x 4096 x 14336 MXFP8, cold: 12.4 us, 17.0
// with such loads four steps ahead, 95 in the 64 x 64 kernel; 48 x 8192 x 8192 MXFP4: 12.9,
// 18.6, 36.7).  A stage is one 128-byte unit of K: AR rows of A (8 suffice
// for M <= 8), 16 FN of B and their scales; every wave has a range of units of its
// own, so that no barrier is needed but the last.  DMAs per stage are constant, so that
// the counter of outstanding ones tells which stages have landed: stages past
// the range's end are asked for past the end of the resources, which reads
// nothing.  A row past M or N is zeros.
#pragma once
#include "small.hpp"

namespace mxg {

// The waves' sums of a tile of at most `rows` rows, in their order, through the epilogue.
template <int SMODE, int FM, int FN, int W>
__device__ inline void rows_finish(const DenseArgs &p, v4f (*part)[FM * FN][64], const v4f (&acc)[FM][FN], int64_t m0,
                                   int64_t n0, int rows) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) part[w][a * FN + b][lane] = acc[a][b];
  __syncthreads();
  float alpha = 1.0f;
  if constexpr (SMODE == SM_TENSOR) alpha = *(const float *)p.sA * *(const float *)p.sB;
  for (int f = w; f < FM * FN; f += W) {
    const int in = 16 * (f / FN) + i16;
    const int64_t r = m0 + in, col = n0 + 16 * (f % FN) + 4 * q;
    if (in >= rows || r >= p.M || col >= p.N) continue;
    const int64_t o = r * p.N + col, room = p.N - col;
    v4f near = {0.f, 0.f, 0.f, 0.f}, bias = {0.f, 0.f, 0.f, 0.f};
    if (p.R) near = load_bf16x4(p.R + o, room);
    if (p.bias) bias = load_bf16x4(p.bias + col, room);
    v4f v = part[0][f][lane];
#pragma unroll
    for (int k = 1; k < W; ++k) v += part[k][f][lane];
    if constexpr (SMODE == SM_TENSOR) v = v * alpha;
    v += bias;
    if (p.Z) store_bf16x4(p.Z + o, v, room);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = activate_select(p.act, v[k]);
    store_bf16x4(p.D + o, v + near, room);
  }
}

template <int FA, int FB, int SMODE, bool PSB, int AR, int FN, int W, int U>
__global__ __launch_bounds__(64 * W) void dense_rows_kernel(DenseArgs p) {
  constexpr bool FP4 = FA == F_E2M1, MX = SMODE == SM_MX;
  constexpr int FM = (AR + 15) / 16, BM = AR, BN = 16 * FN, STEPS = FP4 ? 2 : 1;    // K steps of 128 per unit
  constexpr int SWA = AR * STEPS, SIA = MX ? (SWA + 63) / 64 : 0;                   // scale words of A, DMAs
  constexpr int SWB = BN * STEPS, SIB = !MX ? 0 : PSB ? FN : (SWB + 63) / 64;
  constexpr int A_OFF = 0, B_OFF = AR * 128, SA_OFF = B_OFF + BN * 128, SB_OFF = SA_OFF + SIA * 256;
  constexpr int STAGE = SB_OFF + SIB * 256, RING = U * STAGE;
  constexpr int DMAS = AR / 8 + 2 * FN + SIA + SIB;
  static_assert((U - 2) * DMAS < 64 && W * RING >= W * FM * FN * 1024, "ring");
  constexpr uint32_t NOWHERE = 0x80000000u;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[W * RING];
  const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tn = (int)blockIdx.x / p.tiles_m, tm = (int)blockIdx.x - tn * p.tiles_m;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const uint32_t KB = (uint32_t)(FP4 ? p.K / 2 : p.K), sk = (uint32_t)(p.K / 32);
  const int units = (int)(KB / 128), nst = (int)(p.K / 128);
  const int lo = units * w / W, hi = units * (w + 1) / W;

  const u32x4 ra = rsrc4(p.A + m0 * KB, clamp_records(p.a_bytes - m0 * KB));
  // preshuffled B: column groups of 64 rows, 16 of them (a subtile) in each
  // quarter of a K step; the tile is inside one group or begins one
  constexpr int CG = FP4 ? 4096 : 8192;
  const int64_t bbase = PSB ? n0 / 64 * nst * CG + (n0 % 64) / 16 * (CG / 4) : n0 * KB;
  const u32x4 rb = rsrc4(p.B + bbase, clamp_records(p.b_bytes - bbase));
  u32x4 rsa = rsrc4(p.A, 0), rsb = rsa;
  if constexpr (MX) {
    rsa = rsrc4((const uint8_t *)p.sA + m0 * sk, clamp_records(p.sa_bytes - m0 * sk));
    const int64_t sbb = PSB ? n0 / 64 * ((p.K + 511) / 512) * 1024 + (n0 % 64) / 16 * 256 : n0 * sk;
    rsb = rsrc4((const uint8_t *)p.sB + sbb, clamp_records(p.sb_bytes - sbb));
  }
  uint8_t *ring = smem + w * RING;
  const uint32_t lds0 = lds_addr(smem) + (uint32_t)w * RING;
  const int r8 = lane >> 3;
  const uint32_t vo = (uint32_t)r8 * KB + 16u * ((lane & 7) ^ kswz(r8));
  const uint32_t vsa = (uint32_t)(lane / STEPS) * sk + 4u * (lane % STEPS);
  auto issue = [&](int sl, int u) {
    const uint32_t st = lds0 + (uint32_t)sl * STAGE;
    const bool live = u < hi;
    const uint32_t x = live ? (uint32_t)u : 0u, v = live ? vo : NOWHERE;
    static_for<0, AR / 8>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      dma_asm_v<16, A_OFF + j * 1024>(st, ra, v, 128u * x + 8u * j * KB);
    });
    static_for<0, 2 * FN>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      if constexpr (PSB) {
        // FP8: halves of a K step's subtile; E2M1: the subtile of two K steps
        const uint32_t o = FP4 ? (2u * x + (j & 1)) * CG + (j >> 1) * (CG / 4) : x * CG + (j >> 1) * (CG / 4) + (j & 1) * 1024u;
        dma_asm_v<16, B_OFF + j * 1024>(st, rb, live ? 16u * lane : NOWHERE, o);
      } else {
        dma_asm_v<16, B_OFF + j * 1024>(st, rb, v, 128u * x + 8u * j * KB);
      }
    });
    static_for<0, SIA>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      const bool in = live && 64 * j + lane < SWA;
      dma_asm_v<4, SA_OFF + j * 256>(st, rsa, in ? vsa : NOWHERE, 4u * STEPS * x + (64u / STEPS) * j * sk);
    });
    static_for<0, SIB>([&](auto jc) {
      constexpr int j = decltype(jc)::value;
      if constexpr (PSB) {
        dma_asm_v<4, SB_OFF + j * 256>(st, rsb, live ? 4u * lane : NOWHERE, (STEPS * x >> 2) * 1024u + 256u * j);
      } else {
        const bool in = live && 64 * j + lane < SWB;
        dma_asm_v<4, SB_OFF + j * 256>(st, rsb, in ? vsa : NOWHERE, 4u * STEPS * x + (64u / STEPS) * j * sk);
      }
    });
  };
  v4f acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = (v4f){0.f, 0.f, 0.f, 0.f};
  const uint32_t o0 = (uint32_t)((q ^ kswz(i16)) << 4), o1 = (uint32_t)(((q + 4) ^ kswz(i16)) << 4);
#pragma unroll
  for (int k = 0; k < U - 1; ++k) issue(k, lo + k);
  int sl = 0;
  for (int u = lo; u < hi; ++u) {
    constexpr int N = (U - 2) * DMAS;
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(sl == 0 ? U - 1 : sl - 1, u + U - 1);
    const uint8_t *st = ring + sl * STAGE;
    v4i fa[FM][2], fb[FN][2];
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      const uint8_t *row = st + A_OFF + (AR < 16 ? i16 & (AR - 1) : 16 * a + i16) * 128;
      fa[a][0] = lds_read16(row + o0);
      fa[a][1] = lds_read16(row + o1);
    }
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      if constexpr (PSB) {
        fb[b][0] = lds_read16(st + B_OFF + b * 2048 + lane * 16);
        fb[b][1] = lds_read16(st + B_OFF + b * 2048 + 1024 + lane * 16);
      } else {
        const uint8_t *row = st + B_OFF + (16 * b + i16) * 128;
        fb[b][0] = lds_read16(row + o0);
        fb[b][1] = lds_read16(row + o1);
      }
    }
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      int ea[FM], eb[FN];
#pragma unroll
      for (int a = 0; a < FM; ++a)
        ea[a] = MX ? (int)(lds_load_u32(st + SA_OFF + 4 * ((AR < 16 ? i16 & (AR - 1) : 16 * a + i16) * STEPS + s)) >> (8 * q)) : E8M0_ONE_X4;
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        if constexpr (!MX) eb[b] = E8M0_ONE_X4;
        else if constexpr (PSB) eb[b] = (int)(lds_load_u32(st + SB_OFF + 256 * b + 4 * lane) >> (8 * ((STEPS * u + s) & 3)));
        else eb[b] = (int)(lds_load_u32(st + SB_OFF + 4 * ((16 * b + i16) * STEPS + s)) >> (8 * q));
      }
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b) {
          v8i x, y;
          if constexpr (FP4) {
            x = __builtin_shufflevector(fb[b][s], fb[b][s], 0, 1, 2, 3, -1, -1, -1, -1);
            y = __builtin_shufflevector(fa[a][s], fa[a][s], 0, 1, 2, 3, -1, -1, -1, -1);
          } else {
            x = __builtin_shufflevector(fb[b][0], fb[b][1], 0, 1, 2, 3, 4, 5, 6, 7);
            y = __builtin_shufflevector(fa[a][0], fa[a][1], 0, 1, 2, 3, 4, 5, 6, 7);
          }
          acc[a][b] = mfma_scaled<FB, FA>(x, y, acc[a][b], eb[b], ea[a]);
        }
    }
    sl = sl == U - 1 ? 0 : sl + 1;
  }
  wait_vmem_le<0>();
  __syncthreads();
  rows_finish<SMODE, FM, FN, W>(p, (v4f(*)[FM * FN][64])smem, acc, m0, n0, BM);
}

}  // namespace mxg
