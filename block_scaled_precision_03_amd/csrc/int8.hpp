// 8-bit integer GEMM for gfx950, dense and grouped by expert:
//   D[m,n] = act( sA[m] sB[n] sum_k A[m,k] B[n,k] + bias[n] )
// with signed 8-bit operands, both K-contiguous, exact 32-bit integer sums
// on the matrix cores (v_mfma_i32_16x16x64_i8), FP32 scales per row of A and
// per row of B, BF16 output.
//
// Every kernel below computes the grouped product; a dense call is the one
// group of all M rows (m_sizes null).  Integer sums do not depend on their
// order, so the kernels give the same bits however they cut M, N and K.
//
// K is any multiple of 16.  A K step is 128 bytes of every row; in the last,
// partial one the 16-byte pieces past K are read from past the end of the
// operand A's resource, which gives zeros, so whatever B holds there adds
// nothing.
#pragma once
#include "grouped.hpp"

namespace mxg {

struct Int8Args {
  const uint8_t *A, *B;
  const float *sA, *sB;           // [M], [G, N]
  const uint16_t *bias;           // BF16 [N] or null (dense calls only)
  const int64_t *m_sizes;         // null: one group of M rows
  uint16_t *D;                    // [M, No], No = N or (SwiGLU) N / 2
  int64_t M, N, K, No;
  int G, act, tiles_n;
  const uint16_t *R;              // RES kernels: BF16 [M, No] added after the activation, or null
  uint16_t *Z;                    // RES kernels: the activation's argument in BF16 [M, N], or null
};

// D += the 16x16x64 block of signed bytes: lane (i = lane % 16, q = lane / 16)
// holds bytes 16 q .. 16 q + 15 of row i of either operand; the result lane
// holds rows 4 q .. 4 q + 3 of the first operand and row i of the second.
__device__ inline v4i mfma_i8(const v4i &x, const v4i &y, const v4i &c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
}

// Four columns of a row: scale, bias, activation, all in FP32.  The integer
// sum is rounded to FP32 once (it may have up to 31 bits).
__device__ inline v4f int8_finish(const v4i &acc, float sa, const v4f &sb, const v4f &bias, int act) {
  v4f v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = fmaf((float)acc[k] * sa, sb[k], bias[k]);
  if (act != ACT_NONE && act != ACT_SWIGLU) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = activate(act, v[k]);
  }
  return v;
}

// SwiGLU of two interleaved (gate, up) pairs, packed.
__device__ inline uint32_t swiglu_pack(const v4f &v) {
  return pack_bf16x2(v.x * logistic_f32(v.x) * v.y, v.z * logistic_f32(v.z) * v.w);
}

// The group table of a call (see GroupTable): a dense call is one group.
template <int BM>
__device__ inline void int8_group_table(const Int8Args &p, GroupTable &gt, int lane) {
  if (p.m_sizes) {
    build_group_table<BM>(p.m_sizes, p.G, p.M, gt, lane);
  } else if (lane == 0) {
    gt.rows[0] = 0;
    gt.rows[1] = (int32_t)p.M;
    gt.mtile[0] = 0;
    gt.mtile[1] = (int32_t)((p.M + BM - 1) / BM);
  }
}

__device__ inline v4f unpack_bf16x4(const v2i &w) {
  return (v4f){__uint_as_float((uint32_t)w.x << 16), __uint_as_float((uint32_t)w.x & 0xFFFF0000u),
               __uint_as_float((uint32_t)w.y << 16), __uint_as_float((uint32_t)w.y & 0xFFFF0000u)};
}

// Four consecutive output columns (SwiGLU: two) of one row, from column col
// (a multiple of 4) of the product, in one store at whatever alignment an odd
// row pitch leaves (the hardware takes any).  v is the finished result.
__device__ inline void int8_store4(const Int8Args &p, int act, int64_t row, int64_t col, const v4f &v) {
  if (act == ACT_SWIGLU) {
    const int64_t oc = col >> 1;
    uint16_t *dst = p.D + row * p.No + oc;
    const uint32_t u = swiglu_pack(v);
    if (oc + 2 <= p.No) __builtin_memcpy(dst, &u, 4);
    else if (oc < p.No) dst[0] = (uint16_t)u;
    return;
  }
  uint16_t *dst = p.D + row * p.No + col;
  const uint32_t u[2] = {pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
  if (col + 4 <= p.No) {
    __builtin_memcpy(dst, u, 8);
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (col + k < p.No) dst[k] = (uint16_t)(u[k >> 1] >> (16 * (k & 1)));
  }
}

// The residual beside four consecutive columns of the product (SwiGLU: two of
// D), packed, at any alignment; zeros past the row's end and without one.
__device__ inline v2i int8_near(const Int8Args &p, int act, int64_t row, int64_t col) {
  uint32_t u[2] = {0, 0};
  if (p.R) {
    const bool gated = act == ACT_SWIGLU;
    const int64_t oc = gated ? col >> 1 : col, room = p.No - oc;
    const uint16_t *src = p.R + row * p.No + oc;
    if (gated && room >= 2) {
      __builtin_memcpy(u, src, 4);
    } else if (!gated && room >= 4) {
      __builtin_memcpy(u, src, 8);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < room && (k < 2 || !gated)) u[k >> 1] |= (uint32_t)src[k] << (16 * (k & 1));
    }
  }
  return (v2i){(int)u[0], (int)u[1]};
}

// Four consecutive columns of the product, scaled and biased but not
// activated, to what the call returns; RES: the activation's argument too,
// and the residual added.
template <bool RES>
__device__ inline void int8_emit4(const Int8Args &p, int act, int64_t row, int64_t col, v4f z, const v2i &near) {
  if constexpr (RES) {
    if (p.Z) {
      uint16_t *dst = p.Z + row * p.N + col;
      const uint32_t u[2] = {pack_bf16x2(z.x, z.y), pack_bf16x2(z.z, z.w)};
      if (col + 4 <= p.N) {
        __builtin_memcpy(dst, u, 8);
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (col + k < p.N) dst[k] = (uint16_t)(u[k >> 1] >> (16 * (k & 1)));
      }
    }
    const v4f r = unpack_bf16x4(near);
    if (act == ACT_SWIGLU) {
      const int64_t oc = col >> 1;
      uint16_t *dst = p.D + row * p.No + oc;
      const uint32_t u = pack_bf16x2(z.x * logistic_f32(z.x) * z.y + r.x, z.z * logistic_f32(z.z) * z.w + r.y);
      if (oc + 2 <= p.No) __builtin_memcpy(dst, &u, 4);
      else if (oc < p.No) dst[0] = (uint16_t)u;
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = activate(act, z[k]) + r[k];
    int8_store4(p, ACT_NONE, row, col, z);
  } else {
    if (act != ACT_NONE && act != ACT_SWIGLU) {
#pragma unroll
      for (int k = 0; k < 4; ++k) z[k] = activate(act, z[k]);
    }
    int8_store4(p, act, row, col, z);
  }
}

// The FP32 channel scales and biases of the four consecutive columns n0 + c
// .. from memory (n0 uniform; columns past N read 0, their results are never
// stored), by range-checked loads: with a branch per column their latencies
// add up.
__device__ inline void int8_columns(const Int8Args &p, int g, int64_t n0, int c, v4f &sb, v4f &bias) {
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.sB + (int64_t)g * p.N + n0, clamp_records(4 * (p.N - n0)));
  const __amdgpu_buffer_rsrc_t rb = p.bias ? make_rsrc(p.bias + n0, clamp_records(2 * (p.N - n0))) : make_rsrc(p.D, 0);
  sb = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rs, 4 * c, 0, 0));
  bias = unpack_bf16x4(__builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(rb, 2 * c, 0, 0)));
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles, the matrix-core regime.  Eight waves in a 2 x 4 grid, 128
// x 64 per wave (8 x 4 matrix-core tiles, 128 integer accumulators), two LDS
// stages of 128 bytes of K filled by DMA from waves 4-7 (each SIMD then has
// one wave that starts on the matrix cores right after the barrier while its
// other wave queues the DMAs), a persistent grid whose tiles share one K
// pipeline (an odd count of K steps drains it at the end of every tile: no
// slower, 16384 x 14336 takes 24.2 us per 128 of K with 31, 32 and 33 steps), and
// a finished tile stored during the next tile's first K step: the schedule that
// the block-scaled kernels measured best.
// The tile's 256 row scales, 256 channel scales and 256 biases come into LDS
// with its first stage, in two slots by the tile's parity.  16384 x 14336 x 4096
// takes 735 to 790 us from run to run, 2.4 to 2.6 POP/s, about half of the
// matrix cores' peak.  A K step moves 64 KB into and 192 KB out of a compute
// unit's LDS: 2048 clocks at 128 bytes a clock, as long as its matrix cores take
// for the step, and the two overlap in part.
// The activation is a template argument: as a switch on a kernel argument,
// repeated for each of the tile's 128 accumulators, it made 34 K instructions
// with 216 scratch accesses (5.1 ms for M = 16384, N = 14336, K = 4096).
template <int ACT, bool RES>
struct Int8Loop {
  static constexpr bool SWIGLU = ACT == ACT_SWIGLU;
  static constexpr int FM = 8, FN = 4;
  static constexpr int AB = DBM * 128;                     // bytes of one operand's stage
  static constexpr int B_REG = 2 * AB, S_REG = 4 * AB;
  static constexpr int SB_OFF = 1024, BIAS_OFF = 2048, SCALES = 2560;
  static constexpr int LDS_BYTES = S_REG + 2 * SCALES;
  static constexpr int EPI_STORES = SWIGLU ? FM : 2 * FM;  // stores of a full tile per wave

  struct Ctx {
    const Int8Args *p;
    int lane, w, wm, wn, i16, q, nst;
    uint32_t vo, vo_tail;          // row-tile DMA lane offsets; of A's last K step
    uint32_t lds0;
  };
  struct Tile {
    int64_t m0, n0, lim;
    u32x4 ra, rb;
    int g, slot;
  };

  __device__ static inline void init(Ctx &c, const Int8Args &p, uint8_t *smem) {
    c.p = &p;
    c.lane = threadIdx.x & 63;
    c.w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    c.wm = c.w >> 2;
    c.wn = c.w & 3;
    c.i16 = c.lane & 15;
    c.q = c.lane >> 4;
    c.nst = (int)((p.K + 127) / 128);
    const int rem = (int)(p.K - 128 * (int64_t)(c.nst - 1));
    const int r8 = c.lane >> 3, piece = (c.lane & 7) ^ kswz(r8);
    c.vo = (uint32_t)(r8 * p.K) + (uint32_t)(piece << 4);
    c.vo_tail = 16 * piece < rem ? c.vo : 0x80000000u;     // past any resource: zeros
    c.lds0 = lds_addr(smem);
  }

  __device__ static inline void set_tile(const Ctx &c, const TileId &id, int slot, Tile &t) {
    const Int8Args &p = *c.p;
    t.m0 = id.m0;
    t.n0 = id.n0;
    t.lim = id.lim;
    t.g = id.g;
    t.slot = slot;
    const int64_t abase = id.m0 * p.K, bbase = ((int64_t)id.g * p.N + id.n0) * p.K;
    t.ra = rsrc4(p.A + abase, clamp_records(p.M * p.K - abase));
    t.rb = rsrc4(p.B + bbase, clamp_records((int64_t)p.G * p.N * p.K - bbase));
  }

  // Stage st of tile t into ring slot si.  Waves 4-7: wave 4 + v rows 64 v ..
  // 64 v + 63 of A and of B, eight 1 KiB DMAs each.  With the first stage
  // waves 0-3 bring the tile's scales and biases.
  __device__ static inline void issue(const Ctx &c, const Tile &t, int st, int si) {
    const Int8Args &p = *c.p;
    if (c.w >= 4) {
      const uint32_t dst = c.lds0 + (uint32_t)si * AB + (uint32_t)(c.w - 4) * 8192u;
      const uint32_t va = st == c.nst - 1 ? c.vo_tail : c.vo;
      const uint32_t row0 = (uint32_t)((c.w - 4) * 64);
      static_for<0, 8>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        dma_asm_v<16, j * 1024>(dst, t.ra, va, (uint32_t)((row0 + j * 8) * p.K + 128 * (int64_t)st));
      });
      static_for<0, 8>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        dma_asm_v<16, j * 1024>(dst + B_REG, t.rb, c.vo, (uint32_t)((row0 + j * 8) * p.K + 128 * (int64_t)st));
      });
    } else if (st == 0) {
      const uint32_t dst = c.lds0 + S_REG + (uint32_t)t.slot * SCALES + (uint32_t)c.w * 256u;
      const int64_t nb = (int64_t)t.g * p.N + t.n0;
      dma_asm_v<4>(dst, rsrc4(p.sA + t.m0, clamp_records(4 * (p.M - t.m0))), (uint32_t)(c.lane * 4),
                   (uint32_t)c.w * 256u);
      dma_asm_v<4, SB_OFF>(dst, rsrc4(p.sB + nb, clamp_records(4 * ((int64_t)p.G * p.N - nb))),
                           (uint32_t)(c.lane * 4), (uint32_t)c.w * 256u);
      // without a bias an empty resource: the DMA writes zeros
      if (c.w < 2)
        dma_asm_v<4, BIAS_OFF>(dst, p.bias ? rsrc4(p.bias + t.n0, clamp_records(2 * (p.N - t.n0))) : rsrc4(p.D, 0u),
                               (uint32_t)(c.lane * 4), (uint32_t)c.w * 256u);
    }
  }

  struct Epi {
    u32x4 rd;
    uint32_t voff, rowstride;
    int64_t m0, n0, lim;
    int slot;
    bool full, on;
  };

  __device__ static inline void make_epi(const Ctx &c, const Tile &t, bool on, Epi &e) {
    const Int8Args &p = *c.p;
    e.m0 = t.m0;
    e.n0 = t.n0;
    e.lim = t.lim;
    e.slot = t.slot;
    e.on = on;
    // 16-byte stores through a range-checked 32-bit offset (see DenseLoop), at
    // any alignment
    e.full = t.m0 + DBM <= t.lim && t.n0 + DBN <= p.N && (RES ? p.N : p.No) <= (1 << 22);
    const int64_t org = t.m0 * p.No + (SWIGLU ? t.n0 / 2 : t.n0);
    e.rd = rsrc4(p.D + org, clamp_records(2 * (p.M * p.No - org)));
    e.rowstride = (uint32_t)(32 * p.No);
    const int lane = (int)__lane_id(), i = lane & 15, q = lane >> 4;
    const int64_t r = c.wm * (FM * 16) + i;
    if constexpr (SWIGLU) e.voff = (uint32_t)(2 * (r * p.No + c.wn * 32 + 8 * q));
    else e.voff = (uint32_t)(2 * (r * p.No + c.wn * 64 + 16 * (q & 1) + 8 * (q >> 1)));
  }

  // The residual beside row tile a of a full tile, as its sums lie: four
  // columns per lane and 16-column block, SwiGLU two.  The offsets are those
  // of the stores, so the same sizes bound them.
  typedef v2i ResRow[RES ? FN : 1];
  __device__ static inline void load_residual(const Ctx &c, const Epi &e, int a, ResRow &r) {
    if constexpr (RES) {
      const Int8Args &p = *c.p;
      const int64_t org = e.m0 * p.No + (SWIGLU ? e.n0 / 2 : e.n0);
      const __amdgpu_buffer_rsrc_t rr =
          p.R ? make_rsrc(p.R + org, clamp_records(2 * (p.M * p.No - org))) : make_rsrc(p.D, 0);
      int lane = (int)__lane_id();
      asm volatile("" : "+v"(lane));       // the offset formed here, not kept from row tile to row tile
      const int i = lane & 15, q = lane >> 4;
      const uint32_t row = (uint32_t)(2 * ((c.wm * 128 + a * 16 + i) * p.No));
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        const int col = c.wn * 64 + b * 16 + 4 * q;
        if constexpr (SWIGLU) r[b].x = (int)buf_load_u32(rr, row + (uint32_t)col);
        else r[b] = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(rr, (int)(row + 2u * (uint32_t)col), 0, 0));
      }
    }
  }

  // Row tile a of the finished tile.  Lane (i, q) holds row 16 a + i, columns
  // 16 b + 4 q .. + 3 of the wave's block.  Full tiles: lanes of different q
  // trade their packed pairs (v_permlane16_swap exchanges the odd 16-lane
  // rows of one register with the even rows of another, v_permlane32_swap
  // the halves) until each holds 16 contiguous bytes of its row.
  __device__ static inline void store_rows(const Ctx &c, const Epi &e, int a, const v4i (&row)[FN],
                                           const ResRow &res) {
    const Int8Args &p = *c.p;
    const int lane = (int)__lane_id(), i = lane & 15, q = lane >> 4;
    const uint32_t sc = c.lds0 + S_REG + (uint32_t)e.slot * SCALES;
    const float sa = __uint_as_float(*(const lds_u32_t *)(uintptr_t)(sc + (c.wm * 128 + a * 16 + i) * 4));
    auto finish = [&](int b) -> v4f {
      const uint32_t o = (uint32_t)(c.wn * 64 + b * 16 + 4 * q);
      const v4i s = *(const lds_v4i *)(uintptr_t)(sc + SB_OFF + o * 4);
      const v2i w = *(const lds_v2i *)(uintptr_t)(sc + BIAS_OFF + o * 2);
      return int8_finish(row[b], sa, __builtin_bit_cast(v4f, s), unpack_bf16x4(w), RES ? (int)ACT_NONE : ACT);
    };
    if (e.full) {
      uint32_t rs = e.rowstride;
      asm volatile("" : "+s"(rs));
      // two neighbouring 16-column blocks, 16 contiguous bytes per lane
      auto put = [&](const v4f &x, const v4f &y, const u32x4 &rd, uint32_t voff, uint32_t soff) {
        const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(x.z, x.w), pack_bf16x2(y.z, y.w), false, false);
        store16_asm((v4i){(int)lo[0], (int)hi[0], (int)lo[1], (int)hi[1]}, rd, voff, soff);
      };
      // the activation's argument, [M, N] whatever the activation
      auto put_z = [&](const v4f &x, const v4f &y, int pr) {
        const int64_t org = e.m0 * p.N + e.n0;
        int l = lane;
        asm volatile("" : "+v"(l));
        const int64_t r = c.wm * (FM * 16) + (l & 15);
        put(x, y, rsrc4(p.Z + org, clamp_records(2 * (p.M * p.N - org))),
            (uint32_t)(2 * (r * p.N + c.wn * 64 + 16 * (q & 1) + 8 * (q >> 1))), (uint32_t)(32 * p.N) * (uint32_t)a + 64u * pr);
      };
      if constexpr (SWIGLU) {
        uint32_t d[4];
        if constexpr (RES) {
#pragma unroll
          for (int pr = 0; pr < 2; ++pr) {
            const v4f z[2] = {finish(2 * pr), finish(2 * pr + 1)};
            if (p.Z) put_z(z[0], z[1], pr);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u = (uint32_t)res[2 * pr + k].x;
              d[2 * pr + k] = pack_bf16x2(z[k].x * logistic_f32(z[k].x) * z[k].y + __uint_as_float(u << 16),
                                          z[k].z * logistic_f32(z[k].z) * z[k].w + __uint_as_float(u & 0xFFFF0000u));
            }
          }
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b) d[b] = swiglu_pack(finish(b));
        }
        // 4 x 4 transpose over (b, q)
        const auto s02 = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
        const auto s13 = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
        const auto t01 = __builtin_amdgcn_permlane16_swap(s02[0], s13[0], false, false);
        const auto t23 = __builtin_amdgcn_permlane16_swap(s02[1], s13[1], false, false);
        store16_asm((v4i){(int)t01[0], (int)t01[1], (int)t23[0], (int)t23[1]}, e.rd, e.voff, (uint32_t)a * rs);
      } else {
#pragma unroll
        for (int pr = 0; pr < FN / 2; ++pr) {
          v4f x = finish(2 * pr), y = finish(2 * pr + 1);
          if constexpr (RES) {
            if (p.Z) put_z(x, y, pr);
            const v4f rx = unpack_bf16x4(res[2 * pr]), ry = unpack_bf16x4(res[2 * pr + 1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = activate(ACT, x[k]) + rx[k];
              y[k] = activate(ACT, y[k]) + ry[k];
            }
          }
          put(x, y, e.rd, e.voff, (uint32_t)a * rs + 64u * pr);
        }
      }
    } else {
      const int64_t r = e.m0 + c.wm * (FM * 16) + a * 16 + i;
      if (r < e.lim) {
#pragma unroll
        for (int b = 0; b < FN; ++b) {
          const int64_t col = e.n0 + c.wn * (FN * 16) + b * 16 + 4 * q;
          if constexpr (RES) int8_emit4<true>(p, ACT, r, col, finish(b), int8_near(p, ACT, r, col));
          else int8_store4(p, ACT, r, col, finish(b));
        }
      }
    }
  }

  // All of a finished tile; with a residual between two tiles' steps (see
  // DenseLoop::finish_tile).
  __device__ static inline void finish_tile(const Ctx &c, const Epi &e, const v4i (&acc)[FM][FN]) {
    // As many row tiles' residuals at once as registers allow; a later one's
    // loads are behind the stores of row tiles finished long before its turn.
    constexpr int WIN = SWIGLU ? FM : 5;
    ResRow res[WIN];
    if constexpr (RES) {
      if (e.full) {
#pragma unroll
        for (int a = 0; a < WIN; ++a) load_residual(c, e, a, res[a]);
      }
    }
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      store_rows(c, e, a, acc[a], res[a % WIN]);
      if constexpr (RES) {
        if (e.full && a + WIN < FM) load_residual(c, e, a + WIN, res[a % WIN]);
      }
    }
  }

  __device__ static inline void pin(v4i (&acc)[FM][FN]) {
#pragma unroll
    for (int a = 0; a < FM; ++a)
      asm volatile("" : "+v"(acc[a][0]), "+v"(acc[a][1]), "+v"(acc[a][2]), "+v"(acc[a][3]));
  }

  template <bool EPI>
  __device__ static inline void compute(const Ctx &c, const uint8_t *smem, int si, uint32_t oa0, uint32_t oa1,
                                        uint32_t ob0, uint32_t ob1, v4i (&acc)[FM][FN], const Epi &e) {
    const uint8_t *base = smem + si * AB;
    v4i b0[FN], b1[FN];
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      b0[b] = lds_read16(base + ob0 + b * 2048);
      b1[b] = lds_read16(base + ob1 + b * 2048);
    }
    v4i a0 = lds_read16(base + oa0), a1 = lds_read16(base + oa1);
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      v4i n0, n1;
      if (a + 1 < FM) {
        n0 = lds_read16(base + oa0 + (a + 1) * 2048);
        n1 = lds_read16(base + oa1 + (a + 1) * 2048);
      }
      if (!RES && EPI && e.on) store_rows(c, e, a, acc[a], ResRow{});
      // first operand = B tile: the result lane holds 4 consecutive n
#pragma unroll
      for (int b = 0; b < FN; ++b) acc[a][b] = mfma_i8(b0[b], a0, EPI ? (v4i){0, 0, 0, 0} : acc[a][b]);
#pragma unroll
      for (int b = 0; b < FN; ++b) acc[a][b] = mfma_i8(b1[b], a1, acc[a][b]);
      if (a + 1 < FM) {
        a0 = n0;
        a1 = n1;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // The waits are DenseLoop::run's: the DMAs are invisible to the compiler; a
  // slot is refilled after the barrier that ends the step which read it, and
  // read after the wait and barrier that follow its DMAs.  At the end of a
  // tile's first step up to EPI_STORES stores may still be in flight: they
  // were issued after the stage's DMAs.
  template <class TileAt, class Resolve>
  __device__ static inline void run(const Ctx &c, int ntiles, TileAt tile_at, Resolve resolve, uint8_t *smem) {
    constexpr uint32_t LMASK = 0x3FFFFu;
    const int f = kswz(c.i16);
    const uint32_t p0 = (uint32_t)((c.q ^ f) << 4), p1 = (uint32_t)(((c.q + 4) ^ f) << 4);
    const uint32_t ra = (uint32_t)((c.wm * 128 + c.i16) * 128), rb = (uint32_t)(B_REG + (c.wn * 64 + c.i16) * 128);
    const uint32_t oa0 = (ra + p0) & LMASK, oa1 = (ra + p1) & LMASK;
    const uint32_t ob0 = (rb + p0) & LMASK, ob1 = (rb + p1) & LMASK;

    v4i acc[FM][FN];
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b) acc[a][b] = (v4i){0, 0, 0, 0};

    int tm, tn;
    tile_at(0, tm, tn);
    Tile cur;
    set_tile(c, resolve(tm, tn), 0, cur);
    issue(c, cur, 0, 0);
    wait_vmem_le<0>();
    __syncthreads();

    const int nst = c.nst;
    const bool odd = (nst & 1) != 0;
    Epi e;
    make_epi(c, cur, false, e);
    for (int t = 0; t < ntiles; ++t) {
      const bool more = t + 1 < ntiles;
      if (more) tile_at(t + 1, tm, tn);
      auto step = [&](auto epi, auto slot, int k) {
        constexpr bool EPI = decltype(epi)::value;
        constexpr int SC = decltype(slot)::value, SN = 1 - SC;
        if (k + 1 < nst) {
          issue(c, cur, k + 1, SN);
        } else if (more && !odd) {
          Tile nxt;
          set_tile(c, resolve(tm, tn), (t + 1) & 1, nxt);
          issue(c, nxt, 0, SN);
        }
        compute<EPI>(c, smem, SC, oa0, oa1, ob0, ob1, acc, e);
        pin(acc);
        __builtin_amdgcn_sched_barrier(0);
        if (!RES && EPI && e.on && e.full) wait_vmem_le<EPI_STORES>();
        else wait_vmem_le<0>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
      };
      step(std::true_type{}, std::integral_constant<int, 0>{}, 0);
      int k = 1;
      for (; k + 2 <= nst; k += 2) {
        step(std::false_type{}, std::integral_constant<int, 1>{}, k);
        step(std::false_type{}, std::integral_constant<int, 0>{}, k + 1);
      }
      if (k < nst) step(std::false_type{}, std::integral_constant<int, 1>{}, k);
      make_epi(c, cur, true, e);
      if constexpr (RES) finish_tile(c, e, acc);
      if (more) {
        set_tile(c, resolve(tm, tn), (t + 1) & 1, cur);
        if (odd) {
          issue(c, cur, 0, 0);
          wait_vmem_le<0>();
          __syncthreads();
        }
      }
    }
    if constexpr (!RES) finish_tile(c, e, acc);
  }
};

template <int ACT, bool RES = false>
__global__ __launch_bounds__(DNW8 * 64, 1) void int8_tiled_kernel(Int8Args p) {
  typedef Int8Loop<ACT, RES> L;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[L::LDS_BYTES];
  __shared__ GroupTable gt;
  if (threadIdx.x < 64) int8_group_table<DBM>(p, gt, (int)threadIdx.x);
  __syncthreads();
  const int tiles_m = uni32(gt.mtile[p.G]);
  const int nb = tiles_m * p.tiles_n;
  const int P = (int)gridDim.x, bid = (int)blockIdx.x;
  if (bid >= nb) return;
  const int ntiles = (nb - bid + P - 1) / P;
  typename L::Ctx c;
  L::init(c, p, smem);
  auto tile_at = [&](int k, int &tm, int &tn) {
    int P_ = P, tm_ = tiles_m, tn_ = p.tiles_n;
    asm volatile("" : "+s"(P_), "+s"(tm_), "+s"(tn_));
    persistent_tile(bid, k, P_, tm_, tn_, tm, tn);
  };
  auto resolve = [&](int tm, int tn) -> TileId {
    const int g = group_of_tile(gt, p.G, tm);
    const int64_t start = uni32(gt.rows[g]);
    const int64_t mg = uni32(gt.rows[g + 1]) - start;
    const int64_t m0 = start + (int64_t)(tm - uni32(gt.mtile[g])) * DBM;
    return TileId{m0, (int64_t)tn * DBN, start + mg, start, mg, g};
  };
  L::run(c, ntiles, tile_at, resolve, smem);
}

// ---------------------------------------------------------------------------
// BM x BN tiles (64 x 64 or 128 x 128), for outputs with too few 256 x 256
// tiles to occupy the device: four waves in 2 x 2, a ring of NS stages of KS K
// steps that runs across tile boundaries, two workgroups per compute unit,
// tiles in XCD bands.  Per K step a workgroup takes 0.36 us (64 x 64) or 0.8
// us (128 x 128) where it has the compute unit alone, whatever the ring's
// depth: with one wave per SIMD it is the ~100 instructions of a step, the
// barrier and the latencies between them that count.  With two workgroups
// and full rounds 0.32 and 0.65 us (53 bytes per ns of operands through the
// L2).  Measured for 64 x 64: four one-step stages against two of two steps,
// 128 x 4096 x 9600 27.9 and 31.0 us, 16 x 12000 x 9600 28 and 41, full rounds
// 6 % slower; three stages and three workgroups per unit, 700 rows in 16
// groups x 2048 x 4096 46 against 38.5 us.
template <int BM, int BN, int KS, int NS, bool RES = false>
__global__ __launch_bounds__(256, 2) void int8_stream_kernel(Int8Args p) {
  constexpr int FM = BM / 32, FN = BN / 32, ABLK = BM / 32, BBLK = BN / 32;
  constexpr int AB = BM * 128, BB = BN * 128, STAGE = KS * (AB + BB);
  constexpr int AHEAD = (NS - 2) * KS * (ABLK + BBLK);   // a wave's DMAs of the stages after the next one
  // a tile's scales and biases, in NS + 1 slots (with one stage per tile, NS
  // tiles are in flight when a finished one is stored): [BM row scales][BN channel
  // scales][BN biases].  By DMA like the operands: the compiler's own loads
  // in the loop would make it wait for every DMA behind them.
  constexpr int SB_OFF = 4 * BM, BIAS_OFF = SB_OFF + 4 * BN, SCALES = BIAS_OFF + 256;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NS * STAGE + (NS + 1) * SCALES];
  __shared__ GroupTable gt;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1, i16 = lane & 15, q = lane >> 4;

  if (w == 0) int8_group_table<BM>(p, gt, lane);
  __syncthreads();
  const int P = (int)gridDim.x;
  const int64_t T = (int64_t)uni32(gt.mtile[p.G]) * p.tiles_n;
  const int x = (int)(blockIdx.x & 7), r = (int)(blockIdx.x >> 3);
  const int64_t full = T / P, last = T - full * P;
  auto band_start = [&](int64_t size) -> int64_t { return x * (size >> 3) + (x < (size & 7) ? x : (size & 7)); };
  auto band_count = [&](int64_t size) -> int64_t { return (size >> 3) + (x < (size & 7) ? 1 : 0); };
  const int64_t ntile = (r < band_count(P) ? full : 0) + (r < band_count(last) ? 1 : 0);
  if (ntile == 0) return;
  const int64_t off_full = band_start(P) + r, off_last = band_start(last) + r;
  GroupedArgs ga = {};
  ga.G = p.G;
  ga.tiles_n = p.tiles_n;
  auto tile_at = [&](int64_t i) { return stream_tile<BM, BN>(ga, gt, i * P + (i < full ? off_full : off_last)); };

  const int64_t K = p.K, N = p.N;
  const int nst = (int)((K + 127) / 128), nsg = (nst + KS - 1) / KS;
  const int rem = (int)(K - 128 * (int64_t)(nst - 1));
  constexpr uint32_t NOWHERE = 0x80000000u;    // past any resource: zeros, no memory read
  const int piece = (lane & 7) ^ kswz(lane >> 3);
  const uint32_t vo = (uint32_t)((lane >> 3) * K) + (uint32_t)(piece << 4);
  const uint32_t vo_tail = 16 * piece < rem ? vo : NOWHERE;
  const uint32_t lds0 = lds_addr(smem);
  const uint32_t row8 = (uint32_t)(8 * K), arow = (uint32_t)(ABLK * w) * row8, brow = (uint32_t)(BBLK * w) * row8;

  struct Src {
    int64_t row0, n0;
    int g;
    u32x4 ra, rb;                  // ra ends with the tile's rows: those past them read zeros
  };
  auto make_src = [&](int64_t i) {
    const StreamTile t = tile_at(i);
    Src s;
    const int64_t bbase = ((int64_t)t.g * N + t.n0) * K;
    s.row0 = t.row0;
    s.n0 = t.n0;
    s.g = t.g;
    s.ra = rsrc4(p.A + t.row0 * K, clamp_records((t.lim - t.row0) * K));
    s.rb = rsrc4(p.B + bbase, clamp_records((int64_t)p.G * N * K - bbase));
    return s;
  };
  Src src = make_src(0);
  int64_t iss_i = 0;
  int iss_sg = 0, iss_sc = 0;
  // The next stage into slot sl; K steps past the tile's last and stages
  // past the workgroup's last read nothing.  With a tile's first stage wave 0
  // brings its row scales, wave 1 its channel scales, wave 2 its biases.
  auto issue = [&](int sl) {
    const bool real = iss_i < ntile;
    if (real && iss_sg == 0) {
      const uint32_t dst = lds0 + (uint32_t)(NS * STAGE + iss_sc * SCALES);
      if (w == 0) {
        const u32x4 r = rsrc4(p.sA + src.row0, clamp_records(4 * (p.M - src.row0)));
        static_for<0, BM / 64>([&](auto jc) {
          constexpr int j = decltype(jc)::value;
          dma_asm_v<4, j * 256>(dst, r, (uint32_t)(lane * 4), j * 256u);
        });
      } else if (w == 1) {
        const u32x4 r = rsrc4(p.sB + (int64_t)src.g * N + src.n0, clamp_records(4 * (N - src.n0)));
        static_for<0, BN / 64>([&](auto jc) {
          constexpr int j = decltype(jc)::value;
          dma_asm_v<4, SB_OFF + j * 256>(dst, r, (uint32_t)(lane * 4), j * 256u);
        });
      } else if (w == 2) {
        // without a bias an empty resource: the DMA writes zeros
        const u32x4 r = p.bias ? rsrc4(p.bias + src.n0, clamp_records(2 * (N - src.n0))) : rsrc4(p.D, 0u);
        dma_asm_v<4, BIAS_OFF>(dst, r, (uint32_t)(lane * 4), 0u);
      }
    }
    const uint32_t slot = lds0 + (uint32_t)sl * STAGE;
    static_for<0, KS>([&](auto sc) {
      constexpr int s = decltype(sc)::value;
      const int st = iss_sg * KS + s;
      const bool live = real && st < nst;
      const uint32_t k0 = 128u * (uint32_t)st;
      const uint32_t va = live ? (st == nst - 1 ? vo_tail : vo) + k0 : NOWHERE, vb = live ? vo + k0 : NOWHERE;
      const uint32_t ka = slot + (uint32_t)(s * AB + ABLK * 1024 * w);
      const uint32_t kb = slot + (uint32_t)(KS * AB + s * BB + BBLK * 1024 * w);
      static_for<0, ABLK>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        dma_asm_v<16, j * 1024>(ka, src.ra, va, arow + j * row8);
      });
      static_for<0, BBLK>([&](auto jc) {
        constexpr int j = decltype(jc)::value;
        dma_asm_v<16, j * 1024>(kb, src.rb, vb, brow + j * row8);
      });
    });
    if (++iss_sg == nsg) {
      iss_sg = 0;
      iss_sc = iss_sc == NS ? 0 : iss_sc + 1;
      ++iss_i;
      if (iss_i < ntile) src = make_src(iss_i);
    }
  };

  v4i acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = (v4i){0, 0, 0, 0};
  const int f = kswz(i16);
  const uint32_t p0 = (uint32_t)((q ^ f) << 4), p1 = (uint32_t)(((q + 4) ^ f) << 4);
  const uint32_t oa = (uint32_t)((wm * (BM / 2) + i16) * 128), ob = (uint32_t)((wn * (BN / 2) + i16) * 128);

  auto finish_tile = [&](auto ac, const StreamTile &t, uint32_t sc) {
    constexpr int ACT = decltype(ac)::value;
    v4f sb[FN], bias[FN];
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      const uint32_t o = (uint32_t)(wn * (BN / 2) + b * 16 + 4 * q);
      const v4i s = *(const lds_v4i *)(uintptr_t)(sc + SB_OFF + 4 * o);
      sb[b] = __builtin_bit_cast(v4f, s);
      const v2i u = *(const lds_v2i *)(uintptr_t)(sc + BIAS_OFF + 2 * o);
      bias[b] = unpack_bf16x4(u);
    }
    const int64_t r0 = t.row0 + wm * (BM / 2) + i16;
    // all of the residual before the first store: their latencies together
    v2i near[RES ? FM : 1][FN];
    if constexpr (RES) {
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b) {
          near[a][b] = (v2i){0, 0};
          if (r0 + a * 16 < t.lim) near[a][b] = int8_near(p, ACT, r0 + a * 16, t.n0 + wn * (BN / 2) + b * 16 + 4 * q);
        }
    }
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      const float sa = __uint_as_float(*(const lds_u32_t *)(uintptr_t)(sc + (uint32_t)(4 * (wm * (BM / 2) + a * 16 + i16))));
      if (r0 + a * 16 < t.lim) {
#pragma unroll
        for (int b = 0; b < FN; ++b)
          int8_emit4<RES>(p, ACT, r0 + a * 16, t.n0 + wn * (BN / 2) + b * 16 + 4 * q,
                          int8_finish(acc[a][b], sa, sb[b], bias[b], ACT_NONE), near[RES ? a : 0][b]);
      }
    }
  };

  // Fragments of half h (64 of a step's 128 bytes of K) of the stage at stg.
  // Two register sets: a half is read while the half before it runs on the
  // matrix cores, across the barrier too.
  v4i fa[2][FM], fb[2][FN];
  auto read_half = [&](const uint8_t *stg, auto hc) {
    constexpr int h = decltype(hc)::value, s = h >> 1, set = h & 1;
    const uint32_t pc = set ? p1 : p0;
    const uint8_t *la = stg + s * AB + oa + pc, *lb = stg + KS * AB + s * BB + ob + pc;
#pragma unroll
    for (int b = 0; b < FN; ++b) fb[set][b] = lds_read16(lb + b * 2048);
#pragma unroll
    for (int a = 0; a < FM; ++a) fa[set][a] = lds_read16(la + a * 2048);
  };
  auto multiply = [&](auto sc) {
    constexpr int set = decltype(sc)::value;
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b) acc[a][b] = mfma_i8(fb[set][b], fa[set][a], acc[a][b]);
  };

  // Stage v + NS goes into the slot of stage v once every wave has read v's
  // last half.
  static_for<0, NS>([&](auto sc) { issue(decltype(sc)::value); });
  wait_vmem_le<AHEAD + KS * (ABLK + BBLK)>();
  __syncthreads();
  read_half(smem, std::integral_constant<int, 0>{});
  int64_t ci = 0;
  int csg = 0, slot = 0, csc = 0;
  const int64_t V = ntile * nsg;
  for (int64_t v = 0; v < V; ++v) {
    static_for<1, 2 * KS>([&](auto hc) {
      constexpr int h = decltype(hc)::value;
      read_half(smem + slot * STAGE, std::integral_constant<int, h>{});
      __builtin_amdgcn_sched_barrier(0);
      multiply(std::integral_constant<int, (h - 1) & 1>{});
      __builtin_amdgcn_sched_barrier(0);
    });
    // stage v + 1 has landed (stores of a tile are newer: more is waited for)
    // and this wave's reads of stage v are done
    __builtin_amdgcn_s_waitcnt(0x0070 | (AHEAD & 15) | ((AHEAD >> 4) << 14));
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    issue(slot);
    slot = slot + 1 == NS ? 0 : slot + 1;
    read_half(smem + slot * STAGE, std::integral_constant<int, 0>{});
    __builtin_amdgcn_sched_barrier(0);
    multiply(std::integral_constant<int, 1>{});
    if (++csg == nsg) {
      const StreamTile t = tile_at(ci);
      const uint32_t sc = lds0 + (uint32_t)(NS * STAGE + csc * SCALES);
      if (p.act == ACT_NONE) finish_tile(std::integral_constant<int, ACT_NONE>{}, t, sc);
      else if (p.act == ACT_SWIGLU) finish_tile(std::integral_constant<int, ACT_SWIGLU>{}, t, sc);
      else if (p.act == ACT_GELU_TANH) finish_tile(std::integral_constant<int, ACT_GELU_TANH>{}, t, sc);
      else if (p.act == ACT_SILU) finish_tile(std::integral_constant<int, ACT_SILU>{}, t, sc);
      else finish_tile(std::integral_constant<int, ACT_RELU>{}, t, sc);
#pragma unroll
      for (int a = 0; a < FM; ++a)
#pragma unroll
        for (int b = 0; b < FN; ++b) acc[a][b] = (v4i){0, 0, 0, 0};
      csg = 0;
      csc = csc == NS ? 0 : csc + 1;
      ++ci;
    }
    // accumulators in VGPRs: with one workgroup per compute unit the compiler
    // moved them to AGPRs and back in every step
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b) asm volatile("" : "+v"(acc[a][b]));
  }
  wait_vmem_le<0>();   // no DMA into the LDS of an ended workgroup
}

// ---------------------------------------------------------------------------
// Few rows: BM = 16 FM rows x BN = 16 FN columns per workgroup of W waves that
// split K between them, step st of 128 bytes to wave st % W.  Operands go from
// memory straight to registers in the matrix cores' layout (nothing is shared
// between waves but the final sum, so LDS staging and its barriers would only
// add latency), U steps ahead; the waves' integer partial sums meet in LDS.
// Bound by memory where the weights are large (1 x 14336 x 4096: 12.0 us, 4.9
// TB/s), else by a compute unit's 36 bytes per ns of 64-byte row pieces and
// by latency (16 x 4096 x 4096 7.3 us, 13.8 through LDS in 64 x 64 tiles).
template <int FM, int FN, int W, int U, bool RES = false>
__global__ __launch_bounds__(64 * W) void int8_rows_kernel(Int8Args p) {
  constexpr int BM = 16 * FM, BN = 16 * FN;
  __shared__ v4i part[W][FM * FN][64];
  __shared__ GroupTable gt;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, q = lane >> 4;
  if (w == 0) int8_group_table<BM>(p, gt, lane);
  __syncthreads();
  // eight contiguous bands of tiles, one per XCD: the row tiles of one set of
  // columns read the same weights
  const int64_t T = (int64_t)uni32(gt.mtile[p.G]) * p.tiles_n;
  const int x = (int)(blockIdx.x & 7), r = (int)(blockIdx.x >> 3);
  const int64_t lo = T & 7, band = (T >> 3) + (x < lo ? 1 : 0);
  if (r >= band) return;
  GroupedArgs ga = {};
  ga.G = p.G;
  ga.tiles_n = p.tiles_n;
  const StreamTile t = stream_tile<BM, BN>(ga, gt, x * (T >> 3) + (x < lo ? x : lo) + r);

  const int64_t K = p.K, N = p.N;
  const int nst = (int)((K + 127) / 128);
  const int64_t abase = t.row0 * K, bbase = ((int64_t)t.g * N + t.n0) * K;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + abase, clamp_records(p.M * K - abase));
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.B + bbase, clamp_records((int64_t)p.G * N * K - bbase));
  constexpr uint32_t NOWHERE = 0x80000000u;    // past any resource: zeros, no memory read
  const uint32_t lane_off = (uint32_t)(i16 * K + 16 * q);
  uint32_t rows_a[FM];
#pragma unroll
  for (int a = 0; a < FM; ++a) rows_a[a] = t.row0 + 16 * a + i16 < t.lim ? lane_off + (uint32_t)(16 * a * K) : NOWHERE;

  v4i fa[U][FM][2], fb[U][FN][2];
  auto load = [&](int u, int st) {
    const uint32_t k0 = (uint32_t)st * 128u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = (int64_t)st * 128 + 64 * h + 16 * q < K;
#pragma unroll
      for (int b = 0; b < FN; ++b)
        fb[u][b][h] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(rb, (int)(in ? lane_off + (uint32_t)(16 * b * K) + k0 + 64u * h : NOWHERE), 0, 0));
#pragma unroll
      for (int a = 0; a < FM; ++a)
        fa[u][a][h] = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(
                     ra, (int)(in && rows_a[a] != NOWHERE ? rows_a[a] + k0 + 64u * h : NOWHERE), 0, 0));
    }
  };
  v4i acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = (v4i){0, 0, 0, 0};
#pragma unroll
  for (int u = 0; u < U; ++u) load(u, w + u * W);
  for (int st = w; st < nst; st += U * W) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int a = 0; a < FM; ++a)
#pragma unroll
          for (int b = 0; b < FN; ++b) acc[a][b] = mfma_i8(fb[u][b][h], fa[u][a][h], acc[a][b]);
      if (st + U * W < nst) load(u, st + (u + U) * W);
    }
  }
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) part[w][a * FN + b][lane] = acc[a][b];
  __syncthreads();
#pragma unroll
  for (int f = w; f < FM * FN; f += W) {
    const int a = f / FN, b = f % FN;
    v4i sum = part[0][f][lane];
#pragma unroll
    for (int k = 1; k < W; ++k) sum += part[k][f][lane];
    const int64_t row = t.row0 + 16 * a + i16, col = t.n0 + 16 * b + 4 * q;
    if (row < t.lim) {
      v2i near = {0, 0};
      if constexpr (RES) near = int8_near(p, p.act, row, col);
      v4f sb, bias;
      int8_columns(p, t.g, t.n0, 16 * b + 4 * q, sb, bias);
      int8_emit4<RES>(p, p.act, row, col, int8_finish(sum, p.sA[row], sb, bias, ACT_NONE), near);
    }
  }
}

// K == 0: act(bias) in every row that belongs to a group, plus the residual.
__global__ void int8_fill_kernel(Int8Args p) {
  int64_t covered = p.M;
  if (p.m_sizes) {
    covered = 0;
    for (int g = 0; g < p.G; ++g) {
      const int64_t s = p.m_sizes[g], room = p.M - covered;
      covered += s < 0 ? 0 : (s > room ? room : s);
    }
  }
  const int64_t i = flat_block() * 256 + threadIdx.x;
  if (i >= covered * p.No) return;
  const int64_t c = i % p.No;
  auto bias = [&](int64_t n) { return p.bias ? __uint_as_float((uint32_t)p.bias[n] << 16) : 0.0f; };
  float z;
  if (p.act == ACT_SWIGLU) {
    const float g = bias(2 * c), u = bias(2 * c + 1);
    z = g * logistic_f32(g) * u;
    if (p.Z) ((uint32_t *)p.Z)[i] = pack_bf16x2(g, u);
  } else {
    z = activate(p.act, bias(c));
    if (p.Z) p.Z[i] = (uint16_t)pack_bf16x2(bias(c), 0.0f);
  }
  if (p.R) z += __uint_as_float((uint32_t)p.R[i] << 16);
  p.D[i] = (uint16_t)pack_bf16x2(z, 0.0f);
}

}  // namespace mxg
