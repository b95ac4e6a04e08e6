// The experts of a mixture-of-experts layer for a few tokens, in two kernels:
//   out[t] = R[t] + sum_e share[t,e] W2[e] act( W1[e] x[t] ),
//   share[t,e] = sum of w[t,j] over the slots j with ids[t,j] = e.
// Few tokens make this a stream of the chosen experts' weights: each is read
// once, 128 bytes of K of 16 rows at a time straight into the matrix cores'
// layout, and turned into BF16 there (codes of every format are exact in
// BF16, and so are codes times a power of two inside its range), so that the
// activations stay what they are: x in BF16, sums in FP32.  act's result h is
// kept as two BF16 (its rounding and what that leaves, 16 bits of
// mantissa): rounded to one, it would add as much error as the rounding of
// out; the second costs a second matrix instruction, which the stream hides.
//
// experts_up_kernel: a workgroup per (live expert, tile of W1's rows), its
// waves splitting K; one more workgroup writes the table of live experts and
// their tokens for experts_down_kernel: a workgroup per tile of out's
// columns, its waves taking (live expert, part of K) in turn, each adding
// share * y to sums of its own in LDS; these meet in a fixed order, so a
// call's bits do not change from run to run.
#pragma once
#include "common.hpp"

namespace mxg {

enum : int { WF_INT8 = 0, WF_BF16 = 1, WF_E4M3 = 2, WF_E5M2 = 3, WF_E2M1 = 4, WF_BLOCK = 5 };
constexpr int EXP_MAX_T = 64, EXP_MAX_E = 1024, EXP_MAX_TOPK = 32;

struct ExpertRec {
  int32_t e, base, n, pad;               // expert, its first pair, its tokens
};
struct ExpertPair {
  int32_t t, row;                        // token, row of h
  float share;
  int32_t pad;
};

struct ExpertsArgs {
  const uint16_t *x;                     // [T, D]
  const int32_t *ids;                    // [T, topk]
  const float *w;                        // [T, topk]
  const uint8_t *w1, *w2;
  const void *s1, *s2;
  const uint16_t *residual;              // [T, D] or null
  uint16_t *out;                         // [T, D]
  uint16_t *h;                           // [2][T topk, F]: high parts, low parts
  int32_t *live;                         // number of live experts
  ExpertRec *rec;                        // [live]
  ExpertPair *pair;                      // [<= T topk], by expert, then by token
  int64_t D, F, N1;                      // N1 rows of W1[e]: F or 2 F
  int T, E, topk, act;
  int tiles, parts;                      // row tiles of W1 (up), parts of K per expert (down)
};

// What 16 bytes of a row hold.
template <int WF> struct WeightFormat {
  static constexpr int CODES = WF == WF_BF16 ? 8 : WF == WF_E2M1 ? 32 : 16;   // values in 16 bytes
  static constexpr int UNIT = 8 * CODES;                                      // values in a 128-byte unit
  static constexpr int XL = CODES / 4;                                        // 16-byte pieces of x per lane and unit
  static constexpr bool MX = WF == WF_E4M3 || WF == WF_E5M2 || WF == WF_E2M1;
  static constexpr int SCALES = WF == WF_E2M1 ? 2 : 1;                        // E8M0 scales per lane and unit
  __host__ __device__ static int64_t row_bytes(int64_t K) { return K * 16 / CODES; }
};

// Values 8 m .. 8 m + 7 of 16 bytes of codes, times scale where the format
// has E8M0 scales, in BF16.
template <int WF>
__device__ inline bf16x8_t weight_values(const v4i &raw, int m, float scale) {
  v4i r;
  if constexpr (WF == WF_BF16) {
    r = raw;
  } else if constexpr (WF == WF_E2M1) {
    r[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[m], scale, 0));
    r[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[m], scale, 1));
    r[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[m], scale, 2));
    r[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[m], scale, 3));
  } else {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const int v = raw[2 * m + d];
      if constexpr (WF == WF_INT8) {
        r[2 * d] = (int)pack_bf16x2((float)(int8_t)v, (float)(int8_t)(v >> 8));
        r[2 * d + 1] = (int)pack_bf16x2((float)(int8_t)(v >> 16), (float)(int8_t)(v >> 24));
      } else if constexpr (WF == WF_E5M2) {
        r[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v, scale, false));
        r[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(v, scale, true));
      } else {
        r[2 * d] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, false));
        r[2 * d + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, true));
      }
    }
  }
  return __builtin_bit_cast(bf16x8_t, r);
}

// acc[m][b] += rows 16 b .. of a weight tile times the activation rows xo[m]
// (byte offsets into rx, NOWHERE: none), over the 128-byte units u0, u0 + du,
// .. below u1 of K.  Lane (i = lane % 16, q = lane / 16) holds bytes 32 q .. +
// 31 of a unit of weight row i and the same values of activation row i;
// the result lane holds weight rows 4 q .. + 3 of activation row i.  PL planes of
// activations (plane bytes apart) are summed.  Loads run U units ahead.
constexpr uint32_t EXP_NOWHERE = 0x80000000u;   // past any resource: zeros, no memory read

template <int WF, int FM, int FN, int PL, int U>
__device__ inline void stream_product(__amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rx,
                                      const uint32_t (&xo)[FM], uint32_t plane, int64_t K, int u0, int u1, int du,
                                      v4f (&acc)[FM][FN]) {
  typedef WeightFormat<WF> W;
  const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
  const uint32_t KB = (uint32_t)W::row_bytes(K), SK = (uint32_t)(K / 32);
  const uint32_t wo = (uint32_t)i16 * KB + 32u * q;
  v4i w[U][FN][2], x[U][FM][PL][W::XL];
  uint32_t sc[U][FN][W::SCALES];
  float blk[U];
  auto load = [&](int s, int u) {
    const bool in0 = 128u * u + 32u * q < KB, in1 = 128u * u + 32u * q + 16u < KB;
#pragma unroll
    for (int b = 0; b < FN; ++b) {
      const uint32_t o = wo + 16u * b * KB + 128u * u;
      w[s][b][0] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)(in0 ? o : EXP_NOWHERE), 0, 0));
      w[s][b][1] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)(in1 ? o + 16u : EXP_NOWHERE), 0, 0));
      if constexpr (W::MX) {
        // a lane's 32 (E2M1: 64) values: one E8M0 scale (two)
        const uint32_t so = (16u * b + i16) * SK + (uint32_t)(u * (W::UNIT / 32)) + W::SCALES * q;
        sc[s][b][0] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(in0 ? so : EXP_NOWHERE), 0, 0);
        if constexpr (W::SCALES == 2) sc[s][b][1] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(in1 ? so + 1u : EXP_NOWHERE), 0, 0);
      }
    }
    if constexpr (WF == WF_BLOCK) blk[s] = __uint_as_float(buf_load_u32(rs, 4u * u));
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int p = 0; p < PL; ++p)
#pragma unroll
        for (int j = 0; j < W::XL; ++j) {
          const bool in = xo[m] != EXP_NOWHERE && (j < W::XL / 2 ? in0 : in1);
          const uint32_t o = xo[m] + p * plane + 2u * (uint32_t)(u * W::UNIT + q * 2 * W::CODES) + 16u * j;
          x[s][m][p][j] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(in ? o : EXP_NOWHERE), 0, 0));
        }
  };
#pragma unroll
  for (int s = 0; s < U; ++s)
    if (u0 + s * du < u1) load(s, u0 + s * du);
  for (int u = u0; u < u1; u += U * du) {
#pragma unroll
    for (int s = 0; s < U; ++s) {
      if (u + s * du < u1) {
        v4f part[FM][FN];
        if constexpr (WF == WF_BLOCK) {
#pragma unroll
          for (int m = 0; m < FM; ++m)
#pragma unroll
            for (int b = 0; b < FN; ++b) part[m][b] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int j = 0; j < W::XL; ++j)
#pragma unroll
          for (int b = 0; b < FN; ++b) {
            constexpr int HALF = W::XL / 2;
            float scale = 1.0f;
            if constexpr (W::MX) scale = __uint_as_float(sc[s][b][W::SCALES == 2 ? j / HALF : 0] << 23);
            const bf16x8_t wv = weight_values<WF>(w[s][b][j / HALF], j % HALF, scale);
#pragma unroll
            for (int m = 0; m < FM; ++m)
#pragma unroll
              for (int p = 0; p < PL; ++p) {
                v4f &c = WF == WF_BLOCK ? part[m][b] : acc[m][b];
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8_t, x[s][m][p][j]), c, 0, 0, 0);
              }
          }
        if constexpr (WF == WF_BLOCK) {
          // one FP32 scale for 128 values of K of all of the tile's rows
#pragma unroll
          for (int m = 0; m < FM; ++m)
#pragma unroll
            for (int b = 0; b < FN; ++b) acc[m][b] += part[m][b] * blk[s];
        }
        if (u + (s + U) * du < u1) load(s, u + (s + U) * du);
      }
    }
  }
}

// Resources of rows n0 .. of a weight [N, K] (N rows in all, of expert e) and
// of their scales; past the last row everything reads zero.
template <int WF>
__device__ inline void weight_rsrc(const uint8_t *w, const void *s, int64_t e, int64_t N, int64_t K, int64_t n0,
                                   __amdgpu_buffer_rsrc_t &rw, __amdgpu_buffer_rsrc_t &rs) {
  const int64_t KB = WeightFormat<WF>::row_bytes(K);
  rw = make_rsrc(w + (e * N + n0) * KB, clamp_records((N - n0) * KB));
  if constexpr (WeightFormat<WF>::MX)
    rs = make_rsrc((const uint8_t *)s + (e * N + n0) * (K / 32), clamp_records((N - n0) * (K / 32)));
  else if constexpr (WF == WF_BLOCK)
    rs = make_rsrc((const float *)s + (e * (N / 128) + n0 / 128) * (K / 128), clamp_records(4 * (K / 128)));
  else
    rs = make_rsrc(w, 0);
}

// The channel scales of rows n0 + c .. + 3 (INT8; else 1).
template <int WF>
__device__ inline v4f channel_scales(const void *s, int64_t e, int64_t N, int64_t n0, int c) {
  if constexpr (WF == WF_INT8) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc((const float *)s + e * N + n0, clamp_records(4 * (N - n0)));
    return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * c, 0, 0));
  } else {
    return (v4f){1.f, 1.f, 1.f, 1.f};
  }
}

// The tokens of every expert as bits.
struct ExpertMasks {
  uint32_t bits[EXP_MAX_E][2];
};

__device__ inline void expert_masks(const ExpertsArgs &p, ExpertMasks &mk) {
  for (int i = threadIdx.x; i < 2 * p.E; i += blockDim.x) (&mk.bits[0][0])[i] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < p.T * p.topk; s += blockDim.x) {
    const int e = p.ids[s], t = s / p.topk;
    if (e >= 0 && e < p.E) atomicOr(&mk.bits[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
}

__device__ inline uint64_t expert_mask(const ExpertMasks &mk, int e) {
  return (uint64_t)mk.bits[e][1] << 32 | mk.bits[e][0];
}

// The live expert of this rank (by index), or -1; every wave for itself.
__device__ inline int live_expert(const ExpertsArgs &p, const ExpertMasks &mk, int rank) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    const bool on = e0 + lane < p.E && expert_mask(mk, e0 + lane) != 0;
    const uint64_t b = __ballot(on);
    const int n = __popcll(b);
    if (rank < n) {
      const uint64_t me = __ballot(on && __popcll(b & ((1ull << lane) - 1)) == rank);
      return e0 + __ffsll((unsigned long long)me) - 1;
    }
    rank -= n;
  }
  return -1;
}

// The slot of token t that first names expert e.
__device__ inline int first_slot(const ExpertsArgs &p, int t, int e) {
  int j = 0;
  while (j < p.topk - 1 && p.ids[t * p.topk + j] != e) ++j;
  return j;
}

// The table for the second kernel, by one workgroup.
__device__ inline void expert_table(const ExpertsArgs &p, const ExpertMasks &mk, int32_t (&first)[EXP_MAX_E]) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < 64) {
    int live = 0, base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      const int e = e0 + lane;
      const int n = e < p.E ? __popcll(expert_mask(mk, e)) : 0;
      int sum = n;                         // of the lanes up to this one
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
      }
      const uint64_t b = __ballot(n > 0);
      if (e < p.E) first[e] = base + sum - n;
      if (n > 0) p.rec[live + __popcll(b & ((1ull << lane) - 1))] = ExpertRec{e, base + sum - n, n, 0};
      live += __popcll(b);
      base += __shfl(sum, 63);
    }
    if (lane == 0) *p.live = live;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.T * p.topk; s += blockDim.x) {
    const int e = p.ids[s], t = s / p.topk;
    if (e < 0 || e >= p.E || s != t * p.topk + first_slot(p, t, e)) continue;
    float share = 0.0f;
    for (int j = s - t * p.topk; j < p.topk; ++j)
      if (p.ids[t * p.topk + j] == e) share += p.w[t * p.topk + j];
    p.pair[first[e] + __popcll(expert_mask(mk, e) & ((1ull << t) - 1))] = ExpertPair{t, s, share, 0};
  }
}

// h of four consecutive rows of W1 (two SwiGLU pairs), as two BF16 each.
__device__ inline void store_h(const ExpertsArgs &p, int row, int64_t n, const v4f &z) {
  const int64_t plane = (int64_t)p.T * p.topk * p.F;
  v4f v;
  int cnt = 4;
  int64_t c = n;
  if (p.act == ACT_SWIGLU) {
    v.x = z.x * logistic_f32(z.x) * z.y;
    v.y = z.z * logistic_f32(z.z) * z.w;
    v.z = v.w = 0.0f;
    cnt = 2;
    c = n >> 1;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = activate(p.act, z[k]);
  }
  const uint32_t hi[2] = {pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
  float r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float f = __uint_as_float(k & 1 ? hi[k >> 1] & 0xFFFF0000u : hi[k >> 1] << 16);
    // nothing is left of an infinity or a NaN
    r[k] = fabsf(f) < __builtin_inff() ? v[k] - f : 0.0f;
  }
  const uint32_t lo[2] = {pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3])};
  uint16_t *dst = p.h + (int64_t)row * p.F + c;
  if (cnt == 2) {
    *(uint32_t *)dst = hi[0];
    *(uint32_t *)(dst + plane) = lo[0];
  } else {
    *(v2i *)dst = (v2i){(int)hi[0], (int)hi[1]};
    *(v2i *)(dst + plane) = (v2i){(int)lo[0], (int)lo[1]};
  }
}

constexpr int UP_WAVES = 4, UP_FN = 2;

template <int WF, int FMAX>
__global__ __launch_bounds__(64 * UP_WAVES) void experts_up_kernel(ExpertsArgs p) {
  constexpr int FN = UP_FN, W = UP_WAVES;
  __shared__ union {
    struct {
      ExpertMasks mk;
      int32_t first[EXP_MAX_E];
    } t;
    v4f part[W][FMAX * FN][64];
  } sm;
  __shared__ int32_t row[EXP_MAX_T], tok[EXP_MAX_T];
  const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  expert_masks(p, sm.t.mk);
  if (blockIdx.x == 0) {
    expert_table(p, sm.t.mk, sm.t.first);
    return;
  }
  const int rank = (int)(blockIdx.x - 1) / p.tiles, tile = (int)(blockIdx.x - 1) - rank * p.tiles;
  const int e = __builtin_amdgcn_readfirstlane(live_expert(p, sm.t.mk, rank));
  if (e < 0) return;
  const uint64_t mask = expert_mask(sm.t.mk, e);
  const int n = __popcll(mask);
  if (w == 0 && (mask >> lane & 1)) {
    const int i = __popcll(mask & ((1ull << lane) - 1));
    tok[i] = lane;
    row[i] = lane * p.topk + first_slot(p, lane, e);
  }
  __syncthreads();                         // the masks are free from here on

  const int64_t n0 = (int64_t)tile * (16 * FN);
  __amdgpu_buffer_rsrc_t rw, rs;
  weight_rsrc<WF>(p.w1, p.s1, e, p.N1, p.D, n0, rw, rs);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x, clamp_records(2 * p.T * p.D));
  const int units = (int)((WeightFormat<WF>::row_bytes(p.D) + 127) / 128);
  auto body = [&](auto fc) {
    constexpr int FM = decltype(fc)::value;
    constexpr int U = FM == 1 ? 3 : FM == 2 && WF != WF_E2M1 ? 2 : 1;
    uint32_t xo[FM];
    v4f acc[FM][FN];
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      xo[m] = 16 * m + i16 < n ? (uint32_t)(2 * tok[16 * m + i16] * p.D) : EXP_NOWHERE;
#pragma unroll
      for (int b = 0; b < FN; ++b) acc[m][b] = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    stream_product<WF, FM, FN, 1, U>(rw, rs, rx, xo, 0u, p.D, w, units, W, acc);
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int b = 0; b < FN; ++b) sm.part[w][m * FN + b][lane] = acc[m][b];
    __syncthreads();
    for (int f = w; f < FM * FN; f += W) {
      const int i = 16 * (f / FN) + i16, c = 16 * (f % FN) + 4 * q;
      v4f z = sm.part[0][f][lane];
#pragma unroll
      for (int k = 1; k < W; ++k) z += sm.part[k][f][lane];
      if (i < n && n0 + c < p.N1) store_h(p, row[i], n0 + c, z * channel_scales<WF>(p.s1, e, p.N1, n0, c));
    }
  };
  if (FMAX == 1 || n <= 16) body(std::integral_constant<int, 1>{});
  else if (n <= 32) body(std::integral_constant<int, FMAX == 1 ? 1 : 2>{});
  else body(std::integral_constant<int, FMAX>{});
}

constexpr int DOWN_WAVES = 8, DOWN_FN = 1;
constexpr int DOWN_PITCH = 16 * DOWN_FN + 4;     // floats per token: columns and a skew

inline __host__ __device__ int down_lds_bytes(int T) { return 4 * DOWN_WAVES * T * DOWN_PITCH; }

template <int WF, int FMAX>
__global__ __launch_bounds__(64 * DOWN_WAVES) void experts_down_kernel(ExpertsArgs p) {
  constexpr int FN = DOWN_FN, W = DOWN_WAVES, COLS = 16 * FN;
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [W][T][DOWN_PITCH]
  const int lane = threadIdx.x & 63, i16 = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float *mine = sums + w * p.T * DOWN_PITCH;
  for (int i = lane; i < p.T * DOWN_PITCH; i += 64) mine[i] = 0.0f;
  const int64_t n0 = (int64_t)blockIdx.x * COLS;
  const int live = __builtin_amdgcn_readfirstlane(*p.live);
  const int units = (int)((WeightFormat<WF>::row_bytes(p.F) + 127) / 128);
  const int per = (units + p.parts - 1) / p.parts;
  const int64_t plane = (int64_t)p.T * p.topk * p.F;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.h, clamp_records(4 * plane));
  for (int job = w; job < live * p.parts; job += W) {
    const int a = job / p.parts, part = job - a * p.parts;
    const int e = __builtin_amdgcn_readfirstlane(p.rec[a].e), base = __builtin_amdgcn_readfirstlane(p.rec[a].base);
    const int n = __builtin_amdgcn_readfirstlane(p.rec[a].n);
    __amdgpu_buffer_rsrc_t rw, rs;
    weight_rsrc<WF>(p.w2, p.s2, e, p.D, p.F, n0, rw, rs);
    auto body = [&](auto fc) {
      constexpr int FM = decltype(fc)::value;
      constexpr int U = FM == 1 ? 2 : 1;
      uint32_t xo[FM];
      int t[FM];
      float share[FM];
      v4f acc[FM][FN];
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const bool in = 16 * m + i16 < n;
        const ExpertPair pr = p.pair[base + (in ? 16 * m + i16 : 0)];
        xo[m] = in ? (uint32_t)(2 * pr.row * p.F) : EXP_NOWHERE;
        t[m] = in ? pr.t : -1;
        share[m] = pr.share;
#pragma unroll
        for (int b = 0; b < FN; ++b) acc[m][b] = (v4f){0.f, 0.f, 0.f, 0.f};
      }
      stream_product<WF, FM, FN, 2, U>(rw, rs, rx, xo, (uint32_t)(2 * plane), p.F, part * per, min(units, (part + 1) * per), 1, acc);
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int b = 0; b < FN; ++b)
          if (t[m] >= 0) {
            const int c = 16 * b + 4 * q;
            v4f *s = (v4f *)(mine + t[m] * DOWN_PITCH + c);
            *s += acc[m][b] * channel_scales<WF>(p.s2, e, p.D, n0, c) * share[m];
          }
    };
    if (FMAX == 1 || n <= 16) body(std::integral_constant<int, 1>{});
    else if (n <= 32) body(std::integral_constant<int, FMAX == 1 ? 1 : 2>{});
    else body(std::integral_constant<int, FMAX>{});
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.T * COLS; i += 64 * W) {
    const int t = i / COLS, c = i - t * COLS;
    if (n0 + c >= p.D) continue;
    float v = sums[t * DOWN_PITCH + c];
#pragma unroll
    for (int k = 1; k < W; ++k) v += sums[(k * p.T + t) * DOWN_PITCH + c];
    const int64_t o = (int64_t)t * p.D + n0 + c;
    if (p.residual) v += __uint_as_float((uint32_t)p.residual[o] << 16);
    p.out[o] = (uint16_t)pack_bf16x2(v, 0.0f);
  }
}

}  // namespace mxg
