// The operators of a mixture-of-experts layer around its grouped GEMMs:
// routing and its gradient, per-row 8-bit quantization into the order of the
// experts' rows, and the weighted combine of those rows with its gradient.
// All but the router's choice are memory-bound streams.
#pragma once
#include "common.hpp"

namespace mxg {

enum : int { MOE_SOFTMAX = 0, MOE_SIGMOID = 1 };
enum : int { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 };
constexpr int MOE_MAX_E = 1024, MOE_MAX_TOPK = 32;
constexpr int ROUTE_TG = 64;             // tokens placed at once: one bit each of a 64-bit mask
constexpr int ROUTE_MAX_BLOCKS = 512;

__device__ inline float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ inline float load_elem(const uint16_t *p) { return bf16_to_f32(*p); }
__device__ inline float load_elem(const float *p) { return *p; }
__device__ inline void store_elem(uint16_t *p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }
__device__ inline void store_elem(float *p, float v) { *p = v; }

struct RouteArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *weights;
  int64_t T;
  int E, topk, score, n_group, topk_group, group_score, renorm;
  float scale;
  int lpg, per;                          // lanes per expert group, experts per lane
  int64_t *m_sizes;
  int32_t *row_of, *slot_of;             // null: no maps
  uint16_t *counts;                      // [blocks][Ep]: rows of each expert by block
  int Ep, nblk;
  int64_t tpb;                           // tokens per block, a multiple of ROUTE_TG
};

// LDS of the placement: which tokens of a group of 64 chose each expert.
struct RoutePlace {
  uint32_t mask[MOE_MAX_E][2];
  int32_t base[MOE_MAX_E];               // next row of each expert
  int32_t total[MOE_MAX_E];
  int32_t wave_sum[16];
  int32_t used;
};

// One token's choice by LPT lanes (its lanes hold `per` <= VPT consecutive
// experts each; an expert group owns lpg consecutive lanes, so a group's
// statistics need no more than shuffles among them), `sub` the lane's index
// among them.  Choice values in 64 bits: scores that differ in FP32's last
// bits decide between experts.  Returns the id of rank `sub` (-1: none) in
// lanes sub < topk, and its weight.
template <class IN, int LPT, int VPT>
__device__ inline int route_token(const RouteArgs &p, const IN *row, bool live, int sub, float &weight) {
  const int n = p.E / p.n_group;
  const int gi = sub / p.lpg, part = sub % p.lpg;
  const int e0 = gi * n + part * p.per;
  const int cnt = (live && gi < p.n_group) ? max(0, min(p.per, n - part * p.per)) : 0;
  const double NONE = -__builtin_inf();
  float l[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) l[j] = j < cnt ? load_elem(row + e0 + j) : -__builtin_inff();
  // finite stand-in of an available logit; NaN and -inf are not available
  auto avail = [](float x) { return x > -__builtin_inff(); };
  auto fin = [](float x) { return (double)fminf(x, 3.402823466e38f); };

  double m = NONE, sum = 0.0;
  if (p.score == MOE_SOFTMAX) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (avail(l[j])) m = fmax(m, fin(l[j]));
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) m = fmax(m, __shfl_xor(m, d, 64));
    if (!p.renorm || p.bias || (p.n_group > 1 && p.group_score == MOE_GROUP_TOP2)) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (avail(l[j])) sum += exp(fin(l[j]) - m);
#pragma unroll
      for (int d = 1; d < LPT; d <<= 1) sum += __shfl_xor(sum, d, 64);
    }
  }
  auto score = [&](double x) { return p.score == MOE_SOFTMAX ? exp(x - m) / sum : 1.0 / (1.0 + exp(-x)); };

  double v[VPT];
  double g1 = NONE, g2 = NONE;           // the lane's two best of its group
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    v[j] = NONE;
    if (avail(l[j])) {
      double s = 0.0;
      const bool top2 = p.n_group > 1 && p.group_score == MOE_GROUP_TOP2;
      if (p.bias || top2) s = score(fin(l[j]));
      if (p.bias) s += (double)p.bias[e0 + j];
      v[j] = p.bias ? s : (double)l[j];
      const double gv = top2 ? s : v[j];
      g2 = fmax(g2, fmin(g1, gv));
      g1 = fmax(g1, gv);
    }
  }
  if (p.n_group > 1) {
    for (int d = 1; d < p.lpg; d <<= 1) {
      const double o1 = __shfl_xor(g1, d, 64), o2 = __shfl_xor(g2, d, 64);
      g2 = fmax(fmin(g1, o1), fmax(g2, o2));
      g1 = fmax(g1, o1);
    }
    double gs = g1;
    if (p.group_score == MOE_GROUP_TOP2 && g2 > NONE) gs += g2;
    int rank = 0;
    for (int g = 0; g < p.n_group; ++g) {
      const double o = __shfl(gs, g * p.lpg, LPT);
      rank += (o > gs || (o == gs && g < gi)) ? 1 : 0;
    }
    if (rank >= p.topk_group) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) v[j] = NONE;
    }
  }

  int id = -1;
  for (int r = 0; r < p.topk; ++r) {
    double bv = NONE;
    int be = 0x7FFFFFFF;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (v[j] > bv) {
        bv = v[j];
        be = e0 + j;
      }
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) {
      const double ov = __shfl_xor(bv, d, 64);
      const int oe = __shfl_xor(be, d, 64);
      if (ov > bv || (ov == bv && oe < be)) {
        bv = ov;
        be = oe;
      }
    }
    const int chosen = bv > NONE ? be : -1;
    if (sub == r) id = chosen;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (e0 + j == chosen && j < cnt) v[j] = NONE;
  }

  // weights, one rank per lane
  const bool has = id >= 0;
  const double x = has ? fin(load_elem(row + id)) : 0.0;
  double w;
  if (p.renorm) {
    // shares of the chosen: a common factor e^-top keeps them in range
    const bool sm = p.score == MOE_SOFTMAX;
    double top = has ? (sm ? x : fmin(x, 0.0)) : NONE;
    const double mine = top;
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) top = fmax(top, __shfl_xor(top, d, 64));
    w = 0.0;
    if (has) w = exp(mine - top) / (sm ? 1.0 : 1.0 + exp(-fabs(x)));
    double tot = w;
#pragma unroll
    for (int d = 1; d < LPT; d <<= 1) tot += __shfl_xor(tot, d, 64);
    w = has ? w / tot : 0.0;
  } else {
    w = has ? score(x) : 0.0;
  }
  weight = (float)(w * (double)p.scale);
  return id;
}

// Marks the experts of slots [0, nslot) (ids of up to 64 tokens) in pl.mask.
__device__ inline void route_mark(RoutePlace &pl, const int32_t *ids, int nslot, int topk, int E) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) pl.mask[e][0] = pl.mask[e][1] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < nslot; s += blockDim.x) {
    const int e = ids[s], t = s / topk;
    if (e >= 0) atomicOr(&pl.mask[e][t >> 5], 1u << (t & 31));
  }
  __syncthreads();
}

__device__ inline int route_count(const RoutePlace &pl, int e) {
  return __popc(pl.mask[e][0]) + __popc(pl.mask[e][1]);
}

// pl.base[e] (rows of e in earlier blocks) += first row of e, from
// pl.total[e]; blockDim.x >= 256.  Writes m_sizes in block 0.
__device__ inline void route_bases(const RouteArgs &p, RoutePlace &pl) {
  const int tid = threadIdx.x, lane = tid & 63;
  int c[4], sum = 0;
  if (tid < 256) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = 4 * tid + k;
      c[k] = e < p.E ? pl.total[e] : 0;
      sum += c[k];
    }
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d, 64);
    if (lane >= d) incl += y;
  }
  if (lane == 63 && tid < 256) pl.wave_sum[tid >> 6] = incl;
  __syncthreads();
  if (tid < 256) {
    int first = incl - sum;
    for (int w = 0; w < (tid >> 6); ++w) first += pl.wave_sum[w];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int e = 4 * tid + k;
      if (e < p.E) {
        pl.base[e] += first;
        if (blockIdx.x == 0) p.m_sizes[e] = c[k];
      }
      first += c[k];
    }
    if (tid == 255) pl.used = first;
  }
  __syncthreads();
}

// Rows of the group of tokens t0 .. marked in pl.mask, and -- once all its
// slots are placed -- the experts' next rows.
__device__ inline void route_place(const RouteArgs &p, RoutePlace &pl, const int32_t *ids, int nslot, int64_t t0) {
  for (int s = threadIdx.x; s < nslot; s += blockDim.x) {
    const int e = ids[s], t = s / p.topk;
    int row = -1;
    if (e >= 0) {
      const uint32_t lo = pl.mask[e][0], hi = pl.mask[e][1];
      const uint32_t below = (1u << (t & 31)) - 1;
      row = pl.base[e] + (t < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below));
      p.slot_of[row] = (int32_t)(t0 * p.topk + s);
    }
    p.row_of[t0 * p.topk + s] = row;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) pl.base[e] += route_count(pl, e);
}

__device__ inline void route_tail(const RouteArgs &p, const RoutePlace &pl) {
  const int64_t n = p.T * p.topk;
  for (int64_t r = pl.used + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < n; r += (int64_t)gridDim.x * blockDim.x)
    p.slot_of[r] = -1;
}

// Choice and weights of a block's tokens, 64 at a time, and (COUNT) the
// block's rows of each expert; ONE: the single block of a small call places
// its rows itself.
template <class IN, int LPT, int VPT, bool MAPS, bool ONE>
__global__ void route_kernel(RouteArgs p) {
  __shared__ int32_t ids[MAPS ? ROUTE_TG * MOE_MAX_TOPK : 1];
  __shared__ RoutePlace pl;
  const int tid = threadIdx.x, sub = tid & (LPT - 1);
  const int per_pass = blockDim.x / LPT;
  const int64_t t_end = min(p.T, ((int64_t)blockIdx.x + 1) * p.tpb);
  if constexpr (MAPS) {
    for (int e = tid; e < p.E; e += blockDim.x) pl.total[e] = pl.base[e] = 0;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * p.tpb; t0 < t_end; t0 += ROUTE_TG) {
    const int nt = (int)min((int64_t)ROUTE_TG, t_end - t0);
    for (int tb = 0; tb < nt; tb += per_pass) {
      const int tl = tb + tid / LPT;
      const bool live = tl < nt;
      const int64_t t = t0 + (live ? tl : 0);
      float w;
      const int id = route_token<IN, LPT, VPT>(p, (const IN *)p.logits + t * p.E, live, sub, w);
      if (live && sub < p.topk) {
        p.ids[t * p.topk + sub] = id;
        p.weights[t * p.topk + sub] = w;
        if constexpr (MAPS) ids[tl * p.topk + sub] = id;
      }
    }
    if constexpr (MAPS) {
      __syncthreads();
      route_mark(pl, ids, nt * p.topk, p.topk, p.E);
      for (int e = tid; e < p.E; e += blockDim.x) pl.total[e] += route_count(pl, e);
      __syncthreads();
      if constexpr (ONE) {
        route_bases(p, pl);
        route_place(p, pl, ids, nt * p.topk, t0);
        route_tail(p, pl);
      }
    }
  }
  if constexpr (MAPS && !ONE) {
    for (int e = tid; e < p.E; e += blockDim.x) p.counts[(int64_t)blockIdx.x * p.Ep + e] = (uint16_t)pl.total[e];
  }
}

// The second kernel of a call of more than 64 tokens: every block sums the
// counts of all blocks (its own first rows and the experts' totals), then
// places its tokens.
__global__ __launch_bounds__(256) void route_place_kernel(RouteArgs p) {
  __shared__ int32_t ids[ROUTE_TG * MOE_MAX_TOPK];
  __shared__ RoutePlace pl;
  const int tid = threadIdx.x;
  for (int e = tid; e < MOE_MAX_E; e += 256) pl.total[e] = pl.base[e] = 0;
  __syncthreads();
  const int nv = p.Ep / 8, rows = 256 / nv;       // 16-byte columns, row lanes
  const int col = tid % nv, r0 = tid / nv;
  if (r0 < rows) {
    int tot[8] = {0, 0, 0, 0, 0, 0, 0, 0}, bef[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int b = r0; b < p.nblk; b += rows) {
      const v4i x = *(const v4i *)(p.counts + (int64_t)b * p.Ep + col * 8);
      const bool before = b < (int)blockIdx.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int lo = x[k] & 0xFFFF, hi = (uint32_t)x[k] >> 16;
        tot[2 * k] += lo;
        tot[2 * k + 1] += hi;
        bef[2 * k] += before ? lo : 0;
        bef[2 * k + 1] += before ? hi : 0;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (col * 8 + k < p.E) {
        atomicAdd(&pl.total[col * 8 + k], tot[k]);
        atomicAdd(&pl.base[col * 8 + k], bef[k]);
      }
    }
  }
  __syncthreads();
  route_bases(p, pl);
  const int64_t t_end = min(p.T, ((int64_t)blockIdx.x + 1) * p.tpb);
  for (int64_t t0 = (int64_t)blockIdx.x * p.tpb; t0 < t_end; t0 += ROUTE_TG) {
    const int ns = (int)min((int64_t)ROUTE_TG, t_end - t0) * p.topk;
    __syncthreads();
    for (int s = tid; s < ns; s += 256) ids[s] = p.ids[t0 * p.topk + s];
    __syncthreads();
    route_mark(pl, ids, ns, p.topk, p.E);
    route_place(p, pl, ids, ns, t0);
  }
  route_tail(p, pl);
}

__global__ void moe_zero_sizes_kernel(int64_t *m_sizes, int E) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) m_sizes[e] = 0;
}

// ---------------------------------------------------------------------------
// Gradient of the weights: one wave per token, lane l holds experts l, l +
// 64, ...  One pass: logits in, gradients out.
struct RouteGradArgs {
  const void *logits;
  const int32_t *ids;
  const float *grad;
  void *dlogits;
  int64_t T;
  int E, topk, score, renorm;
  float scale;
};

__device__ inline float wave_sum(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}
__device__ inline float wave_max(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = fmaxf(x, __shfl_xor(x, d, 64));
  return x;
}

// A logit's finite stand-in; -inf where the expert is not available (-inf
// or NaN).
__device__ inline float avail_logit(float x) {
  return x > -__builtin_inff() ? fminf(x, 3.402823466e38f) : -__builtin_inff();
}

template <class IN, int VPT>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.T) return;
  const IN *row = (const IN *)p.logits + t * p.E;
  IN *drow = (IN *)p.dlogits + t * p.E;
  const float NI = -__builtin_inff();
  float l[VPT], ds[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 64 * j;
    l[j] = avail_logit(e < p.E ? load_elem(row + e) : NI);
    ds[j] = 0.0f;
  }
  // lane r holds choice r
  int id = -1;
  float c = 0.0f, x = NI;
  if (lane < p.topk) {
    id = p.ids[t * p.topk + lane];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      x = avail_logit(load_elem(row + id));
      if (x > NI) c = p.scale * p.grad[t * p.topk + lane];
      else id = -1;
    }
  }
  const bool sm = p.score == MOE_SOFTMAX;
  float mine = 0.0f;                     // the chosen expert's own share of the gradient
  float m = 0.0f, inv = 0.0f, dot = 0.0f;
  if (p.renorm) {
    const float z = id >= 0 ? (sm ? x : fminf(x, 0.0f)) : NI;
    const float top = wave_max(z);
    float w = id >= 0 ? expf(z - top) / (sm ? 1.0f : 1.0f + expf(-fabsf(x))) : 0.0f;
    const float tot = wave_sum(w);
    w = id >= 0 ? w / tot : 0.0f;
    dot = wave_sum(c * w);
    mine = w * (c - dot);
    if (!sm) mine *= 1.0f / (1.0f + expf(x));             // 1 - s
  } else if (sm) {
    float mm = NI;
#pragma unroll
    for (int j = 0; j < VPT; ++j) mm = fmaxf(mm, l[j]);
    m = wave_max(mm);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) s += l[j] > NI ? expf(l[j] - m) : 0.0f;
    s = wave_sum(s);
    inv = s > 0.0f ? 1.0f / s : 0.0f;
    dot = wave_sum(id >= 0 ? c * (expf(x - m) * inv) : 0.0f);
    mine = c;
  } else {
    // s (1 - s) = 1 / ((1 + e^x) (1 + e^-x)), e^-|x| <= 1
    const float ex = expf(-fabsf(x)), s1 = 1.0f / (1.0f + ex);
    mine = id >= 0 ? c * ex * s1 * s1 : 0.0f;
  }
  for (int r = 0; r < p.topk; ++r) {
    const int e = __shfl(id, r, 64);
    const float g = __shfl(mine, r, 64);
#pragma unroll
    for (int j = 0; j < VPT; ++j) ds[j] = e == lane + 64 * j ? g : ds[j];
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int e = lane + 64 * j;
    float d = ds[j];
    if (!p.renorm && sm) d = l[j] > NI ? expf(l[j] - m) * inv * (d - dot) : 0.0f;
    if (e < p.E) store_elem(drow + e, d);
  }
}

// ---------------------------------------------------------------------------
// Rows -> int8 codes and one scale.  GROUP lanes (a wave, or a workgroup of
// 256) hold one row in registers, NV pieces of 16 values per lane, so x is
// read once; a row wider than that is read twice (WIDE).
//
// The codes are rint(q) of the correctly rounded FP32 quotient q = x / s.
// With inv = 1 / s correctly rounded, q0 = x inv is within two units of q's
// last place; one residual step q0 + (x - q0 s) inv leaves a value within
// one, and a second gives the correctly rounded quotient (Markstein's
// theorem), in five instructions instead of the division's dozen.  That
// needs inv and the residuals in the normal range: rows whose scale is
// below 2^-96 or above 2^96 divide.
struct QuantArgs {
  const void *x;
  int8_t *codes;
  float *scales;
  int64_t T, K;
  const int32_t *row_of;
  int topk;
};

// Rows in registers stay in their own type: two BF16 values per register.
template <class IN> struct Piece;
template <> struct Piece<float> {
  float4 u[4];
  __device__ inline void load(const float *p) {
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = ((const float4 *)p)[k];
  }
  __device__ inline float get(int i) const { return (&u[i >> 2].x)[i & 3]; }
};
template <> struct Piece<uint16_t> {
  v4i u[2];
  __device__ inline void load(const uint16_t *p) {
    u[0] = ((const v4i *)p)[0];
    u[1] = ((const v4i *)p)[1];
  }
  __device__ inline float get(int i) const {
    const uint32_t w = (uint32_t)u[i >> 3][(i & 7) >> 1];
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
};

template <class IN>
__device__ inline float piece_amax(const Piece<IN> &x) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x.get(i)));
  return m;
}

template <class IN>
__device__ inline v4i piece_codes(const Piece<IN> &x, float s, float inv, bool divide) {
  v4i out;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = x.get(4 * k + j);
      float q;
      if (divide) {
        q = v / s;
      } else {
        q = v * inv;
        q = fmaf(fmaf(-q, s, v), inv, q);
        q = fmaf(fmaf(-q, s, v), inv, q);
      }
      q = fminf(fmaxf(rintf(q), -127.0f), 127.0f);
      w |= ((uint32_t)(int)q & 0xFFu) << (8 * j);
    }
    out[k] = (int)w;
  }
  return out;
}

template <class IN, int GROUP, int NV, bool WIDE>
__global__ __launch_bounds__(256) void quant_int8_kernel(QuantArgs p) {
  __shared__ float part[4];
  const int tid = threadIdx.x, gl = tid & (GROUP - 1);
  const int64_t t = (int64_t)blockIdx.x * (256 / GROUP) + tid / GROUP;
  if (GROUP == 64 && t >= p.T) return;
  const IN *row = (const IN *)p.x + t * p.K;
  const int np = (int)(p.K / 16);
  Piece<IN> x[NV];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = gl + j * GROUP;
    if (c < np) x[j].load(row + 16 * c);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (gl + j * GROUP < np) m = fmaxf(m, piece_amax(x[j]));
  if constexpr (WIDE) {
    for (int c = gl + NV * GROUP; c < np; c += GROUP) {
      Piece<IN> y;
      y.load(row + 16 * c);
      m = fmaxf(m, piece_amax(y));
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
  if constexpr (GROUP == 256) {
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  }
  float s = m / 127.0f;
  if (!(s > 0.0f)) s = 1.0f;
  const bool divide = !(s >= 0x1p-96f && s <= 0x1p96f);
  const float inv = 1.0f / s;
  auto put = [&](int c, const v4i &q) {
    if (p.row_of == nullptr) {
      *(v4i *)(p.codes + t * p.K + 16 * c) = q;
      return;
    }
    for (int k = 0; k < p.topk; ++k) {
      const int64_t r = p.row_of[t * p.topk + k];
      if (r >= 0 && r < p.T * p.topk) *(v4i *)(p.codes + r * p.K + 16 * c) = q;
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = gl + j * GROUP;
    if (c < np) put(c, piece_codes(x[j], s, inv, divide));
  }
  if constexpr (WIDE) {
    for (int c = gl + NV * GROUP; c < np; c += GROUP) {
      Piece<IN> y;
      y.load(row + 16 * c);
      put(c, piece_codes(y, s, inv, divide));
    }
  }
  if (p.row_of == nullptr) {
    if (gl == 0) p.scales[t] = s;
  } else if (gl < p.topk) {
    const int64_t r = p.row_of[t * p.topk + gl];
    if (r >= 0 && r < p.T * p.topk) p.scales[r] = s;
  }
}

__global__ void fill_f32_kernel(float *x, int64_t n, float v) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) x[i] = v;
}

// ---------------------------------------------------------------------------
// Combine: one workgroup per token and stripe of columns, VEC values per
// lane (8: 16-byte accesses; 1 where N is not a multiple of 8).
struct CombineArgs {
  const uint16_t *y;
  const float *w;
  const int32_t *row_of;
  uint16_t *out;
  int64_t T, N, rows;
  int topk;
};

template <int VEC>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs p) {
  const int64_t t = blockIdx.y + (int64_t)blockIdx.z * 65535;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * VEC;
  if (t >= p.T || c >= p.N) return;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
#pragma unroll 4
  for (int k = 0; k < p.topk; ++k) {
    const int64_t r = p.row_of[t * p.topk + k];
    if (r < 0 || r >= p.rows) continue;
    const float w = p.w[t * p.topk + k];
    const uint16_t *src = p.y + r * p.N + c;
    if constexpr (VEC == 8) {
      const v4i u = *(const v4i *)src;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w, __uint_as_float((uint32_t)u[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, __uint_as_float((uint32_t)u[i] & 0xFFFF0000u), acc[2 * i + 1]);
      }
    } else {
      acc[0] = fmaf(w, bf16_to_f32(*src), acc[0]);
    }
  }
  uint16_t *dst = p.out + t * p.N + c;
  if constexpr (VEC == 8) {
    v4i o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (int)pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
    *(v4i *)dst = o;
  } else {
    store_elem(dst, acc[0]);
  }
}

struct CombineGradArgs {
  const uint16_t *dout, *y;
  const float *w;
  const int32_t *row_of;
  uint16_t *dy;
  float *dw;
  int64_t T, N, rows;
  int topk;
};

// One wave per (token, slot): its row of y and the token's row of dout
// (shared through the caches by the token's slots) in, its row of dy out,
// the dot product in registers and one wave reduction.
template <int VEC>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineGradArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t s = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (s >= p.T * p.topk) return;
  const int64_t t = s / p.topk;
  const int64_t r = p.row_of[s];
  if (r < 0 || r >= p.rows) {
    if (lane == 0) p.dw[s] = 0.0f;
    return;
  }
  const float w = p.w[s];
  const uint16_t *d = p.dout + t * p.N, *y = p.y + r * p.N;
  uint16_t *o = p.dy + r * p.N;
  float acc = 0.0f;
#pragma unroll 4
  for (int64_t c = lane * VEC; c < p.N; c += 64 * VEC) {
    if constexpr (VEC == 8) {
      const v4i a = *(const v4i *)(d + c), b = *(const v4i *)(y + c);
      v4i g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = __uint_as_float((uint32_t)a[i] << 16), a1 = __uint_as_float((uint32_t)a[i] & 0xFFFF0000u);
        const float b0 = __uint_as_float((uint32_t)b[i] << 16), b1 = __uint_as_float((uint32_t)b[i] & 0xFFFF0000u);
        acc = fmaf(a0, b0, acc);
        acc = fmaf(a1, b1, acc);
        g[i] = (int)pack_bf16x2(w * a0, w * a1);
      }
      *(v4i *)(o + c) = g;
    } else {
      const float a0 = bf16_to_f32(d[c]);
      acc = fmaf(a0, bf16_to_f32(y[c]), acc);
      store_elem(o + c, w * a0);
    }
  }
  acc = wave_sum(acc);
  if (lane == 0) p.dw[s] = acc;
}

}  // namespace mxg
