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
  int64_t tpb;                           // tokens per row of counts, a multiple of ROUTE_TG
  int64_t tpc;                           // tokens per block of the choice: tpb, or half of it
  bool halves;                           // a count is the sum of two bytes, one per block of the choice
};

// LDS of the placement: which tokens of a group of 64 chose each expert.
struct RoutePlace {
  uint32_t mask[MOE_MAX_E][2];
  int32_t base[MOE_MAX_E];               // next row of each expert
  int32_t total[MOE_MAX_E];
  int32_t wave_sum[16];
  int32_t used;
};

// x of the lane that the DPP control names (within 16 lanes).
template <int CTRL>
__device__ inline int dpp(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ inline float dpp(float x) {
  return __int_as_float(dpp<CTRL>(__float_as_int(x)));
}
template <int CTRL>
__device__ inline double dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = (uint32_t)dpp<CTRL>((int)(uint32_t)u), hi = (uint32_t)dpp<CTRL>((int)(u >> 32));
  return __builtin_bit_cast(double, hi << 32 | lo);
}
// x of both members of the lane's pair of 16-lane rows (HALF: of wave halves).
template <bool HALF>
__device__ inline void both(int x, int &y0, int &y1) {
  if constexpr (HALF) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    y0 = r[0], y1 = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    y0 = r[0], y1 = r[1];
  }
}
template <bool HALF>
__device__ inline void both(double x, double &y0, double &y1) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  int l0, l1, h0, h1;
  both<HALF>((int)(uint32_t)u, l0, l1);
  both<HALF>((int)(u >> 32), h0, h1);
  y0 = __builtin_bit_cast(double, (uint64_t)(uint32_t)h0 << 32 | (uint32_t)l0);
  y1 = __builtin_bit_cast(double, (uint64_t)(uint32_t)h1 << 32 | (uint32_t)l1);
}
// op over each run of LPT (16 or 64) lanes, in all of them: lane exchanges
// in registers (neighbours, pairs, mirrored eights and sixteens, rows,
// halves), with no trip through LDS.
template <bool HALF>
__device__ inline void both(float x, float &y0, float &y1) {
  int a, b;
  both<HALF>(__float_as_int(x), a, b);
  y0 = __int_as_float(a), y1 = __int_as_float(b);
}
template <int LPT, class T, class Op>
__device__ inline T lanes_reduce(T x, Op op) {
  x = op(x, dpp<0xB1>(x));               // quad_perm 1 0 3 2
  x = op(x, dpp<0x4E>(x));               // quad_perm 2 3 0 1
  x = op(x, dpp<0x141>(x));              // row_half_mirror
  x = op(x, dpp<0x140>(x));              // row_mirror
  if constexpr (LPT == 64) {
    T a, b;
    both<false>(x, a, b);
    x = op(a, b);
    both<true>(x, a, b);
    x = op(a, b);
  }
  return x;
}
struct OpMax {
  __device__ double operator()(double a, double b) const { return fmax(a, b); }
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct OpAdd {
  __device__ double operator()(double a, double b) const { return a + b; }
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct OpMin {
  __device__ int operator()(int a, int b) const { return min(a, b); }
  __device__ float operator()(float a, float b) const { return fminf(a, b); }
};

// e^-t for t >= 0 in 64 bits, within about an ulp: -t = n ln 2 + r, |r| <=
// ln 2 / 2, with ln 2 in two parts as Cody and Waite reduce arguments (its first
// 32 bits, n times which is exact, and the rest rounded to 64 bits), then the
// exponential series of r to r^13 (what follows is below 2^-57).
__device__ inline double exp_neg(double t) {
  t = fmin(t, 750.0);                    // e^-750 < 2^-1075
  const double n = rint(t * -1.4426950408889634);
  const double r = fma(n, -0x1.a39ef35793c76p-33, fma(n, -0x1.62e42feep-1, -t));
  double q = 1.0 / 6227020800.0;
  q = fma(q, r, 1.0 / 479001600.0);
  q = fma(q, r, 1.0 / 39916800.0);
  q = fma(q, r, 1.0 / 3628800.0);
  q = fma(q, r, 1.0 / 362880.0);
  q = fma(q, r, 1.0 / 40320.0);
  q = fma(q, r, 1.0 / 5040.0);
  q = fma(q, r, 1.0 / 720.0);
  q = fma(q, r, 1.0 / 120.0);
  q = fma(q, r, 1.0 / 24.0);
  q = fma(q, r, 1.0 / 6.0);
  q = fma(q, r, 0.5);
  q = fma(q, r, 1.0);
  q = fma(q, r, 1.0);
  return __builtin_ldexp(q, (int)n);
}

// 1 / d for d in [1, 2^1000] by two Newton steps from the hardware's estimate
// (exact for d = 1).
__device__ inline double recip(double d) {
  double r = __builtin_amdgcn_rcp(d);
  r = fma(fma(-d, r, 1.0), r, r);
  return fma(fma(-d, r, 1.0), r, r);
}

// 1 / (1 + e^-x); 0 where e^-x is past 64 bits.
__device__ inline double logistic(double x) {
  const double t = fabs(x), e = exp_neg(t), r = recip(1.0 + e);
  return x >= 0.0 ? r : (t > 709.78 ? 0.0 : e * r);
}

// The lane's `cnt` <= VPT consecutive logits, -inf past them: four at a time
// (at any alignment) where all four are there.
template <class IN, int VPT>
__device__ inline void load_logits(const IN *p, int cnt, float (&l)[VPT]) {
#pragma unroll
  for (int j = 0; j < VPT; j += 4) {
    if (j + 4 <= cnt) {
      IN u[4];
      __builtin_memcpy(u, p + j, sizeof(u));
#pragma unroll
      for (int k = 0; k < 4; ++k) l[j + k] = load_elem(u + k);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) l[j + k] = j + k < cnt ? load_elem(p + j + k) : -__builtin_inff();
    }
  }
}

// A token's LPT lanes hold `per` <= VPT consecutive experts each; an expert
// group owns lpg consecutive lanes, so a group's statistics need no more than
// shuffles among them.
struct LaneSpan {
  int gi, e0, cnt;                       // group, first expert, experts of this lane
};
__device__ inline LaneSpan lane_span(const RouteArgs &p, bool live, int sub) {
  const int n = p.E / p.n_group;
  LaneSpan s;
  s.gi = sub / p.lpg;
  const int part = sub % p.lpg;
  s.e0 = s.gi * n + part * p.per;
  s.cnt = (live && s.gi < p.n_group) ? max(0, min(p.per, n - part * p.per)) : 0;
  return s;
}

// An available logit (not -inf, not NaN) and its finite stand-in.
__device__ inline bool avail(float x) { return x > -__builtin_inff(); }
__device__ inline float fin(float x) { return fminf(x, 3.402823466e38f); }

// The largest available logit and 1 / (sum of e^(l - m)).
template <int LPT, int VPT>
__device__ inline void softmax_stats(const float (&l)[VPT], double &m, double &inv) {
  float mm = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < VPT; ++j) mm = fmaxf(mm, avail(l[j]) ? fin(l[j]) : -__builtin_inff());
  m = (double)lanes_reduce<LPT>(mm, OpMax());
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) sum += avail(l[j]) ? exp_neg(m - (double)fin(l[j])) : 0.0;
  inv = recip(fmax(lanes_reduce<LPT>(sum, OpAdd()), 1.0));
}

// The largest two of the lane's group, from the lane's own.
template <class T>
__device__ inline void group_best(const RouteArgs &p, T &g1, T &g2) {
  for (int d = 1; d < p.lpg; d <<= 1) {
    const T o1 = __shfl_xor(g1, d, 64), o2 = __shfl_xor(g2, d, 64);
    g2 = fmax(fmin(g1, o1), fmax(g2, o2));
    g1 = fmax(g1, o1);
  }
}

// How many groups come before the lane's.
template <int LPT, class T>
__device__ inline int group_rank(const RouteArgs &p, T gs, int gi) {
  int rank = 0;
  for (int g = 0; g < p.n_group; ++g) {
    const T o = __shfl(gs, g * p.lpg, LPT);
    rank += (o > gs || (o == gs && g < gi)) ? 1 : 0;
  }
  return rank;
}

// One rank of the choice: the largest value over the lanes, then the lowest
// expert that holds it, which becomes NaN (no maximum takes it); -1: none.
// (Where `at` is past a lane's experts it names a value that is -inf.)
template <int LPT, int VPT, class T>
__device__ inline int take_best(T (&v)[VPT], int e0, T &best) {
  T bv = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < VPT; ++j) bv = fmax(bv, v[j]);
  bv = lanes_reduce<LPT>(bv, OpMax());
  int jl = 0x7FFF;
#pragma unroll
  for (int j = VPT - 1; j >= 0; --j) jl = v[j] == bv ? j : jl;
  const int be = lanes_reduce<LPT>(jl < VPT ? e0 + jl : 0x7FFFFFFF, OpMin());
  best = bv;
  const int chosen = bv > -__builtin_inff() ? be : -1, at = chosen - e0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) v[j] = at == j ? (T)__builtin_nanf("") : v[j];
  return chosen;
}

// The choice with every value in 64 bits.  Lane `sub` < topk returns the id
// of rank `sub`.
template <class IN, int LPT, int VPT>
__device__ inline int choose64(const RouteArgs &p, const IN *row, const LaneSpan &sp, int sub) {
  const double NONE = -__builtin_inf();
  float l[VPT];
  load_logits<IN, VPT>(row + sp.e0, sp.cnt, l);
  const bool top2 = p.n_group > 1 && p.group_score == MOE_GROUP_TOP2;
  double m = 0.0, inv = 0.0;
  if (p.score == MOE_SOFTMAX) softmax_stats<LPT>(l, m, inv);
  double v[VPT];
  double g1 = NONE, g2 = NONE;           // the lane's two best of its group
  float b[VPT];
  if (p.bias) load_logits<float, VPT>(p.bias + sp.e0, sp.cnt, b);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    v[j] = NONE;
    if (avail(l[j])) {
      const double x = (double)fin(l[j]);
      double s = p.score == MOE_SOFTMAX ? exp_neg(m - x) * inv : logistic(x);
      if (p.bias) s += (double)b[j];
      v[j] = p.bias ? s : (double)l[j];
      const double gv = top2 ? s : v[j];
      g2 = fmax(g2, fmin(g1, gv));
      g1 = fmax(g1, gv);
    }
  }
  if (p.n_group > 1) {
    group_best(p, g1, g2);
    if (group_rank<LPT>(p, top2 && g2 > NONE ? g1 + g2 : g1, sp.gi) >= p.topk_group) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) v[j] = NONE;
    }
  }
  int id = -1;
  for (int r = 0; r < p.topk; ++r) {
    double best;
    const int c = take_best<LPT>(v, sp.e0, best);
    if (sub == r) id = c;
  }
  return id;
}

// How many groups come before the lane's by 64-bit values of the lane's best
// three experts (by v, its 32-bit choice values); `open` where its fourth is
// too close to its second to leave it out.
template <class IN, int LPT, int VPT, class Apart>
__device__ inline int groups64(const RouteArgs &p, const IN *row, const LaneSpan &sp, const float (&v)[VPT],
                               Apart apart, bool &open) {
  const float NONE = -__builtin_inff();
  float a[4] = {NONE, NONE, NONE, NONE};
  int at[3] = {0, 0, 0};
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const float x = v[j];
    const bool b0 = x > a[0], b1 = x > a[1], b2 = x > a[2];
    a[3] = b2 ? a[2] : fmaxf(a[3], x);
    at[2] = b1 ? at[1] : (b2 ? j : at[2]);
    a[2] = b1 ? a[1] : (b2 ? x : a[2]);
    at[1] = b0 ? at[0] : (b1 ? j : at[1]);
    a[1] = b0 ? a[0] : (b1 ? x : a[1]);
    at[0] = b0 ? j : at[0];
    a[0] = b0 ? x : a[0];
  }
  open = p.bias && !apart(a[1], a[3]);
  double g1 = -__builtin_inf(), g2 = g1;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (a[k] > NONE) {
      const int e = sp.e0 + at[k];
      const double x = logistic((double)fin(load_elem(row + e))) + (p.bias ? (double)p.bias[e] : 0.0);
      g2 = fmax(g2, fmin(g1, x));
      g1 = fmax(g1, x);
    }
  }
  group_best(p, g1, g2);
  const bool top2 = p.group_score == MOE_GROUP_TOP2;
  return group_rank<LPT>(p, top2 && g2 > -__builtin_inf() ? g1 + g2 : g1, sp.gi);
}

// The choice from values in 32 bits, where they can decide it.  Without a
// bias they are the logits themselves.  A sigmoid's score plus bias is within
// 4e-7 + 6e-8 |value| of the exact sum (the exponential and the reciprocal
// one unit in the last place each, one rounding for the sum), so values
// further apart than `apart` are in their exact order: the best topk + 1
// experts by 32 bits hold the topk best wherever the topk-th is so far from
// the first one left, and 64-bit values of these candidates alone, one per
// lane, give the choice and its order.  Groups are decided by 32 bits where
// every kept one stays before every dropped one whatever their errors, else by
// groups64; the error of a sum of two is that of its terms, which may be far
// larger than the sum: 8e-7 + 1.2e-7 (|g1| + |g2|), and a rounding more for
// the interval's ends.
// `open` is set where this does not decide, for choose64: that takes several
// values within 1e-6 of each other at one border.
// 16384 tokens of 256 experts in 8 groups, 8 chosen by sigmoid and bias: the
// whole call 34 us with all values in 64 bits, 25 us this way.
template <class IN, int LPT, int VPT>
__device__ inline int choose32(const RouteArgs &p, const IN *row, const LaneSpan &sp, int sub, bool &open) {
  const float NONE = -__builtin_inff();
  float v[VPT];
  load_logits<IN, VPT>(row + sp.e0, sp.cnt, v);
  const bool top2 = p.n_group > 1 && p.group_score == MOE_GROUP_TOP2;
  auto apart = [](float hi, float lo) { return lo == -__builtin_inff() || hi - lo > 1.6e-6f + 2.5e-7f * (fabsf(hi) + fabsf(lo)); };
  float g1 = NONE, g2 = NONE;
  if (p.bias || top2) {
    float b[VPT];
    if (p.bias) load_logits<float, VPT>(p.bias + sp.e0, sp.cnt, b);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const bool ok = avail(v[j]);
      const float s = logistic_f32(v[j]) + (p.bias ? b[j] : 0.0f);
      v[j] = ok ? (p.bias ? s : v[j]) : NONE;
      const float gv = ok ? (top2 ? s : v[j]) : NONE;
      g2 = fmaxf(g2, fminf(g1, gv));
      g1 = fmaxf(g1, gv);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      v[j] = avail(v[j]) ? v[j] : NONE;
      g1 = fmaxf(g1, v[j]);
    }
  }
  open = false;
  if (p.n_group > 1) {
    group_best(p, g1, g2);
    const float gs = top2 && g2 > NONE ? g1 + g2 : g1;
    bool out = group_rank<LPT>(p, gs, sp.gi) >= p.topk_group;
    if (p.bias || top2) {
      const bool some = g1 > NONE;       // else no available expert: comes last
      const float err = 8e-7f + 2.5e-7f * (fabsf(g1) + (top2 && g2 > NONE ? fabsf(g2) : 0.0f));
      const bool known = err < -NONE;    // the sum is in 32-bit range
      const float lo = some && known ? gs - err : NONE, hi = some ? (known ? gs + err : -NONE) : NONE;
      const float kept = lanes_reduce<LPT>(out ? -NONE : lo, OpMin());
      const float left = lanes_reduce<LPT>(out ? hi : NONE, OpMax());
      if (__any(left > NONE && !(kept > left))) out = groups64<IN, LPT, VPT>(p, row, sp, v, apart, open) >= p.topk_group;
    }
    if (out) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) v[j] = NONE;
    }
  }
  int id = -1;
  float last = NONE, next;
  for (int r = 0; r < p.topk; ++r) {
    const int c = take_best<LPT>(v, sp.e0, last);
    if (sub == r) id = c;
  }
  if (!p.bias) return id;
  int cand = p.topk;
  if (cand < LPT) {
    const int c = take_best<LPT>(v, sp.e0, next);
    if (sub == cand) id = c;
    ++cand;
  }
  float rest = NONE;
#pragma unroll
  for (int j = 0; j < VPT; ++j) rest = fmaxf(rest, v[j]);
  open |= !apart(last, lanes_reduce<LPT>(rest, OpMax()));
  // order by the 64-bit values; lanes past the last chosen stay where they are
  double x = -__builtin_inf();
  if (id >= 0) x = logistic((double)fin(load_elem(row + id))) + (double)p.bias[id];
  int rank = 0;
  for (int r = 0; r < cand; ++r) {
    const double o = __shfl(x, r, LPT);
    const int oid = __shfl(id, r, LPT);
    rank += (o > x || (o == x && oid < id)) ? 1 : 0;
  }
  if (id < 0) rank = sub;
  const int base = (int)(threadIdx.x & 63) - sub;
  id = __builtin_amdgcn_ds_permute((base + rank) * 4, id);
  return sub < p.topk ? id : -1;
}

// One token's choice and weights by LPT lanes: the id of rank `sub` (-1:
// none) in lanes sub < topk, and its weight.  Scores that differ in FP32's
// last bits decide between experts.  Softmax with a bias, or with groups by
// their best two, has no 32-bit path: 16384 x 256, top 8, takes 33 us with a bias
// and 24 with sigmoid scores.
template <class IN, int LPT, int VPT>
__device__ inline int route_token(const RouteArgs &p, const IN *row, bool live, int sub, float &weight) {
  const LaneSpan sp = lane_span(p, live, sub);
  const bool sm = p.score == MOE_SOFTMAX;
  bool open = true;
  int id = -1;
  if (!(sm && (p.bias || (p.n_group > 1 && p.group_score == MOE_GROUP_TOP2))))
    id = choose32<IN, LPT, VPT>(p, row, sp, sub, open);
  if (__any(open)) id = choose64<IN, LPT, VPT>(p, row, sp, sub);

  // weights, one rank per lane
  const bool has = id >= 0;
  const double x = has ? (double)fin(load_elem(row + id)) : 0.0;
  double w;
  if (p.renorm) {
    // shares of the chosen: a common factor e^-top keeps them in range
    const double mine = has ? (sm ? x : fmin(x, 0.0)) : -__builtin_inf();
    const double top = lanes_reduce<LPT>(mine, OpMax());
    w = 0.0;
    if (has) w = exp_neg(top - mine) * (sm ? 1.0 : recip(1.0 + exp_neg(fabs(x))));
    const double tot = lanes_reduce<LPT>(w, OpAdd());
    w = has ? w / tot : 0.0;
  } else if (sm) {
    float l[VPT];
    load_logits<IN, VPT>(row + sp.e0, sp.cnt, l);
    double m, inv;
    softmax_stats<LPT>(l, m, inv);
    w = has ? exp_neg(m - x) * inv : 0.0;
  } else {
    w = has ? logistic(x) : 0.0;
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
// its rows itself.  Blocks of up to 1024 threads leave a lane 128 registers:
// choose64's doubles spill 56 to 87 of them with 32 experts per lane and about
// 12 with 16 and ONE (16384 x 1000 in 20 groups 125 us, 64 x 1000 98, 64 x 256 in 8
// groups 18).
template <class IN, int LPT, int VPT, bool MAPS, bool ONE>
__global__ void route_kernel(RouteArgs p) {
  __shared__ int32_t ids[MAPS ? ROUTE_TG * MOE_MAX_TOPK : 1];
  __shared__ RoutePlace pl;
  const int tid = threadIdx.x, sub = tid & (LPT - 1);
  const int per_pass = blockDim.x / LPT;
  const int64_t t_end = min(p.T, ((int64_t)blockIdx.x + 1) * p.tpc);
  if constexpr (MAPS) {
    for (int e = tid; e < p.E; e += blockDim.x) pl.total[e] = pl.base[e] = 0;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * p.tpc; t0 < t_end; t0 += ROUTE_TG) {
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
    for (int e = tid; e < p.E; e += blockDim.x) {
      if (p.halves) ((uint8_t *)p.counts)[((int64_t)(blockIdx.x >> 1) * p.Ep + e) * 2 + (blockIdx.x & 1)] = (uint8_t)pl.total[e];
      else p.counts[(int64_t)blockIdx.x * p.Ep + e] = (uint16_t)pl.total[e];
    }
  }
}

// The second kernel of a call of more than 64 tokens: every block sums the
// counts of all blocks (its own first rows and the experts' totals), then
// places its tokens.
// Up to 16 waves per block: with 256 threads a block of 16384 tokens' call
// read the 128 KB of counts in 32 dependent rounds, 9.6 us.  It takes 8.1 us now;
// beside the reads of the counts it is LDS accesses that count, half of which
// conflict (the sums' atomics at a stride of four words, from as many row lanes
// as a column has, and the two words of a mask).
__global__ __launch_bounds__(1024) void route_place_kernel(RouteArgs p) {
  __shared__ int32_t ids[ROUTE_TG * MOE_MAX_TOPK];
  __shared__ RoutePlace pl;
  const int tid = threadIdx.x;
  const int nthr = (int)blockDim.x;
  for (int e = tid; e < MOE_MAX_E; e += nthr) pl.total[e] = pl.base[e] = 0;
  __syncthreads();
  // the block's first ids are on their way while the counts are summed
  const int64_t first = (int64_t)blockIdx.x * p.tpb, t_end = min(p.T, first + p.tpb);
  {
    const int ns = (int)min((int64_t)ROUTE_TG, t_end - first) * p.topk;
    for (int s = tid; s < ns; s += nthr) ids[s] = p.ids[first * p.topk + s];
  }
  const int nv = p.Ep / 4, rows = nthr / nv;       // columns of four experts, row lanes
  const int col = tid % nv, r0 = tid / nv;
  if (r0 < rows) {
    int tot[4] = {0, 0, 0, 0}, bef[4] = {0, 0, 0, 0};
    // every block starts at its own row: in step they would read one row of
    // counts, one L2 channel, at a time
    const int turn = (int)blockIdx.x;
#pragma unroll 8
    for (int i = r0; i < p.nblk; i += rows) {
      const int b = i + turn < p.nblk ? i + turn : i + turn - p.nblk;
      const v2i x = *(const v2i *)(p.counts + (int64_t)b * p.Ep + col * 4);
      const bool before = b < (int)blockIdx.x;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t u = (uint32_t)x[k];
        const uint32_t c = p.halves ? (u & 0x00FF00FFu) + ((u >> 8) & 0x00FF00FFu) : u;
        const int lo = (int)(c & 0xFFFF), hi = (int)(c >> 16);
        tot[2 * k] += lo;
        tot[2 * k + 1] += hi;
        bef[2 * k] += before ? lo : 0;
        bef[2 * k + 1] += before ? hi : 0;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (col * 4 + k < p.E) {
        atomicAdd(&pl.total[col * 4 + k], tot[k]);
        atomicAdd(&pl.base[col * 4 + k], bef[k]);
      }
    }
  }
  __syncthreads();
  route_bases(p, pl);
  for (int64_t t0 = first; t0 < t_end; t0 += ROUTE_TG) {
    const int ns = (int)min((int64_t)ROUTE_TG, t_end - t0) * p.topk;
    if (t0 != first) {
      __syncthreads();
      for (int s = tid; s < ns; s += nthr) ids[s] = p.ids[t0 * p.topk + s];
      __syncthreads();
    }
    route_mark(pl, ids, ns, p.topk, p.E);
    route_place(p, pl, ids, ns, t0);
  }
  route_tail(p, pl);
}

__global__ void moe_zero_sizes_kernel(int64_t *m_sizes, int E) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) m_sizes[e] = 0;
}

// ---------------------------------------------------------------------------
// Gradient of the weights: LPT lanes (16, or 64 where 16 do not hold the
// experts or choices) per token, each with up to VPT consecutive experts.  One
// pass: logits in, gradients out.  The chosen experts' own shares, one per
// lane, reach the lanes of their experts through LDS.  What bounds it is
// instructions rather than bytes: with a wave per token 16384 tokens of 128
// experts took 9.4 us, with four tokens per
// wave 6.6.
struct RouteGradArgs {
  const void *logits;
  const int32_t *ids;
  const float *grad;
  void *dlogits;
  int64_t T;
  int E, topk, score, renorm;
  float scale;
  int per;                               // experts per lane
};

__device__ inline float wave_sum(float x) { return lanes_reduce<64>(x, OpAdd()); }

// A logit's finite stand-in; -inf where the expert is not available (-inf
// or NaN).
__device__ inline float avail_logit(float x) {
  return x > -__builtin_inff() ? fminf(x, 3.402823466e38f) : -__builtin_inff();
}

// Four consecutive values in one store, at any alignment.
__device__ inline void store4(float *p, const float *v) { __builtin_memcpy(p, v, 16); }
__device__ inline void store4(uint16_t *p, const float *v) {
  const uint32_t u[2] = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  __builtin_memcpy(p, u, 8);
}

template <class IN, int LPT, int VPT>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradArgs p) {
  // expert j of lane i at j LPT + i, tokens 16 banks apart: no conflicts
  __shared__ float share[256 / LPT][LPT * VPT + 16];
  const int tid = threadIdx.x, sub = tid & (LPT - 1);
  const int64_t tw = (int64_t)blockIdx.x * (256 / LPT) + tid / LPT;
  const bool live = tw < p.T;
  const int64_t t = live ? tw : 0;
  const IN *row = (const IN *)p.logits + t * p.E;
  const float NI = -__builtin_inff();
  const int e0 = sub * p.per, cnt = max(0, min(p.per, p.E - e0));
  float l[VPT];
  load_logits<IN, VPT>(row + e0, cnt, l);
  float *mine_row = share[tid / LPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    l[j] = avail_logit(l[j]);
    mine_row[j * LPT + sub] = 0.0f;
  }
  // lane r holds choice r
  int id = -1;
  float c = 0.0f, x = NI;
  if (sub < p.topk) {
    id = p.ids[t * p.topk + sub];
    if (id < 0 || id >= p.E) id = -1;
    if (id >= 0) {
      x = avail_logit(load_elem(row + id));
      if (x > NI) c = p.scale * p.grad[t * p.topk + sub];
      else id = -1;
    }
  }
  const bool sm = p.score == MOE_SOFTMAX;
  float mine = 0.0f;                     // the chosen expert's own share of the gradient
  float m = 0.0f, inv = 0.0f, dot = 0.0f;
  if (p.renorm) {
    const float z = id >= 0 ? (sm ? x : fminf(x, 0.0f)) : NI;
    const float top = lanes_reduce<LPT>(z, OpMax());
    float w = id >= 0 ? expf(z - top) / (sm ? 1.0f : 1.0f + expf(-fabsf(x))) : 0.0f;
    const float tot = lanes_reduce<LPT>(w, OpAdd());
    w = id >= 0 ? w / tot : 0.0f;
    dot = lanes_reduce<LPT>(c * w, OpAdd());
    mine = w * (c - dot);
    if (!sm) mine *= 1.0f / (1.0f + expf(x));             // 1 - s
  } else if (sm) {
    float mm = NI;
#pragma unroll
    for (int j = 0; j < VPT; ++j) mm = fmaxf(mm, l[j]);
    m = lanes_reduce<LPT>(mm, OpMax());
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      l[j] = l[j] > NI ? expf(l[j] - m) : 0.0f;
      s += l[j];
    }
    s = lanes_reduce<LPT>(s, OpAdd());
    inv = s > 0.0f ? 1.0f / s : 0.0f;
    dot = lanes_reduce<LPT>(id >= 0 ? c * (expf(x - m) * inv) : 0.0f, OpAdd());
    mine = c;
  } else {
    // s (1 - s) = 1 / ((1 + e^x) (1 + e^-x)), e^-|x| <= 1
    const float ex = expf(-fabsf(x)), s1 = 1.0f / (1.0f + ex);
    mine = id >= 0 ? c * ex * s1 * s1 : 0.0f;
  }
  __syncthreads();
  if (id >= 0) mine_row[id % p.per * LPT + id / p.per] = mine;
  __syncthreads();
  if (!live) return;
  IN *drow = (IN *)p.dlogits + t * p.E + e0;
#pragma unroll
  for (int j = 0; j < VPT; j += 4) {
    float d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      d[k] = mine_row[(j + k) * LPT + sub];
      if (!p.renorm && sm) d[k] = l[j + k] > 0.0f ? l[j + k] * inv * (d[k] - dot) : 0.0f;
    }
    if (j + 4 <= cnt) {
      store4(drow + j, d);
    } else {
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (j + k < cnt) store_elem(drow + j + k, d[k]);
    }
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
//
// A stream: 4096 x 14336 BF16 in 34.4 us (5.1 TB/s), 2049 x 7168 to eight rows
// each in 27.0 (5.5 TB/s); the codes bypass the caches (36.3 and 30.2 through
// them), x does not (bypassing cost 2 %).
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
  const int64_t t = flat_block() * (256 / GROUP) + tid / GROUP;
  if (t >= p.T) return;                  // GROUP 256: the whole workgroup
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
      __builtin_nontemporal_store(q, (v4i *)(p.codes + t * p.K + 16 * c));
      return;
    }
    for (int k = 0; k < p.topk; ++k) {
      const int64_t r = p.row_of[t * p.topk + k];
      if (r >= 0 && r < p.T * p.topk) __builtin_nontemporal_store(q, (v4i *)(p.codes + r * p.K + 16 * c));
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
// lane (8: 16-byte accesses; 1 where N is not a multiple of 8).  A stream: 4096
// tokens x 8 rows of 7168 in 89.5 us, 5.9 TB/s (a copy of 1 GiB reaches 5.04),
// 104 us with its reads and writes through the caches.
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
#pragma unroll 8
  for (int k = 0; k < p.topk; ++k) {
    const int64_t r = p.row_of[t * p.topk + k];
    if (r < 0 || r >= p.rows) continue;
    const float w = p.w[t * p.topk + k];
    const uint16_t *src = p.y + r * p.N + c;
    if constexpr (VEC == 8) {
      const v4i u = __builtin_nontemporal_load((const v4i *)src);
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
    __builtin_nontemporal_store(o, (v4i *)dst);
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

// One workgroup (up to four waves) per token: its row of dout stays in
// registers for eight slots at a time, whose rows of y are in flight
// together; the dot products end in a wave reduction and one sum over the
// waves.  With a wave per (token, slot) instead, dout came from the caches
// once per slot: 2049 tokens x 8 x 4096 62.1 us.
template <int VEC>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineGradArgs p) {
  constexpr int S = 8;
  __shared__ float part[4][S];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = (int)blockDim.x >> 6;
  const int64_t t = flat_block();
  if (t >= p.T) return;
  const uint16_t *d = p.dout + t * p.N;
  for (int k0 = 0; k0 < p.topk; k0 += S) {
    int64_t row[S];                      // -1: no row
    float w[S], acc[S];
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const bool in = k0 + k < p.topk;
      const int64_t s = t * p.topk + (in ? k0 + k : 0), r = p.row_of[s];
      row[k] = in && r >= 0 && r < p.rows ? r : -1;
      w[k] = p.w[s];
      acc[k] = 0.0f;
    }
    for (int64_t c = (int64_t)tid * VEC; c < p.N; c += (int64_t)blockDim.x * VEC) {
      if constexpr (VEC == 8) {
        const v4i a = *(const v4i *)(d + c);
        v4i y[S];
#pragma unroll
        for (int k = 0; k < S; ++k)
          y[k] = row[k] >= 0 ? __builtin_nontemporal_load((const v4i *)(p.y + row[k] * p.N + c)) : (v4i){0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < S; ++k) {
          if (row[k] < 0) continue;
          v4i g;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = __uint_as_float((uint32_t)a[i] << 16), a1 = __uint_as_float((uint32_t)a[i] & 0xFFFF0000u);
            acc[k] = fmaf(a0, __uint_as_float((uint32_t)y[k][i] << 16), acc[k]);
            acc[k] = fmaf(a1, __uint_as_float((uint32_t)y[k][i] & 0xFFFF0000u), acc[k]);
            g[i] = (int)pack_bf16x2(w[k] * a0, w[k] * a1);
          }
          __builtin_nontemporal_store(g, (v4i *)(p.dy + row[k] * p.N + c));
        }
      } else {
        const float a0 = bf16_to_f32(d[c]);
#pragma unroll
        for (int k = 0; k < S; ++k) {
          if (row[k] < 0) continue;
          acc[k] = fmaf(a0, bf16_to_f32(p.y[row[k] * p.N + c]), acc[k]);
          store_elem(p.dy + row[k] * p.N + c, w[k] * a0);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const float sum = wave_sum(acc[k]);
      if (lane == 0) part[wave][k] = sum;
    }
    __syncthreads();
    if (tid < S && k0 + tid < p.topk) {
      float sum = part[0][tid];
      for (int v = 1; v < waves; ++v) sum += part[v][tid];
      p.dw[t * p.topk + k0 + tid] = sum;
    }
    __syncthreads();
  }
}

}  // namespace mxg
