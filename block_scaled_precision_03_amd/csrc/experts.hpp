// The experts of a mixture-of-experts layer for a few tokens, in two kernels:
//   out[t] = R[t] + sum_e share[t,e] W2[e] act( W1[e] x[t] ),
//   share[t,e] = sum of w[t,j] over the slots j with ids[t,j] = e.
// Few tokens make this a stream of the chosen experts' weights: each comes from
// memory once, in units of 128 bytes of K, and is turned into BF16 in
// registers (codes of every format are exact in BF16, and so are codes times a
// power of two inside its range), so that the activations stay what they are: x
// in BF16, sums in FP32.  act's result h is kept as two BF16 (its rounding
// and the rounding of what that leaves, 16 bits of mantissa): rounded to one, it
// would add as much error as the rounding of out (2.3e-3 instead of 1.7e-3 of
// the result's norm); the second costs a matrix instruction, which the stream hides.
// The two parts' products have sums of their own: an infinite weight times the low
// part is an infinity of either sign, or NaN, beside the high part's infinity (see
// join_planes).
//
// Tokens of an expert beyond 16 make further records of up to 16 of it.
// experts_up_kernel: a workgroup per (record, tile of W1's rows); one more
// writes the records and their tokens for experts_down_kernel: a workgroup per
// tile of out's columns (and split of the records), which walks the records'
// units of K as one list and adds share * y to sums in LDS when a record ends.
// No sum's order depends on timing.
//
// Two ways of sharing the work of a workgroup's four waves:
//   private (one or two tokens): each wave has a ring of stages of its own; up:
//     64 rows of the weight, 16 per wave, or, where that makes too few
//     workgroups, 16 rows with K split over the waves; down: 16 rows (columns
//     of out), the list split over the waves, whose sums meet at the end.
//   shared: 64 rows, 16 per wave, one ring; the activations of a stage, up to 16
//     rows of them, are brought once for all four waves.
// Both sides for one token, the call's us (copies of the weights in turn, none of
// them cached), private and shared: 4 of 1024 x 512 INT8 10.2, 13.5; 8 of 7168 x 2304
// MXFP4 53.7, 61.8.
//
// Bound by memory where the experts are large: 16 tokens, 8 each, 64 experts of
// 7168 x 2304 INT8, SwiGLU 487 to 493 us, 5.7 TB/s of weights (records of up to 8 tokens;
// a fifth wave that does the loads made the two kernels a third and a quarter
// slower); 1 token, 8 of them in MXFP4 53 us, 4.0 TB/s.  By the two kernels' starts
// where they are small (1 token, 4 of 1024 x 512: 9.7 us).
#pragma once
#include "small.hpp"

namespace mxg {

enum : int { WF_INT8 = 0, WF_BF16 = 1, WF_E4M3 = 2, WF_E5M2 = 3, WF_E2M1 = 4, WF_BLOCK = 5 };
constexpr int EXP_MAX_T = 64, EXP_MAX_E = 1024, EXP_MAX_TOPK = 32;
constexpr int EXP_ROWS = 16;                   // tokens of a record at most
constexpr int EXP_WAVES = 4;
constexpr int EXP_SPLIT_BLOCKS = 512;          // workgroups of the second kernel that splits of the list may make

struct ExpertRec {
  int32_t e, base, n, pad;                     // expert, its first pair, its tokens (1 .. 16)
};
struct ExpertPair {
  int32_t t;
  float share;
};

struct ExpertsArgs {
  const uint16_t *x;                           // [T, D]
  const int32_t *ids;                          // [T, topk]
  const float *w;                              // [T, topk]
  const uint8_t *w1, *w2;
  const void *s1, *s2;
  const uint16_t *residual;                    // [T, D] or null
  uint16_t *out;                               // [T, D]
  uint16_t *h;                                 // [2][T topk, F]: high parts, low parts, by pair
  int32_t *count;                              // number of records
  int32_t *arrived;                            // [tiles of the second kernel]: splits that are done
  ExpertRec *rec;                              // [records]
  ExpertPair *pair;                            // [<= T topk], by expert, then by token
  float *part;                                 // [splits][T][D]: sums of the list's splits
  int64_t D, F, N1;                            // N1 rows of W1[e]: F or 2 F
  int T, E, topk, act;
  int up_tiles, down_tiles, splits;
  int rows;                                    // tokens of a record at most: 8 or 16
  bool split_k;                                // private, up: K split over the waves, else 16 rows each
};

// What 16 bytes of a row hold.
template <int WF> struct WeightFormat {
  static constexpr int CODES = WF == WF_BF16 ? 8 : WF == WF_E2M1 ? 32 : 16;   // values in 16 bytes
  static constexpr int UNIT = 8 * CODES;                                      // values in a 128-byte unit
  static constexpr int XPITCH = 2 * UNIT;                                     // bytes of an activation row's unit
  static constexpr int SUB = CODES / 8;                                       // matrix instructions per 16 bytes
  static constexpr bool MX = WF == WF_E4M3 || WF == WF_E5M2 || WF == WF_E2M1;
  // tokens up to which the waves work apart: what one DMA brings of them, in
  // two planes
  static constexpr int PRIVATE_T = WF == WF_E2M1 ? 1 : 2;
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

// A wave's stream of stages through a ring in LDS.  A stage is one 128-byte
// unit of K of the wave's 16 weight rows, with its scales, and the same
// values of up to RC activation rows in PL planes (private: as many as make
// 1 KiB, one DMA); DOWN: the record's pairs too.
// All of it comes by DMA (nothing in registers while it is in flight), a
// constant number of DMAs per stage, so that the counter of outstanding ones tells
// which stages have landed: stages that do not exist are asked for past the end
// of their resources, which writes zeros and reads no memory.
//
// LDS of a stage: [W: 4 x 2 KiB][X][S: 4 x 256 B][pairs],
// a quarter of W and S per wave; X and the pairs a quarter per wave (private)
// or for all (shared).
//   W: row r of 128 bytes, 16-byte piece p at position p ^ kswz(r); lane (i, q)
//     of a matrix instruction takes pieces q and q + 4 of row i.
//   X: rows of XPITCH bytes, piece p at position p ^ xswz(r): the values beside
//     weight piece p are pieces SUB p ..; each read's 16-lane phases (see kswz)
//     land on 16 different 16-byte bank groups: rows {0-3, 12-15} at one value of
//     q and {4-11} at the next, so the set of xswz of the first eight must not change
//     when it is shifted by the XOR of their pieces (1, 2 or 4).  That is not so with
//     8 rows of 256 bytes (records of up to 8 tokens of INT8, E4M3, E5M2 and block
//     weights), where both halves of a phase are the same 8 rows on the same 8 groups,
//     two accesses each: 0.4 of the LDS cycles of kernels that memory bounds.
//   S: the aligned dwords around a row's E8M0 scales of the unit (2 per row,
//     E2M1 4); the channel scales (INT8, DOWN); the unit's block scale.
template <int WF, int PL, int ROWS, bool DOWN, int U>
struct ExpertStream {
  static constexpr bool SHARED = ROWS > 0;     // activation rows of a shared stage; 0: private
  typedef WeightFormat<WF> F;
  static constexpr int RC = SHARED ? ROWS : F::PRIVATE_T;
  // the rows of one plane after the other, in DMAs of 1 KiB: shared, a share
  // of them per wave (the same number for each); private, one
  static constexpr int XPLANE = RC * F::XPITCH;
  static constexpr int XD = SHARED ? (PL * XPLANE + EXP_WAVES * 1024 - 1) / (EXP_WAVES * 1024) : 1;   // DMAs per wave
  static constexpr int XSIZE = EXP_WAVES * XD * 1024;
  static_assert(SHARED || PL * XPLANE <= 1024, "one DMA");
  static constexpr bool S = F::MX || WF == WF_BLOCK || (DOWN && WF == WF_INT8);
  static constexpr int W_OFF = 0, X_OFF = EXP_WAVES * 2048;
  static constexpr int S_OFF = X_OFF + XSIZE;
  static constexpr int P_OFF = S_OFF + (S ? EXP_WAVES * 256 : 0);
  // every wave brings the record's pairs, shared to the same place
  static constexpr int STAGE = P_OFF + (DOWN ? (SHARED ? 256 : EXP_WAVES * 256) : 0);
  static constexpr int LDS_BYTES = U * STAGE;
  static constexpr int DMAS = 2 + XD + (S ? 1 : 0) + (DOWN ? 1 : 0);
  static_assert((U - 1) * DMAS < 64, "vmcnt is 6 bits");

  __device__ static inline int xswz(int r) {
    if constexpr (WF == WF_BF16) return kswz(r);
    else if constexpr (WF == WF_E2M1) return (r & 3) ^ (r & 4 ? 12 : 0) ^ (r & 8);
    else return r;
  }

  int lane, w, i16, q;
  uint32_t lds0;
  uint32_t KB, K, SK, units;
  uint32_t vo, vo_tail;                        // weight rows: lane offsets; in the last unit
  uint32_t xv[XD], xv_tail[XD];                // activation rows
  uint32_t xplane;                             // bytes between planes in memory
  u32x4 rw, rs, rx, rp;
  uint32_t pair0;                              // byte offset of the record's pairs

  __device__ inline void init(uint8_t *smem, int64_t K_, u32x4 rx_, uint32_t xplane_) {
    lane = threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    i16 = lane & 15;
    q = lane >> 4;
    lds0 = lds_addr(smem);
    K = (uint32_t)K_;
    KB = (uint32_t)F::row_bytes(K_);
    SK = K / 32;
    units = (KB + 127) / 128;
    const int r8 = lane >> 3, piece = (lane & 7) ^ kswz(r8);
    vo = (uint32_t)r8 * KB + 16u * piece;
    vo_tail = 128u * (units - 1) + 16u * piece < KB ? vo : NOWHERE;
    rx = rx_;
    xplane = xplane_;
    rw = rs = rp = rsrc4(smem, 0);             // until the first record: nothing
    pair0 = 0;
#pragma unroll
    for (int k = 0; k < XD; ++k) xv[k] = xv_tail[k] = NOWHERE;
  }
  static constexpr uint32_t NOWHERE = 0x80000000u;

  // The wave's weight rows: n0 .. n0 + 15 of [N, K] of expert e, and their scales.
  __device__ inline void set_weight(const uint8_t *wt, const void *s, int64_t e, int64_t N, int64_t n0) {
    rw = rsrc4(wt + (e * N + n0) * KB, clamp_records((N - n0) * KB));
    if constexpr (F::MX) rs = rsrc4((const uint8_t *)s + (e * N + n0) * SK, clamp_records((N - n0) * SK));
    else if constexpr (WF == WF_BLOCK)
      rs = rsrc4((const float *)s + (e * (N / 128) + n0 / 128) * (K / 128), n0 < N ? 4 * (K / 128) : 0u);
    else if constexpr (S) rs = rsrc4((const float *)s + e * N + n0, clamp_records(4 * (N - n0)));
  }

  // The activation rows: row_at(r) is row r's byte offset, r < n.
  template <class RowAt>
  __device__ inline void set_rows(int n, RowAt row_at) {
#pragma unroll
    for (int k = 0; k < XD; ++k) {
      const int at = ((SHARED ? w * XD : 0) + k) * 1024 + 16 * lane, row = at / F::XPITCH;
      const int pl = row / RC, r = row % RC, piece = (at % F::XPITCH / 16) ^ xswz(r);
      xv[k] = r < n && pl < PL ? row_at(r) + pl * xplane + 16u * piece : NOWHERE;
      xv_tail[k] = (units - 1) * F::UNIT + 8u * piece < K ? xv[k] : NOWHERE;
    }
  }

  // Unit u (live: it exists) into ring slot sl.
  __device__ inline void issue(int sl, uint32_t u, bool live) {
    const uint32_t st = lds0 + (uint32_t)sl * STAGE;
    const bool last = u + 1 == units;
    const uint32_t vw = !live ? NOWHERE : last ? vo_tail : vo;
    const uint32_t wd = st + W_OFF + 2048u * w;
    dma_asm_v<16, 0>(wd, rw, vw, live ? 128u * u : 0u);
    dma_asm_v<16, 1024>(wd, rw, vw, live ? 128u * u + 8u * KB : 0u);
    const uint32_t xd = st + X_OFF + 1024u * XD * (uint32_t)w;
    static_for<0, XD>([&](auto kc) {
      constexpr int k = decltype(kc)::value;
      dma_asm_v<16, k * 1024>(xd, rx, !live ? NOWHERE : last ? xv_tail[k] : xv[k], live ? u * F::XPITCH : 0u);
    });
    if constexpr (S) {
      uint32_t v = NOWHERE;
      if constexpr (WF == WF_E2M1) v = (((uint32_t)(lane >> 2) * SK + 8u * u) & ~3u) + 4u * (lane & 3);
      else if constexpr (F::MX) v = lane < 32 ? (((uint32_t)(lane >> 1) * SK + 4u * u) & ~3u) + 4u * (lane & 1) : NOWHERE;
      else if constexpr (WF == WF_BLOCK) v = lane == 0 ? 4u * u : NOWHERE;
      else v = lane < 16 ? 4u * lane : NOWHERE;
      dma_asm_v<4>(st + S_OFF + 256u * w, rs, live ? v : NOWHERE, 0u);
    }
    if constexpr (DOWN)
      dma_asm_v<4>(st + P_OFF + (SHARED ? 0u : 256u * w), rp, live && lane < 32 ? 4u * lane : NOWHERE, live ? pair0 : 0u);
  }

  // Stage v has landed once at most the later stages' DMAs are outstanding
  // (U - 2 of them are in flight); the reads of the stage before it are done.
  __device__ static inline void wait() {
    constexpr int N = (U - 2) * DMAS;
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
    if constexpr (SHARED) __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  }

  // acc += the stage's product, plane by plane: the result lane holds weight
  // rows 4 q .. + 3 of activation row i.
  __device__ inline void consume(const uint8_t *smem, int sl, uint32_t u, v4f (&acc)[PL]) const {
    const uint8_t *st = smem + sl * STAGE;
    const uint8_t *wt = st + W_OFF + 2048 * w + i16 * 128;
    const int ri = i16 & (RC - 1), f = xswz(ri);
    const uint8_t *xt = st + X_OFF + (SHARED ? 0 : w * 1024) + ri * F::XPITCH;
    const uint8_t *sc = st + S_OFF + 256 * w;
    const v4i raw[2] = {lds_read16(wt + ((q ^ kswz(i16)) << 4)), lds_read16(wt + (((q + 4) ^ kswz(i16)) << 4))};
    v4f part[PL];
#pragma unroll
    for (int p = 0; p < PL; ++p) part[p] = WF == WF_BLOCK ? (v4f){0.f, 0.f, 0.f, 0.f} : acc[p];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int piece = q + 4 * h;
      float scale = 1.0f;
      if constexpr (F::MX) {
        const uint32_t skew = ((uint32_t)i16 * SK + u * (F::UNIT / 32)) & 3u;
        const int at = WF == WF_E2M1 ? i16 * 16 + piece : i16 * 8 + (piece >> 1);
        // past K the codes are zero and the byte is not this row's
        if (128u * u + 16u * piece < KB) scale = __uint_as_float((uint32_t)sc[at + skew] << 23);
      }
#pragma unroll
      for (int m = 0; m < F::SUB; ++m) {
        const bf16x8_t wv = weight_values<WF>(raw[h], m, scale);
#pragma unroll
        for (int p = 0; p < PL; ++p) {
          const v4i xr = lds_read16(xt + p * XPLANE + (((piece * F::SUB + m) ^ f) << 4));
          part[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(bf16x8_t, xr), part[p], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      // one FP32 scale for 128 values of K of all of the tile's rows
      if constexpr (WF == WF_BLOCK) acc[p] += part[p] * *(const float *)sc;
      else acc[p] = part[p];
    }
  }
};

// The sum of the two planes' products.  Where the high plane's is infinite or NaN
// it stands alone: a high part is zero only where its argument is (or is below
// FP32's normal range), and has its sign, so that beside infinite weights it gives
// what the argument itself does.
__device__ inline v4f join_planes(const v4f (&acc)[2]) {
  v4f v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = fabsf(acc[0][k]) < __builtin_inff() ? acc[0][k] + acc[1][k] : acc[0][k];
  return v;
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

// For 64 experts, one per lane: their tokens n, and before each of them the
// records (p.rows tokens or fewer each) and the pairs, of these 64.
__device__ inline void expert_scan(const ExpertsArgs &p, const ExpertMasks &mk, int e, int &n, int &recs, int &pairs,
                                   int &all_recs, int &all_pairs) {
  const int lane = threadIdx.x & 63;
  n = e < p.E ? __popcll(expert_mask(mk, e)) : 0;
  const int mine = (n + p.rows - 1) / p.rows << 16 | n;     // both counts stay below 2^12
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(sum, d);
    if (lane >= d) sum += o;
  }
  const int all = __shfl(sum, 63);
  recs = (sum - mine) >> 16;
  pairs = (sum - mine) & 0xFFFF;
  all_recs = all >> 16;
  all_pairs = all & 0xFFFF;
}

// Record `rank` and its tokens as bits (n = 0: there is none); every wave for itself.
__device__ inline ExpertRec find_record(const ExpertsArgs &p, const ExpertMasks &mk, int rank, uint64_t &tokens) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += 64) {
    int n, recs, pairs, all_recs, all_pairs;
    expert_scan(p, mk, e0 + lane, n, recs, pairs, all_recs, all_pairs);
    if (rank < all_recs) {
      const uint64_t me = __ballot(n > 0 && recs <= rank && rank < recs + (n + p.rows - 1) / p.rows);
      const int l = __ffsll((unsigned long long)me) - 1;
      const int skip = p.rows * (rank - __shfl(recs, l));
      tokens = expert_mask(mk, e0 + l);
      for (int k = 0; k < skip; ++k) tokens &= tokens - 1;
      const int left = __shfl(n, l) - skip;
      return ExpertRec{e0 + l, base + __shfl(pairs, l) + skip, left < p.rows ? left : p.rows, 0};
    }
    rank -= all_recs;
    base += all_pairs;
  }
  tokens = 0;
  return ExpertRec{0, 0, 0, 0};
}

// The tables for the second kernel, by one workgroup.
__device__ inline void expert_table(const ExpertsArgs &p, const ExpertMasks &mk, int32_t (&first)[EXP_MAX_E]) {
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < p.down_tiles; i += blockDim.x)
    if (p.splits > 1) p.arrived[i] = 0;
  if (threadIdx.x < 64) {
    int rec0 = 0, pair0 = 0;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
      int n, recs, pairs, all_recs, all_pairs;
      expert_scan(p, mk, e0 + lane, n, recs, pairs, all_recs, all_pairs);
      if (e0 + lane < p.E) first[e0 + lane] = pair0 + pairs;
      for (int k = 0; k < n; k += p.rows)
        p.rec[rec0 + recs + k / p.rows] = ExpertRec{e0 + lane, pair0 + pairs + k, n - k < p.rows ? n - k : p.rows, 0};
      rec0 += all_recs;
      pair0 += all_pairs;
    }
    if (lane == 0) *p.count = rec0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.T * p.topk; s += blockDim.x) {
    const int e = p.ids[s], t = s / p.topk, j0 = s - t * p.topk;
    if (e < 0 || e >= p.E) continue;
    float share = 0.0f;
    bool again = false;                        // the token named this expert before
    for (int j = 0; j < p.topk; ++j) {
      if (p.ids[t * p.topk + j] != e) continue;
      again |= j < j0;
      share += p.w[t * p.topk + j];
    }
    if (!again) p.pair[first[e] + __popcll(expert_mask(mk, e) & ((1ull << t) - 1))] = ExpertPair{t, share};
  }
}

// The same for at most 64 slots (one or two tokens), in the registers of every
// wave, without LDS or barriers: lane s holds slot s.  Records come in the
// order of the slots that first name their experts.
struct SlotTable {
  int e, t;                                    // expert (-1: none) and token of the lane's slot
  int head;                                    // first lane with this expert
  uint32_t tokens;                             // tokens that name it
  int base;                                    // its first pair
  uint64_t heads;                              // lanes that are their expert's first
};

__device__ inline SlotTable slot_table(const ExpertsArgs &p) {
  const int lane = threadIdx.x & 63, P = p.T * p.topk;
  const uint64_t below = (1ull << lane) - 1;
  SlotTable s;
  s.e = -1;
  s.t = lane / p.topk;
  if (lane < P) s.e = p.ids[lane];
  if (s.e < 0 || s.e >= p.E) s.e = -1;
  s.head = lane;
  s.tokens = 0;
  for (int k = P - 1; k >= 0; --k) {
    const int e = __builtin_amdgcn_readlane(s.e, k), t = k >= p.topk;
    if (s.e >= 0 && e == s.e) {
      s.head = k < s.head ? k : s.head;
      s.tokens |= 1u << t;
    }
  }
  s.heads = __ballot(s.e >= 0 && s.head == lane);
  const uint64_t both = __ballot(s.tokens == 3u) & s.heads;
  s.base = __popcll(s.heads & below) + __popcll(both & below);
  return s;
}

// Record `rank` (n = 0: there is none) and its tokens as bits.
__device__ inline ExpertRec find_record(const SlotTable &s, int rank, uint64_t &tokens) {
  const int lane = threadIdx.x & 63;
  tokens = 0;
  if (rank >= __popcll(s.heads)) return ExpertRec{0, 0, 0, 0};
  const uint64_t me = __ballot((s.heads >> lane & 1) && __popcll(s.heads & ((1ull << lane) - 1)) == rank);
  const int l = __ffsll((unsigned long long)me) - 1;
  tokens = (uint32_t)__shfl((int)s.tokens, l);
  return ExpertRec{__shfl(s.e, l), __shfl(s.base, l), (int32_t)__popcll(tokens), 0};
}

__device__ inline void expert_table(const ExpertsArgs &p, const SlotTable &s) {
  const int lane = threadIdx.x & 63;
  const int base = __shfl(s.base, s.head), P = p.T * p.topk;
  for (int i = threadIdx.x; i < p.down_tiles; i += blockDim.x)
    if (p.splits > 1) p.arrived[i] = 0;
  if (threadIdx.x >= 64) return;
  const float w = lane < P ? p.w[lane] : 0.0f;
  float share = 0.0f;                          // of the lane's token
  bool lead = s.e >= 0;                        // first slot of its token with this expert
  for (int k = 0; k < P; ++k) {
    const int e = __builtin_amdgcn_readlane(s.e, k), t = k >= p.topk;
    const float wk = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), k));
    if (s.e < 0 || e != s.e || t != s.t) continue;
    share += wk;
    lead &= k >= lane;
  }
  if (lane == 0) *p.count = __popcll(s.heads);
  if (s.heads >> lane & 1) p.rec[__popcll(s.heads & ((1ull << lane) - 1))] = ExpertRec{s.e, s.base, (int32_t)__popc(s.tokens), 0};
  if (lead) p.pair[base + (s.t == 1 && (s.tokens & 1u) ? 1 : 0)] = ExpertPair{s.t, share};
}

// h of four consecutive rows of W1 (two SwiGLU pairs), as two BF16 each.
__device__ inline void store_h(const ExpertsArgs &p, int row, int64_t n, const v4f &z) {
  const int64_t plane = (int64_t)p.T * p.topk * p.F;
  const bool gated = p.act == ACT_SWIGLU;
  v4f v = {0.f, 0.f, 0.f, 0.f};
  if (gated) {
    v.x = z.x * logistic_f32(z.x) * z.y;
    v.y = z.z * logistic_f32(z.z) * z.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = activate_select(p.act, z[k]);
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
  uint16_t *dst = p.h + (int64_t)row * p.F + (gated ? n >> 1 : n);
  if (gated) {
    *(uint32_t *)dst = hi[0];
    *(uint32_t *)(dst + plane) = lo[0];
  } else {
    *(v2i *)dst = (v2i){(int)hi[0], (int)hi[1]};
    *(v2i *)(dst + plane) = (v2i){(int)lo[0], (int)lo[1]};
  }
}

// ROWS: the most tokens of a record, shared; 0: private.
template <int WF, int ROWS>
__global__ __launch_bounds__(64 * EXP_WAVES) void experts_up_kernel(ExpertsArgs p) {
  constexpr bool SHARED = ROWS > 0;
  constexpr int U = 4;
  typedef ExpertStream<WF, 1, ROWS, false, U> Stream;
  __shared__ __attribute__((aligned(1024))) union {
    struct {
      ExpertMasks mk;
      int32_t first[EXP_MAX_E];
    } t;
    uint8_t ring[Stream::LDS_BYTES];
    v4f part[EXP_WAVES][64];
  } sm;
  __shared__ int32_t tok[EXP_ROWS];
  const int rank = (int)(blockIdx.x - 1) / max(p.up_tiles, 1), tile = (int)(blockIdx.x - 1) - rank * p.up_tiles;
  uint64_t tokens;
  ExpertRec rec;
  if constexpr (SHARED) {
    expert_masks(p, sm.t.mk);
    if (blockIdx.x == 0) {
      expert_table(p, sm.t.mk, sm.t.first);
      return;
    }
    rec = find_record(p, sm.t.mk, rank, tokens);
  } else {
    const SlotTable slots = slot_table(p);
    if (blockIdx.x == 0) {
      expert_table(p, slots);
      return;
    }
    rec = find_record(slots, rank, tokens);
  }
  rec.e = __builtin_amdgcn_readfirstlane(rec.e);
  rec.n = __builtin_amdgcn_readfirstlane(rec.n);
  if (rec.n == 0) return;
  if constexpr (SHARED) {
    const int lane = threadIdx.x & 63, place = __popcll(tokens & ((1ull << lane) - 1));
    if (threadIdx.x < 64 && (tokens >> lane & 1) && place < p.rows) tok[place] = lane;
    __syncthreads();                           // and the masks' memory is free from here on
  }

  Stream s;
  s.init(sm.ring, p.D, rsrc4(p.x, clamp_records(2 * p.T * p.D)), 0u);
  const bool split = !SHARED && p.split_k;
  const int64_t n0 = (int64_t)tile * (split ? 16 : 64) + (split ? 0 : 16 * s.w);
  s.set_weight(p.w1, p.s1, rec.e, p.N1, n0);
  s.set_rows(rec.n, [&](int r) {
    const int t = SHARED ? tok[r] : (tokens & 1) ? r : 1;
    return (uint32_t)(2 * t * p.D);
  });
  const int c = 4 * s.q;
  v4f chan = {1.f, 1.f, 1.f, 1.f};
  if constexpr (WF == WF_INT8) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc((const float *)p.s1 + rec.e * p.N1 + n0, clamp_records(4 * (p.N1 - n0)));
    chan = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(r, 4 * c, 0, 0));
    // here, not among the ring's DMAs
#pragma unroll
    for (int k = 0; k < 4; ++k) asm volatile("" : "+v"(chan[k]));
  }
  const int units = (int)s.units;
  const int lo = split ? s.w * units / EXP_WAVES : 0, hi = split ? (s.w + 1) * units / EXP_WAVES : units;
#pragma unroll
  for (int k = 0; k < U - 1; ++k) s.issue(k, lo + k, lo + k < hi);
  v4f acc[1] = {{0.f, 0.f, 0.f, 0.f}};
  int sl = 0;
  for (int v = lo; v < hi; ++v) {
    Stream::wait();
    s.issue(sl == 0 ? U - 1 : sl - 1, v + U - 1, v + U - 1 < hi);
    s.consume(sm.ring, sl, v, acc);
    sl = sl == U - 1 ? 0 : sl + 1;
  }
  wait_vmem_le<0>();                           // no DMA into LDS that is used for something else
  if (split) {
    __syncthreads();
    sm.part[s.w][s.lane] = acc[0];
    __syncthreads();
    if (s.w != 0) return;
#pragma unroll
    for (int k = 1; k < EXP_WAVES; ++k) acc[0] += sm.part[k][s.lane];
  }
  if (s.i16 < rec.n && n0 + c < p.N1) store_h(p, rec.base + s.i16, n0 + c, acc[0] * chan);
}

// TM: the most tokens (the sums' rows).
template <int WF, int ROWS, int TM>
__global__ __launch_bounds__(64 * EXP_WAVES) void experts_down_kernel(ExpertsArgs p) {
  constexpr bool SHARED = ROWS > 0;
  constexpr int U = !SHARED ? 5 : TM > 16 && ROWS > 8 ? 3 : 4, COLS = SHARED ? 16 * EXP_WAVES : 16, SETS = SHARED ? 1 : EXP_WAVES;
  constexpr int PITCH = COLS + 4;              // floats per token: columns and a skew
  typedef ExpertStream<WF, 2, ROWS, true, U> Stream;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[Stream::LDS_BYTES];
  __shared__ __attribute__((aligned(16))) float sums[SETS][TM][PITCH];
  __shared__ int32_t done;
  for (int i = threadIdx.x; i < SETS * TM * PITCH; i += 64 * EXP_WAVES) (&sums[0][0][0])[i] = 0.0f;
  __syncthreads();
  const int tile = (int)blockIdx.x / p.splits, split = (int)blockIdx.x - tile * p.splits;
  const int64_t tile0 = (int64_t)tile * COLS, plane = (int64_t)p.T * p.topk * p.F;
  Stream s;
  s.init(ring, p.F, rsrc4(p.h, clamp_records(4 * plane)), (uint32_t)(2 * plane));
  const int64_t n0 = tile0 + (SHARED ? 16 * s.w : 0);
  s.rp = rsrc4(p.pair, (uint32_t)(8 * p.T * p.topk));
  // read as constants, through the scalar cache: the kernel before wrote them
  typedef const __attribute__((address_space(4))) ExpertRec *RecPtr;
  const RecPtr recs = (RecPtr)(uintptr_t)p.rec;
  const int units = (int)s.units;
  const int total = __builtin_amdgcn_readfirstlane(*p.count) * units;
  const int pieces = SHARED ? p.splits : p.splits * EXP_WAVES, mine = SHARED ? split : split * EXP_WAVES + s.w;
  const int lo = (int)((int64_t)total * mine / pieces), hi = (int)((int64_t)total * (mine + 1) / pieces);

  // the stage to issue, and the one to use: record and unit
  int ia = units > 0 ? lo / units : 0, iu = lo - ia * units;
  int ca = ia, cu = iu, at = lo;
  auto enter = [&](int a) {
    const int e = recs[a].e, base = recs[a].base, n = recs[a].n;
    s.set_weight(p.w2, p.s2, e, p.D, n0);
    s.set_rows(n, [&](int r) { return (uint32_t)(2 * (base + r) * p.F); });
    s.pair0 = 8u * base;
  };
  auto issue = [&](int sl) {
    s.issue(sl, iu, at < hi);
    ++at;
    if (++iu == units) {
      iu = 0;
      ++ia;
      if (at < hi) enter(ia);
    }
  };
  if (lo < hi) enter(ia);
#pragma unroll
  for (int k = 0; k < U - 1; ++k) issue(k);
  v4f acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  int sl = 0;
  for (int v = lo; v < hi; ++v) {
    Stream::wait();
    issue(sl == 0 ? U - 1 : sl - 1);
    s.consume(ring, sl, cu, acc);
    if (++cu == units || v + 1 == hi) {
      // the record's part of this list is done: its tokens' sums
      const uint8_t *st = ring + sl * Stream::STAGE;
      const int t = *(const int32_t *)(st + Stream::P_OFF + (SHARED ? 0 : 256 * s.w) + 8 * s.i16);
      const float share = *(const float *)(st + Stream::P_OFF + (SHARED ? 0 : 256 * s.w) + 8 * s.i16 + 4);
      v4f y = join_planes(acc);
      if constexpr (WF == WF_INT8) y *= *(const v4f *)(st + Stream::S_OFF + 256 * s.w + 16 * s.q);
      if (s.i16 < recs[ca].n) {
        v4f *sum = (v4f *)&sums[SHARED ? 0 : s.w][t][(SHARED ? 16 * s.w : 0) + 4 * s.q];
        *sum += y * share;
      }
      acc[0] = acc[1] = (v4f){0.f, 0.f, 0.f, 0.f};
      cu = 0;
      ++ca;
    }
    sl = sl == U - 1 ? 0 : sl + 1;
  }
  wait_vmem_le<0>();                           // no DMA into the LDS of an ended workgroup
  __syncthreads();
  if (p.splits == 1) {
    for (int i = threadIdx.x; i < p.T * COLS; i += 64 * EXP_WAVES) {
      const int t = i / COLS, c = i - t * COLS;
      if (tile0 + c >= p.D) continue;
      const int64_t o = (int64_t)t * p.D + tile0 + c;
      float v = sums[0][t][c];
#pragma unroll
      for (int k = 1; k < SETS; ++k) v += sums[k][t][c];
      if (p.residual) v += __uint_as_float((uint32_t)p.residual[o] << 16);
      p.out[o] = (uint16_t)pack_bf16x2(v, 0.0f);
    }
    return;
  }
  // Splits of the list: the workgroup that is done last adds their sums, in the
  // splits' order.  The sums go through device-scope accesses, which do not
  // stay in an XCD's own L2: each wave waits for its stores, the workgroup for
  // its waves, and then it counts itself.  (A release fence in place of the
  // wait writes back the whole L2, once per workgroup: 100 instead of 27 us for
  // 37 tokens, 24 experts of 2080 x 1440.)
  const int64_t size = p.T * p.D;
  constexpr int DEVICE = 16;                   // the sc1 bit of a buffer access: device scope
  const __amdgpu_buffer_rsrc_t rp = make_rsrc(p.part, clamp_records(4 * p.splits * size));
  auto place = [&](int k, int t, int c) { return (int)(4 * (k * size + (int64_t)t * p.D + tile0 + c)); };
  constexpr int QUADS = COLS / 4, GROUP = 64 * EXP_WAVES / QUADS, MT = (TM + GROUP - 1) / GROUP;
  const int c = 4 * (threadIdx.x % QUADS), t0 = threadIdx.x / QUADS;
  const bool in = tile0 + c < p.D;             // D is a multiple of 8
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int t = t0 + j * GROUP;
    if (in && t < p.T) {
      v4f v = *(const v4f *)&sums[0][t][c];
#pragma unroll
      for (int k = 1; k < SETS; ++k) v += *(const v4f *)&sums[k][t][c];
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4v, v), rp, place(split, t, c), 0, DEVICE);
    }
  }
  wait_vmem_le<0>();
  __syncthreads();
  if (threadIdx.x == 0) done = __hip_atomic_fetch_add(p.arrived + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (done != p.splits - 1) return;
  if (!in) return;
  // four columns and up to four tokens per thread, the loads of eight splits
  // in flight together (past the last split: zeros)
  v4f v[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) v[j] = (v4f){0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < p.splits; k0 += 8) {
    v4f u[8][MT];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int t = t0 + j * GROUP;
        const bool real = k0 + k < p.splits && t < p.T;
        u[k][j] = __builtin_bit_cast(
            v4f, __builtin_amdgcn_raw_buffer_load_b128(rp, real ? place(k0 + k, t, c) : (int)Stream::NOWHERE, 0, DEVICE));
      }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < MT; ++j) v[j] += u[k][j];
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int t = t0 + j * GROUP;
    if (t >= p.T) break;
    const int64_t o = (int64_t)t * p.D + tile0 + c;
    if (p.residual) v[j] += load_bf16x4(p.residual + o, 4);
    store_bf16x4(p.out + o, v[j], 4);
  }
}

}  // namespace mxg
