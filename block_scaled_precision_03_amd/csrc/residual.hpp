// The gradient of the residual epilogue D = act(z) + R, z = sum + bias:
//   dz = dD act'(z),  dbias[n] = sum_m dz[m,n]  (of the unrounded dz),
// R's gradient being dD itself.  SwiGLU, D = g s(g) u with g = z[2j], u =
// z[2j+1] and s the logistic function: dg = dD u s (1 + g (1 - s)), du = dD g s.
//
// A stream over dD, z and dz; the column sums are formed beside it: a
// workgroup walks the rows of its part for its columns and leaves FP32
// partial sums in the workspace, which a second kernel adds in order.
#pragma once
#include "common.hpp"

namespace mxg {

struct ResidualGradArgs {
  const uint16_t *dD;              // [M, No]
  const uint16_t *z;               // [M, N]
  uint16_t *dz;                    // [M, N] or null
  float *part;                     // [parts, N] or null (no bias gradient)
  int64_t M, N, No, rows;          // rows per part
};

// act'(z) of the activations that have one everywhere.
//   GELU (tanh form): z s(2u), u = sqrt(2/pi) (z + 0.044715 z^3):
//     s + z s (1 - s) 2u',  u' = sqrt(2/pi) (1 + 0.134145 z^2)
//   SiLU: s + z s (1 - s)
//   (ReLU's gradient is dD where z > 0 and 0 elsewhere, chosen, not multiplied: a
//   dead unit has none even where dD is infinite or NaN.)
// 1 - s is formed as the logistic function of the negated argument, which
// keeps its leading bits where s is near 1, and z s (1 - s) as 0 where it
// vanishes (|z| large), not as infinity times zero.
template <int ACT>
__device__ inline float act_slope(float z) {
  if constexpr (ACT == ACT_GELU_TANH) {
    const float c = fminf(fmaxf(z, -16.0f), 16.0f);        // beyond: exactly 0 or 1
    const float u2 = 1.5957691216057308f * fmaf(0.044715f * c, c * c, c);
    const float s = logistic_f32(u2), t = logistic_f32(-u2);
    const float d = fmaf(c * s * t, 1.5957691216057308f * fmaf(0.134145f * c, c, 1.0f), s);
    return z == z ? d : z;
  }
  if constexpr (ACT == ACT_SILU) {
    const float c = fminf(fmaxf(z, -126.0f), 126.0f);
    const float s = logistic_f32(c), t = logistic_f32(-c);
    const float d = fmaf(c * s, t, s);
    return z == z ? d : z;
  }
  return 1.0f;
}

// N BF16 values of a row of which `room` are left, at any alignment (an odd
// pitch leaves rows at two bytes; the hardware takes any); read and written past
// the caches, which they would only pass through.
template <int N>
struct RowPiece {
  typedef uint16_t Any __attribute__((ext_vector_type(N), aligned(2)));
  __device__ static inline void load(const uint16_t *src, int64_t room, float (&v)[N]) {
    Any h;
    if (room >= N) {
      h = __builtin_nontemporal_load((const Any *)src);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) h[k] = k < room ? src[k] : (uint16_t)0;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __uint_as_float((uint32_t)h[k] << 16);
  }
  __device__ static inline void store(uint16_t *dst, int64_t room, const float (&v)[N]) {
    Any h;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const uint32_t u = pack_bf16x2(v[k], v[k + 1]);
      h[k] = (uint16_t)u;
      h[k + 1] = (uint16_t)(u >> 16);
    }
    if (room >= N) {
      __builtin_nontemporal_store(h, (Any *)dst);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < room) dst[k] = h[k];
    }
  }
};

// V columns of z per lane, RG_ROWS rows at a time (their loads in flight
// together); block (x, y): columns 64 V x .., the rows of part y, row r of them to
// wave r % W.  Many rows: V 8, four waves, parts that a second kernel sums; few:
// V 2, sixteen waves and one part, one kernel (V 4: 129 x 5002 11.6 us, 7.2), whose
// grid is folded (flat_grid): 2^29 columns would make 2^32 work-items in one dimension.
constexpr int RG_ROWS = 4, RG_FEW_V = 2, RG_FEW_WAVES = 16;

template <int ACT, int V, int W>
__global__ __launch_bounds__(64 * W) void residual_grad_kernel(ResidualGradArgs p) {
  constexpr bool GATED = ACT == ACT_SWIGLU;
  constexpr int DV = GATED ? V / 2 : V, COLS = 64 * V;
  __shared__ float sums[W][COLS];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c0 = (W == RG_FEW_WAVES ? flat_block() : (int64_t)blockIdx.x) * COLS, c = c0 + lane * V, room = p.N - c;
  const int64_t cd = GATED ? c / 2 : c, roomd = GATED ? room / 2 : room;
  const int64_t part = W == RG_FEW_WAVES ? 0 : blockIdx.y, m0 = part * p.rows, m1 = min(p.M, m0 + p.rows);
  float sum[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = 0.0f;
  if (room > 0) {
    for (int64_t m = m0 + w; m < m1; m += W * RG_ROWS) {
      float d[RG_ROWS][DV], z[RG_ROWS][V];
#pragma unroll
      for (int i = 0; i < RG_ROWS; ++i) {
        const int64_t r = m + W * i;
        if (r < m1) {
          RowPiece<DV>::load(p.dD + r * p.No + cd, roomd, d[i]);
          if constexpr (ACT != ACT_NONE) RowPiece<V>::load(p.z + r * p.N + c, room, z[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < RG_ROWS; ++i) {
        const int64_t r = m + W * i;
        if (r >= m1) break;
        float g[V];
        if constexpr (GATED) {
#pragma unroll
          for (int k = 0; k < DV; ++k) {
            const float a = z[i][2 * k], u = z[i][2 * k + 1];
            g[2 * k] = d[i][k] * (u * act_slope<ACT_SILU>(a));
            g[2 * k + 1] = d[i][k] * (a * logistic_f32(a));
          }
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) {
            if constexpr (ACT == ACT_RELU) g[k] = z[i][k] > 0.0f ? d[i][k] : 0.0f;
            else g[k] = ACT == ACT_NONE ? d[i][k] : d[i][k] * act_slope<ACT>(z[i][k]);
          }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) sum[k] += g[k];
        if (p.dz) RowPiece<V>::store(p.dz + r * p.N + c, room, g);
      }
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int k = 0; k < V; ++k) sums[w][lane * V + k] = sum[k];
  __syncthreads();
  for (int i = threadIdx.x; i < COLS; i += 64 * W) {
    const int64_t col = c0 + i;
    if (col >= p.N) continue;
    float t = sums[0][i];
#pragma unroll
    for (int k = 1; k < W; ++k) t += sums[k][i];
    p.part[part * p.N + col] = t;
  }
}

// out[n] = sum of the parts; none: 0.  64 columns per workgroup, part k to wave
// k % 16, eight parts' loads in flight together, the waves' sums in their order
// (one thread per column through all parts: 9327 x 146 took 140 us, 13 so).
constexpr int CS_WAVES = 16;
__global__ __launch_bounds__(64 * CS_WAVES) void column_sums_kernel(const float *part, float *out, int64_t N, int parts) {
  __shared__ float sums[CS_WAVES][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = flat_block() * 64 + lane;
  float s = 0.0f;
  if (n < N) {
    for (int k0 = w; k0 < parts; k0 += 8 * CS_WAVES) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = k0 + j * CS_WAVES;
        v[j] = k < parts ? part[(int64_t)k * N + n] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
  }
  sums[w][lane] = s;
  __syncthreads();
  if (w != 0 || n >= N) return;
#pragma unroll
  for (int k = 1; k < CS_WAVES; ++k) s += sums[k][lane];
  out[n] = s;
}

}  // namespace mxg
