// Host-side helpers shared by the translation units of the C ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxgemm.h"
#include "common.hpp"

namespace mxg {

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Largest operand extents the 32-bit in-kernel offsets support.
constexpr int64_t MAX_DIM = 1ll << 31;

inline int launch_status() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MXG_OK : MXG_ERR_HIP;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A grid of at least n workgroups for kernels that use flat_block().
inline dim3 flat_grid(int64_t n) {
  const int64_t row = 1ll << FLAT_LOG2;
  return n <= row ? dim3((unsigned)n) : dim3((unsigned)row, (unsigned)cdiv(n, row));
}

// Compute units of the current device: the grid size of the persistent
// kernels.  Queried once per device.
inline int cu_count() {
  static int cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cache[dev] <= 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cache[dev] = n;
  }
  return cache[dev];
}

// The 8-bit integer GEMM (k_int8.hip): host checks, kernel choice and
// launch of a dense call with MXG_INT8 operands.
int int8_validate(int fmtA, int fmtB, int layout, const void *A, const void *sA, const void *B, const void *sB,
                  const void *D, int64_t M, int64_t N, int64_t K);
int int8_dense_variant(int64_t M, int64_t N, int64_t K);
int int8_run(const void *A, const void *sA, const void *B, const void *sB, void *D, int64_t M, int64_t N,
             int64_t K, const void *bias, int act, const void *residual, void *z, hipStream_t stream);
int int8_init();
int moe_init();                          // k_moe.hip
int experts_init();                      // k_experts.hip
int residual_init();                     // k_residual.hip

}  // namespace mxg
