// The kernels for few rows or columns, every MX and tensor-wise format.
#include "kernels.hpp"
#include "rows.hpp"

namespace mxg {
namespace {
template <int FA, int FB, int SMODE, bool PSB>
dense_fn pick_rows_tile(int tile) {
  switch (tile) {
    case 0: return dense_rows_kernel<FA, FB, SMODE, PSB, 8, 1, 4, 5>;
    case 1: return dense_rows_kernel<FA, FB, SMODE, PSB, 16, 1, 8, 4>;
    case 2: return dense_rows_kernel<FA, FB, SMODE, PSB, 32, 2, 4, 4>;
    case 3: return dense_rows_kernel<FA, FB, SMODE, PSB, 64, 2, 4, 3>;
    default: return dense_rows_kernel<FA, FB, SMODE, PSB, 64, 4, 4, 2>;
  }
}
template <int FA, int FB>
dense_fn pick_rows_fmt(bool mx, bool psb, int tile) {
  if (mx) return psb ? pick_rows_tile<FA, FB, SM_MX, true>(tile) : pick_rows_tile<FA, FB, SM_MX, false>(tile);
  if constexpr (FA != F_E2M1)
    return psb ? pick_rows_tile<FA, FB, SM_TENSOR, true>(tile) : pick_rows_tile<FA, FB, SM_TENSOR, false>(tile);
  return nullptr;
}
}  // namespace

dense_fn pick_rows(int ea, int eb, bool mx, bool psb, int tile) {
  if (ea == F_E2M1 && eb == F_E2M1) return pick_rows_fmt<F_E2M1, F_E2M1>(mx, psb, tile);
  if (ea == F_E4M3 && eb == F_E4M3) return pick_rows_fmt<F_E4M3, F_E4M3>(mx, psb, tile);
  if (ea == F_E4M3 && eb == F_E5M2) return pick_rows_fmt<F_E4M3, F_E5M2>(mx, psb, tile);
  if (ea == F_E5M2 && eb == F_E4M3) return pick_rows_fmt<F_E5M2, F_E4M3>(mx, psb, tile);
  if (ea == F_E5M2 && eb == F_E5M2) return pick_rows_fmt<F_E5M2, F_E5M2>(mx, psb, tile);
  return nullptr;
}
}  // namespace mxg
