// The kernels for few rows, every MX and tensor-wise format.
#include "kernels.hpp"
#include "rows.hpp"

namespace mxg {
namespace {
template <int FA, int FB, int SMODE, bool PSB>
dense_fn pick_rows_tile(int fm) {
  constexpr int U = FA == F_E2M1 ? 4 : 3;
  return fm == 1   ? dense_rows_kernel<FA, FB, SMODE, PSB, 1, 1, 4>
         : fm == 2 ? dense_rows_kernel<FA, FB, SMODE, PSB, 2, 2, U>
                   : dense_rows_kernel<FA, FB, SMODE, PSB, 4, 2, U - 1>;
}
template <int FA, int FB>
dense_fn pick_rows_fmt(bool mx, bool psb, int fm) {
  if (mx) return psb ? pick_rows_tile<FA, FB, SM_MX, true>(fm) : pick_rows_tile<FA, FB, SM_MX, false>(fm);
  if constexpr (FA != F_E2M1)
    return psb ? pick_rows_tile<FA, FB, SM_TENSOR, true>(fm) : pick_rows_tile<FA, FB, SM_TENSOR, false>(fm);
  return nullptr;
}
}  // namespace

dense_fn pick_rows(int ea, int eb, bool mx, bool psb, int fm) {
  if (ea == F_E2M1 && eb == F_E2M1) return pick_rows_fmt<F_E2M1, F_E2M1>(mx, psb, fm);
  if (ea == F_E4M3 && eb == F_E4M3) return pick_rows_fmt<F_E4M3, F_E4M3>(mx, psb, fm);
  if (ea == F_E4M3 && eb == F_E5M2) return pick_rows_fmt<F_E4M3, F_E5M2>(mx, psb, fm);
  if (ea == F_E5M2 && eb == F_E4M3) return pick_rows_fmt<F_E5M2, F_E4M3>(mx, psb, fm);
  if (ea == F_E5M2 && eb == F_E5M2) return pick_rows_fmt<F_E5M2, F_E5M2>(mx, psb, fm);
  return nullptr;
}
}  // namespace mxg
