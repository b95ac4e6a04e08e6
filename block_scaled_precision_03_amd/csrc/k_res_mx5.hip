// Dense kernels with the residual epilogue: MX FP8 with A in E5M2.
#include "kernels.hpp"

namespace mxg {
dense_fn pick_residual_mx_a5(int eb, bool psb, int fuse) {
  if (eb == F_E4M3) return pick_residual<F_E5M2, F_E4M3, SM_MX>(psb, fuse);
  if (eb == F_E5M2) return pick_residual<F_E5M2, F_E5M2, SM_MX>(psb, fuse);
  return nullptr;
}
}  // namespace mxg
