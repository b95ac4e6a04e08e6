// Dense kernels with the residual epilogue: tensor-wise FP8 with A in E4M3.
#include "kernels.hpp"

namespace mxg {
dense_fn pick_residual_tw_a4(int eb, bool psb, int fuse) {
  if (eb == F_E4M3) return pick_residual<F_E4M3, F_E4M3, SM_TENSOR>(psb, fuse);
  if (eb == F_E5M2) return pick_residual<F_E4M3, F_E5M2, SM_TENSOR>(psb, fuse);
  return nullptr;
}
}  // namespace mxg
