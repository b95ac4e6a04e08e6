// Dense kernels with the residual epilogue: MXFP4.
#include "kernels.hpp"

namespace mxg {
dense_fn pick_residual_fp4(bool psb, int fuse) { return pick_residual<F_E2M1, F_E2M1, SM_MX>(psb, fuse); }
}  // namespace mxg
