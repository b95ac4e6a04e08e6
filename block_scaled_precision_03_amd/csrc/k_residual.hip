// C ABI of the residual epilogue's gradient: argument checks and launch.
#include <algorithm>

#include "host.hpp"
#include "residual.hpp"

namespace mxg {
namespace {

// Parts of the rows, from sizes alone (the workspace's size must not depend on
// the device): about 2048 workgroups of at least 32 rows each; one part of
// sixteen waves up to 256 rows (129 x 5002, GELU: 7.2 us, 9.9 in parts of 16; 379 x 8966,
// SwiGLU: 16.0 and 16.8).
struct GradShape {
  bool few;
  int64_t stripes, parts, rows;
};
GradShape grad_shape(int64_t M, int64_t N) {
  GradShape s;
  s.few = M <= 256;
  s.stripes = cdiv(N, s.few ? 64 * RG_FEW_V : 512);
  s.rows = s.few ? M : std::max<int64_t>(32, cdiv(M, std::max<int64_t>(1, 2048 / s.stripes)));
  s.parts = cdiv(M, s.rows);
  return s;
}

template <int V, int W>
void (*pick_grad(int act))(ResidualGradArgs) {
  return act == ACT_SWIGLU      ? residual_grad_kernel<ACT_SWIGLU, V, W>
         : act == ACT_RELU      ? residual_grad_kernel<ACT_RELU, V, W>
         : act == ACT_GELU_TANH ? residual_grad_kernel<ACT_GELU_TANH, V, W>
         : act == ACT_SILU      ? residual_grad_kernel<ACT_SILU, V, W>
                                : residual_grad_kernel<ACT_NONE, V, W>;
}

}  // namespace

int residual_init() {
  hipFuncAttributes attr;
  return hipFuncGetAttributes(&attr, (const void *)column_sums_kernel) == hipSuccess ? MXG_OK : MXG_ERR_HIP;
}

}  // namespace mxg

using namespace mxg;

extern "C" int64_t mxgemm_residual_backward_workspace_bytes(int64_t M, int64_t N) {
  if (M < 0 || N < 0 || M >= MAX_DIM || N >= MAX_DIM) return -1;
  if (M == 0 || N == 0) return 0;
  const GradShape s = grad_shape(M, N);
  return s.parts == 1 ? 0 : 4 * s.parts * N;
}

extern "C" int mxgemm_residual_backward_validate(int activation, const void *dD, const void *z, const void *dz,
                                                 const float *dbias, int64_t M, int64_t N, const void *workspace,
                                                 int64_t workspace_bytes) {
  if ((activation < MXG_ACT_NONE || activation > MXG_ACT_SILU) && activation != MXG_ACT_SWIGLU) return MXG_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || (!dz && !dbias)) return MXG_ERR_INVALID_ARG;
  const bool gated = activation == MXG_ACT_SWIGLU;
  if (M >= MAX_DIM || N >= MAX_DIM || (gated && N % 2 != 0)) return MXG_ERR_UNSUPPORTED;
  if (!aligned(dbias, 4)) return MXG_ERR_MISALIGNED;
  if (M == 0 || N == 0) return MXG_OK;
  if (!dD || (activation != MXG_ACT_NONE && !z)) return MXG_ERR_INVALID_ARG;
  // rows of another pitch than dz's: not in place
  if (gated && dz == dD) return MXG_ERR_INVALID_ARG;
  if (!aligned(dD, 16) || !aligned(dz, 16) || (activation != MXG_ACT_NONE && !aligned(z, 16))) return MXG_ERR_MISALIGNED;
  if (dbias) {
    const int64_t need = mxgemm_residual_backward_workspace_bytes(M, N);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MXG_ERR_INVALID_ARG;
    if (need > 0 && !aligned(workspace, 16)) return MXG_ERR_MISALIGNED;
  }
  return MXG_OK;
}

extern "C" int mxgemm_residual_backward(int activation, const void *dD, const void *z, void *dz, float *dbias, int64_t M,
                                        int64_t N, void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  const int v = mxgemm_residual_backward_validate(activation, dD, z, dz, dbias, M, N, workspace, workspace_bytes);
  if (v != MXG_OK || N == 0) return v;
  const dim3 sums = flat_grid(cdiv(N, 64));
  if (M == 0) {
    if (dbias) hipLaunchKernelGGL(column_sums_kernel, sums, dim3(64 * CS_WAVES), 0, stream, nullptr, dbias, N, 0);
    return launch_status();
  }
  const GradShape s = grad_shape(M, N);
  ResidualGradArgs a = {};
  a.dD = (const uint16_t *)dD;
  a.z = (const uint16_t *)z;
  a.dz = (uint16_t *)dz;
  a.part = !dbias ? nullptr : s.parts == 1 ? dbias : (float *)workspace;
  a.M = M;
  a.N = N;
  a.No = activation == MXG_ACT_SWIGLU ? N / 2 : N;
  a.rows = s.rows;
  if (s.few)
    hipLaunchKernelGGL((pick_grad<RG_FEW_V, RG_FEW_WAVES>(activation)), flat_grid(s.stripes), dim3(64 * RG_FEW_WAVES), 0, stream, a);
  else
    hipLaunchKernelGGL((pick_grad<8, 4>(activation)), dim3((unsigned)s.stripes, (unsigned)s.parts), dim3(256), 0, stream, a);
  if (dbias && s.parts > 1)
    hipLaunchKernelGGL(column_sums_kernel, sums, dim3(64 * CS_WAVES), 0, stream, (const float *)workspace, dbias, N, (int)s.parts);
  return launch_status();
}
