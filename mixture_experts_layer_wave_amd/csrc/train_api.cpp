// Host side of the training part of include/moe.h: argument validation,
// workspace layout and the launch sequence on the caller's stream.  As in
// moe_api.cpp, nothing here allocates device memory or synchronises.
#include "moe.h"

#include <hip/hip_runtime.h>

#include "api_internal.h"
#include "kernels.h"

using namespace moe;

namespace {

int check_norm(int32_t n, int32_t d, int act) {
  if (n < 0 || n >= (1 << 30) || d < 1 || d > kLayerNormMaxD) return MOE_ERR_SHAPE;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_DTYPE;
  if (act == MOE_BF16 && d % 8) return MOE_ERR_SHAPE;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_layer_norm(int32_t n, int32_t d, const void *x, int act, const float *weight,
                   const float *bias, float eps, void *y, float *mean, float *rstd, void *stream) {
  const int st = check_norm(n, d, act);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f)) return MOE_ERR_SHAPE;
  if (n == 0) return MOE_OK;
  if (!x || !weight || !y) return MOE_ERR_NULL;
  if (act == MOE_BF16 && (!aligned16(x) || !aligned16(y))) return MOE_ERR_ALIGN;
  return hip_status(launch_layer_norm(x, act == MOE_BF16, weight, bias, eps, n, d, y, mean, rstd,
                                      (hipStream_t)stream));
}

size_t moe_layer_norm_backward_workspace_bytes(int32_t n, int32_t d) {
  if (check_norm(n, d, MOE_F32) != MOE_OK) return 0;
  return align_up(layer_norm_grad_bytes(n, d));
}

int moe_layer_norm_backward(int32_t n, int32_t d, const void *dy, const void *x, int act,
                            const float *weight, const float *mean, const float *rstd, void *dx,
                            float *dweight, float *dbias, void *ws, size_t ws_bytes, void *stream) {
  const int st = check_norm(n, d, act);
  if (st != MOE_OK) return st;
  if (n > 0) {
    if (!dy || !x || !weight || !mean || !rstd || !dx) return MOE_ERR_NULL;
    if (act == MOE_BF16 && (!aligned16(dy) || !aligned16(x) || !aligned16(dx))) return MOE_ERR_ALIGN;
    if (!ws || ws_bytes < moe_layer_norm_backward_workspace_bytes(n, d)) return MOE_ERR_WORKSPACE;
    if (!aligned16(ws)) return MOE_ERR_ALIGN;
  }
  return hip_status(launch_layer_norm_grad(dy, x, act == MOE_BF16, weight, mean, rstd, n, d, dx,
                                           dweight, dbias, (float *)ws, (hipStream_t)stream));
}

}  // extern "C"
