// What the host sides of the C ABI share: moe_forward's body (moe_api.cpp and
// noalloc.hip) and the argument checks (moe_api.cpp and train_api.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include "kernels.h"
#include "moe.h"

namespace moe {

// Workspace regions start at multiples of 256 bytes.
constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Shape limits; activation and weight dtypes with the shape rules each
// needs; the weights' pointers (act_mx8: activations already MXFP8).
int check_shape(const moe_shape *s);
int check_dtypes(const moe_shape *s, int act, int wdt);
int check_weights(const moe_shape *s, int act, const moe_expert_weights *w, bool act_mx8 = false);
bool renorm_of(const moe_shape *s);
// The FFN's arguments as the launchers take them.
FfnArgs ffn_args(const moe_shape *s, const void *a, const int32_t *perm, const int32_t *offsets,
                 const moe_expert_weights *w, void *h, float *yp);

// moe_forward: every argument check, then the launches, with the workspace
// ws of ws_bytes bytes (MOE_ERR_WORKSPACE when it is NULL or too small; the
// other checks run first).
int forward_impl(const moe_shape *s, const void *x, int act, const void *wg, const float *bias,
                 const moe_expert_weights *w, void *y, int out, int32_t *topk_idx,
                 float *topk_w, void *ws, size_t ws_bytes, void *stream);

}  // namespace moe
