// Grouped products of the expert FFN's gradient: host launch interface
// (bf16: gemm_grad.hip, float32: gemm_f32.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// The FFN's gradient over piles.  With r a pile row, e its expert and
// t = perm[r] (t = r without perm):
//   dh0_r = dy_t W2_e                    dw_r = <dh0_r, h_r>, h = silu(g) u
//   dg_r  = w_r dh0_r u_r silu'(g_r)     du_r = w_r dh0_r silu(g_r)
//   da_r  = dg_r W1_e + du_r W3_e
//   dW1_e = dg^T a,  dW3_e = du^T a,  dW2_e = dy^T (w h)   (sums over the pile)
struct FfnGradArgs {
  const void *dy, *a;      // [n][d] token rows (perm given) or [R][d] pile rows
  const int32_t *perm;     // pile row -> token, or NULL
  const int32_t *inv;      // [n][k] pile row of each pair (with perm)
  const float *topk_w;     // [n][k] combine weights (with perm)
  const int32_t *offsets;  // [E+1]
  int n, k, E, R, d, d_ff;
  bool bf16;               // else float32 throughout
  const void *w1, *w3, *w2;
  const int32_t *slot;
  int n_slots;
  const void *g, *u;       // [R][d_ff]
  void *da;                // [R][d]
  void *dw1, *dw3, *dw2;   // by logical expert; all of them are written
  float *dtopk_w;          // [n][k] (with perm)
  void *ws;                // ffn_grad_bytes(a)
};
size_t ffn_grad_bytes(const FfnGradArgs &a);
hipError_t launch_ffn_grad(const FfnGradArgs &a, hipStream_t st);

// What a gradient pass leaves for its last kernel, by shape alone: planes of
// <dh0, h> row sums, one for each column range of the dh product, and planes
// of da when its product is split along K (1: da is written directly).
struct GradPlan {
  int dw_planes, dx_splits;
};

// Workspace regions: dg, du and w h, [R][d_ff] each in the activations' type;
// part [dw_planes][R] and dx_part [dx_splits][R][d], float32.
struct FfnGradWs {
  GradPlan plan;
  void *dg, *du, *hs;
  float *part, *dx_part;
};

// The products, in order on the stream.
GradPlan grad_plan_bf16(const FfnGradArgs &a);
hipError_t launch_grad_bf16(const FfnGradArgs &a, const FfnGradWs &w, hipStream_t st);
GradPlan grad_plan_f32(const FfnGradArgs &a);
hipError_t launch_grad_f32(const FfnGradArgs &a, const FfnGradWs &w, hipStream_t st);

}  // namespace moe
