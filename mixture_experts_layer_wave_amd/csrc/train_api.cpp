// Host side of the training part of include/moe.h: argument validation,
// workspace layout and the launch sequence on the caller's stream.  As in
// moe_api.cpp, nothing here allocates device memory or synchronises.
#include "moe.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_internal.h"
#include "gemm_grad.h"
#include "kernels.h"

using namespace moe;

namespace {

int check_norm(int32_t n, int32_t d, int act) {
  if (n < 0 || n >= (1 << 30) || d < 1 || d > kLayerNormMaxD) return MOE_ERR_SHAPE;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_DTYPE;
  if (act == MOE_BF16 && d % 8) return MOE_ERR_SHAPE;
  return MOE_OK;
}

// The training FFN's largest grids, in threads: those of the products over pile
// rows (512 a block at most), of da and the three weight gradients together
// (256 a block; larger tiles have fewer blocks), and of the last kernel (1024 a
// block).  A launch takes less than 2^32.  Only a d or d_ff of a few elements
// beside a very long other side, or piles of hundreds of millions of rows, come
// near it.
bool grids_fit(const moe_shape *s, int wdt) {
  const long long T = wdt == MOE_F32 ? 64 : 128;  // the smallest tiles
  auto tiles = [](long long v, long long t) { return (v + t - 1) / t; };
  const long long R = (long long)s->n * s->k, ft = tiles(s->d_ff, T), dt = tiles(s->d, T);
  const long long rt = tiles(R, T) + std::min<long long>(s->E, R);
  // (two of da's K ranges; there are more only where its blocks are a few hundred)
  const long long rest = 2 * rt * dt + 2048 + 3 * s->E * ft * dt + 16ll * s->E;
  const long long last = tiles(R, 64) + tiles(R * s->d, 1024);
  return std::max({rt * ft * 512, rest * 256, last * 1024}) < (1ll << 32);
}

// Shapes and weights of the training FFN: weights that are trained (F32 or
// BF16), sizes that every product's grid and buffer offsets take.
int check_ffn_shape(const moe_shape *s, int act, int wdt) {
  int st = check_shape(s);
  if (st != MOE_OK) return st;
  if (wdt != MOE_F32 && wdt != MOE_BF16) return MOE_ERR_DTYPE;
  st = check_dtypes(s, act, wdt);
  if (st != MOE_OK) return st;
  if (s->d >= (1 << 20) || s->d_ff >= (1 << 20)) return MOE_ERR_SHAPE;
  // 32-bit byte offsets, as check_dtypes asks of bf16
  const long long R = (long long)s->n * s->k, bytes = wdt == MOE_F32 ? 4 : 2;
  if (R * std::max(s->d, s->d_ff) * bytes >= (1ll << 31) || (long long)s->d * s->d_ff * bytes >= (1ll << 31))
    return MOE_ERR_SHAPE;
  return grids_fit(s, wdt) ? MOE_OK : MOE_ERR_SHAPE;
}

int check_ffn(const moe_shape *s, int act, const moe_expert_weights *w) {
  if (!s || !w) return MOE_ERR_NULL;
  const int st = check_ffn_shape(s, act, w->dtype);
  return st == MOE_OK ? check_weights(s, act, w) : st;
}

FfnGradArgs grad_args(const moe_shape *s, int wdt) {
  FfnGradArgs a{};
  a.n = s->n;
  a.k = s->k;
  a.E = s->E;
  a.R = s->n * s->k;
  a.d = s->d;
  a.d_ff = s->d_ff;
  a.bf16 = wdt == MOE_BF16;
  return a;
}

int check_router(const moe_shape *s) {
  const int st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->n >= (1 << 24) || s->d >= (1 << 20) || (long long)s->E * s->d >= (1ll << 29)) return MOE_ERR_SHAPE;
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

int moe_expert_up_save(const moe_shape *s, const void *a, int act, const int32_t *perm,
                       const int32_t *offsets, const moe_expert_weights *w, void *h, void *g, void *u,
                       void *stream) {
  const int st = check_ffn(s, act, w);
  if (st != MOE_OK) return st;
  if (!a || !offsets || !h || !g || !u) return MOE_ERR_NULL;
  if (act == MOE_BF16 && (!aligned16(a) || !aligned16(h) || !aligned16(g) || !aligned16(u)))
    return MOE_ERR_ALIGN;
  return hip_status(launch_expert_up_save(ffn_args(s, a, perm, offsets, w, h, nullptr), g, u,
                                          (hipStream_t)stream));
}

size_t moe_grouped_ffn_backward_workspace_bytes(const moe_shape *s, int w_dtype) {
  if (!s || check_ffn_shape(s, w_dtype, w_dtype) != MOE_OK) return 0;
  return align_up(ffn_grad_bytes(grad_args(s, w_dtype)));
}

int moe_grouped_ffn_backward(const moe_shape *s, const void *dy, const void *a, int act,
                             const int32_t *perm, const int32_t *inv, const float *topk_w,
                             const int32_t *offsets, const moe_expert_weights *w, const void *g,
                             const void *u, void *da_perm, void *dw1, void *dw3, void *dw2,
                             float *dtopk_w, void *ws, size_t ws_bytes, void *stream) {
  const int st = check_ffn(s, act, w);
  if (st != MOE_OK) return st;
  if (!dy || !a || !offsets || !g || !u || !da_perm || !dw1 || !dw3 || !dw2) return MOE_ERR_NULL;
  const int given = (perm != nullptr) + (inv != nullptr) + (topk_w != nullptr) + (dtopk_w != nullptr);
  if (given != 0 && given != 4) return MOE_ERR_NULL;
  if (act == MOE_BF16)
    for (const void *p : {dy, a, g, u, (const void *)da_perm, (const void *)dw1, (const void *)dw3,
                          (const void *)dw2})
      if (!aligned16(p)) return MOE_ERR_ALIGN;
  if (!ws || ws_bytes < moe_grouped_ffn_backward_workspace_bytes(s, w->dtype)) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  FfnGradArgs f = grad_args(s, w->dtype);
  f.dy = dy;
  f.a = a;
  f.perm = perm;
  f.inv = inv;
  f.topk_w = topk_w;
  f.offsets = offsets;
  f.w1 = w->w1;
  f.w3 = w->w3;
  f.w2 = w->w2;
  f.slot = w->slot;
  f.n_slots = w->slot ? w->n_slots : s->E;
  f.g = g;
  f.u = u;
  f.da = da_perm;
  f.dw1 = dw1;
  f.dw3 = dw3;
  f.dw2 = dw2;
  f.dtopk_w = dtopk_w;
  f.ws = ws;
  return hip_status(launch_ffn_grad(f, (hipStream_t)stream));
}

size_t moe_router_backward_workspace_bytes(const moe_shape *s) {
  if (check_router(s) != MOE_OK) return 0;
  return align_up(router_grad_bytes(s->n, s->d, s->E));
}

int moe_router_backward(const moe_shape *s, const float *logits, const int32_t *topk_idx,
                        const float *topk_w, const float *dtopk_w, const float *f, float alpha,
                        const void *x, int act, const void *wg, const void *da_perm,
                        const int32_t *inv, float *dlogits, void *dx, void *dwg, float *dbias, void *ws,
                        size_t ws_bytes, void *stream) {
  const int st = check_router(s);
  if (st != MOE_OK) return st;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_DTYPE;
  if (act == MOE_BF16 && s->d % 8) return MOE_ERR_SHAPE;
  if (!logits || !topk_idx || !topk_w || !dtopk_w || !x || !wg || !dlogits || !dx || !dwg)
    return MOE_ERR_NULL;
  if ((da_perm != nullptr) != (inv != nullptr)) return MOE_ERR_NULL;
  if (act == MOE_BF16)
    for (const void *p : {x, wg, da_perm, (const void *)dx, (const void *)dwg})
      if (!aligned16(p)) return MOE_ERR_ALIGN;
  if (!ws || ws_bytes < moe_router_backward_workspace_bytes(s)) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  RouterGradArgs a{};
  a.logits = logits;
  a.idx = topk_idx;
  a.topk_w = topk_w;
  a.dtopk_w = dtopk_w;
  a.f = f;
  a.alpha = alpha;
  a.n = s->n;
  a.d = s->d;
  a.E = s->E;
  a.k = s->k;
  a.renorm = renorm_of(s);
  a.bf16 = act == MOE_BF16;
  a.x = x;
  a.wg = wg;
  a.da = da_perm;
  a.inv = inv;
  a.dlogits = dlogits;
  a.dx = dx;
  a.dwg = dwg;
  a.dbias = dbias;
  a.ws = ws;
  return hip_status(launch_router_grad(a, (hipStream_t)stream));
}

}  // extern "C"
