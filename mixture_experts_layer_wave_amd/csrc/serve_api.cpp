// Host side of the last part of include/moe.h: the MXFP4 codec and product, the
// layer for a few tokens, and the norms around a block.  As in moe_api.cpp,
// nothing here allocates device memory or synchronises.
#include "moe.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_internal.h"
#include "kernels.h"

using namespace moe;

namespace {

// rows x cols values in MXFP4: whole blocks, and a count that 64 bits hold.
int check_mx4(int64_t rows, int32_t cols, int dtype) {
  if (rows < 0 || rows > (1ll << 31) - 1 || cols <= 0 || cols % 32) return MOE_ERR_SHAPE;
  return dtype == MOE_F32 || dtype == MOE_BF16 ? MOE_OK : MOE_ERR_DTYPE;
}

int check_linear(int32_t n, int32_t d, int32_t m, int act) {
  if (n < 0 || d < 32 || d % 32 || m < 1) return MOE_ERR_SHAPE;
  if (act != MOE_BF16 && act != MOE_MXFP4) return MOE_ERR_DTYPE;
  // 32-bit byte offsets into x, y and W as bf16, as moe_shape asks of them
  if ((long long)n * std::max(d, m) >= (1ll << 30) || (long long)m * d >= (1ll << 30)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int check_few(const moe_shape *s, int wdt) {
  int st = check_shape(s);
  if (st != MOE_OK) return st;
  if (s->n > MOE_FEW_MAX_TOKENS) return MOE_ERR_SHAPE;
  st = check_dtypes(s, wdt == MOE_F32 ? MOE_F32 : MOE_BF16, wdt);
  if (st != MOE_OK) return st;
  // A group of eight weight rows is read by 32-bit byte offsets (wave_stream.h); bf16 and
  // MXFP4 matrices are small enough by check_dtypes.
  if (wdt == MOE_F32 && std::max(s->d, s->d_ff) >= (1 << 26)) return MOE_ERR_SHAPE;
  // the hidden columns of all chosen experts are counted in 32 bits
  if ((long long)s->n * s->k * s->d_ff >= (1ll << 30)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int check_block_norm(int32_t n, int32_t d, int act, const moe_norm *post, const moe_norm *pre) {
  if (n < 0 || n >= (1 << 30) || d < 1 || d > kLayerNormMaxD) return MOE_ERR_SHAPE;
  if (act != MOE_F32 && act != MOE_BF16) return MOE_ERR_DTYPE;
  if (act == MOE_BF16 && d % 8) return MOE_ERR_SHAPE;
  for (const moe_norm *v : {post, pre})
    if (v) {
      if (v->kind != MOE_NORM_LAYER && v->kind != MOE_NORM_RMS) return MOE_ERR_DTYPE;
      if (!(v->eps >= 0.f)) return MOE_ERR_SHAPE;
      if (!v->weight) return MOE_ERR_NULL;
    }
  return MOE_OK;
}

BlockNorm norm_of(const moe_norm *v) {
  return v ? BlockNorm{v->kind == MOE_NORM_RMS ? 2 : 1, v->eps, v->weight, v->bias} : BlockNorm{0, 0.f, nullptr, nullptr};
}

}  // namespace

extern "C" {

int moe_quantize_mxfp4(int64_t rows, int32_t cols, const void *x, int act, uint8_t *q, uint8_t *s, void *stream) {
  const int st = check_mx4(rows, cols, act);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !s) return MOE_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return MOE_ERR_ALIGN;
  return hip_status(launch_quantize_mx4(x, act == MOE_BF16, (size_t)rows * (cols / 32), q, s, (hipStream_t)stream));
}

int moe_dequantize_mxfp4(int64_t rows, int32_t cols, const uint8_t *q, const uint8_t *s, void *y, int out,
                         void *stream) {
  const int st = check_mx4(rows, cols, out);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!q || !s || !y) return MOE_ERR_NULL;
  if (!aligned16(q) || !aligned16(s) || !aligned16(y)) return MOE_ERR_ALIGN;
  return hip_status(launch_dequantize_mx4(q, s, (size_t)rows * (cols / 32), y, out == MOE_BF16, (hipStream_t)stream));
}

size_t moe_mxfp4_linear_workspace_bytes(int32_t n, int32_t d, int32_t m, int act) {
  if (check_linear(n, d, m, act) != MOE_OK || n == 0) return 0;
  return align_up(mxfp4_linear_bytes(n, d, m, act == MOE_MXFP4));
}

int moe_mxfp4_linear(int32_t n, int32_t d, int32_t m, const void *x, const uint8_t *x_s, int act, const uint8_t *w,
                     const uint8_t *w_s, const float *bias, void *y, int out, void *ws, size_t ws_bytes,
                     void *stream) {
  const int st = check_linear(n, d, m, act);
  if (st != MOE_OK) return st;
  if (out != MOE_F32 && out != MOE_BF16) return MOE_ERR_DTYPE;
  if (n == 0) return MOE_OK;
  if (!x || !w || !w_s || !y || (act == MOE_MXFP4 && !x_s)) return MOE_ERR_NULL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(w_s) || !aligned16(y)) return MOE_ERR_ALIGN;
  if (act == MOE_MXFP4 && !aligned16(x_s)) return MOE_ERR_ALIGN;
  const size_t need = moe_mxfp4_linear_workspace_bytes(n, d, m, act);
  if (need > 0) {
    if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned16(ws)) return MOE_ERR_ALIGN;
  }
  LinearArgs a{};
  a.n = n;
  a.d = d;
  a.m = m;
  a.x = x;
  a.x_s = x_s;
  a.x_mx4 = act == MOE_MXFP4;
  a.w = w;
  a.w_s = w_s;
  a.bias = bias;
  a.y = y;
  a.out_bf16 = out == MOE_BF16;
  a.ws = ws;
  return hip_status(launch_mxfp4_linear(a, (hipStream_t)stream));
}

size_t moe_forward_few_workspace_bytes(const moe_shape *s, int w_dtype) {
  if (check_few(s, w_dtype) != MOE_OK) return 0;
  return forward_few_bytes(s->n, s->E, s->k, s->d_ff, w_dtype == MOE_F32);
}

int moe_forward_few(const moe_shape *s, const void *x, int act, const void *wg, const float *bias,
                    const moe_expert_weights *w, void *y, int out, int32_t *topk_idx, float *topk_w, void *ws,
                    size_t ws_bytes, void *stream) {
  int st = check_shape(s);
  if (st != MOE_OK) return st;
  st = check_weights(s, act, w);
  if (st != MOE_OK) return st;
  if (w->act_quant) return MOE_ERR_DTYPE;
  st = check_few(s, w->dtype);
  if (st != MOE_OK) return st;
  if (!x || !wg || !y) return MOE_ERR_NULL;
  if (out != MOE_F32 && out != MOE_BF16) return MOE_ERR_DTYPE;
  if (act == MOE_BF16 && (!aligned16(x) || !aligned16(wg))) return MOE_ERR_ALIGN;
  if (s->d % 4 == 0 && !aligned16(y)) return MOE_ERR_ALIGN;
  if (!ws || ws_bytes < moe_forward_few_workspace_bytes(s, w->dtype)) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_ALIGN;
  FewArgs a{};
  a.x = x;
  a.wg = wg;
  a.bias = bias;
  a.n = s->n;
  a.d = s->d;
  a.E = s->E;
  a.k = s->k;
  a.d_ff = s->d_ff;
  a.renorm = renorm_of(s) ? 1 : 0;
  a.w_dtype = w->dtype;
  a.w1 = w->w1;
  a.w3 = w->w3;
  a.w2 = w->w2;
  a.s1 = w->s1;
  a.s3 = w->s3;
  a.s2 = w->s2;
  a.slot = w->slot;
  a.n_slots = w->slot ? w->n_slots : s->E;
  a.y = y;
  a.out_bf16 = out == MOE_BF16;
  a.idx = topk_idx;
  a.w = topk_w;
  a.ws = ws;
  return hip_status(launch_forward_few(a, (hipStream_t)stream));
}

int moe_block_norm(int32_t n, int32_t d, const void *x, const void *z, int act, float scale, const float *gate,
                   const moe_norm *post, const moe_norm *pre, void *h, void *u, float *stats, void *stream) {
  const int st = check_block_norm(n, d, act, post, pre);
  if (st != MOE_OK) return st;
  if (n == 0) return MOE_OK;
  if (!x || !z || !h || (pre && !u)) return MOE_ERR_NULL;
  if (act == MOE_BF16 && (!aligned16(x) || !aligned16(z) || !aligned16(h) || (pre && !aligned16(u))))
    return MOE_ERR_ALIGN;
  BlockNormArgs a{};
  a.n = n;
  a.d = d;
  a.bf16 = act == MOE_BF16;
  a.scale = scale;
  a.gate = gate;
  a.post = norm_of(post);
  a.pre = norm_of(pre);
  a.x = x;
  a.z = z;
  a.h = h;
  a.u = u;
  a.stats = stats;
  return hip_status(launch_block_norm(a, (hipStream_t)stream));
}

size_t moe_block_norm_backward_workspace_bytes(int32_t n, int32_t d) {
  if (check_block_norm(n, d, MOE_F32, nullptr, nullptr) != MOE_OK) return 0;
  return align_up(block_norm_grad_bytes(n, d));
}

int moe_block_norm_backward(int32_t n, int32_t d, const void *dh, const void *du, const void *z, const void *h,
                            int act, float scale, const float *gate, const moe_norm *post, const moe_norm *pre,
                            const float *stats, void *dx, void *dz, float *dgate, float *dpost_weight,
                            float *dpost_bias, float *dpre_weight, float *dpre_bias, void *ws, size_t ws_bytes,
                            void *stream) {
  const int st = check_block_norm(n, d, act, post, pre);
  if (st != MOE_OK) return st;
  // gradients of parameters that the call does not have
  if ((!gate && dgate) || (!post && (dpost_weight || dpost_bias)) || (!pre && (dpre_weight || dpre_bias)))
    return MOE_ERR_NULL;
  if (n > 0) {
    if (!dx || !dz || (!dh && !pre)) return MOE_ERR_NULL;
    if (pre && (!du || !h)) return MOE_ERR_NULL;
    if ((post || gate) && !z) return MOE_ERR_NULL;
    if ((post || pre) && !stats) return MOE_ERR_NULL;
    if (act == MOE_BF16)
      for (const void *v : {dh, du, z, h, (const void *)dx, (const void *)dz})
        if (!aligned16(v)) return MOE_ERR_ALIGN;  // (NULL is)
    if (!ws || ws_bytes < moe_block_norm_backward_workspace_bytes(n, d)) return MOE_ERR_WORKSPACE;
    if (!aligned16(ws)) return MOE_ERR_ALIGN;
  }
  BlockNormArgs a{};
  a.n = n;
  a.d = d;
  a.bf16 = act == MOE_BF16;
  a.scale = scale;
  a.gate = gate;
  a.post = norm_of(post);
  a.pre = norm_of(pre);
  a.z = z;
  a.h = const_cast<void *>(h);
  a.stats = const_cast<float *>(stats);
  a.dh = dh;
  a.du = du;
  a.dx = dx;
  a.dz = dz;
  a.dgate = dgate;
  a.dpost_w = dpost_weight;
  a.dpost_b = dpost_bias;
  a.dpre_w = dpre_weight;
  a.dpre_b = dpre_bias;
  a.part = (float *)ws;
  return hip_status(launch_block_norm_grad(a, (hipStream_t)stream));
}

}  // extern "C"
