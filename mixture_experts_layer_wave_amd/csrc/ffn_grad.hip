// The expert FFN's gradient: workspace layout, the products (gemm_grad.hip,
// gemm_f32.hip) and the sum that gives the combine weights' gradient.
//
// y_t = sum_j w_tj yp_r with yp_r = h_r W2^T gives
//   d w_tj = <dy_t, yp_r> = <dy_t W2, h_r> = <dh0_r, h_r>,
// so the weights' gradient falls out of the dh product, whose epilogue has
// both factors in registers: the pile outputs yp need not be kept for it,
// and dy needs no copy scaled by w (the epilogue scales the product's rows).
#include "common.h"
#include "gemm_grad.h"
#include "kernels.h"

namespace moe {
namespace {

struct FinishParams {
  const float *part;
  int P, R, E, k, d;
  const int32_t *offsets, *perm, *inv;
  float *dw;
  const float *dx_part;
  int S, bf16;
  void *da;
  int w_blocks;  // blocks of the weights' gradient (0 without a combine)
};

// The last kernel of the pass.  Blocks 0 .. w_blocks - 1: dtopk_w from the
// partial row sums part[P][R], 64 pile rows a block, 16 waves the planes w,
// w + 16, ... of each; the 16 sums are added in wave order, so the result
// does not depend on scheduling.  The sum of row r goes to the pair whose row
// it is; pairs without a row (inv outside [0, R)) get 0.  The other blocks:
// the piled rows of da, four elements a thread (bf16) or one, as the sum of
// their S planes in order (4096 rows of 1024, three planes: 11.1 us).
__global__ __launch_bounds__(1024) void ffn_grad_finish_kernel(FinishParams p) {
  __shared__ float s_p[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x < p.w_blocks) {
    const int r = blockIdx.x * 64 + lane;
    const bool piled = r < p.R && r < p.offsets[p.E];
    float v = 0.f;
    if (piled)
      for (int q = wave; q < p.P; q += 16) v += p.part[(size_t)q * p.R + r];
    s_p[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && piled) {
      v = 0.f;
      for (int i = 0; i < 16; ++i) v += s_p[i][lane];
      const int t = p.perm[r];
      for (int j = 0; j < p.k; ++j)
        if (p.inv[(size_t)t * p.k + j] == r) p.dw[(size_t)t * p.k + j] = v;
    }
    if (wave == 1 && r < p.R && (unsigned)p.inv[r] >= (unsigned)p.R) p.dw[r] = 0.f;  // pair r
    return;
  }
  const size_t total = (size_t)p.offsets[p.E] * p.d, plane = (size_t)p.R * p.d;
  const size_t i = (size_t)(blockIdx.x - p.w_blocks) * 1024 + threadIdx.x;
  if (p.bf16) {
    if (i * 4 >= total) return;
    f32x4 v = *(const f32x4 *)(p.dx_part + i * 4);
#pragma unroll 4
    for (int s = 1; s < p.S; ++s) v += *(const f32x4 *)(p.dx_part + s * plane + i * 4);
    *(u32x2 *)((uint16_t *)p.da + i * 4) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  } else {
    if (i >= total) return;
    float v = p.dx_part[i];
#pragma unroll 8
    for (int s = 1; s < p.S; ++s) v += p.dx_part[s * plane + i];
    ((float *)p.da)[i] = v;
  }
}

struct Layout {
  GradPlan plan;
  size_t du, hs, part, dx_part, total;
};

Layout layout(const FfnGradArgs &a) {
  Layout L{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t mat = up((size_t)a.R * a.d_ff * (a.bf16 ? 2 : 4));
  L.plan = a.bf16 ? grad_plan_bf16(a) : grad_plan_f32(a);
  L.du = mat;
  L.hs = 2 * mat;
  L.part = 3 * mat;
  L.dx_part = L.part + up((size_t)L.plan.dw_planes * a.R * 4);
  L.total = L.dx_part + (L.plan.dx_splits > 1 ? up((size_t)L.plan.dx_splits * a.R * a.d * 4) : 0);
  return L;
}

}  // namespace

size_t ffn_grad_bytes(const FfnGradArgs &a) { return layout(a).total; }

hipError_t launch_ffn_grad(const FfnGradArgs &a, hipStream_t st) {
  const Layout L = layout(a);
  char *base = (char *)a.ws;
  const FfnGradWs w{L.plan, base, base + L.du, base + L.hs, (float *)(base + L.part), (float *)(base + L.dx_part)};
  const hipError_t e = a.bf16 ? launch_grad_bf16(a, w, st) : launch_grad_f32(a, w, st);
  if (e != hipSuccess) return e;
  FinishParams p{};
  p.part = w.part;
  p.P = L.plan.dw_planes;
  p.R = a.R;
  p.E = a.E;
  p.k = a.k;
  p.d = a.d;
  p.offsets = a.offsets;
  p.perm = a.perm;
  p.inv = a.inv;
  p.dw = a.dtopk_w;
  p.dx_part = w.dx_part;
  p.S = L.plan.dx_splits;
  p.da = a.da;
  p.bf16 = a.bf16;
  p.w_blocks = a.perm ? (a.R + 63) / 64 : 0;
  const size_t sums = p.S > 1 ? ((size_t)a.R * a.d / (a.bf16 ? 4 : 1) + 1023) / 1024 : 0;
  if (p.w_blocks + sums == 0) return hipSuccess;
  ffn_grad_finish_kernel<<<(unsigned)(p.w_blocks + sums), 1024, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
