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

// dtopk_w from the partial row sums part[P][R].  A block takes 64 pile rows,
// 16 waves the planes w, w + 16, ... of each; the 16 sums are added in wave
// order, so the result does not depend on scheduling.  The sum of row r goes
// to the pair whose row it is; pairs without a row (inv outside [0, R)) get 0.
__global__ __launch_bounds__(1024) void weight_grad_kernel(const float *__restrict__ part, int P, int R,
                                                           int E, const int32_t *__restrict__ offsets,
                                                           const int32_t *__restrict__ perm,
                                                           const int32_t *__restrict__ inv, int k,
                                                           float *__restrict__ dw) {
  __shared__ float s_p[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = blockIdx.x * 64 + lane;
  const bool piled = r < R && r < offsets[E];
  float v = 0.f;
  if (piled)
    for (int q = wave; q < P; q += 16) v += part[(size_t)q * R + r];
  s_p[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && piled) {
    v = 0.f;
    for (int i = 0; i < 16; ++i) v += s_p[i][lane];
    const int t = perm[r];
    for (int j = 0; j < k; ++j)
      if (inv[(size_t)t * k + j] == r) dw[(size_t)t * k + j] = v;
  }
  if (wave == 1 && r < R && (unsigned)inv[r] >= (unsigned)R) dw[r] = 0.f;  // pair r
}

struct Layout {
  size_t du, hs, part, total;
};

Layout layout(const FfnGradArgs &a) {
  Layout L{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t mat = up((size_t)a.R * a.d_ff * (a.bf16 ? 2 : 4));
  const int planes = a.bf16 ? grad_planes_bf16(a.d_ff) : grad_planes_f32(a.d_ff);
  L.du = mat;
  L.hs = 2 * mat;
  L.part = 3 * mat;
  L.total = L.part + up((size_t)planes * a.R * 4);
  return L;
}

}  // namespace

size_t ffn_grad_bytes(const FfnGradArgs &a) { return layout(a).total; }

hipError_t launch_ffn_grad(const FfnGradArgs &a, hipStream_t st) {
  const Layout L = layout(a);
  char *base = (char *)a.ws;
  const FfnGradWs w{base, base + L.du, base + L.hs, (float *)(base + L.part)};
  int planes = 0;
  const hipError_t e = a.bf16 ? launch_grad_bf16(a, w, &planes, st) : launch_grad_f32(a, w, &planes, st);
  if (e != hipSuccess || !a.perm) return e;
  weight_grad_kernel<<<(a.R + 63) / 64, 1024, 0, st>>>(w.part, planes, a.R, a.E, a.offsets, a.perm,
                                                       a.inv, a.k, a.dtopk_w);
  return hipGetLastError();
}

}  // namespace moe
