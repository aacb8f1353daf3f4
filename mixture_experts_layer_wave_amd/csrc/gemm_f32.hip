// Grouped float32 products of training: the up projection that keeps its
// pre-activations, and the expert FFN's gradient (formulas in gemm_grad.h).
// Everything stays float32 (v_mfma_f32_32x32x2_f32 accumulates each product
// in float32), so dg, du and w h are not rounded between the products.
// Any d and d_ff; pointers need no alignment beyond a float's.
#include "common.h"
#include "gemm_common.h"
#include "gemm_f32.h"
#include "gemm_grad.h"
#include "kernels.h"
#include "route_dev.h"

namespace moe {
namespace {

using namespace f32gemm;
// K groups of a block: the products that everything waits for often have few
// blocks, the rest of the gradient many (5 experts, 501 x 709, 666 rows: the
// rest 57.8 us with Two, 44.4 with One; dh 19.0 with Two, about 23 with One.
// 16 times the rows and six times the weights: dh and the up projection 3%
// slower with Two).
using One = Groups<1>;
using Two = Groups<2>;
using gemm::TileSlot;

struct F32Params {
  const float *a, *dy;
  const int32_t *perm, *inv, *offsets, *slot;
  const float *topk_w;
  int n_slots, src_rows, k, E, R, d, f, n_nt;  // src_rows: rows of a and dy
  const float *w1, *w3, *w2, *g, *u;
  float *dg, *du, *hs, *part;  // gradient
  float *o0, *o1, *o2, *o3;    // up: h, g, u; gradient: da's planes, dW1, dW3, dW2
  int splits;                  // da's planes
};

// A row-major matrix as a buffer (under 2^31 bytes, checked on the host), and
// the byte offset of an element.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t f32_rsrc(const float *p, int rows, int cols) {
  return gemm::rsrc(p, (uint32_t)rows * (uint32_t)cols * 4u);
}
__device__ __forceinline__ uint32_t at(int row, int cols, int col) {
  return ((uint32_t)row * (uint32_t)cols + (uint32_t)col) * 4u;
}

__device__ __forceinline__ float sigmoid_f32(float g) { return 1.0f / (1.0f + expf(-g)); }

// The tile's pile, first row, rows, column tile and K range, from the pile
// sizes; false for a block without work.
__device__ __forceinline__ bool row_tile(const F32Params &p, TileSlot &s_t, int block, int splits) {
  if (threadIdx.x < 64)
    gemm::map_block<kT>(p.offsets, p.E, p.n_nt, splits, threadIdx.x, &s_t, splits, 0, block);
  __syncthreads();
  return s_t.e >= 0;
}

// Rows of this thread's pieces of an operand contiguous along K, gathered or
// not (past the tile's rows: -1).
__device__ __forceinline__ void source_rows(int (&src)[kFour], const int32_t *perm, int row0, int rows) {
#pragma unroll
  for (int i = 0; i < kFour; ++i) {
    int k, r;
    place<false>(i, k, r);
    src[i] = r < rows ? (perm ? perm[row0 + r] : row0 + r) : -1;
  }
}

// g = a W1^T, u = a W3^T, h = silu(g) u.
__global__ __launch_bounds__(Two::THREADS, 4) void up_save_f32_kernel(F32Params p) {
  __shared__ __attribute__((aligned(16))) float smem[Two::SMEM];
  __shared__ TileSlot s_t;
  if (!row_tile(p, s_t, blockIdx.x, 1)) return;
  const int row0 = s_t.row0, rows = s_t.rows, n0 = s_t.nt * kT;
  const size_t mat = (size_t)phys_slot(p.slot, p.n_slots, s_t.e) * p.f * p.d;
  int src[kFour];
  source_rows(src, p.perm, row0, rows);
  const auto ra = f32_rsrc(p.a, p.src_rows, p.d);
  auto fa = [&](int i, int k, int) { return Piece{ra, at(src[i], p.d, k), src[i] >= 0 ? 4 : 0}; };
  auto weights = [&](const float *w) {
    const auto rw = f32_rsrc(w + mat, p.f, p.d);
    return [=](int, int k, int c) { return Piece{rw, at(n0 + c, p.d, k), n0 + c < p.f ? 4 : 0}; };
  };
  f32x4 g[Two::LINES], u[Two::LINES];
  f32x16 sum = {};
  product<2, false, false>(sum, smem, p.d, fa, weights(p.w1));
  lines<2>(sum, smem, g);
  sum = f32x16{};
  product<2, false, false>(sum, smem, p.d, fa, weights(p.w3));
  lines<2>(sum, smem, u);
  const int c = n0 + Two::col();
#pragma unroll
  for (int i = 0; i < Two::LINES; ++i) {
    if (Two::row(i) >= rows) continue;
    const size_t o = (size_t)(row0 + Two::row(i)) * p.f + c;
    f32x4 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = g[i][j] * sigmoid_f32(g[i][j]) * u[i][j];
    store4(p.o0 + o, p.f - c, h);
    store4(p.o1 + o, p.f - c, g[i]);
    store4(p.o2 + o, p.f - c, u[i]);
  }
}

// dh0 = dy W2 and what follows from it; row sums of dh0 h over the tile's 64
// columns go to part[column tile][row].
__global__ __launch_bounds__(Two::THREADS, 4) void dh_f32_kernel(F32Params p) {
  __shared__ __attribute__((aligned(16))) float smem[Two::SMEM];
  __shared__ float s_w[kT];
  __shared__ TileSlot s_t;
  if (!row_tile(p, s_t, blockIdx.x, 1)) return;
  const int row0 = s_t.row0, rows = s_t.rows, n0 = s_t.nt * kT;
  const float *w2 = p.w2 + (size_t)phys_slot(p.slot, p.n_slots, s_t.e) * p.d * p.f;
  int src[kFour];
  source_rows(src, p.perm, row0, rows);
  if (threadIdx.x < kT) {  // combine weight of a row, that of the pair whose row it is
    const int r = row0 + threadIdx.x;
    float w = 1.f;
    if (p.perm && (int)threadIdx.x < rows) {
      const size_t t = p.perm[r];
      w = 0.f;
      for (int j = 0; j < p.k; ++j)
        if (p.inv[t * p.k + j] == r) w = p.topk_w[t * p.k + j];
    }
    s_w[threadIdx.x] = w;
  }
  const auto ra = f32_rsrc(p.dy, p.src_rows, p.d), rw = f32_rsrc(w2, p.d, p.f);
  f32x16 dot = {};
  product<2, false, true>(
      dot, smem, p.d, [&](int i, int k, int) { return Piece{ra, at(src[i], p.d, k), src[i] >= 0 ? 4 : 0}; },
      [&](int, int k, int c) { return Piece{rw, at(k, p.f, n0 + c), p.f - n0 - c}; });
  const int c = n0 + Two::col();
  const size_t base = (size_t)row0 * p.f;
  const auto rg = f32_rsrc(p.g + base, rows, p.f), ru = f32_rsrc(p.u + base, rows, p.f);
  f32x4 acc[Two::LINES], g[Two::LINES], u[Two::LINES];
#pragma unroll
  for (int i = 0; i < Two::LINES; ++i) {
    const int r = Two::row(i), n = r < rows ? p.f - c : 0;
    g[i] = fetch4(Piece{rg, at(r, p.f, c), n});
    u[i] = fetch4(Piece{ru, at(r, p.f, c), n});
  }
  lines<2>(dot, smem, acc);
#pragma unroll
  for (int i = 0; i < Two::LINES; ++i) {
    const int r = Two::row(i);
    const float wr = s_w[r];
    f32x4 dg, du, hs;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = sigmoid_f32(g[i][j]), a = g[i][j] * s, h = a * u[i][j], dh = acc[i][j] * wr;
      sum = fmaf(acc[i][j], h, sum);
      dg[j] = dh * u[i][j] * fmaf(a, 1.0f - s, s);
      du[j] = dh * a;
      hs[j] = wr * h;
    }
    sum = group_sum(sum, 16);
    if (r >= rows) continue;
    const size_t o = base + (size_t)r * p.f + c;
    store4(p.dg + o, p.f - c, dg);
    store4(p.du + o, p.f - c, du);
    store4(p.hs + o, p.f - c, hs);
    if (p.perm && (threadIdx.x & 15) == 0) p.part[(size_t)s_t.nt * p.R + row0 + r] = sum;
  }
}

// One K range of da = dg W1 + du W3: split 2 s + h of 2 S is range s of half
// h (0: dg W1, 1: du W3); its sums go to plane dx_part[split][R][d].
__device__ __forceinline__ void dx_tile(const F32Params &p, int block, float *smem, TileSlot &s_t) {
  if (!row_tile(p, s_t, block, p.splits)) return;
  const int row0 = s_t.row0, rows = s_t.rows, n0 = s_t.nt * kT;
  const size_t mat = (size_t)phys_slot(p.slot, p.n_slots, s_t.e) * p.f * p.d;
  const int half = s_t.split & 1, S = p.splits / 2, steps = (p.f + kK - 1) / kK;
  const int k0 = (int)((long long)(s_t.split / 2) * steps / S) * kK;
  const int k1 = min(p.f, (int)((long long)(s_t.split / 2 + 1) * steps / S) * kK);
  const auto rz = f32_rsrc((half ? p.du : p.dg) + (size_t)row0 * p.f, rows, p.f);
  const auto rw = f32_rsrc((half ? p.w3 : p.w1) + mat, p.f, p.d);
  f32x4 acc[One::LINES];
  f32x16 sum = {};
  product<1, false, true>(
      sum, smem, k1 - k0, [&](int, int k, int m) { return Piece{rz, at(m, p.f, k0 + k), m < rows ? 4 : 0}; },
      [&](int, int k, int c) { return Piece{rw, at(k0 + k, p.d, n0 + c), p.d - n0 - c}; });
  lines<1>(sum, smem, acc);
  float *out = p.o0 + ((size_t)s_t.split * p.R + row0) * p.d;
  const int c = n0 + One::col();
#pragma unroll
  for (int i = 0; i < One::LINES; ++i)
    if (One::row(i) < rows) store4(out + (size_t)One::row(i) * p.d + c, p.d - c, acc[i]);
}

constexpr int kTokens = 1024;

// Weight gradients: dW1 and dW3 (f x d; row tiles of dW1, then of dW3), or
// dW2 (d x f).  Blocks run over an expert's column tiles, then its row tiles.
template <bool W2>
__device__ __forceinline__ void dw_tile(const F32Params &p, int block, float *smem, int32_t *s_tok) {
  const int M = W2 ? p.d : p.f, N = W2 ? p.f : p.d, mt = (M + kT - 1) / kT, nt = (N + kT - 1) / kT;
  const int per = (W2 ? mt : 2 * mt) * nt, e = block / per, tile = block % per;
  const int n0 = tile % nt * kT;
  const bool second = !W2 && tile / nt >= mt;
  const int m0 = (tile / nt - (second ? mt : 0)) * kT;
  const int row0 = p.offsets[e], rows = p.offsets[e + 1] - row0;
  f32x4 acc[One::LINES];
  f32x16 sum = {};
  // 1024 of the pile's rows at a time, their tokens in LDS (a fetch that
  // waited for a token from memory would drain the fetches before it); an
  // empty pile's weight gradients are zeros.
  for (int q0 = 0; q0 < rows; q0 += kTokens) {
    const int q = min(kTokens, rows - q0), first = row0 + q0;
    __syncthreads();
    for (int i = threadIdx.x; i < q; i += One::THREADS) s_tok[i] = p.perm ? p.perm[first + i] : first + i;
    __syncthreads();
    const auto rf = f32_rsrc((W2 ? p.hs : second ? p.du : p.dg) + (size_t)first * p.f, q, p.f);
    const auto rd = f32_rsrc(W2 ? p.dy : p.a, p.src_rows, p.d);
    auto token = [&](int k) { return s_tok[min(k, q - 1)]; };
    product<1, true, true>(
        sum, smem, q,
        [&](int, int k, int m) {
          return W2 ? Piece{rd, at(token(k), p.d, m0 + m), M - m0 - m} : Piece{rf, at(k, p.f, m0 + m), M - m0 - m};
        },
        [&](int, int k, int c) {
          return W2 ? Piece{rf, at(k, p.f, n0 + c), N - n0 - c} : Piece{rd, at(token(k), p.d, n0 + c), N - n0 - c};
        });
  }
  lines<1>(sum, smem, acc);
  float *out = (W2 ? p.o3 : second ? p.o2 : p.o1) + (size_t)e * M * N;
  const int c = n0 + One::col();
#pragma unroll
  for (int i = 0; i < One::LINES; ++i) {
    const int r = m0 + One::row(i);
    if (r < M) store4(out + (size_t)r * N + c, N - c, acc[i]);
  }
}

// Everything that waits for dg, du and w h, in one grid: da, then dW1 and
// dW3, then dW2.
__global__ __launch_bounds__(One::THREADS, 4) void rest_f32_kernel(F32Params p, int end_dx, int end_dw13) {
  __shared__ __attribute__((aligned(16))) float smem[One::SMEM];
  __shared__ int32_t s_tok[kTokens];
  __shared__ TileSlot s_t;
  const int b = blockIdx.x;
  if (b < end_dx)
    dx_tile(p, b, smem, s_t);
  else if (b < end_dw13)
    dw_tile<false>(p, b - end_dx, smem, s_tok);
  else
    dw_tile<true>(p, b - end_dw13, smem, s_tok);
}

int row_tiles(int R, int E) { return (R + kT - 1) / kT + (E < R ? E : R); }

}  // namespace

// da's K ranges, two at least (one for each of its two products), more until
// its blocks fill the chip two to a CU, each range 128 deep at least.
GradPlan grad_plan_f32(const FfnGradArgs &a) {
  const int blocks = row_tiles(a.R, a.E) * ((a.d + kT - 1) / kT) * 2;
  int S = blocks < 512 ? 512 / blocks : 1;
  if (S > a.d_ff / 128) S = a.d_ff / 128;
  return {(a.d_ff + kT - 1) / kT, 2 * (S < 1 ? 1 : S)};
}

hipError_t launch_up_save_f32(const FfnArgs &a, void *g, void *u, hipStream_t st) {
  F32Params p{};
  p.a = (const float *)a.a;
  p.src_rows = a.perm ? a.n : a.R;
  p.perm = a.perm;
  p.offsets = a.offsets;
  p.slot = a.slot;
  p.n_slots = a.n_slots;
  p.E = a.E;
  p.R = a.R;
  p.d = a.d;
  p.f = a.d_ff;
  p.w1 = (const float *)a.w1;
  p.w3 = (const float *)a.w3;
  p.o0 = (float *)a.h;
  p.o1 = (float *)g;
  p.o2 = (float *)u;
  p.n_nt = (p.f + kT - 1) / kT;
  up_save_f32_kernel<<<row_tiles(p.R, p.E) * p.n_nt, Two::THREADS, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_grad_f32(const FfnGradArgs &a, const FfnGradWs &w, hipStream_t st) {
  F32Params p{};
  p.a = (const float *)a.a;
  p.src_rows = a.perm ? a.n : a.R;
  p.dy = (const float *)a.dy;
  p.perm = a.perm;
  p.inv = a.inv;
  p.topk_w = a.topk_w;
  p.offsets = a.offsets;
  p.slot = a.slot;
  p.n_slots = a.n_slots;
  p.k = a.k;
  p.E = a.E;
  p.R = a.R;
  p.d = a.d;
  p.f = a.d_ff;
  p.w1 = (const float *)a.w1;
  p.w3 = (const float *)a.w3;
  p.w2 = (const float *)a.w2;
  p.g = (const float *)a.g;
  p.u = (const float *)a.u;
  p.dg = (float *)w.dg;
  p.du = (float *)w.du;
  p.hs = (float *)w.hs;
  p.part = w.part;
  const int ft = (p.f + kT - 1) / kT, dt = (p.d + kT - 1) / kT;
  const int rt = row_tiles(p.R, p.E);
  p.n_nt = ft;
  dh_f32_kernel<<<rt * ft, Two::THREADS, 0, st>>>(p);
  p.n_nt = dt;
  p.splits = w.plan.dx_splits;
  p.o0 = w.dx_part;
  p.o1 = (float *)a.dw1;
  p.o2 = (float *)a.dw3;
  p.o3 = (float *)a.dw2;
  const int end_dx = (rt * dt * p.splits + 7) / 8 * 8, dw = p.E * ft * dt;
  rest_f32_kernel<<<end_dx + 3 * dw, One::THREADS, 0, st>>>(p, end_dx, end_dx + 2 * dw);
  return hipGetLastError();
}

}  // namespace moe
