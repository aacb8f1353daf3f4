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

namespace moe {
namespace {

using namespace f32gemm;
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
__global__ __launch_bounds__(kThreads) void up_save_f32_kernel(F32Params p) {
  __shared__ float smem[kSmem];
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
  f32x16 ga = {}, ua = {};
  product<false, false>(ga, smem, p.d, fa, weights(p.w1));
  product<false, false>(ua, smem, p.d, fa, weights(p.w3));
  const int r = out_row();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = n0 + out_col(i);
    if (r < rows && c < p.f) {
      const size_t o = (size_t)(row0 + r) * p.f + c;
      p.o1[o] = ga[i];
      p.o2[o] = ua[i];
      p.o0[o] = ga[i] * sigmoid_f32(ga[i]) * ua[i];
    }
  }
}

// dh0 = dy W2 and what follows from it; row sums of dh0 h over each wave's 32
// columns go to part[plane][row].
__global__ __launch_bounds__(kThreads) void dh_f32_kernel(F32Params p) {
  __shared__ float smem[kSmem];
  __shared__ TileSlot s_t;
  if (!row_tile(p, s_t, blockIdx.x, 1)) return;
  const int row0 = s_t.row0, rows = s_t.rows, n0 = s_t.nt * kT;
  const float *w2 = p.w2 + (size_t)phys_slot(p.slot, p.n_slots, s_t.e) * p.d * p.f;
  int src[kFour];
  source_rows(src, p.perm, row0, rows);
  const auto ra = f32_rsrc(p.dy, p.src_rows, p.d), rw = f32_rsrc(w2, p.d, p.f);
  f32x16 acc = {};
  product<false, true>(
      acc, smem, p.d, [&](int i, int k, int) { return Piece{ra, at(src[i], p.d, k), src[i] >= 0 ? 4 : 0}; },
      [&](int, int k, int c) { return Piece{rw, at(k, p.f, n0 + c), p.f - n0 - c}; });
  const int r = out_row();
  float wr = 1.f, sum = 0.f;
  if (p.perm && r < rows) {
    const int t = p.perm[row0 + r];
    wr = 0.f;
    for (int j = 0; j < p.k; ++j)
      if (p.inv[(size_t)t * p.k + j] == row0 + r) wr = p.topk_w[(size_t)t * p.k + j];
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = n0 + out_col(i);
    if (r < rows && c < p.f) {
      const size_t o = (size_t)(row0 + r) * p.f + c;
      const float g = p.g[o], u = p.u[o], s = sigmoid_f32(g), a = g * s, h = a * u;
      sum = fmaf(acc[i], h, sum);
      const float dh = acc[i] * wr;
      p.dg[o] = dh * u * fmaf(a, 1.0f - s, s);
      p.du[o] = dh * a;
      p.hs[o] = wr * h;
    }
  }
  sum += __shfl_xor(sum, 32, 64);
  const int plane = s_t.nt * 2 + ((threadIdx.x >> 6) & 1);
  if (p.perm && (threadIdx.x & 63) < 32 && r < rows) p.part[(size_t)plane * p.R + row0 + r] = sum;
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
  f32x16 acc = {};
  product<false, true>(
      acc, smem, k1 - k0, [&](int, int k, int m) { return Piece{rz, at(m, p.f, k0 + k), m < rows ? 4 : 0}; },
      [&](int, int k, int c) { return Piece{rw, at(k0 + k, p.d, n0 + c), p.d - n0 - c}; });
  float *out = p.o0 + ((size_t)s_t.split * p.R + row0) * p.d;
  const int r = out_row();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = n0 + out_col(i);
    if (r < rows && c < p.d) out[(size_t)r * p.d + c] = acc[i];
  }
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
  f32x16 acc = {};
  // 1024 of the pile's rows at a time, their tokens in LDS (a fetch that
  // waited for a token from memory would drain the fetches before it); an
  // empty pile's weight gradients are zeros.
  for (int q0 = 0; q0 < rows; q0 += kTokens) {
    const int q = min(kTokens, rows - q0), first = row0 + q0;
    __syncthreads();
    for (int i = threadIdx.x; i < q; i += kThreads) s_tok[i] = p.perm ? p.perm[first + i] : first + i;
    __syncthreads();
    const auto rf = f32_rsrc((W2 ? p.hs : second ? p.du : p.dg) + (size_t)first * p.f, q, p.f);
    const auto rd = f32_rsrc(W2 ? p.dy : p.a, p.src_rows, p.d);
    auto token = [&](int k) { return s_tok[min(k, q - 1)]; };
    product<true, true>(
        acc, smem, q,
        [&](int, int k, int m) {
          return W2 ? Piece{rd, at(token(k), p.d, m0 + m), M - m0 - m} : Piece{rf, at(k, p.f, m0 + m), M - m0 - m};
        },
        [&](int, int k, int c) {
          return W2 ? Piece{rf, at(k, p.f, n0 + c), N - n0 - c} : Piece{rd, at(token(k), p.d, n0 + c), N - n0 - c};
        });
  }
  float *out = (W2 ? p.o3 : second ? p.o2 : p.o1) + (size_t)e * M * N;
  const int r = m0 + out_row();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = n0 + out_col(i);
    if (r < M && c < N) out[(size_t)r * N + c] = acc[i];
  }
}

// Everything that waits for dg, du and w h, in one grid: da, then dW1 and
// dW3, then dW2.
__global__ __launch_bounds__(kThreads) void rest_f32_kernel(F32Params p, int end_dx, int end_dw13) {
  __shared__ float smem[kSmem];
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
// its blocks fill the chip four to a CU, each range 128 deep at least.
GradPlan grad_plan_f32(const FfnGradArgs &a) {
  const int blocks = row_tiles(a.R, a.E) * ((a.d + kT - 1) / kT) * 2;
  int S = blocks < 1024 ? 1024 / blocks : 1;
  if (S > a.d_ff / 128) S = a.d_ff / 128;
  return {(a.d_ff + kT - 1) / kT * 2, 2 * (S < 1 ? 1 : S)};
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
  up_save_f32_kernel<<<row_tiles(p.R, p.E) * p.n_nt, kThreads, 0, st>>>(p);
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
  dh_f32_kernel<<<rt * ft, kThreads, 0, st>>>(p);
  p.n_nt = dt;
  p.splits = w.plan.dx_splits;
  p.o0 = w.dx_part;
  p.o1 = (float *)a.dw1;
  p.o2 = (float *)a.dw3;
  p.o3 = (float *)a.dw2;
  const int end_dx = (rt * dt * p.splits + 7) / 8 * 8, dw = p.E * ft * dt;
  rest_f32_kernel<<<end_dx + 3 * dw, kThreads, 0, st>>>(p, end_dx, end_dx + 2 * dw);
  return hipGetLastError();
}

}  // namespace moe
