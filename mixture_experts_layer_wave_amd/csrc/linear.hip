// Product with an MXFP4 matrix (moe_mxfp4_linear): y = x W^T + bias, x in bf16 or
// MXFP4.
//
// Few rows are bound by reading W: the weight rows go straight into the matrix
// cores (wave_stream.h).  A workgroup takes an equal run of output columns in
// tiles of at most 16; its waves share out the tiles and, where there are fewer
// tiles than waves, a tile's K steps.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "wave_stream.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;

struct LinearParams {
  const uint8_t *x, *xs, *w, *ws;
  const float *bias;
  void *y;
  int n, d, m, out_bf16;
  int G;  // workgroups of one group of 16 rows
};

__device__ __forceinline__ void put(const LinearParams &p, int t, int c, float v) {
  if (p.bias) v += p.bias[c];
  const size_t at = (size_t)t * p.m + c;
  if (p.out_bf16)
    ((uint16_t *)p.y)[at] = (uint16_t)f32_to_bf16_bits(v);
  else
    ((float *)p.y)[at] = v;
}

template <int WT, int ARING, int PF>
__global__ __launch_bounds__(kThreads) void linear_rows_kernel(LinearParams p) {
  using F = Form<WT>;
  constexpr int NF = F::kActBytes / 16;
  __shared__ __attribute__((aligned(16))) uint8_t s_stage[WT == kMx ? kWaves * 1024 * ARING : 16];
  __shared__ __attribute__((aligned(16))) float s_red[kWaves][64][4];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = blockIdx.x % p.G, t0 = blockIdx.x / p.G * 16, rows = min(16, p.n - t0);
  const int d = p.d, m = p.m;
  const int c_lo = (int)((long long)m * part / p.G), c_hi = (int)((long long)m * (part + 1) / p.G);
  const int cols = c_hi - c_lo, tiles = (cols + 15) / 16;
  int KS = kWaves;  // waves on one tile
  while (KS > 1 && tiles > kWaves / KS) KS >>= 1;
  const int mine = wave / KS, step = kWaves / KS, kp = wave % KS;  // this wave's tiles: mine, mine + step, ..
  const int S = (F::blocks(d) + 3) / 4, s_lo = S * kp / KS, s_hi = S * (kp + 1) / KS;
  const int segs = tiles > mine ? (tiles - mine + step - 1) / step : 0;
  const size_t rb = F::row_bytes(d), xb = WT == kMx4 ? (size_t)d / 2 : (size_t)d * 2;
  auto col = [&](int tile) { return c_lo + (int)((long long)cols * tile / max(tiles, 1)); };
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  stream<WT, PF, ARING>(
      segs * (s_hi - s_lo), S, s_lo, d, s_stage + (WT == kMx ? wave * 1024 * ARING : 0),
      [&](int i, const uint8_t *&row, const uint8_t *&srow, const uint8_t *(&arow)[ARING], const uint8_t *&asrow) {
        const int tile = mine + i * step, c = col(tile), cnt = col(tile + 1) - c;
        const size_t wr = (size_t)c + min(r, cnt - 1);
        row = p.w + wr * rb;
        srow = p.ws + wr * (d / 32);
#pragma unroll
        for (int j = 0; j < ARING; ++j)
          arow[j] = p.x + (size_t)(t0 + min(WT == kMx ? g + 4 * j : r, rows - 1)) * xb;
        if constexpr (WT == kMx4) asrow = p.xs + (size_t)(t0 + min(r, rows - 1)) * (d / 32);
      },
      [&](int, int, u32x4 (&)[NF]) {}, [&](int) { return min(r, rows - 1); },
      [&](int i, f32x4 v) {
        if (KS > 1) {
          sum = v;
          return;
        }
        const int tile = mine + i * step, c = col(tile), cnt = col(tile + 1) - c;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r < cnt && 4 * g + q < rows) put(p, t0 + 4 * g + q, c + r, v[q]);
      });
  if (KS == 1) return;
  // (KS > 1: a wave has one tile at most)
  *(f32x4 *)s_red[wave][lane] = sum;
  __syncthreads();
  if (kp == 0 && segs > 0) {
    const int c = col(mine), cnt = col(mine + 1) - c;
    for (int j = 1; j < KS; ++j) sum += *(const f32x4 *)s_red[wave + j][lane];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (r < cnt && 4 * g + q < rows) put(p, t0 + 4 * g + q, c + r, sum[q]);
  }
}

}  // namespace

size_t mxfp4_linear_bytes(int n, int d, int m, bool x_mx4) { return 0; }

hipError_t launch_mxfp4_linear(const LinearArgs &a, hipStream_t st) {
  LinearParams p{};
  p.x = (const uint8_t *)a.x;
  p.xs = a.x_s;
  p.w = a.w;
  p.ws = a.w_s;
  p.bias = a.bias;
  p.y = a.y;
  p.n = a.n;
  p.d = a.d;
  p.m = a.m;
  p.out_bf16 = a.out_bf16;
  p.G = std::min(cu_count(), a.m);
  const int grid = p.G * ((a.n + 15) / 16);
  if (a.x_mx4)
    linear_rows_kernel<kMx4, 1, 12><<<grid, kThreads, 0, st>>>(p);
  else if (a.n <= 4)
    linear_rows_kernel<kMx, 1, 12><<<grid, kThreads, 0, st>>>(p);
  else if (a.n <= 8)
    linear_rows_kernel<kMx, 2, 8><<<grid, kThreads, 0, st>>>(p);
  else
    linear_rows_kernel<kMx, 4, 6><<<grid, kThreads, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
