// Product with an MXFP4 matrix (moe_mxfp4_linear): y = x W^T + bias, x in bf16 or
// MXFP4.
//
// Few rows are bound by reading W: the weight rows go straight into the matrix
// cores (wave_stream.h).  A workgroup takes an equal run of output columns in
// tiles of at most 16; its waves share out the tiles and, where there are fewer
// tiles than waves, a tile's K steps.
#include <algorithm>
#include <atomic>

#include "common.h"
#include "kernels.h"
#include "wave_stream.h"

namespace moe {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kRows = 16;  // the M of the MFMA
constexpr int kRowsLds = 76 * 1024;  // x in LDS where it fits

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

// XL: the rows of x fit LDS.
template <int WT, bool XL, bool NARROW, int PC>
__global__ __launch_bounds__(kThreads) void linear_rows_kernel(LinearParams p) {
  using F = Form<WT>;
  constexpr int NF = F::kActBytes / 16, RC = kRowChunk<WT>, SL = (RC - 16) / 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];
  __shared__ __attribute__((aligned(16))) uint8_t s_ex[kWaves][kExchange];
  __shared__ __attribute__((aligned(16))) float s_red[kWaves][64][4];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = blockIdx.x % p.G, t0 = blockIdx.x / p.G * kRows, rows = min(kRows, p.n - t0);
  const int d = p.d, m = p.m;
  const int c_lo = (int)((long long)m * part / p.G), c_hi = (int)((long long)m * (part + 1) / p.G);
  const int cols = c_hi - c_lo, tiles = (cols + 15) / 16;
  int KS = kWaves;  // waves on one tile
  while (KS > 1 && tiles > kWaves / KS) KS >>= 1;
  const int mine = wave / KS, step = kWaves / KS, kp = wave % KS;  // this wave's tiles: mine, mine + step, ..
  const int C = (F::blocks(d) + kChunkBlocks - 1) / kChunkBlocks, k_lo = C * kp / KS, k_hi = C * (kp + 1) / KS;
  const int segs = tiles > mine ? (tiles - mine + step - 1) / step : 0;
  const size_t xb = WT == kMx4 ? (size_t)d / 2 : (size_t)d * 2;
  auto col = [&](int tile) { return c_lo + (int)((long long)cols * tile / max(tiles, 1)); };
  const int tok = min(r, rows - 1);
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  // (KS > 1: a wave has one tile at most, and its part k_lo .. k_hi - 1 of the chunks)
  stream<WT, PC, NARROW>(
      C, d, s_ex[wave],
      [&](int i, Segment &w) {
        if (i >= segs || k_lo == k_hi) return false;
        const int tile = mine + i * step, c = col(tile);
        rows_of_one<WT>(w, p.w, p.ws, c, col(tile + 1) - c, d);
        w.first = k_lo;
        w.count = k_hi - k_lo;
        return true;
      },
      [&] {  // the first weights are on their way
        if constexpr (XL) {
          for (int i = tid / SL; i < rows * C; i += kThreads / SL) {
            const int c = i / rows, t = i - c * rows;
            stage_row_chunk<WT>(s_x + i * RC, p.x + (t0 + t) * xb, c, d, tid % SL);
          }
          lds_barrier();
        }
      },
      [&](int, int &c, int &left) {
        c = k_lo;
        left = k_hi - k_lo;
      },
      [&](int, int c, int b, u32x4 (&a)[NF], uint32_t &as) {
        if constexpr (XL) {
          const uint8_t *px = s_x + (c * rows + tok) * RC + b * F::kActBytes;
#pragma unroll
          for (int q = 0; q < NF; ++q) a[q] = *(const u32x4 *)(px + q * 16);
        } else {
          load_block<WT>(p.x + (t0 + tok) * xb, c * kChunkBlocks + b, d, a);
        }
        if constexpr (WT == kMx4) as = p.xs[(size_t)(t0 + tok) * (d / 32) + min(c * kChunkBlocks + b, d / 32 - 1)];
      },
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

template <int WT, bool XL, bool NARROW, int PC>
hipError_t launch_rows(const LinearParams &p, hipStream_t st) {
  auto kern = linear_rows_kernel<WT, XL, NARROW, PC>;
  int lds = 0;
  if constexpr (XL) {
    lds = std::min(kRows, p.n) * ((Form<WT>::blocks(p.d) + kChunkBlocks - 1) / kChunkBlocks) * kRowChunk<WT>;
    // The LDS limit is raised once per device (a per-device kernel attribute).
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load(std::memory_order_acquire) & bit)) {
      err = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, kRowsLds);
      if (err != hipSuccess) return err;
      attr_done.fetch_or(bit, std::memory_order_release);
    }
  }
  kern<<<p.G * ((p.n + kRows - 1) / kRows), kThreads, lds, st>>>(p);
  return hipGetLastError();
}

template <int WT>
bool rows_fit(int n, int d) {
  return (long long)std::min(kRows, n) * ((Form<WT>::blocks(d) + kChunkBlocks - 1) / kChunkBlocks) * kRowChunk<WT> <=
         kRowsLds;
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
  if (a.x_mx4) {
    if (a.d < 128) return launch_rows<kMx4, true, true, 2>(p, st);
    return rows_fit<kMx4>(a.n, a.d) ? launch_rows<kMx4, true, false, 2>(p, st) : launch_rows<kMx4, false, false, 2>(p, st);
  }
  if (a.d < 128) return launch_rows<kMx, true, true, 2>(p, st);
  return rows_fit<kMx>(a.n, a.d) ? launch_rows<kMx, true, false, 2>(p, st) : launch_rows<kMx, false, false, 2>(p, st);
}

}  // namespace moe
