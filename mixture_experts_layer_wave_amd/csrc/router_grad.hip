// The router's gradient ("How Mixture of Experts Scales Model Parameters",
// sections "Routing", "Top-K" and "Load balancing").
//
// With p = softmax(z) over all E logits of a token, c_j its chosen experts,
// w_j their weights and dw_j the loss's gradient with respect to them:
//   renormalised (w = p_c / sum p_c, a softmax over the chosen logits)
//     dz_c += w_j (dw_j - D)                     D = sum_j w_j dw_j
//   raw (w = p_c)
//     dz_e  = p_e (sum_{j: c_j = e} dw_j - D)
//   and, for the auxiliary loss alpha E sum_i f_i P_i with f held constant,
//     dz_e += alpha E / n p_e (f_e - sum_i f_i p_i).
// Then  dx = dz W_g (+ the token's expert rows da[inv]),  dW_g = dz^T x,
// dbias = sum_t dz.
//
// dz is float32.  For bf16 x and W_g the two products run on the bf16 matrix
// cores with dz split into a bf16 value and the bf16 rest, two MFMAs in place
// of one: the operand keeps 16 of float32's 24 bits, so dx and dW_g are
// rounded only on their way out.  Both products are too narrow (E) to matter
// beside their traffic: dx reads n k + writes n rows of d, dW_g reads n.
//
// Measured: 8192 tokens of 4096, 8 experts top-2 67.0 us (269 MB, 53 us at a
// copy's rate); 4096 of 2880, 128 experts top-4 53.7 us (29 us: there W_g's
// tiles from L2 and the two halves of dz weigh as much as the rows, and the dz
// and sum launches take 10 us).  float32, the same two: 268 and 189 us (106 and
// 57: the gathered rows come four separate dwords at a time, after the product).
#include <atomic>

#include "common.h"
#include "gemm_f32.h"
#include "kernels.h"
#include "kmajor.h"
#include "route_dev.h"

namespace moe {
namespace {

// x = hi + lo + rest, the rest below 2^-16 of x.
__device__ __forceinline__ void split_bf16(float x, uint16_t &hi, uint16_t &lo) {
  hi = (uint16_t)f32_to_bf16_bits(x);
  const float r = x - bf16_bits_to_f32(hi);
  // (an infinite or NaN x keeps its value in hi; the rest would be NaN)
  lo = __builtin_isfinite(x) ? (uint16_t)f32_to_bf16_bits(r) : 0;
}

// Experts of dz's bf16 halves, padded with zeros.
__host__ __device__ constexpr int padded(int E) { return (E + 31) & ~31; }

// ---- dz: one group of G = topk_group(E) lanes per token -----------------------
// Lane l owns experts l, l + G, ... (PER of them at most) and, as k <= 32 and
// k <= E make k <= G, slot l: every load of a token is one of a few that do
// not wait for each other.  split (bf16 rows): dz's two halves too, hi
// [n][padded(E)], then lo, which the dW_g product reads once per column tile.
template <int PER>
__global__ __launch_bounds__(256) void router_dz_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ idx, const float *__restrict__ w,
    const float *__restrict__ dw, const float *__restrict__ f, float aux, int n, int E, int k, int renorm,
    float *__restrict__ dz, uint16_t *__restrict__ split) {
  const int G = topk_group(E);
  const int lane = threadIdx.x & 63, gl = lane & (G - 1), g0 = lane - gl;
  const int t = (blockIdx.x * 256 + threadIdx.x) / G;
  if ((blockIdx.x * 256 + (threadIdx.x & ~63)) / G >= n) return;  // whole wave idle
  const bool live = t < n;
  const int Ep = padded(E);
  const size_t row = live ? t : 0;
  float z[PER], fv[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = gl + i * G;
    z[i] = e < E ? logits[row * E + e] : -__builtin_inff();
    fv[i] = f && e < E ? f[e] : 0.f;
  }
  int c = -1;  // this lane's slot: expert, weight and the weight's gradient
  float wj = 0.f, dj = 0.f;
  if (gl < k) {
    c = idx[row * k + gl];
    wj = w[row * k + gl];
    dj = dw[row * k + gl];
  }
  const float D = group_sum((unsigned)c < (unsigned)E ? wj * dj : 0.f, G);
  // A token whose logits are all -inf has no expert and no gradient.  The
  // maximum cannot tell: fmaxf drops a NaN beside -inf, which lanes without an
  // expert hold too.
  float m = z[0];
  bool some = false;  // one of this lane's logits is not -inf (NaN counts)
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    m = fmaxf(m, z[i]);
    some |= !(z[i] == -__builtin_inff());
  }
  m = group_max(m, G);
  const bool any = (__ballot(some) >> g0 & (G == 64 ? ~0ull : (1ull << G) - 1)) != 0;
  float q[PER], s = 0.f, fp = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    q[i] = gl + i * G < E ? expf(z[i] - m) : 0.f;
    s += q[i];
    fp = fmaf(q[i], fv[i], fp);
  }
  s = group_sum(s, G);
  fp = group_sum(fp, G) / s;
  // Renormalised: sum over the expert's slots of w_j (dw_j - D); else of dw_j.
  float g[PER] = {};
  if (renorm) dj = wj * (dj - D);
  for (int j = 0; j < k; ++j) {
    const int cj = __shfl(c, g0 + j);
    const float vj = __shfl(dj, g0 + j);
#pragma unroll
    for (int i = 0; i < PER; ++i) g[i] += cj == gl + i * G ? vj : 0.f;
  }
  if (!live) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = gl + i * G;
    if (e >= E) {
      if (split && e < Ep) split[row * Ep + e] = split[(size_t)n * Ep + row * Ep + e] = 0;
      continue;
    }
    float v = 0.f;
    if (any) {
      const float p = q[i] / s;
      v = renorm ? g[i] : p * (g[i] - D);
      if (f) v = fmaf(aux * p, fv[i] - fp, v);
    }
    dz[row * E + e] = v;
    if (split) split_bf16(v, split[row * Ep + e], split[(size_t)n * Ep + row * Ep + e]);
  }
  // (the padding past PER G experts)
  if (split)
    for (int e = gl + PER * G; e < Ep; e += G) split[row * Ep + e] = split[(size_t)n * Ep + row * Ep + e] = 0;
}

// ---- dx, bf16 -------------------------------------------------------------------
// Block: 8 waves, 32 tokens x 512 columns (64 a wave), 32 experts a step; the
// products go through LDS as float32, after which a wave takes four whole
// row pieces of 1 KB.  Which rows those are is known from the start: their
// tokens are uniform (the pile rows come by scalar loads) and the gathered
// rows of the first two slots are already on their way during the products.
// (Waves that each keep to 32 x 128 and meet nowhere were slower: 89 against
// 72 us on 8 experts, each wave's chain of loads being its own.)
constexpr int kXT = 32, kXC = 512, kXE = 32, kXPitch = kXC + 4, kZPitch = kXE + 8, kXRows = kXT / 8;

__device__ __forceinline__ void router_dx_tile(
    const float *__restrict__ dz, const uint16_t *__restrict__ wg, const uint16_t *__restrict__ da,
    const int32_t *__restrict__ inv, int n, int d, int E, int k, uint16_t *__restrict__ dx, int tx, int ty,
    uint8_t *smem) {
  union Lds {
    struct {
      uint8_t w[kXE * kXC * 2];
      uint16_t hi[kXT * kZPitch], lo[kXT * kZPitch];
    } in;
    float out[kXT * kXPitch];
  };
  Lds &s = *(Lds *)smem;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = tx * kXT, c0 = ty * kXC;
  const int col = c0 + lane * 8, safe = col < d ? col : 0;
  const unsigned R = (unsigned)n * (unsigned)k;
  const int first = t0 + wave * kXRows;  // this wave's tokens first .. first + 3

  // The rows of slots j and j + 1 of the wave's tokens; slots past k and pairs
  // without a row read row 0 and give zeros.
  auto gather = [&](u32x4 (&q)[2][kXRows], int j) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < kXRows; ++i) {
        const int t = min(first + i, n - 1);
        const unsigned r = j + b < k ? (unsigned)inv[(size_t)t * k + j + b] : ~0u;
        const uint32_t keep = r < R ? ~0u : 0u;
        q[b][i] = *(const u32x4 *)(da + (size_t)(r & keep) * d + safe) & u32x4{keep, keep, keep, keep};
      }
  };
  // This thread's pieces of a step's rows of W_g and values of dz.
  u32x4 wr[kXE / 8];
  float zr[kXT * kXE / 512];
  auto fetch = [&](int e0) {
#pragma unroll
    for (int i = 0; i < kXE / 8; ++i) {
      const int e = e0 + wave + 8 * i;
      wr[i] = *(const u32x4 *)(wg + (size_t)min(e, E - 1) * d + safe);
      if (e >= E || col >= d) wr[i] = u32x4{};
    }
#pragma unroll
    for (int i = 0; i < kXT * kXE / 512; ++i) {
      const int e = e0 + (tid & 31), t = t0 + (tid >> 5) + 16 * i;
      zr[i] = dz[(size_t)min(t, n - 1) * E + min(e, E - 1)];
      if (e >= E || t >= n) zr[i] = 0.f;
    }
  };
  fetch(0);
  u32x4 q[2][kXRows] = {};
  if (da) gather(q, 0);

  f32x16 acc[2] = {};
  int b_lane[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) b_lane[j] = kmaj_lane<kXC>(wave * 64 + j * 32, lane);
  for (int e0 = 0; e0 < E; e0 += kXE) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kXE / 8; ++i) {
      const int e = wave + 8 * i;
      *(u32x4 *)(s.in.w + e * kXC * 2 + ((lane ^ kmaj_key<kXC>(e)) << 4)) = wr[i];
    }
#pragma unroll
    for (int i = 0; i < kXT * kXE / 512; ++i) {
      const int at = ((tid >> 5) + 16 * i) * kZPitch + (tid & 31);
      split_bf16(zr[i], s.in.hi[at], s.in.lo[at]);
    }
    __syncthreads();
    if (e0 + kXE < E) fetch(e0 + kXE);
#pragma unroll
    for (int kk = 0; kk < kXE / 16; ++kk) {
      if (e0 + kk * 16 >= E) break;
      const int at = (lane & 31) * kZPitch + kk * 16 + (lane >> 5) * 8;
      const bf16x8 hi = *(const bf16x8 *)(s.in.hi + at), lo = *(const bf16x8 *)(s.in.lo + at);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bf16x8 b = kmaj_frag<kXC>(s.in.w, b_lane[j], kk);
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, hi, acc[j], 0, 0, 0);
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, lo, acc[j], 0, 0, 0);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *(f32x4 *)(s.out + (lane & 31) * kXPitch + wave * 64 + j * 32 + g * 8 + (lane >> 5) * 4) =
          f32x4{acc[j][g * 4], acc[j][g * 4 + 1], acc[j][g * 4 + 2], acc[j][g * 4 + 3]};
  __syncthreads();
  f32x4 v[kXRows][2];
#pragma unroll
  for (int i = 0; i < kXRows; ++i) {
    const float *p = s.out + (wave * kXRows + i) * kXPitch + lane * 8;
    v[i][0] = *(const f32x4 *)p;
    v[i][1] = *(const f32x4 *)(p + 4);
  }
  // the slots' rows are added in slot order
  auto add = [&](const u32x4 (&q)[2][kXRows]) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < kXRows; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          v[i][x >> 1][(2 * x) & 3] += __uint_as_float(q[b][i][x] << 16);
          v[i][x >> 1][(2 * x + 1) & 3] += __uint_as_float(q[b][i][x] & 0xffff0000u);
        }
  };
  add(q);
  if (da)
    for (int j = 2; j < k; j += 2) {
      gather(q, j);
      add(q);
    }
  if (col >= d) return;
#pragma unroll
  for (int i = 0; i < kXRows; ++i)
    if (first + i < n)
      *(u32x4 *)(dx + (size_t)(first + i) * d + col) =
          u32x4{pack_bf16x2(v[i][0][0], v[i][0][1]), pack_bf16x2(v[i][0][2], v[i][0][3]),
                pack_bf16x2(v[i][1][0], v[i][1][1]), pack_bf16x2(v[i][1][2], v[i][1][3])};
}

// ---- dW_g, bf16 -----------------------------------------------------------------
// Block: 8 waves, EW experts x WC columns over a range of the tokens, 64 at a
// step, the next step's pieces of x and of dz's halves on their way.  A wave
// takes 32 columns and up to 64 experts (EW = 128: four waves each for the
// lower and the upper half).  The ranges' float32 planes part[s][E][d] are
// added in order by router_sum_kernel.  The blocks past the last column tile
// take the bias's sums bias_part[s][E] instead, from the float32 dz.
constexpr int kWT = 64;
template <int EW>
struct DwTile {
  static constexpr int TM = EW < 64 ? 1 : 2, NE = EW / (32 * TM), WC = 32 * (8 / NE);
  static constexpr int LDS = kWT * WC * 2 + 2 * kWT * EW * 2;
};

template <int EW>
__device__ __forceinline__ void router_dw_tile(const float *__restrict__ dz, const uint16_t *__restrict__ split,
                                               const uint16_t *__restrict__ x, int n, int d, int E, int range,
                                               float *__restrict__ part, float *__restrict__ bias_part, int bx,
                                               int by, int bz, uint8_t *smem) {
  using T = DwTile<EW>;
  constexpr int TM = T::TM, WC = T::WC, NT = 512;
  constexpr int ZC = EW / 8, ZN = kWT * ZC / NT > 0 ? kWT * ZC / NT : 1;  // 16-B pieces of a dz row; per thread
  constexpr int XC = WC / 8, XN = kWT * XC / NT;
  uint8_t *s_x = smem, *s_z = smem + kWT * WC * 2;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c0 = bx * WC, e0 = bz * EW, Ep = padded(E);
  const int tb = by * range, te = min(n, tb + range);
  if (c0 >= d) {
    constexpr int ZR = NT / EW;
    float *s_b = (float *)smem;
    const int e = e0 + tid % EW;
    float v = 0.f;
    if (e < E)
#pragma unroll 16
      for (int t = tb + tid / EW; t < te; t += ZR) v += dz[(size_t)t * E + e];
    s_b[tid] = v;
    __syncthreads();
    if (tid < EW && e < E) {
      for (int i = 1; i < ZR; ++i) v += s_b[i * EW + tid];
      bias_part[(size_t)by * E + e] = v;
    }
    return;
  }
  const int xcol = c0 + tid % XC * 8, zt = tid / ZC, ze = e0 + tid % ZC * 8;
  const bool zin = ZC * kWT >= NT || zt < kWT;  // (EW = 32: half of the threads hold pieces of dz)
  u32x4 xr[XN], zr[2][ZN];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int t = t0 + tid / XC + (NT / XC) * i;
      xr[i] = *(const u32x4 *)(x + (size_t)min(t, te - 1) * d + (xcol < d ? xcol : 0));
      if (t >= te || xcol >= d) xr[i] = u32x4{};
    }
    if (zin)
#pragma unroll
      for (int i = 0; i < ZN; ++i) {
        const int t = t0 + zt + (NT / ZC) * i;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          zr[h][i] = *(const u32x4 *)(split + ((size_t)h * n + min(t, te - 1)) * Ep + (ze < Ep ? ze : 0));
          if (t >= te || ze >= Ep) zr[h][i] = u32x4{};
        }
      }
  };
  const int half = wave % T::NE, cg = wave / T::NE;  // this wave's experts and columns
  f32x16 acc[TM] = {};
  int a_lane[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) a_lane[i] = kmaj_lane<EW>(half * 64 + i * 32, lane);
  const int b_lane = kmaj_lane<WC>(cg * 32, lane);
  fetch(tb);
  for (int t0 = tb; t0 < te; t0 += kWT) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < XN; ++i) {
      const int t = tid / XC + (NT / XC) * i;
      *(u32x4 *)(s_x + t * WC * 2 + (((tid % XC) ^ kmaj_key<WC>(t)) << 4)) = xr[i];
    }
    if (zin)
#pragma unroll
      for (int i = 0; i < ZN; ++i) {
        const int t = zt + (NT / ZC) * i;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *(u32x4 *)(s_z + (h * kWT + t) * EW * 2 + (((tid % ZC) ^ kmaj_key<EW>(t)) << 4)) = zr[h][i];
      }
    __syncthreads();
    if (t0 + kWT < te) fetch(t0 + kWT);
#pragma unroll
    for (int kk = 0; kk < kWT / 16; ++kk) {
      const bf16x8 b = kmaj_frag<WC>(s_x, b_lane, kk);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              b, kmaj_frag<EW>(s_z + h * kWT * EW * 2, a_lane[i], kk), acc[i], 0, 0, 0);
    }
  }
  float *out = part + (size_t)by * E * d;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int e = e0 + half * 64 + i * 32 + (lane & 31);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int col = c0 + cg * 32 + g * 8 + (lane >> 5) * 4;
      if (e < E && col < d)
        *(f32x4 *)(out + (size_t)e * d + col) =
            f32x4{acc[i][g * 4], acc[i][g * 4 + 1], acc[i][g * 4 + 2], acc[i][g * 4 + 3]};
    }
  }
}

// Both products in one grid: they read different things, and the few long
// blocks of dW_g start first and end under dx's many short ones.
struct BothParams {
  const float *dz;
  const uint16_t *split, *x, *wg, *da;
  const int32_t *inv;
  uint16_t *dx;
  float *part, *bias_part;
  int n, d, E, k, range;
  int dw_cols, dw_S, dw_blocks;  // column tiles (with the bias's), token ranges, all blocks
  int dx_rows;                   // token tiles
};

template <int EW>
__global__ __launch_bounds__(512, 4) void router_both_kernel(BothParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int b = blockIdx.x;
  if (b < p.dw_blocks) {
    const int bx = b % p.dw_cols, q = b / p.dw_cols;
    router_dw_tile<EW>(p.dz, p.split, p.x, p.n, p.d, p.E, p.range, p.part, p.bias_part, bx, q % p.dw_S,
                       q / p.dw_S, smem);
  } else {
    b -= p.dw_blocks;
    router_dx_tile(p.dz, p.wg, p.da, p.inv, p.n, p.d, p.E, p.k, p.dx, b % p.dx_rows, b / p.dx_rows, smem);
  }
}

// dW_g = the sum of S planes, in order; dbias likewise (threads past E d).
template <bool BF>
__global__ __launch_bounds__(256) void router_sum_kernel(const float *__restrict__ part,
                                                         const float *__restrict__ bias_part, int S, int E,
                                                         int d, void *__restrict__ dwg,
                                                         float *__restrict__ dbias) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, ed = (size_t)E * d;
  if (i < ed) {
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < S; ++s) v += part[(size_t)s * ed + i];
    if constexpr (BF)
      ((uint16_t *)dwg)[i] = (uint16_t)f32_to_bf16_bits(v);
    else
      ((float *)dwg)[i] = v;
  } else if (i < ed + E && dbias) {
    float v = 0.f;
    for (int s = 0; s < S; ++s) v += bias_part[(size_t)s * E + (i - ed)];
    dbias[i - ed] = v;
  }
}

// ---- float32 ----------------------------------------------------------------------
using namespace f32gemm;
// (the whole pass, E = 8, 1024 wide, 4096 tokens: 35.3 us with dx in One, 41.9
// with it in Two; E = 128, 2880 wide, 8000 tokens: 348 us with dW_g in Two, 363
// with it in One)
using One = Groups<1>;
using Two = Groups<2>;

__global__ __launch_bounds__(One::THREADS, 4) void router_dx_f32_kernel(
    const float *__restrict__ dz, const float *__restrict__ wg, const float *__restrict__ da,
    const int32_t *__restrict__ inv, int n, int d, int E, int k, float *__restrict__ dx) {
  __shared__ __attribute__((aligned(16))) float smem[One::SMEM];
  const int t0 = blockIdx.x * kT, c0 = blockIdx.y * kT;
  const auto rz = gemm::rsrc(dz + (size_t)t0 * E, (uint32_t)min(kT, n - t0) * (uint32_t)E * 4u);
  const auto rw = gemm::rsrc(wg, (uint32_t)E * (uint32_t)d * 4u);
  f32x4 acc[One::LINES];
  f32x16 sum = {};
  product<1, false, true>(
      sum, smem, E,
      [&](int, int e, int t) { return Piece{rz, ((uint32_t)t * E + e) * 4u, t0 + t < n ? 4 : 0}; },
      [&](int, int e, int c) { return Piece{rw, ((uint32_t)e * d + c0 + c) * 4u, d - c0 - c}; });
  lines<1>(sum, smem, acc);
  const unsigned R = (unsigned)n * (unsigned)k;
  const int c = c0 + One::col();
#pragma unroll
  for (int i = 0; i < One::LINES; ++i) {
    const int t = t0 + One::row(i);
    if (t >= n) continue;
    if (da)
      for (int j = 0; j < k; ++j) {
        const int pr = inv[(size_t)t * k + j];
        if ((unsigned)pr >= R) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + q < d) acc[i][q] += da[(size_t)pr * d + c + q];
      }
    store4(dx + (size_t)t * d + c, d - c, acc[i]);
  }
}

__global__ __launch_bounds__(Two::THREADS, 4) void router_dw_f32_kernel(const float *__restrict__ dz,
                                                                 const float *__restrict__ x, int n, int d,
                                                                 int E, int range, float *__restrict__ part,
                                                                 float *__restrict__ bias_part) {
  __shared__ __attribute__((aligned(16))) float smem[Two::SMEM];
  __shared__ float s_b[Two::THREADS];
  const int c0 = blockIdx.x * kT, e0 = blockIdx.z * kT;
  const int tb = blockIdx.y * range, te = min(n, tb + range);
  const auto rz = gemm::rsrc(dz + (size_t)tb * E, (uint32_t)(te - tb) * (uint32_t)E * 4u);
  const auto rx = gemm::rsrc(x + (size_t)tb * d, (uint32_t)(te - tb) * (uint32_t)d * 4u);
  f32x4 acc[Two::LINES];
  f32x16 sum = {};
  product<2, true, true>(
      sum, smem, te - tb,
      [&](int, int t, int e) { return Piece{rz, ((uint32_t)t * E + e0 + e) * 4u, E - e0 - e}; },
      [&](int, int t, int c) { return Piece{rx, ((uint32_t)t * d + c0 + c) * 4u, d - c0 - c}; });
  lines<2>(sum, smem, acc);
  const int c = c0 + Two::col();
#pragma unroll
  for (int i = 0; i < Two::LINES; ++i) {
    const int e = e0 + Two::row(i);
    if (e < E) store4(part + ((size_t)blockIdx.y * E + e) * d + c, d - c, acc[i]);
  }
  if (blockIdx.x == 0) {
    constexpr int W = Two::THREADS / 64;
    const int be = e0 + (threadIdx.x & 63), s = threadIdx.x >> 6;
    float v = 0.f;
    if (be < E)
      for (int t = tb + s; t < te; t += W) v += dz[(size_t)t * E + be];
    s_b[threadIdx.x] = v;
    __syncthreads();
    if (s == 0 && be < E) {
      for (int i = 1; i < W; ++i) v += s_b[i * 64 + threadIdx.x];
      bias_part[(size_t)blockIdx.y * E + be] = v;
    }
  }
}

// Token ranges of the dW_g product: blocks for three CUs of four beside dx's
// (128 experts, 2880 wide, 4096 tokens: 54.2 us; for every CU, whose planes
// cost more, 60, for every second 55.4, for every fourth 60), but planes of at
// most the bytes of x (S E 4 <= n 2), and whole steps; a range's rows
// of x and dz stay under 2^30 bytes (32-bit buffer offsets, float32).
struct Ranges {
  int S, range;
};
Ranges dw_ranges(int n, int d, int E) {
  const int cols = E <= 64 ? 256 : 128, tiles = ((d + cols - 1) / cols) * ((E + 127) / 128);
  int S = (192 + tiles - 1) / tiles;
  const int most = n / (2 * E) > 1 ? n / (2 * E) : 1;
  if (S > most) S = most;
  const long long bytes = (long long)n * (d > E ? d : E) * 4;
  if (S < (bytes >> 29)) S = (int)(bytes >> 29);
  int range = (n + S - 1) / S;
  range = (range + kWT - 1) / kWT * kWT;
  return {(n + range - 1) / range, range};
}

template <int EW>
hipError_t launch_both(const RouterGradArgs &a, const uint16_t *split, const Ranges &q, float *part,
                       float *bias_part, hipStream_t st) {
  using T = DwTile<EW>;
  constexpr int dx_lds = kXT * kXPitch * 4, lds = dx_lds > T::LDS ? dx_lds : T::LDS;
  static_assert(dx_lds >= kXE * kXC * 2 + 2 * kXT * kZPitch * 2, "both uses of dx's LDS fit");
  static std::atomic<uint64_t> allowed{0};  // devices on which LDS above 64 KB is allowed
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    err = hipFuncSetAttribute((const void *)router_both_kernel<EW>, hipFuncAttributeMaxDynamicSharedMemorySize,
                              lds);
    if (err != hipSuccess) return err;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  BothParams p{};
  p.dz = a.dlogits;
  p.split = split;
  p.x = (const uint16_t *)a.x;
  p.wg = (const uint16_t *)a.wg;
  p.da = (const uint16_t *)a.da;
  p.inv = a.inv;
  p.dx = (uint16_t *)a.dx;
  p.part = part;
  p.bias_part = bias_part;
  p.n = a.n;
  p.d = a.d;
  p.E = a.E;
  p.k = a.k;
  p.range = q.range;
  p.dw_cols = (a.d + T::WC - 1) / T::WC + 1;
  p.dw_S = q.S;
  p.dw_blocks = p.dw_cols * q.S * ((a.E + EW - 1) / EW);
  p.dx_rows = (a.n + kXT - 1) / kXT;
  router_both_kernel<EW><<<p.dw_blocks + p.dx_rows * ((a.d + kXC - 1) / kXC), 512, lds, st>>>(p);
  return hipGetLastError();
}

}  // namespace

namespace {
size_t plane_bytes(int n, int d, int E) {
  return ((size_t)dw_ranges(n, d, E).S * ((size_t)E * d + E) * sizeof(float) + 255) / 256 * 256;
}
}  // namespace

size_t router_grad_bytes(int n, int d, int E) {
  // the planes, then (bf16 rows) dz's two halves
  return plane_bytes(n, d, E) + (size_t)2 * n * padded(E) * sizeof(uint16_t);
}

hipError_t launch_router_grad(const RouterGradArgs &a, hipStream_t st) {
  uint16_t *split = a.bf16 ? (uint16_t *)((char *)a.ws + plane_bytes(a.n, a.d, a.E)) : nullptr;
  const int per_block = 256 / topk_group(a.E);
  // (E <= 64: one expert a lane, E <= 128: two)
  auto dz = a.E <= 64 ? router_dz_kernel<1> : a.E <= 128 ? router_dz_kernel<2> : router_dz_kernel<16>;
  dz<<<(a.n + per_block - 1) / per_block, 256, 0, st>>>(
      a.logits, a.idx, a.topk_w, a.dtopk_w, a.f, a.alpha * (float)a.E / (float)a.n, a.n, a.E, a.k,
      a.renorm ? 1 : 0, a.dlogits, split);
  const Ranges q = dw_ranges(a.n, a.d, a.E);
  float *part = (float *)a.ws, *bias_part = part + (size_t)q.S * a.E * a.d;
  if (a.bf16) {
    // experts of a dW_g block: as many 32-wide groups as there are, up to 128
    const hipError_t e = a.E <= 32   ? launch_both<32>(a, split, q, part, bias_part, st)
                         : a.E <= 64 ? launch_both<64>(a, split, q, part, bias_part, st)
                                     : launch_both<128>(a, split, q, part, bias_part, st);
    if (e != hipSuccess) return e;
  } else {
    router_dx_f32_kernel<<<dim3((a.n + kT - 1) / kT, (a.d + kT - 1) / kT), One::THREADS, 0, st>>>(
        a.dlogits, (const float *)a.wg, (const float *)a.da, a.inv, a.n, a.d, a.E, a.k, (float *)a.dx);
    router_dw_f32_kernel<<<dim3((a.d + kT - 1) / kT, q.S, (a.E + kT - 1) / kT), Two::THREADS, 0, st>>>(
        a.dlogits, (const float *)a.x, a.n, a.d, a.E, q.range, part, bias_part);
  }
  const size_t outs = (size_t)a.E * a.d + a.E;
  auto sum = a.bf16 ? router_sum_kernel<true> : router_sum_kernel<false>;
  sum<<<(unsigned)((outs + 255) / 256), 256, 0, st>>>(part, bias_part, q.S, a.E, a.d, a.dwg, a.dbias);
  return hipGetLastError();
}

}  // namespace moe
