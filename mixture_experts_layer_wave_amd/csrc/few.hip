// The whole layer for at most 16 tokens in two kernels (moe_forward_few).
//
//   z = x Wg^T + b, top-k and weights as in the router,
//   y[t] = sum_j w_tj (silu(x_t W1_e) (x_t W3_e)) W2_e,  e = idx[t][j]
//
// With a few tokens the layer is bound by reading the chosen experts' weights
// once, and by the launches, barriers and round trips between the steps that
// depend on each other.  few_router_kernel takes the logits (one workgroup per
// expert).  few_layer_kernel does the rest: every workgroup takes the top-k of
// all tokens by itself (cheaper than a launch), then its part of the up
// projections, and once all parts are done, its part of the outputs.
//
// The parts are tickets from one counter: 0 .. G-1 are the up parts, G .. 2G-1
// the output parts.  A workgroup takes a ticket, does it and takes the next; an
// output part waits until all G up parts are done.  A ticket is only ever taken
// by a running workgroup, up parts never wait, and a workgroup does its tickets
// in order, so when an output part waits, every up part is done or in the hands
// of a running workgroup that does not wait: the wait ends however few of the
// workgroups are resident and whatever else runs on the GPU (two calls at once
// among it).  What a part computes depends on its ticket alone, so results do
// not depend on who takes it.
//
// A wave streams weight rows straight into registers: one 16-byte load per lane
// and step, 16 rows by 4 blocks (of 32 MXFP4, 8 bf16 or 4 float32 elements) to a
// step, PF steps in flight.  The products run on 16x16 MFMAs with the tokens as
// rows (M) and the 16 weight rows as columns.  Up: a tile is 8 rows of W1 and the
// same 8 of W3, over all of K, so gate and value meet in one wave; every wave of
// the grid takes an equal run of hidden columns.  Output: a workgroup takes an
// equal run of output columns over all chosen experts, its waves equal runs of
// (expert, K step); each wave adds an expert's product to its tokens' sums where
// the expert's K range ends, and the waves' sums meet in LDS in a fixed order.
// The hidden is multiplied by its combine weight before its one rounding, so
// that the output needs no pass of its own.
#include <algorithm>
#include <atomic>

#include "common.h"
#include "kernels.h"
#include "route_dev.h"
#include "wave_stream.h"

namespace moe {
namespace {

constexpr int kT = kFewMaxTokens;  // 16: the M of the MFMA
constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kFewLds = 160 * 1024;
constexpr int kMaxXBytes = 112 * 1024;  // the tokens' rows in LDS, else read through the ring
// Tries of a waiting output part (each at least a microsecond): seconds, where a
// call takes microseconds.  Past it the part writes NaN.
constexpr int kMaxTries = 1 << 23;

struct FewLds {
  int x, pitch;     // tokens' rows (pitch bytes each); the output part's staging lies over it
  int red, idx, w, mask, aidx, act, pile, misc, total;
};

struct FewParams {
  const void *x;
  const float *logits;
  const uint8_t *w1, *w3, *w2, *s1, *s3, *s2;
  const int32_t *slot;
  int n_slots;
  int n, d, E, k, f;
  int renorm, out_bf16;
  void *h;         // [n k][f], bf16 or f32
  void *y;
  int32_t *idx;    // [n][k] or NULL
  float *w;
  int *count;      // ticket counter, parts done
  int G;
  FewLds lds;
};

template <int WT, int PER, int ARU, int ARD, int PFU, int PFD>
__global__ __launch_bounds__(kThreads) void few_layer_kernel(FewParams p) {
  using F = Form<WT>;
  constexpr int NF = F::kActBytes / 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const FewLds &L = p.lds;
  int *s_idx = (int *)(smem + L.idx), *s_mask = (int *)(smem + L.mask), *s_act = (int *)(smem + L.act);
  float *s_w = (float *)(smem + L.w), *s_red = (float *)(smem + L.red);
  uint16_t *s_aidx = (uint16_t *)(smem + L.aidx), *s_pile = (uint16_t *)(smem + L.pile);
  int *s_misc = (int *)(smem + L.misc);  // active experts, ticket, whether the wait ended
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = p.n, k = p.k, E = p.E, d = p.d, f = p.f, R = n * k, G = p.G;
  const size_t xrow = (size_t)d * (F::f32 ? 4 : 2), hrow = (size_t)f * (F::f32 ? 4 : 2);

  auto take = [&]() {
    return __hip_atomic_fetch_add(p.count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  int first = 0;
  if (tid == 0) first = take();
  if constexpr (ARU == 0)  // the tokens' rows
    for (int i = tid; i < n * (d / 8); i += kThreads) {
      const int t = i / (d / 8), c = i % (d / 8);
      *(u32x4 *)(smem + L.x + t * L.pitch + c * 16) = *(const u32x4 *)((const uint8_t *)p.x + t * xrow + c * 16);
    }
  for (int e = tid; e < E; e += kThreads) s_mask[e] = 0;
  const int TG = topk_group(E);
  for (int t0 = 0; t0 < n; t0 += kThreads / TG)
    topk_token_t<PER>(p.logits, 1, 0, t0 + tid / TG, n, E, k, p.renorm, s_idx, s_w, nullptr, nullptr);
  if (tid == 0) s_misc[1] = first;
  __syncthreads();
  // ---- who takes which expert ------------------------------------------------
  for (int q = tid; q < R; q += kThreads) atomicOr(&s_mask[s_idx[q]], 1 << (q / k));
  __syncthreads();
  if (wave == 0) {
    int a = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane;
      const bool on = e < E && s_mask[e] != 0;
      const uint64_t bits = __ballot(on);
      if (on) {
        const int at = a + __popcll(bits & ((1ull << lane) - 1));
        s_aidx[e] = (uint16_t)at;
        s_act[at] = e;
      }
      a += __popcll(bits);
    }
    if (lane == 0) s_misc[0] = a;
  }
  __syncthreads();
  for (int q = tid; q < R; q += kThreads) {
    const int e = s_idx[q], t = q / k;
    s_pile[s_aidx[e] * kT + __popc(s_mask[e] & ((1 << t) - 1))] = (uint16_t)q;
  }
  __syncthreads();
  const int A = s_misc[0];
  int ticket = s_misc[1];

  if (ticket == 0 && p.idx)
    for (int q = tid; q < R; q += kThreads) p.idx[q] = s_idx[q];
  if (ticket == 0 && p.w)
    for (int q = tid; q < R; q += kThreads) p.w[q] = s_w[q];

  // (a block's tickets ascend, so no up part follows an output part, whose
  // staging overwrites the tokens' rows)
  while (ticket < 2 * G) {
    if (ticket < G) {
      // ---- up: hidden columns [u0, u1) of the chosen experts' A f -----------
      const long long U = (long long)A * f, NW = (long long)G * kWaves, wv = (long long)ticket * kWaves + wave;
      const int u0 = (int)(U * wv / NW), u1 = (int)(U * (wv + 1) / NW);
      // Tiles: runs of at most 8 columns of one expert.
      auto tile_at = [&](int u, int &a, int &c, int &cnt) {
        a = u / f;
        c = u - a * f;
        cnt = min(8, min(u1 - u, f - c));
      };
      int tiles = 0;
      for (int u = u0; u < u1;) {
        int a, c, cnt;
        tile_at(u, a, c, cnt);
        u += cnt;
        ++tiles;
      }
      const int S = (F::blocks(d) + 3) / 4;
      int lu = u0, eu = u0;  // first column of the tile to load, to finish
      const size_t rb = F::row_bytes(d);
      stream<WT, PFU, ARU>(
          tiles * S, S, 0, d, smem + L.x + wave * 1024 * (ARU ? ARU : 1),
          [&](int, const uint8_t *&row, const uint8_t *&srow, const uint8_t *(&arow)[ARU ? ARU : 1],
              const uint8_t *&) {
            int a, c, cnt;
            tile_at(lu, a, c, cnt);
            lu += cnt;
            const int e = s_act[a];
            const size_t wr = (size_t)phys_slot(p.slot, p.n_slots, e) * f + c + min(r & 7, cnt - 1);
            row = (r < 8 ? p.w1 : p.w3) + wr * rb;
            if constexpr (WT == kMx) srow = (r < 8 ? p.s1 : p.s3) + wr * (d / 32);
            if constexpr (ARU > 0)
#pragma unroll
              for (int i = 0; i < ARU; ++i)
                arow[i] = (const uint8_t *)p.x + min(WT == kMx ? g + 4 * i : r, n - 1) * xrow;
          },
          [&](int, int b, u32x4 (&a)[NF]) {
            const uint8_t *px = smem + L.x + min(r, n - 1) * L.pitch + b * F::kActBytes;
#pragma unroll
            for (int q = 0; q < NF; ++q) a[q] = *(const u32x4 *)(px + q * 16);
          },
          [&](int) { return min(r, n - 1); },
          [&](int, f32x4 v) {
            int a, c, cnt;
            tile_at(eu, a, c, cnt);
            eu += cnt;
            const int mask = s_mask[s_act[a]];
            // lane (r, g): token 4 g + i, column c + r (r < 8: gate, r + 8: value)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = __shfl_xor(v[i], 8, 64);
              const int t = 4 * g + i;
              if (r < cnt && r < 8 && ((mask >> t) & 1)) {
                const int q = s_pile[a * kT + __popc(mask & ((1 << t) - 1))];
                const float hv = s_w[q] * (silu(v[i]) * u);
                if constexpr (F::f32)
                  __hip_atomic_store((float *)p.h + (size_t)q * f + c + r, hv, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
                else
                  __hip_atomic_store((uint16_t *)p.h + (size_t)q * f + c + r, (uint16_t)f32_to_bf16_bits(hv),
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
              }
            }
          });
      __syncthreads();  // the block's hidden is on its way out
      if (tid == 0) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
        __hip_atomic_fetch_add(p.count + 1, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_misc[1] = take();
      }
      __syncthreads();
      ticket = s_misc[1];
      continue;
    }
    // ---- output columns [c_lo, c_hi) ------------------------------------------
    __syncthreads();  // everyone has read s_misc
    if (tid == 0) {
      int tries = 0;
      while (__hip_atomic_load(p.count + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < G && ++tries < kMaxTries)
        __builtin_amdgcn_s_sleep(1);
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      s_misc[2] = tries < kMaxTries;
      s_misc[1] = take();
    }
    __syncthreads();
    const bool whole = s_misc[2];
    const int part = ticket - G;
    ticket = s_misc[1];
    const int c_lo = (int)((long long)d * part / G), c_hi = (int)((long long)d * (part + 1) / G);
    const int S = (F::blocks(f) + 3) / 4;
    const long long steps = (long long)A * S;
    const int i0 = (int)(steps * wave / kWaves), i1 = (int)(steps * (wave + 1) / kWaves);
    const size_t rb = F::row_bytes(f);
    for (int c0 = c_lo; c0 < c_hi; c0 += 16) {
      const int cnt = min(16, c_hi - c0), a0 = i0 / S;
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      stream<WT, PFD, ARD>(
          i1 - i0, S, i0 - a0 * S, f, smem + L.x + wave * 1024 * ARD,
          [&](int i, const uint8_t *&row, const uint8_t *&srow, const uint8_t *(&arow)[ARD], const uint8_t *&) {
            const int a = a0 + i, e = s_act[a], mask = s_mask[e], m = __popc(mask);
            const size_t wr = (size_t)phys_slot(p.slot, p.n_slots, e) * d + c0 + min(r, cnt - 1);
            row = p.w2 + wr * rb;
            if constexpr (WT == kMx) srow = p.s2 + wr * (f / 32);
            const int own = min(__popc(mask & ((1 << r) - 1)), m - 1);
#pragma unroll
            for (int j = 0; j < ARD; ++j)
              arow[j] = (const uint8_t *)p.h + s_pile[a * kT + (WT == kMx ? min(g + 4 * j, m - 1) : own)] * hrow;
          },
          [&](int, int, u32x4 (&)[NF]) {},
          [&](int i) {
            const int mask = s_mask[s_act[a0 + i]];
            return min(__popc(mask & ((1 << r) - 1)), __popc(mask) - 1);
          },
          [&](int i, f32x4 v) {  // only the expert's own tokens: 0 times a NaN weight is NaN
            const int mask = s_mask[s_act[a0 + i]];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if ((mask >> (4 * g + q)) & 1) sum[q] += v[q];
          });
      *(f32x4 *)(s_red + (wave * 64 + lane) * 4) = sum;
      __syncthreads();
      if (wave < 4) {  // wave i: token 4 g + i
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < kWaves; ++j) v += s_red[(j * 64 + lane) * 4 + wave];
        if (!whole) v = __builtin_nanf("");
        const int t = 4 * g + wave;
        if (t < n && r < cnt) {
          const size_t at = (size_t)t * d + c0 + r;
          if (p.out_bf16)
            ((uint16_t *)p.y)[at] = (uint16_t)f32_to_bf16_bits(v);
          else
            ((float *)p.y)[at] = v;
        }
      }
      __syncthreads();
    }
  }
}

// logits[t][e] = x_t . wg_e + bias_e, one workgroup per expert; the first also
// clears the next kernel's counters.  Rows of bf16 in 16-byte pieces.
template <bool BF>
__global__ __launch_bounds__(256) void few_router_kernel(const void *__restrict__ x, const void *__restrict__ wg,
                                                         const float *__restrict__ bias, int n, int d, int E,
                                                         float *__restrict__ logits, int *__restrict__ count) {
  __shared__ float s_sum[4][kT];
  const int e = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (e == 0 && tid < 2) count[tid] = 0;
  float acc[kT] = {};
  if constexpr (BF) {
    const u32x4 *wr = (const u32x4 *)((const uint16_t *)wg + (size_t)e * d);
    for (int c = tid; c < d / 8; c += 256) {
      const u32x4 w = wr[c];
#pragma unroll
      for (int t = 0; t < kT; ++t)
        if (t < n) {
          const u32x4 v = ((const u32x4 *)((const uint16_t *)x + (size_t)t * d))[c];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[t] = fmaf(__uint_as_float(w[i] << 16), __uint_as_float(v[i] << 16), acc[t]);
            acc[t] = fmaf(__uint_as_float(w[i] & 0xffff0000u), __uint_as_float(v[i] & 0xffff0000u), acc[t]);
          }
        }
    }
  } else {
    const float *wr = (const float *)wg + (size_t)e * d;
    for (int c = tid; c < d; c += 256) {
      const float w = wr[c];
#pragma unroll
      for (int t = 0; t < kT; ++t)
        if (t < n) acc[t] = fmaf(w, ((const float *)x)[(size_t)t * d + c], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kT; ++t)
    if (t < n) {
      const float v = group_sum(acc[t], 64);
      if (lane == 0) s_sum[wave][t] = v;
    }
  __syncthreads();
  if (tid < n) {
    const float v = (s_sum[0][tid] + s_sum[1][tid]) + (s_sum[2][tid] + s_sum[3][tid]);
    logits[(size_t)tid * E + e] = bias ? v + bias[e] : v;
  }
}

int up16(int v) { return (v + 15) / 16 * 16; }

struct FewPlan {
  size_t logits, count, h, total;  // workspace
};

FewPlan plan_of(int n, int E, int k, int d_ff, bool f32) {
  FewPlan P{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  P.logits = 0;
  P.count = up((size_t)n * E * 4);
  P.h = P.count + 256;
  P.total = P.h + up((size_t)n * k * d_ff * (f32 ? 4 : 2));
  return P;
}

template <int WT, int PER, int ARU, int ARD, int PFU, int PFD>
hipError_t launch(FewParams &p, hipStream_t st) {
  auto kern = few_layer_kernel<WT, PER, ARU, ARD, PFU, PFD>;
  FewLds &L = p.lds;
  const int R = p.n * p.k, A = std::min(R, p.E);
  int o = 0;
  auto put = [&](int bytes) {
    const int at = o;
    o += up16(bytes);
    return at;
  };
  // an odd number of 16-byte pieces a row: the 16 rows' reads meet different banks
  L.pitch = WT >= kF4 ? 0 : ((p.d / 8) | 1) * 16;
  const int stage = WT == kMx ? kWaves * 1024 * std::max(ARU, ARD) : 0;
  L.x = put(std::max(ARU == 0 ? p.n * L.pitch : 0, stage));
  L.red = put(kWaves * 64 * 16);
  L.idx = put(R * 4);
  L.w = put(R * 4);
  L.mask = put(p.E * 4);
  L.aidx = put(p.E * 2);
  L.act = put(A * 4);
  L.pile = put(A * kT * 2);
  L.misc = put(16);
  L.total = o;
  if (L.total > kFewLds) return hipErrorInvalidValue;
  if (L.total > 64 * 1024) {
    // The LDS limit is raised once per device (a per-device kernel attribute).
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load(std::memory_order_acquire) & bit)) {
      err = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, kFewLds);
      if (err != hipSuccess) return err;
      attr_done.fetch_or(bit, std::memory_order_release);
    }
  }
  kern<<<p.G, kThreads, L.total, st>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t forward_few_bytes(int n, int E, int k, int d_ff, bool f32) { return plan_of(n, E, k, d_ff, f32).total; }

hipError_t launch_forward_few(const FewArgs &a, hipStream_t st) {
  const bool f32 = a.w_dtype == 0;
  const FewPlan P = plan_of(a.n, a.E, a.k, a.d_ff, f32);
  char *base = (char *)a.ws;
  FewParams p{};
  p.x = a.x;
  p.logits = (float *)(base + P.logits);
  p.count = (int *)(base + P.count);
  p.h = base + P.h;
  p.w1 = (const uint8_t *)a.w1;
  p.w3 = (const uint8_t *)a.w3;
  p.w2 = (const uint8_t *)a.w2;
  p.s1 = a.s1;
  p.s3 = a.s3;
  p.s2 = a.s2;
  p.slot = a.slot;
  p.n_slots = a.n_slots;
  p.n = a.n;
  p.d = a.d;
  p.E = a.E;
  p.k = a.k;
  p.f = a.d_ff;
  p.renorm = a.renorm;
  p.out_bf16 = a.out_bf16;
  p.y = a.y;
  p.idx = a.idx;
  p.w = a.w;
  p.G = cu_count();
  float *logits = (float *)(base + P.logits);
  if (f32)
    few_router_kernel<false><<<a.E, 256, 0, st>>>(a.x, a.wg, a.bias, a.n, a.d, a.E, logits, p.count);
  else
    few_router_kernel<true><<<a.E, 256, 0, st>>>(a.x, a.wg, a.bias, a.n, a.d, a.E, logits, p.count);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool few_experts = topk_per(a.E) == 2, in_lds = a.n * (size_t)(a.d / 8 + 1) * 16 <= kMaxXBytes;
  if (a.w_dtype == 2) {
    if (!in_lds) return launch<kMx, 16, 4, 4, 6, 6>(p, st);
    if (a.n <= 4) return few_experts ? launch<kMx, 2, 0, 1, 12, 12>(p, st) : launch<kMx, 16, 0, 1, 12, 12>(p, st);
    if (a.n <= 8) return few_experts ? launch<kMx, 2, 0, 2, 12, 8>(p, st) : launch<kMx, 16, 0, 2, 12, 8>(p, st);
    return few_experts ? launch<kMx, 2, 0, 4, 12, 6>(p, st) : launch<kMx, 16, 0, 4, 12, 6>(p, st);
  }
  if (a.w_dtype == 1) {
    if (!in_lds) return launch<kBf, 16, 1, 1, 12, 12>(p, st);
    return few_experts ? launch<kBf, 2, 0, 1, 16, 12>(p, st) : launch<kBf, 16, 0, 1, 16, 12>(p, st);
  }
  if (a.d % 4 || a.d_ff % 4) return launch<kF4Tail, 16, 1, 1, 4, 4>(p, st);
  return launch<kF4, 16, 1, 1, 12, 12>(p, st);
}

}  // namespace moe
