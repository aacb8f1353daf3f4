// Streaming a few rows' products with a weight matrix: one wave's pass over
// weight rows that go straight from memory to the matrix cores, and the forms
// of weights it takes.  Used by the few-token layer (few.hip) and the MXFP4
// product of few rows (linear.hip).
#pragma once

#include "common.h"

namespace moe {

// Forms of weights and activations: MXFP4 with bf16, MXFP4 with MXFP4, bf16,
// float32, and float32 rows of any length (the others' rows are whole blocks).
enum { kMx = 0, kMx4 = 1, kBf = 2, kF4 = 3, kF4Tail = 4 };

template <int WT>
struct Form {
  static constexpr bool f32 = WT >= kF4, mx = WT <= kMx4;
  static constexpr int V = mx ? 32 : (WT == kBf ? 8 : 4);  // elements of a block (16 B of weights)
  static constexpr int kActBytes = WT == kMx4 ? 16 : V * (f32 ? 4 : 2);  // the block's activations
  __host__ __device__ static int blocks(int K) { return (K + V - 1) / V; }
  __host__ __device__ static size_t row_bytes(int K) { return mx ? (size_t)K / 2 : (size_t)K * (f32 ? 4 : 2); }
};

typedef int v8i __attribute__((ext_vector_type(8)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// 16 bytes of block b of a weight row of K elements.
template <int WT>
__device__ __forceinline__ u32x4 load_weights(const uint8_t *row, int b, int K) {
  if constexpr (WT == kF4Tail) {
    const float *p = (const float *)row;
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = p[min(b * 4 + j, K - 1)];
    return __builtin_bit_cast(u32x4, v);
  } else if constexpr (WT == kF4) {
    return __builtin_bit_cast(u32x4, __builtin_nontemporal_load((const f32x4_any *)(row + (size_t)b * 16)));
  } else {
    return __builtin_nontemporal_load((const u32x4 *)(row + (size_t)b * 16));
  }
}

template <int WT>
__device__ __forceinline__ u32x4 load_act(const uint8_t *row, int b, int K) {
  if constexpr (WT == kF4Tail) {
    return load_weights<WT>(row, b, K);
  } else if constexpr (WT == kF4) {
    return __builtin_bit_cast(u32x4, *(const f32x4_any *)(row + (size_t)b * 16));
  } else {
    return *(const u32x4 *)(row + (size_t)b * 16);
  }
}

// acc += (the tokens' block) x (the weights' block); a: NF 16-byte pieces.
template <int WT>
__device__ __forceinline__ void multiply(const u32x4 *a, uint32_t ascale, u32x4 w, uint32_t scale,
                                         f32x4 (&acc)[2]) {
  if constexpr (WT == kMx4) {
    const v8i av = {(int)a[0].x, (int)a[0].y, (int)a[0].z, (int)a[0].w, 0, 0, 0, 0};
    const v8i wv = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    acc[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, wv, acc[0], 4, 4, 0, (int)ascale, 0, (int)scale);
  } else if constexpr (WT == kMx) {
    const float sc = e8m0_to_f32(scale);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const u32x4 bw = {
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], sc, 0)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], sc, 1)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], sc, 2)),
          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], sc, 3))};
      acc[q & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[q]),
                                                           __builtin_bit_cast(bf16x8, bw), acc[q & 1], 0, 0, 0);
    }
  } else if constexpr (WT == kBf) {
    acc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[0]),
                                                     __builtin_bit_cast(bf16x8, w), acc[0], 0, 0, 0);
  } else {
    const f32x4 av = __builtin_bit_cast(f32x4, a[0]), wv = __builtin_bit_cast(f32x4, w);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[j & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[j], wv[j], acc[j & 1], 0, 0, 0);
  }
}

// One wave's pass over `total` steps: segments (rows of weights with the tokens'
// rows that meet them) of S steps each, the first one entered at step s0.  Lane
// (r, g) = (lane % 16, lane / 16) holds weight row r and block 4 s + g.
//   seg(i, row, srow, arow[], asrow)  the lane's weight row, its scales and, where
//                 the activations come through the ring, its rows to fetch (and
//                 with kMx4 their scales)
//   acts(i, s, a) the lane's pieces of token r, block 4 s + g, from LDS
//                 (ARING = 0), or nothing
//   rank(i)       with ARING and kMx: which fetched row is token r's
//   end(i, acc)   a segment's last step is done
// With ARING the rows come through the ring, at its depth (in-order loads: a
// shallower one for them would hold up the weights).  kMx4, bf16 and float32: lane
// (r, g) fetches its own piece.  kMx: a step is 16 pieces of each row; lane l
// fetches piece l % 16 of rows l / 16 + 4 i, i < ARING, and the pieces change
// lanes through abuf, the wave's own LDS.
template <int WT, int PF, int ARING, class Seg, class Acts, class Rank, class End>
__device__ __forceinline__ void stream(int total, int S, int s0, int K, uint8_t *abuf, Seg seg, Acts acts,
                                       Rank rank, End end) {
  using F = Form<WT>;
  constexpr int NF = F::kActBytes / 16;
  constexpr int NA = ARING ? ARING : 1;
  if (total <= 0) return;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int KB = F::blocks(K);
  u32x4 w[PF], ar[ARING ? PF : 1][NA];
  uint32_t sc[PF], asc[PF];
  const uint8_t *row, *srow, *arow[NA], *asrow = nullptr;
  int ld_seg = 0, ld_s = s0, left = total;
  seg(0, row, srow, arow, asrow);
  auto load = [&](int j) {  // the next step (the last one again when none is left)
    const int b = min(4 * ld_s + g, KB - 1);
    w[j] = load_weights<WT>(row, b, K);
    if constexpr (F::mx) sc[j] = srow[b];
    if constexpr (WT == kMx4) asc[j] = asrow[b];
    if constexpr (ARING > 0) {
      if constexpr (WT == kMx) {
        const int ab = min(4 * ld_s + (r >> 2), KB - 1);
#pragma unroll
        for (int i = 0; i < NA; ++i) ar[j][i] = load_act<WT>(arow[i], ab * 4 + (r & 3), K);
      } else {
        ar[j][0] = load_act<WT>(arow[0], b, K);
      }
    }
    if (left > 1) {
      --left;
      if (++ld_s == S) {
        ld_s = 0;
        seg(++ld_seg, row, srow, arow, asrow);
      }
    }
  };
  f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
  int cur = 0, s = s0;
  auto use = [&](int j, bool last) {
    u32x4 a[NF], wj = w[j];
    uint32_t scale = F::mx ? sc[j] : 0u, ascale = WT == kMx4 ? asc[j] : 0u;
    if constexpr (ARING == 0) {
      acts(cur, min(4 * s + g, KB - 1), a);
    } else if constexpr (WT == kMx) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < NA; ++i) {
        const int ai = g + 4 * i;
        *(u32x4 *)(abuf + (ai * 16 + (r ^ ai)) * 16) = ar[j][i];
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
      const int at = rank(cur);
#pragma unroll
      for (int q = 0; q < NF; ++q) a[q] = *(const u32x4 *)(abuf + (at * 16 + ((g * 4 + q) ^ at)) * 16);
    } else {
      a[0] = ar[j][0];
    }
    if (s == S - 1 && (KB % 4 || WT == kF4Tail)) {  // blocks past the row's end
      const u32x4 z = {0u, 0u, 0u, 0u};
      const int b = 4 * s + g;
      if constexpr (WT == kF4Tail) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (b * 4 + i >= K) wj[i] = 0u, a[0][i] = 0u;
      } else if (b >= KB) {
        wj = z;
        scale = ascale = 127u;
#pragma unroll
        for (int q = 0; q < NF; ++q) a[q] = z;
      }
    }
    multiply<WT>(a, ascale, wj, scale, acc);
    if (++s == S || last) {
      end(cur, acc[0] + acc[1]);
      acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
      s = 0;
      ++cur;
    }
  };
  const int groups = (total + PF - 1) / PF;
#pragma unroll
  for (int j = 0; j < PF; ++j) load(j);
  for (int gi = 0; gi + 1 < groups; ++gi)
#pragma unroll
    for (int j = 0; j < PF; ++j) {
      use(j, false);
      load(j);
    }
  const int rest = total - (groups - 1) * PF;
#pragma unroll
  for (int j = 0; j < PF; ++j)
    if (j < rest) use(j, j == rest - 1);
}

}  // namespace moe
