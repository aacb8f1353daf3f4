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
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
struct __attribute__((packed, aligned(1))) u32_any {
  uint32_t v;
};

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

// One wave's pass over segments: two groups of 1 to 8 consecutive rows of weights, with
// the tokens' rows that meet them, over `count` chunks of K from chunk `first` on.  A
// chunk is kSteps steps, a step four blocks of each row; in the products lane (r, g) =
// (lane % 16, lane / 16) holds row r % 8 of group r / 8 and the step's block g.
//   seg(i, s)     segment i; false where there is none (asked for in order, up to
//                 PC segments ahead of the products)
//   ready()       called once by every wave behind its first loads, also by a wave
//                 without segments
//   begin(i, first, count)  the products of segment i begin: its chunks
//   acts(i, c, b, a, as)  the lane's NF pieces (and with kMx4 the scale) of its token
//                 r, block b of chunk c of segment i; zeros past K
//   end(i, acc)   they are done
// A load takes 256 consecutive bytes of four rows (16 lanes a row) and the pieces
// change lanes through xbuf, the wave's own kExchange bytes of LDS: loads of 64 bytes
// of 16 rows, straight into the lanes that multiply, streamed 128 MXFP4 experts' up
// projections at 3.9 TB/s.  PC chunks of weights are in flight, in registers.  Every
// load of the loop is unconditional (the last chunk again when none is left): a load
// behind a branch makes the compiler wait for all of them at the join.
constexpr int kSteps = 4, kChunkBlocks = 4 * kSteps;
constexpr int kExchange = 16 * 256 + 256;  // a chunk's codes and scales

struct Segment {
  const uint8_t *row[2], *scale[2];
  int cnt[2];
  int first, count;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The rows of a segment: 1 to 16 rows of one matrix as two groups (the first row again
// as the second group where there are no more than 8).
template <int WT>
__device__ __forceinline__ void rows_of_one(Segment &g, const uint8_t *w, const uint8_t *s, size_t row, int cnt,
                                            int K) {
  using F = Form<WT>;
  const size_t rb = F::row_bytes(K), next = cnt > 8 ? 8 : 0;
  g.row[0] = w + row * rb;
  g.row[1] = w + (row + next) * rb;
  g.scale[0] = F::mx ? s + row * (K / 32) : nullptr;
  g.scale[1] = F::mx ? s + (row + next) * (K / 32) : nullptr;
  g.cnt[0] = min(cnt, 8);
  g.cnt[1] = max(cnt - 8, 1);
}

template <int WT, int PC, bool NARROW, class Seg, class Ready, class Begin, class Acts, class End>
__device__ __forceinline__ void stream(int C, int K, uint8_t *xbuf, Seg seg, Ready ready, Begin begin, Acts acts,
                                       End end) {
  using F = Form<WT>;
  constexpr int NF = F::kActBytes / 16;
  constexpr bool kTail = WT == kF4Tail;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int KB = F::blocks(K), last = KB - 1 - kChunkBlocks * (C - 1);  // the last chunk's last block
  const int rb = (int)F::row_bytes(K);
  // Scales: lane l fetches four of row l / 4.  Where a row ends inside them they are
  // the row's last four, moved down; NARROW (some row has under four): one by one.
  const int sback = max(0, 4 * (lane & 3) + 3 - last);  // in the last chunk
  u32x4 w[PC][kSteps];
  uint32_t sc[PC];
  Segment rows;
  if (!seg(0, rows)) {
    ready();
    return;
  }
  uint32_t off[kSteps];  // of the lane's pieces, from its group's first row (callers keep 8 rows below 2^31 bytes)
  const uint8_t *sp = nullptr;
  int ld_seg = 0, ld_c = 0, ld_left = 0, issued = 1;  // the chunk to load next, and its number
  bool more = true;
  auto open = [&] {
    const int c = ld_c = rows.first;
    ld_left = rows.count;
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
      off[u] = (uint32_t)(min(4 * (u & 1) + g, rows.cnt[u >> 1] - 1) * rb);
    if constexpr (F::mx) {
      const int h = lane >> 5;
      sp = (h ? rows.scale[1] : rows.scale[0]) +
           (min((lane >> 2) & 7, (h ? rows.cnt[1] : rows.cnt[0]) - 1) * KB + c * kChunkBlocks);
    }
    if constexpr (!kTail)
#pragma unroll
      for (int i = 0; i < 2; ++i) rows.row[i] += (size_t)c * kChunkBlocks * 16;
  };
  auto load = [&](int j) {
    const bool end_of_row = ld_c == C - 1;
    const uint32_t piece = min(r, end_of_row ? last : kChunkBlocks - 1) * 16;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const uint8_t *p = rows.row[u >> 1];
      if constexpr (kTail) {
        const uint32_t *v = (const uint32_t *)(p + off[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[j][u][i] = v[min((ld_c * kChunkBlocks + r) * 4 + i, K - 1)];
      } else if constexpr (WT == kF4) {
        w[j][u] = __builtin_bit_cast(u32x4, __builtin_nontemporal_load((const f32x4_any *)(p + (off[u] + piece))));
      } else {
        w[j][u] = __builtin_nontemporal_load((const u32x4 *)(p + (off[u] + piece)));
      }
    }
    if constexpr (F::mx) {
      const int at = 4 * (lane & 3);
      if constexpr (NARROW) {
        const int most = end_of_row ? last : kChunkBlocks - 1;
        sc[j] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[j] |= (uint32_t)sp[min(at + i, most)] << (8 * i);
      } else {
        sc[j] = ((const u32_any *)(sp + (at - (end_of_row ? sback : 0))))->v;
      }
    }
    if (--ld_left > 0) {
      ++ld_c;
      ++issued;
      if constexpr (!kTail)
#pragma unroll
        for (int i = 0; i < 2; ++i) rows.row[i] += kChunkBlocks * 16;
      if constexpr (F::mx) sp += kChunkBlocks;
    } else if (more) {
      Segment next;
      if (seg(ld_seg + 1, next)) {
        rows = next;
        ++ld_seg;
        ++issued;
        open();
      } else {
        more = false;
      }
    }
  };
  f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
  int cur = -1, c = 0, c_left = 0;
  auto use = [&](int j) {
    if (c_left == 0) begin(++cur, c, c_left);
    // piece q of row i lies in slot q ^ i of the row's 16
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int row = 4 * u + g;
      *(u32x4 *)(xbuf + (row * 16 + (r ^ row)) * 16) = w[j][u];
    }
    if constexpr (F::mx) *(uint32_t *)(xbuf + 4096 + lane * 4) = (!NARROW && c == C - 1) ? sc[j] >> (8 * min(sback, 3)) : sc[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    u32x4 wj[kSteps], sj = {0u, 0u, 0u, 0u};
    if constexpr (F::mx) sj = *(const u32x4 *)(xbuf + 4096 + r * 16);
#pragma unroll
    for (int u = 0; u < kSteps; ++u) wj[u] = *(const u32x4 *)(xbuf + (r * 16 + ((4 * u + g) ^ r)) * 16);
    uint32_t scale[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) scale[u] = (sj[u] >> (8 * g)) & 255u;
    if (c == C - 1) {  // what lies past the row's end
#pragma unroll
      for (int u = 0; u < kSteps; ++u) {
        if (4 * u + g > last) scale[u] = 127u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (kTail ? (c * kChunkBlocks + 4 * u + g) * 4 + i >= K : 4 * u + g > last) wj[u][i] = 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      u32x4 a[NF];
      uint32_t as = 127u;
      acts(cur, c, 4 * u + g, a, as);
      multiply<WT>(a, as, wj[u], scale[u], acc);
    }
    ++c;
    if (--c_left == 0) {
      end(cur, acc[0] + acc[1]);
      acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  };
  open();
#pragma unroll
  for (int j = 0; j < PC; ++j) load(j);
  ready();
  int used = 0;
  while (used + PC < issued) {  // at least one more load after these
#pragma unroll
    for (int j = 0; j < PC; ++j) {
      use(j);
      load(j);
    }
    used += PC;
  }
  const int rest = issued - used;
#pragma unroll
  for (int j = 0; j < PC; ++j)
    if (j < rest) use(j);
}

// Rows of activations in LDS, cut into row chunks: the kChunkBlocks blocks that one
// chunk meets, and 16 bytes more, which puts 16 rows' reads into different banks.
template <int WT>
constexpr int kRowChunk = kChunkBlocks * Form<WT>::kActBytes + 16;

// Lane l's 16 bytes of row chunk c of a row of K elements, 0 past K (16 or 64 lanes a
// row chunk).
template <int WT>
__device__ __forceinline__ u32x4 row_chunk_piece(const uint8_t *row, int c, int K, int l) {
  using F = Form<WT>;
  constexpr int P = F::kActBytes / 16;  // pieces of a block
  u32x4 v = {0u, 0u, 0u, 0u};
  if constexpr (WT == kF4Tail) {
    const int at = c * kChunkBlocks * 4 + l * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i < K) v[i] = ((const uint32_t *)row)[at + i];
  } else {
    const int b = c * kChunkBlocks + l / P;
    const bool in = b < F::blocks(K);
    const uint8_t *p = row + (in ? (size_t)b * F::kActBytes + (l % P) * 16 : 0);
    const u32x4 q = F::f32 ? __builtin_bit_cast(u32x4, *(const f32x4_any *)p) : *(const u32x4 *)p;
    if (in) v = q;
  }
  return v;
}

template <int WT>
__device__ __forceinline__ void stage_row_chunk(uint8_t *dst, const uint8_t *row, int c, int K, int l) {
  *(u32x4 *)(dst + l * 16) = row_chunk_piece<WT>(row, c, K, l);
}

// The lane's pieces of block b of a row of K elements, from global memory, 0 past K.
template <int WT>
__device__ __forceinline__ void load_block(const uint8_t *row, int b, int K, u32x4 (&a)[Form<WT>::kActBytes / 16]) {
  using F = Form<WT>;
  if constexpr (WT == kF4Tail) {
    const uint32_t *v = (const uint32_t *)row;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[0][i] = b * 4 + i < K ? v[b * 4 + i] : 0u;
  } else {
    const bool in = b < F::blocks(K);
    const uint8_t *p = row + (in ? (size_t)b * F::kActBytes : 0);
#pragma unroll
    for (int q = 0; q < F::kActBytes / 16; ++q) {
      const u32x4 v = F::f32 ? __builtin_bit_cast(u32x4, *(const f32x4_any *)(p + q * 16)) : *(const u32x4 *)(p + q * 16);
      a[q] = in ? v : u32x4{0u, 0u, 0u, 0u};
    }
  }
}

}  // namespace moe
