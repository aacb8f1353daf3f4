// A float32 product tile on the matrix cores, shared by the float32 kernels
// of the training operators (gemm_f32.hip, router_grad.hip).
//
// Block: G groups of 4 waves (2 x 2, each 32 x 32 on v_mfma_f32_32x32x2_f32)
// compute the same 64 x 64 output tile, group g over the K steps of 32 that
// are g mod G.  G = 2 is for grids of few blocks, which have two waves per
// SIMD all the same (one group's LDS and barrier waits lie under the other's
// products); with many blocks G = 1 has four of them on a CU, each at its own
// place.
// Both operands lie in LDS K row by K row, 66 floats apart: the stores of
// operands contiguous along K (8 pieces of four K, 8 rows) and the fragment
// reads (32 rows of K rows k and k + 16) meet 64 different banks.  Two stages
// a group, one barrier a step; a thread fetches four consecutive elements at
// a time, two steps ahead.  A 16-byte fetch needs 4-byte alignment only, so
// every size and layout takes it.
//
// A sum over K is taken in runs of eight steps, each from zero, added to a
// total: the error of a long sum then grows with the runs, not with K.
#pragma once

#include <type_traits>

#include "common.h"
#include "gemm_common.h"

namespace moe {
namespace f32gemm {

constexpr int kT = 64, kK = 32, kPitch = kT + 2;
constexpr int kFour = kT * kK / 4 / 256;       // pieces a thread fetches per operand and step
constexpr int kStage = 2 * kK * kPitch;        // floats of both tiles of a stage
constexpr int kOutPitch = kT + 4;
template <int G>
struct Groups {
  static constexpr int THREADS = 256 * G;
  static constexpr int SMEM = 2 * G * kStage;            // floats: two stages a group
  static constexpr int LINES = kT * kT / 4 / THREADS;    // pieces of the result a thread holds
  // Row and first column (in the tile) of the result's piece i of this
  // thread: 16 lanes hold a row.
  static __device__ __forceinline__ int row(int i) { return (threadIdx.x >> 4) + i * (THREADS / 16); }
  static __device__ __forceinline__ int col() { return (threadIdx.x & 15) * 4; }
};

// Four consecutive elements at byte offset `off` of a buffer, of which the
// first `n` (<= 0: none, >= 4: all) belong to the operand.  Dwords past the
// buffer's record count read as zero one by one; elements past n (the next
// row's) are replaced by zero.  No branch: the fetches in flight stay
// countable.
struct Piece {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off;
  int n;
};
__device__ __forceinline__ f32x4 fetch4(Piece q) {
  f32x4 v = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                          q.r, q.n > 0 ? q.off : gemm::kOOB, 0, 0));
#pragma unroll
  for (int j = 1; j < 4; ++j) v[j] = j < q.n ? v[j] : 0.f;
  return v;
}
// The first n of four elements to dst (4-byte aligned).
__device__ __forceinline__ void store4(float *dst, int n, f32x4 v) {
  typedef f32x4 f32x4_any __attribute__((aligned(4)));
  if (n >= 4) {
    *(f32x4_any *)dst = v;
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < n) dst[j] = v[j];
  }
}

// (k, row) of the first element of piece i of this thread (of its group) in a
// step: pieces run along the rows' index for K-major operands, along K
// otherwise.
template <bool KMAJ>
__device__ __forceinline__ void place(int i, int &k, int &r) {
  const int t = threadIdx.x & 255;
  if constexpr (KMAJ) {
    r = (t & 15) * 4;
    k = (t >> 4) + i * 16;
  } else {
    k = (t & 7) * 4;
    r = (t >> 3) + i * 32;
  }
}
template <bool KMAJ>
__device__ __forceinline__ void put(float *tile, int i, f32x4 v) {
  int k, r;
  place<KMAJ>(i, k, r);
#pragma unroll
  for (int j = 0; j < 4; ++j) tile[KMAJ ? k * kPitch + r + j : (k + j) * kPitch + r] = v[j];
}

// This group's part of total += sum over k < K of A(k, m) B(k, n).
// piece_a(i, k, m) and piece_b(i, k, n) give the thread's piece i at tile row
// m or column n; k may be past K (the piece is cut here).  smem:
// Groups<G>::SMEM floats.  Every thread of the block calls it.
template <int G, bool A_KMAJ, bool B_KMAJ, typename FA, typename FB>
__device__ __forceinline__ void product(f32x16 &total, float *smem, int K, FA piece_a, FB piece_b) {
  const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) & 3, kg = G > 1 ? threadIdx.x >> 8 : 0;
  const int am = (wave >> 1) * 32 + (lane & 31), bn = (wave & 1) * 32 + (lane & 31), kh = lane >> 5;
  auto get = [&](auto kmaj, auto f, int i, int k0) {
    constexpr bool KMAJ = decltype(kmaj)::value;
    int k, r;
    place<KMAJ>(i, k, r);
    Piece q = f(i, k0 + k, r);
    if (KMAJ)
      q.n = k0 + k < K ? q.n : 0;
    else
      q.n = q.n > 0 ? K - k0 - k : 0;
    return fetch4(q);
  };
  f32x4 ra[2][kFour], rb[2][kFour];
  // step s of this group
  auto fetch = [&](f32x4 *a, f32x4 *b, int s) {
    const int k0 = (G * s + kg) * kK;
#pragma unroll
    for (int i = 0; i < kFour; ++i) {
      a[i] = get(std::integral_constant<bool, A_KMAJ>{}, piece_a, i, k0);
      b[i] = get(std::integral_constant<bool, B_KMAJ>{}, piece_b, i, k0);
    }
  };
  f32x16 acc = {};
  const int steps = (K + G * kK - 1) / (G * kK);  // of every group
  fetch(ra[0], rb[0], 0);
  fetch(ra[1], rb[1], 1);
  __syncthreads();  // smem's readers before this call are done
  auto step = [&](int s, auto odd) {
    constexpr int P = decltype(odd)::value;
    // (stage P was last read in step s - 2, before the barrier of s - 1)
    float *sa = smem + (2 * kg + P) * kStage, *sb = sa + kK * kPitch;
#pragma unroll
    for (int i = 0; i < kFour; ++i) {
      put<A_KMAJ>(sa, i, ra[P][i]);
      put<B_KMAJ>(sb, i, rb[P][i]);
    }
    fetch(ra[P], rb[P], s + 2);
    __syncthreads();
    // half of the step's fragments first, so that the products wait for the
    // first of them only
    constexpr int H = kK / 4;
#pragma unroll
    for (int h = 0; h < kK / 2; h += H) {
      float fa[H], fb[H];
#pragma unroll
      for (int k = 0; k < H; ++k) {
        fa[k] = sa[(h + k + 16 * kh) * kPitch + am];
        fb[k] = sb[(h + k + 16 * kh) * kPitch + bn];
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < H; ++k) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[k], fa[k], acc, 0, 0, 0);
    }
    if ((s & 7) == 7) {
      total += acc;
      acc = f32x16{};
    }
  };
  for (int s = 0; s < steps; s += 2) {
    step(s, std::integral_constant<int, 0>{});
    if (s + 1 < steps) step(s + 1, std::integral_constant<int, 1>{});
  }
  total += acc;
}

// The groups' totals, added, as pieces of four columns (Groups::row, col).
template <int G>
__device__ __forceinline__ void lines(const f32x16 &total, float *smem, f32x4 (&out)[Groups<G>::LINES]) {
  using L = Groups<G>;
  const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) & 3, kg = G > 1 ? threadIdx.x >> 8 : 0;
  const int am = (wave >> 1) * 32 + (lane & 31), kh = lane >> 5;
  // Lane l of wave (wm, wn) holds row 32 wm + l % 32 and columns 32 wn +
  // 8 g + 4 (l / 32) + 0 .. 3: the groups' sums, in order.
#pragma unroll
  for (int half = 0; half < G; ++half) {
    __syncthreads();
    if (kg == half)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float *q = smem + am * kOutPitch + (wave & 1) * 32 + g * 8 + kh * 4;
        f32x4 v = {total[g * 4], total[g * 4 + 1], total[g * 4 + 2], total[g * 4 + 3]};
        if (half) v += *(const f32x4 *)q;
        *(f32x4 *)q = v;
      }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < L::LINES; ++i) out[i] = *(const f32x4 *)(smem + L::row(i) * kOutPitch + L::col());
}

}  // namespace f32gemm
}  // namespace moe
