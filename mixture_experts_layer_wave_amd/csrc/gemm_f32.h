// A float32 product tile on the matrix cores, shared by the float32 kernels
// of the training operators (gemm_f32.hip, router_grad.hip).
//
// Block of 256 threads (4 waves, 2 x 2), output tile 64 x 64 (each wave
// 32 x 32 on v_mfma_f32_32x32x2_f32), K steps of 32.  Both operands lie in
// LDS K row by K row, 65 floats apart, in two stages with one barrier a step;
// a thread fetches four consecutive elements at a time, two steps ahead
// (these products are small, so the trip to memory is most of a step).  A
// 16-byte fetch needs 4-byte alignment only, so every size and layout takes
// it.
//
// A sum over K is taken in runs of 256, each from zero, added to a total:
// the error of a long sum then grows with the runs, not with K.
#pragma once

#include <type_traits>

#include "common.h"
#include "gemm_common.h"

namespace moe {
namespace f32gemm {

constexpr int kT = 64, kK = 32, kPitch = kT + 1, kThreads = 256;
constexpr int kFour = kT * kK / 4 / kThreads;  // pieces a thread fetches per operand and step
constexpr int kStage = 2 * kK * kPitch;        // floats of both tiles of a stage
constexpr int kSmem = 2 * kStage;

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

// (k, row) of the first element of piece i of this thread in a step: pieces
// run along the rows' index for K-major operands, along K otherwise.
template <bool KMAJ>
__device__ __forceinline__ void place(int i, int &k, int &r) {
  const int t = threadIdx.x;
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

// total += sum over k < K of A(k, m) B(k, n): lane l of wave (wm, wn) holds
// row m = 32 wm + l % 32 and columns n = 32 wn + (i / 4) 8 + (l / 32) 4 + i % 4.
// fa(i, k, m) and fb(i, k, n) give the thread's piece i at tile row m or
// column n; k may be past K (the piece is cut here).  smem: kSmem floats.
template <bool A_KMAJ, bool B_KMAJ, typename FA, typename FB>
__device__ __forceinline__ void product(f32x16 &total, float *smem, int K, FA fa, FB fb) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
  auto fetch = [&](f32x4 *a, f32x4 *b, int k0) {
#pragma unroll
    for (int i = 0; i < kFour; ++i) {
      a[i] = get(std::integral_constant<bool, A_KMAJ>{}, fa, i, k0);
      b[i] = get(std::integral_constant<bool, B_KMAJ>{}, fb, i, k0);
    }
  };
  f32x16 acc = {};
  const int steps = (K + kK - 1) / kK;
  fetch(ra[0], rb[0], 0);
  fetch(ra[1], rb[1], kK);
  __syncthreads();  // smem's readers before this call are done
  auto step = [&](int s, auto odd) {
    constexpr int P = decltype(odd)::value;
    // (stage P was last read in step s - 2, before the barrier of s - 1)
    float *sa = smem + P * kStage, *sb = sa + kK * kPitch;
#pragma unroll
    for (int i = 0; i < kFour; ++i) {
      put<A_KMAJ>(sa, i, ra[P][i]);
      put<B_KMAJ>(sb, i, rb[P][i]);
    }
    fetch(ra[P], rb[P], (s + 2) * kK);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kK; k += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sb[(k + kh) * kPitch + bn], sa[(k + kh) * kPitch + am],
                                                 acc, 0, 0, 0);
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

// Tile-relative row and column of accumulator element i.
__device__ __forceinline__ int out_row() {
  return ((threadIdx.x >> 6) >> 1) * 32 + (threadIdx.x & 31);
}
__device__ __forceinline__ int out_col(int i) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  return (wave & 1) * 32 + (i >> 2) * 8 + (lane >> 5) * 4 + (i & 3);
}

}  // namespace f32gemm
}  // namespace moe
