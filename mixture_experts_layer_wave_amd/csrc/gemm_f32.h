// A float32 product tile on the matrix cores, shared by the float32 kernels
// of the training operators (gemm_f32.hip, router_grad.hip).
//
// Block of 256 threads (4 waves, 2 x 2), output tile 64 x 64 (each wave
// 32 x 32 on v_mfma_f32_32x32x2_f32), K steps of 32.  Both operands lie in
// LDS K row by K row, 65 floats apart, so that the stores of operands that
// are contiguous along K (32 K of one row by 32 lanes) and the fragment
// reads (32 rows of one K) both meet 64 different banks.  Elements come
// through a function of (k, row), zero outside the operand, so every size,
// gather and layout runs through the same loop; the next step's elements are
// fetched while this step is multiplied.
#pragma once

#include "common.h"

namespace moe {
namespace f32gemm {

constexpr int kT = 64, kK = 32, kPitch = kT + 1, kThreads = 256;
constexpr int kPer = kT * kK / kThreads;  // elements a thread fetches per operand and step

// (k, row) of element i of this thread in a step: lanes run along K for
// operands contiguous along K, along the rows otherwise.
template <bool KMAJ>
__device__ __forceinline__ void place(int i, int &k, int &r) {
  const int t = threadIdx.x;
  if constexpr (KMAJ) {
    r = t & (kT - 1);
    k = (t >> 6) + i * (kThreads / kT);
  } else {
    k = t & (kK - 1);
    r = (t >> 5) + i * (kThreads / kK);
  }
}

// acc += sum over k < K of A(k, m) B(k, n): lane l of wave (wm, wn) holds row
// m = 32 wm + l % 32 and columns n = 32 wn + (i / 4) 8 + (l / 32) 4 + i % 4.
// fa(i, k, m) and fb(i, k, n) give element i of the thread at tile rows m, n;
// they are called with k < K only.  smem: 2 * kK * kPitch floats.
template <bool A_KMAJ, bool B_KMAJ, typename FA, typename FB>
__device__ __forceinline__ void product(f32x16 &acc, float *smem, int K, FA fa, FB fb) {
  float *sa = smem, *sb = smem + kK * kPitch;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int am = (wave >> 1) * 32 + (lane & 31), bn = (wave & 1) * 32 + (lane & 31), kh = lane >> 5;
  float ra[kPer], rb[kPer];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      int k, r;
      place<A_KMAJ>(i, k, r);
      ra[i] = k0 + k < K ? fa(i, k0 + k, r) : 0.f;
      place<B_KMAJ>(i, k, r);
      rb[i] = k0 + k < K ? fb(i, k0 + k, r) : 0.f;
    }
  };
  fetch(0);
  for (int k0 = 0; k0 < K; k0 += kK) {
    __syncthreads();  // the tiles of the step before have been read
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      int k, r;
      place<A_KMAJ>(i, k, r);
      sa[k * kPitch + r] = ra[i];
      place<B_KMAJ>(i, k, r);
      sb[k * kPitch + r] = rb[i];
    }
    __syncthreads();
    if (k0 + kK < K) fetch(k0 + kK);
#pragma unroll
    for (int k = 0; k < kK; k += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sb[(k + kh) * kPitch + bn], sa[(k + kh) * kPitch + am],
                                                 acc, 0, 0, 0);
  }
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
