// What the row norms share (norm.hip, block_norm.hip): a row in registers in
// chunks, columns of float32 parameters, sums over a row's threads.
#pragma once

#include <type_traits>

#include "common.h"
#include "route_dev.h"

namespace moe {

// A row's elements in chunks of V, as float32: bf16 rows are multiples of 8
// wide, float32 rows of any width (TAIL: not a multiple of 4).  float32
// chunks are 16-B accesses on 4-B boundaries, which global memory takes; a
// row's last, partial chunk goes element by element, its missing elements
// staying 0.
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <bool BF, bool TAIL>
struct Chunk {
  static constexpr int V = BF ? 8 : 4;
  typedef typename std::conditional<BF, u32x4, f32x4>::type Raw;
  Raw q = {};
  __device__ __forceinline__ void load(const void *p, size_t row, int col, int d) {
    if (col >= d) return;
    if constexpr (BF) {
      q = *(const u32x4 *)((const uint16_t *)p + row * d + col);
    } else {
      const float *f = (const float *)p + row * d + col;
      if (!TAIL || col + 4 <= d)
        q = *(const f32x4_any *)f;
      else
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (col + j < d) q[j] = f[j];
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (BF)
      return __uint_as_float((j & 1) ? (q[j / 2] & 0xffff0000u) : (q[j / 2] << 16));
    else
      return q[j];
  }
  // Element j of the chunk at col is inside the row.
  static __device__ __forceinline__ bool in(int col, int j, int d) { return TAIL ? col + j < d : col < d; }
  // NT: a store that leaves the caches to others.
  template <bool NT = false>
  static __device__ __forceinline__ void store(void *p, size_t row, int col, int d, const float *v) {
    if (col >= d) return;
    if constexpr (BF) {
      const u32x4 o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
      u32x4 *at = (u32x4 *)((uint16_t *)p + row * d + col);
      if constexpr (NT)
        __builtin_nontemporal_store(o, at);
      else
        *at = o;
    } else {
      float *f = (float *)p + row * d + col;
      if (!TAIL || col + 4 <= d)
        if constexpr (NT)
          __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, (f32x4_any *)f);
        else
          *(f32x4_any *)f = f32x4{v[0], v[1], v[2], v[3]};
      else
#pragma unroll
        for (int j = 0; j < 3; ++j)
          if (col + j < d) f[j] = v[j];
    }
  }
};

// w's (or b's) values for the chunk at col, 0 past the row's end.  In 16-B
// loads: with one load per value, a chunk's stride apart over the lanes, the
// norm of one row of 16384 took 16.8 us instead of 5.7, that of 8192 rows of
// 4096 34.0 instead of 29.4.
template <bool TAIL, int V>
__device__ __forceinline__ void load_columns(const float *__restrict__ p, int col, int d, float (&o)[V]) {
#pragma unroll
  for (int h = 0; h < V; h += 4) {
    f32x4 q = {0.f, 0.f, 0.f, 0.f};
    if (!TAIL ? col < d : col + h + 4 <= d)
      q = *(const f32x4_any *)(p + col + h);
    else if (TAIL)
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (col + h + j < d) q[j] = p[col + h + j];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[h + j] = q[j];
  }
}

// Likewise V sums to part.
template <bool TAIL, int V>
__device__ __forceinline__ void store_columns(float *__restrict__ p, int col, int d, const float (&v)[V]) {
#pragma unroll
  for (int h = 0; h < V; h += 4) {
    if (!TAIL ? col < d : col + h + 4 <= d)
      *(f32x4_any *)(p + col + h) = f32x4{v[h], v[h + 1], v[h + 2], v[h + 3]};
    else if (TAIL)
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (col + h + j < d) p[col + h + j] = v[h + j];
  }
}

// fn on each 32-bit half of a double.
template <typename Fn>
__device__ __forceinline__ double by_halves(double v, Fn fn) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)fn((int)(uint32_t)b), hi = (uint32_t)fn((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// group_sum of float64 values over 16 or 64 lanes: the same lane permutations,
// half by half.
__device__ __forceinline__ double group_sum_f64(double v, int G) {
  v += by_halves(v, [](int h) { return dpp_i<kDppXor1>(h); });
  v += by_halves(v, [](int h) { return dpp_i<kDppXor2>(h); });
  v += by_halves(v, [](int h) { return dpp_i<kDppHalfMirror>(h); });
  v += by_halves(v, [](int h) { return dpp_i<kDppMirror>(h); });
  if (G == 64) {
    auto row = [&](int lane) {
      return by_halves(v, [=](int h) { return __builtin_amdgcn_readlane(h, lane); });
    };
    v = (row(0) + row(16)) + (row(32) + row(48));
  }
  return v;
}

// Sums over the TPR threads of a row, in every thread.  Up to a wave the
// sum is lane permutations; above that the waves' sums meet in LDS, in two
// buffers used in turn: a wave can write a buffer again only after the
// barrier of the sum in between, which every reader of the old values has
// passed.  N values at once.
template <typename T, int TPR, int NT, int N>
struct RowSum {
  T (*buf)[N][NT / 64];
  int turn = 0;
  __device__ __forceinline__ explicit RowSum(T (*b)[N][NT / 64]) : buf(b) {}
  __device__ __forceinline__ void operator()(T (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      constexpr int L = TPR < 64 ? TPR : 64;
      static_assert(L == 16 || L == 64, "lanes of a row in a wave");
      if constexpr (std::is_same<T, double>::value)
        v[i] = group_sum_f64(v[i], L);
      else
        v[i] = group_sum(v[i], L);
    }
    if constexpr (TPR > 64) {
      constexpr int W = TPR / 64;
      const int wave = threadIdx.x >> 6, first = wave / W * W;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[turn][i][wave] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < N; ++i) {
        T s = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) s += buf[turn][i][first + j];
        v[i] = s;
      }
      turn ^= 1;
    }
  }
};

// Threads per row and chunks per thread for rows of d: the fewest threads
// that hold a row in one 16-B chunk each (two above 1024 threads, four for
// float32 above 8192), so narrow rows share a block.
template <bool BF, bool TAIL, typename Launch>
hipError_t with_layout(int d, Launch go) {
  constexpr int V = Chunk<BF, TAIL>::V;
#define MOE_LN(C_, T_) \
  if (d <= V * C_ * T_) return go(std::integral_constant<int, C_>{}, std::integral_constant<int, T_>{});
  MOE_LN(1, 16)
  MOE_LN(1, 64)
  MOE_LN(1, 128)
  MOE_LN(1, 256)
  MOE_LN(1, 512)
  MOE_LN(1, 1024)
  MOE_LN(2, 1024)
  if constexpr (!BF) MOE_LN(4, 1024)
#undef MOE_LN
  return hipErrorInvalidValue;
}

}  // namespace moe
