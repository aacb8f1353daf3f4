// K-major operand tiles in LDS and their MFMA fragments: the operand lies as
// in memory, K row by K row, W columns each, and ds_read_b64_tr_b16
// transposes 4 x 16 blocks of 16-bit values on the way to the registers.
#pragma once

#include "common.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// 16-B chunk c of K row k is stored at chunk c ^ key(k).  A transposing read
// takes 64 consecutive bytes of four consecutive rows per half wave; the key
// puts those in four different quarters of the 64 banks (rows of 64 bytes
// fall there by themselves, rows of 128 bytes need the halves swapped in
// every other pair of rows).
template <int W>
__device__ __forceinline__ int kmaj_key(int k) {
  static_assert(W == 32 || W == 64 || W % 128 == 0, "columns of a K-major tile");
  if constexpr (W == 32) return 0;
  if constexpr (W == 64) return ((k >> 1) & 1) << 2;
  return (k & 3) << 2;
}

// Byte offset in a K-major tile of W columns that this lane hands to the
// transposing reads of the 32-column fragment at column `col`: 16-lane group
// g of the wave covers columns 16 (g % 2) .. + 15 and K rows 8 (g / 2) .. + 3
// of the slice; lane i of it reads four columns of row i / 4.
template <int W>
__device__ __forceinline__ int kmaj_lane(int col, int lane) {
  const int grp = lane >> 4, i = lane & 15;
  const int chunk = ((col + (grp & 1) * 16) >> 3) + ((i & 3) >> 1);
  return ((grp >> 1) * 8 + (i >> 2)) * (W * 2) + ((chunk ^ kmaj_key<W>(i >> 2)) << 4) + (i & 1) * 8;
}

// The fragment of slice kk: column lane % 32, K rows 16 kk + 8 (lane / 32) + 0 .. 7.
template <int W>
__device__ __forceinline__ bf16x8 kmaj_frag(const uint8_t *tile, int lane_off, int kk) {
  const uint8_t *p = tile + lane_off + kk * 16 * (W * 2);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * (W * 2)));
  const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}

}  // namespace moe
