// MXFP4 encoder and decoder (OCP MX v1.0: E2M1 elements, one E8M0 scale for 32
// consecutive ones).
//
//   X = max(floor(log2 max|v|) - 2, -127) over a block (code X + 127; 0 for a
//   block of zeros), element = v / 2^X to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6
//   with its sign, ties to the even code, at most 6.
//
// A block holding an infinity or a NaN has no such X: its scale code is 255, the
// format's NaN, and its elements are 0.
//
// A row's blocks follow one another and rows do too, so a matrix is one run of
// blocks.  Both directions are bound by HBM; four lanes share a block, eight
// values each.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// The eight values of lane `i` (32 consecutive ones to four lanes).
template <bool BF>
__device__ __forceinline__ void load8(const void *x, size_t i, float (&v)[8]) {
  if constexpr (BF) {
    const u32x4 q = ((const u32x4 *)x)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(q[j] << 16);
      v[2 * j + 1] = __uint_as_float(q[j] & 0xffff0000u);
    }
  } else {
    const f32x4 a = ((const f32x4 *)x)[2 * i], b = ((const f32x4 *)x)[2 * i + 1];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
  }
}

template <bool BF>
__global__ __launch_bounds__(kThreads) void quantize_mx4_kernel(const void *__restrict__ x, size_t lanes,
                                                                uint32_t *__restrict__ q, uint8_t *__restrict__ s) {
  const size_t stride = (size_t)gridDim.x * kThreads;
  // (lanes is a multiple of 4: a block's four lanes take part together)
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < lanes; i += stride) {
    float v[8];
    load8<BF>(x, i, v);
    // the bit pattern of a magnitude grows with it, infinities and NaN on top
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp((int)top, (int)top, 0xB1, 0xF, 0xF, false));
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp((int)top, (int)top, 0x4E, 0xF, 0xF, false));
    const uint32_t ef = top >> 23;  // biased exponent; 0 for float32 subnormals, whose X is below -127
    const bool bad = ef == 255u;
    const uint32_t code = bad ? 255u : (ef > 2u ? ef - 2u : 0u);
    const float inv = __uint_as_float(bad ? 0u : (254u - code) << 23);
    uint32_t w = 0;
    if (!bad) {
      float c[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = fminf(fmaxf(v[j] * inv, -6.f), 6.f);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[0], c[1], 1.0f, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[2], c[3], 1.0f, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[4], c[5], 1.0f, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, c[6], c[7], 1.0f, 3);
    }
    q[i] = w;
    if ((threadIdx.x & 3) == 0) s[i >> 2] = (uint8_t)code;
  }
}

// The conversion instructions take the scale; a bf16 or float32 value is exact down to
// 2^-128.
template <bool BF>
__global__ __launch_bounds__(kThreads) void dequantize_mx4_kernel(const uint32_t *__restrict__ q,
                                                                  const uint8_t *__restrict__ s, size_t lanes,
                                                                  void *__restrict__ y) {
  const size_t stride = (size_t)gridDim.x * kThreads;
  for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < lanes; i += stride) {
    const uint32_t w = q[i];
    const float sc = e8m0_to_f32(s[i >> 2]);
    if constexpr (BF) {
      ((u32x4 *)y)[i] = u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0)),
                              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1)),
                              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2)),
                              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3))};
    } else {
      const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 1);
      const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, sc, 3);
      ((f32x4 *)y)[2 * i] = f32x4{a[0], a[1], b[0], b[1]};
      ((f32x4 *)y)[2 * i + 1] = f32x4{c[0], c[1], e[0], e[1]};
    }
  }
}

int grid_of(size_t lanes) {
  const size_t want = (lanes + kThreads - 1) / kThreads, cap = 256 * 8;
  return (int)(want < cap ? want : cap);
}

}  // namespace

hipError_t launch_quantize_mx4(const void *x, bool is_bf16, size_t blocks, uint8_t *q, uint8_t *s, hipStream_t st) {
  const size_t lanes = blocks * 4;
  if (is_bf16)
    quantize_mx4_kernel<true><<<grid_of(lanes), kThreads, 0, st>>>(x, lanes, (uint32_t *)q, s);
  else
    quantize_mx4_kernel<false><<<grid_of(lanes), kThreads, 0, st>>>(x, lanes, (uint32_t *)q, s);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx4(const uint8_t *q, const uint8_t *s, size_t blocks, void *y, bool out_bf16,
                                 hipStream_t st) {
  const size_t lanes = blocks * 4;
  if (out_bf16)
    dequantize_mx4_kernel<true><<<grid_of(lanes), kThreads, 0, st>>>((const uint32_t *)q, s, lanes, y);
  else
    dequantize_mx4_kernel<false><<<grid_of(lanes), kThreads, 0, st>>>((const uint32_t *)q, s, lanes, y);
  return hipGetLastError();
}

}  // namespace moe
