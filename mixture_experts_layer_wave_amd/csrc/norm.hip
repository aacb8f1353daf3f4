// Layer norm and its gradient (the norm in front of the layer's router and
// experts, and what training it needs).
//
//   mean = sum_c x_c / d,  rstd = (sum_c (x_c - mean)^2 / d + eps)^-1/2,
//   xh = (x - mean) rstd,  y = xh w + b
//
//   dx = rstd (w dy - m1 - xh m2),  m1 = sum_c w_c dy_c / d,
//                                   m2 = sum_c w_c dy_c xh_c / d
//   dw_c = sum_t dy_tc xh_tc,  db_c = sum_t dy_tc
//
// Both are bound by HBM: a row is read once (x, or x and dy) and written
// once.  TPR threads hold a row in registers, C chunks of V consecutive
// elements each (16-B accesses where rows allow), so the variance is the sum
// of squared differences from the mean, not a difference of sums, and
// nothing is read twice.  A thread owns the same columns of every row it
// meets: w and b stay in its registers, and so do its columns' partial dw
// and db in the gradient.  Those are added over the block's rows and row
// groups, then, by a second kernel, over the blocks, always in the same
// order.  Sums are float32, but for the mean of float32 rows (float64); rows
// are rounded once on their way out.
//
// Measured, 8192 rows of 4096 in bf16: forward 27.6 us (134 MB, 4.9 TB/s),
// gradient 43 us (201 MB, 4.7 TB/s) with 4.7 us of it for the sum over the
// blocks; a 1 GiB copy reaches 5.07 TB/s.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "route_dev.h"

namespace moe {
namespace {

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
  static __device__ __forceinline__ void store(void *p, size_t row, int col, int d, const float *v) {
    if (col >= d) return;
    if constexpr (BF) {
      const u32x4 o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7])};
      *(u32x4 *)((uint16_t *)p + row * d + col) = o;
    } else {
      float *f = (float *)p + row * d + col;
      if (!TAIL || col + 4 <= d)
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

template <bool BF, bool TAIL, int C, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void layer_norm_kernel(
    const void *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b, float eps,
    int n, int d, void *__restrict__ y, float *__restrict__ mean, float *__restrict__ rstd) {
  using K = Chunk<BF, TAIL>;
  constexpr int V = K::V;
  constexpr int NT = TPR > 256 ? TPR : 256, G = NT / TPR;  // G rows at a time
  // A float32 row's values are added in float64: the mean is then exact to
  // float32's last bit, and what that bit leaves (rest) is taken off as well, so
  // that y depends on the row's spread only, however far from zero it lies.
  // (Added in float32, y of a row 1e5 from zero took over the rounding of 1e5,
  // and rows of equal values had differences other than 0; that took 49.7 us for
  // 8192 rows of 4096, 36.7 of 2880, 19.0 for 65536 of 128, this 50.9, 40.3 and
  // 20.7.)
  // bf16 values carry few enough bits for float32.
  typedef typename std::conditional<BF, float, double>::type Sum;
  __shared__ Sum s_mean[2][1][NT / 64];
  __shared__ float s_var[2][1][NT / 64];
  RowSum<Sum, TPR, NT, 1> mean_sum(s_mean);
  RowSum<float, TPR, NT, 1> var_sum(s_var);
  const double inv_d = 1.0 / (double)d;
  const int grp = threadIdx.x / TPR, gl = threadIdx.x % TPR;
  const int stride = gridDim.x * G;
  K next[C];  // the row to come
  auto load_row = [&](int row) {
    if (row < n)
#pragma unroll
      for (int c = 0; c < C; ++c) next[c].load(x, row, (c * TPR + gl) * V, d);
  };
  load_row(blockIdx.x * G + grp);
  float wv[C][V], bv[C][V] = {};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_columns<TAIL>(w, (c * TPR + gl) * V, d, wv[c]);
    if (b) load_columns<TAIL>(b, (c * TPR + gl) * V, d, bv[c]);
  }
  // (every thread of a block takes the same number of turns: the sums of a
  // row over several waves meet at barriers)
  for (int base = blockIdx.x * G; base < n; base += stride) {
    const int row = base + grp;
    float v[C][V], s[1] = {0.f};
    Sum total[1] = {0};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[c][j] = next[c].get(j);  // 0 past the row's end
        total[0] += (Sum)v[c][j];
      }
    load_row(row + stride);  // runs under this row's sums
    mean_sum(total);
    // The mean of equal values, whose sum is exact, is that value: bf16 sums are
    // divided, as s * (1 / d) may be off by a bit; of float64 ones rounding to
    // float32 drops that bit, and rest is 0 because s - d mu is.
    float mu, rest = 0.f;
    if constexpr (BF) {
      mu = total[0] / (float)d;
    } else {
      mu = (float)(total[0] * inv_d);
      rest = (float)(fma(-(double)mu, (double)d, total[0]) * inv_d);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float away = BF ? v[c][j] - mu : v[c][j] - mu - rest;
        v[c][j] = K::in((c * TPR + gl) * V, j, d) ? away : 0.f;
        s[0] = fmaf(v[c][j], v[c][j], s[0]);
      }
    var_sum(s);
    const float rs = 1.0f / sqrtf(s[0] / (float)d + eps);
    if (row < n) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = fmaf(v[c][j] * rs, wv[c][j], bv[c][j]);
        K::store(y, row, (c * TPR + gl) * V, d, o);
      }
      if (gl == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
      }
    }
  }
}

// Gradient: dx, and the block's partial dw and db in part[block][2][d].
constexpr int kGradThreads = 1024;

template <bool BF, bool TAIL, int C, int TPR>
__global__ __launch_bounds__(kGradThreads) void layer_norm_grad_kernel(
    const void *__restrict__ dy, const void *__restrict__ x, const float *__restrict__ w,
    const float *__restrict__ mean, const float *__restrict__ rstd, int n, int d,
    void *__restrict__ dx, float *__restrict__ part) {
  using K = Chunk<BF, TAIL>;
  constexpr int V = K::V, NT = kGradThreads, G = NT / TPR;
  __shared__ float s_buf[2][2][NT / 64];
  // Row groups' column sums: within a wave by lane permutations, then over WG
  // groups of TW threads in halves through LDS.
  constexpr int TW = TPR < 64 ? 64 : TPR, WG = NT / TW, COLS = TPR * C * V;
  __shared__ __attribute__((aligned(16))) float s_col[2][WG > 1 ? WG / 2 * COLS : 4];
  RowSum<float, TPR, NT, 2> row_sum(s_buf);
  const int grp = threadIdx.x / TPR, gl = threadIdx.x % TPR;
  const int stride = gridDim.x * G;
  const float inv_d = 1.0f / (float)d;
  // (w is read again for every row, from L1 or L2, where a thread's columns
  // are too many to keep beside their sums)
  constexpr bool kKeepW = C * V <= 8;
  float wv[C][V], dw[C][V] = {}, db[C][V] = {};
#pragma unroll
  for (int c = 0; c < C; ++c)
    if constexpr (kKeepW) load_columns<TAIL>(w, (c * TPR + gl) * V, d, wv[c]);
  K cx[C], cy[C];
  float mu = 0.f, rs = 0.f;
  auto load_row = [&](int row) {
    if (row < n) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        cx[c].load(x, row, (c * TPR + gl) * V, d);
        cy[c].load(dy, row, (c * TPR + gl) * V, d);
      }
      mu = mean[row];
      rs = rstd[row];
    }
  };
  load_row(blockIdx.x * G + grp);
  for (int base = blockIdx.x * G; base < n; base += stride) {
    const int row = base + grp;
    const bool live = row < n;
    float t[C][V], xh[C][V], s[2] = {0.f, 0.f};
    const float r = rs;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (!kKeepW) load_columns<TAIL>(w, (c * TPR + gl) * V, d, wv[c]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = live && K::in((c * TPR + gl) * V, j, d);
        const float g = in ? cy[c].get(j) : 0.f;
        xh[c][j] = in ? (cx[c].get(j) - mu) * r : 0.f;
        db[c][j] += g;
        dw[c][j] = fmaf(g, xh[c][j], dw[c][j]);
        t[c][j] = g * wv[c][j];
        s[0] += t[c][j];
        s[1] = fmaf(t[c][j], xh[c][j], s[1]);
      }
    }
    load_row(row + stride);
    row_sum(s);
    const float m1 = s[0] * inv_d, m2 = s[1] * inv_d;
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = r * (t[c][j] - m1 - xh[c][j] * m2);
        K::store(dx, row, (c * TPR + gl) * V, d, o);
      }
    }
  }
  if constexpr (TPR < 64)
#pragma unroll
    for (int off = TPR; off < 64; off *= 2)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dw[c][j] += __shfl_xor(dw[c][j], off);
          db[c][j] += __shfl_xor(db[c][j], off);
        }
  const int wg = threadIdx.x / TW;
  const bool mine = (int)threadIdx.x % TW < TPR;  // (below 64 threads a row: the wave's first group)
#pragma unroll
  for (int half = WG / 2; half > 0; half /= 2) {
    auto each = [&](int at, auto fn) {
      if (mine)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < V; j += 4) fn(c, j, at * COLS + (c * TPR + gl) * V + j);
    };
    if (wg >= half && wg < 2 * half)
      each(wg - half, [&](int c, int j, int i) {
        *(f32x4 *)&s_col[0][i] = f32x4{dw[c][j], dw[c][j + 1], dw[c][j + 2], dw[c][j + 3]};
        *(f32x4 *)&s_col[1][i] = f32x4{db[c][j], db[c][j + 1], db[c][j + 2], db[c][j + 3]};
      });
    __syncthreads();
    if (wg < half)
      each(wg, [&](int c, int j, int i) {
        const f32x4 p = *(const f32x4 *)&s_col[0][i], q = *(const f32x4 *)&s_col[1][i];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          dw[c][j + x] += p[x];
          db[c][j + x] += q[x];
        }
      });
    __syncthreads();
  }
  float *out = part + (size_t)blockIdx.x * 2 * d;
  if (wg == 0 && mine)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      store_columns<TAIL>(out, (c * TPR + gl) * V, d, dw[c]);
      store_columns<TAIL>(out + d, (c * TPR + gl) * V, d, db[c]);
    }
}

// dw | db [2 d] = the sum of P partial rows [P][2 d], in a fixed order: a
// block takes 64 columns, 16 threads of four columns for each of 64 slabs of
// the rows (slab s: rows s, s + 64, ...), then the slabs' sums in order.
__global__ __launch_bounds__(1024) void column_sum_kernel(const float *__restrict__ part, int P,
                                                          int d, float *__restrict__ dw,
                                                          float *__restrict__ db) {
  __shared__ __attribute__((aligned(16))) float s_p[64][64];
  __shared__ float s_q[4][64];
  const int tid = threadIdx.x, slab = tid >> 4, c4 = (tid & 15) * 4;
  const int base = blockIdx.x * 64, left = 2 * d - base - c4;  // columns from this thread's first on
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int p = slab; p < P; p += 64) {
    const float *q = part + (size_t)p * 2 * d + base + c4;
    if (left >= 4) {
      v += *(const f32x4_any *)q;
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < left) v[j] += q[j];
    }
  }
  *(f32x4 *)&s_p[slab][c4] = v;
  __syncthreads();
  const int col = tid & 63;
  if (tid < 256) {
    float a = 0.f;
    for (int i = 0; i < 16; ++i) a += s_p[(tid >> 6) * 16 + i][col];
    s_q[tid >> 6][col] = a;
  }
  __syncthreads();
  const int c = base + col;
  if (tid < 64 && c < 2 * d) {
    const float a = s_q[0][col] + s_q[1][col] + s_q[2][col] + s_q[3][col];
    if (c < d) {
      if (dw) dw[c] = a;
    } else if (db) {
      db[c - d] = a;
    }
  }
}

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

// Blocks of the gradient: one per CU (1024 threads, about 100 VGPRs each),
// fewer for few rows; each writes one partial row of 2 d floats.
int grad_blocks(int n) { return n < 256 ? n : 256; }

// Threads per CU of the forward pass: all that fit (8192 rows of 4096 bf16: 512
// threads 35.7, 1024 29.4, 2048 27.6 us; 8192 rows of 2880: 33.3, 26.0, 22.9).
constexpr int kRowThreads = 2048;

template <bool BF, bool TAIL>
hipError_t launch_fwd(const void *x, const float *w, const float *b, float eps, int n, int d, void *y,
                      float *mean, float *rstd, hipStream_t st) {
  return with_layout<BF, TAIL>(d, [&](auto cc, auto tt) {
    constexpr int C = decltype(cc)::value, TPR = decltype(tt)::value;
    constexpr int NT = TPR > 256 ? TPR : 256, G = NT / TPR;
    const int want = (n + G - 1) / G, cap = 256 * kRowThreads / NT;
    layer_norm_kernel<BF, TAIL, C, TPR><<<want < cap ? want : cap, NT, 0, st>>>(x, w, b, eps, n, d, y,
                                                                             mean, rstd);
    return hipGetLastError();
  });
}

template <bool BF, bool TAIL>
hipError_t launch_grad(const void *dy, const void *x, const float *w, const float *mean,
                       const float *rstd, int n, int d, void *dx, float *dw, float *db, float *part,
                       hipStream_t st) {
  int P = 0;
  const hipError_t e = with_layout<BF, TAIL>(d, [&](auto cc, auto tt) {
    constexpr int C = decltype(cc)::value, TPR = decltype(tt)::value;
    constexpr int G = kGradThreads / TPR;
    P = grad_blocks((n + G - 1) / G);
    if (P > 0)
      layer_norm_grad_kernel<BF, TAIL, C, TPR><<<P, kGradThreads, 0, st>>>(dy, x, w, mean, rstd, n, d, dx,
                                                                        part);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  if (!dw && !db) return hipSuccess;
  column_sum_kernel<<<(2 * d + 63) / 64, 1024, 0, st>>>(part, P, d, dw, db);
  return hipGetLastError();
}

}  // namespace

size_t layer_norm_grad_bytes(int n, int d) { return (size_t)grad_blocks(n) * 2 * d * sizeof(float); }

hipError_t launch_layer_norm(const void *x, bool bf16, const float *w, const float *b, float eps, int n,
                             int d, void *y, float *mean, float *rstd, hipStream_t st) {
  if (n == 0) return hipSuccess;
  if (bf16) return launch_fwd<true, false>(x, w, b, eps, n, d, y, mean, rstd, st);
  if (d % 4 == 0) return launch_fwd<false, false>(x, w, b, eps, n, d, y, mean, rstd, st);
  return launch_fwd<false, true>(x, w, b, eps, n, d, y, mean, rstd, st);
}

hipError_t launch_layer_norm_grad(const void *dy, const void *x, bool bf16, const float *w,
                                  const float *mean, const float *rstd, int n, int d, void *dx,
                                  float *dw, float *db, float *part, hipStream_t st) {
  if (bf16) return launch_grad<true, false>(dy, x, w, mean, rstd, n, d, dx, dw, db, part, st);
  if (d % 4 == 0) return launch_grad<false, false>(dy, x, w, mean, rstd, n, d, dx, dw, db, part, st);
  return launch_grad<false, true>(dy, x, w, mean, rstd, n, d, dx, dw, db, part, st);
}

}  // namespace moe
