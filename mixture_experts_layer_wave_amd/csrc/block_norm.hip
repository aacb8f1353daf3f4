// The norms before and after a block, with the block's gate and the residual's
// scale, and their gradient (moe_block_norm, moe_block_norm_backward).
//
//   h = a x + gate * post(z),  u = pre(h),   post, pre: a layer norm, an RMS norm
//   (layer norm without mean and bias), or nothing
//
// A norm's rows: xh = (v - mean) rstd, norm(v) = xh w + b, and for t = w dy
//   dv = rstd (t - avg(t) - xh avg(t xh))     (without avg(t) for an RMS norm)
//
// Gradient, with dh and du given:
//   D  = dh + pre'(du),  dx = a D,  dz = post'(gate D)
//   dw_pre = sum du hh,  db_pre = sum du,  dw_post = gate sum D zh,
//   db_post = gate sum D,  dgate = w_post sum D zh + b_post sum D
//   (sums over rows; without a norm behind it, dgate = sum D z)
//
// Both are bound by HBM: a row is read once and written once, and held in
// registers in between as in the layer norm (norm_dev.h).  The column sums are
// four, S1 = sum du hh, S2 = sum du, S3 = sum D zh, S4 = sum D: a thread adds its
// columns over the rows it meets, the block its row groups, and a second kernel
// the blocks, always in the same order.  u is taken from h before its rounding.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "norm_dev.h"

namespace moe {
namespace {

constexpr bool kNt = true;  // rows leave the caches to the parameters (8192 x 4096: forward 2 us less, gradient 105 -> 102)

enum { kNone = 0, kLayer = 1, kRms = 2 };

struct NormRef {
  int kind;
  float eps;
  const float *w, *b;
};

struct BlockNormParams {
  const void *x, *z, *dh, *du, *h_in;
  float scale;
  const float *gate;
  NormRef post, pre;
  void *h, *u, *dx, *dz;
  float *stats;  // [4][n]
  float *part;   // [blocks][4][d]
  int n, d;
};

// Mean (as value and rest, see norm.hip) and rstd of the rows held in v; v turns
// into the differences from the mean, 0 past the row's end.  Sum: what the mean's
// sum is taken in.  float does for values of bf16 precision, whose sums lose
// nothing where they lie close together; float32 values, which the norm in front
// gets in calls of either type, need double: with float a row of equal values
// near 1e4 came out 0.3 weight off its bias (8192 x 4096 bf16, two layer norms:
// 57.6 us with float for both, 60.5 so; eight values added in float before their
// conversion 59.6).
template <bool BF, bool TAIL, int TPR, class Sum, int C, int V, class Mean, class Var>
__device__ __forceinline__ void center(int kind, float eps, int d, int gl, float (&v)[C][V], Mean &mean_sum,
                                       Var &var_sum, float &mu, float &rs) {
  using K = Chunk<BF, TAIL>;
  constexpr bool kRest = std::is_same<Sum, double>::value;
  mu = 0.f;
  if (kind == kLayer) {
    Sum total[1] = {0};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) total[0] += (Sum)v[c][j];
    mean_sum(total);
    float rest = 0.f;
    if constexpr (!kRest) {
      mu = total[0] / (float)d;
    } else {
      const double inv_d = 1.0 / (double)d;
      mu = (float)(total[0] * inv_d);
      rest = (float)(fma(-(double)mu, (double)d, total[0]) * inv_d);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float away = kRest ? v[c][j] - mu - rest : v[c][j] - mu;
        v[c][j] = K::in((c * TPR + gl) * V, j, d) ? away : 0.f;
      }
  }
  float s[1] = {0.f};
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < V; ++j) s[0] = fmaf(v[c][j], v[c][j], s[0]);
  var_sum(s);
  rs = 1.0f / sqrtf(s[0] / (float)d + eps);
}

template <bool BF, bool TAIL, int C, int TPR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_kernel(BlockNormParams p) {
  using K = Chunk<BF, TAIL>;
  constexpr int V = K::V;
  constexpr int NT = TPR > 256 ? TPR : 256, G = NT / TPR;
  typedef typename std::conditional<BF, float, double>::type Sum;  // of z's mean; h's is double
  __shared__ Sum s_post[2][1][NT / 64];
  __shared__ double s_pre[2][1][NT / 64];
  __shared__ float s_var[2][1][NT / 64];
  RowSum<Sum, TPR, NT, 1> post_sum(s_post);
  RowSum<double, TPR, NT, 1> pre_sum(s_pre);
  RowSum<float, TPR, NT, 1> var_sum(s_var);
  const int n = p.n, d = p.d, grp = threadIdx.x / TPR, gl = threadIdx.x % TPR, stride = gridDim.x * G;
  const int post = p.post.kind, pre = p.pre.kind;
  K nx[C], nz[C];
  auto load_row = [&](int row) {
    if (row < n)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        nx[c].load(p.x, row, (c * TPR + gl) * V, d);
        nz[c].load(p.z, row, (c * TPR + gl) * V, d);
      }
  };
  load_row(blockIdx.x * G + grp);
  // h = scale x + (z or zh) a1 + a2
  float a1[C][V], a2[C][V] = {}, pw[C][V] = {}, pb[C][V] = {};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * TPR + gl) * V;
    float gt[V];
#pragma unroll
    for (int j = 0; j < V; ++j) a1[c][j] = gt[j] = 1.f;
    if (p.gate) load_columns<TAIL>(p.gate, col, d, gt);
    if (post) load_columns<TAIL>(p.post.w, col, d, a1[c]);
    if (post && p.post.b) load_columns<TAIL>(p.post.b, col, d, a2[c]);
#pragma unroll
    for (int j = 0; j < V; ++j) a1[c][j] *= gt[j], a2[c][j] *= gt[j];
    if (pre) load_columns<TAIL>(p.pre.w, col, d, pw[c]);
    if (pre && p.pre.b) load_columns<TAIL>(p.pre.b, col, d, pb[c]);
  }
  for (int base = blockIdx.x * G; base < n; base += stride) {
    const int row = base + grp;
    float v[C][V], xv[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j) v[c][j] = nz[c].get(j), xv[c][j] = nx[c].get(j);
    load_row(row + stride);  // runs under this row's sums
    float mu, rs = 1.f;
    if (post) {
      center<BF, TAIL, TPR, Sum>(post, p.post.eps, d, gl, v, post_sum, var_sum, mu, rs);
      if (row < n && gl == 0 && p.stats) {
        p.stats[row] = mu;
        p.stats[(size_t)n + row] = rs;
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float o = fmaf(v[c][j] * rs, a1[c][j], a2[c][j]);
        v[c][j] = K::in((c * TPR + gl) * V, j, d) ? fmaf(p.scale, xv[c][j], o) : 0.f;
      }
      if (row < n) K::template store<kNt>(p.h, row, (c * TPR + gl) * V, d, v[c]);
    }
    if (pre) {
      center<BF, TAIL, TPR, double>(pre, p.pre.eps, d, gl, v, pre_sum, var_sum, mu, rs);
      if (row < n) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float o[V];
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = fmaf(v[c][j] * rs, pw[c][j], pb[c][j]);
          K::template store<kNt>(p.u, row, (c * TPR + gl) * V, d, o);
        }
        if (gl == 0 && p.stats) {
          p.stats[2 * (size_t)n + row] = mu;
          p.stats[3 * (size_t)n + row] = rs;
        }
      }
    }
  }
}

constexpr int kGradThreads = 1024;  // of a gradient block

template <bool BF, bool TAIL, int C, int TPR>
__global__ __launch_bounds__(kGradThreads) void block_norm_grad_kernel(BlockNormParams p) {
  using K = Chunk<BF, TAIL>;
  constexpr int V = K::V, NT = kGradThreads, G = NT / TPR;
  __shared__ float s_buf[2][2][NT / 64];
  // Row groups' column sums: within a wave by lane permutations, then over WG
  // groups of TW threads in halves through LDS.
  constexpr int TW = TPR < 64 ? 64 : TPR, WG = NT / TW, COLS = TPR * C * V;
  __shared__ __attribute__((aligned(16))) float s_col[2][WG > 1 ? WG / 2 * COLS : 4];
  RowSum<float, TPR, NT, 2> row_sum(s_buf);
  const int n = p.n, d = p.d, grp = threadIdx.x / TPR, gl = threadIdx.x % TPR, stride = gridDim.x * G;
  const int post = p.post.kind, pre = p.pre.kind;
  const bool need_z = post || p.gate;
  const float inv_d = 1.0f / (float)d;
  float S[4][C][V] = {};
  K ch[C], cu[C], cz[C], cd[C];
  float m0 = 0.f, r0 = 1.f, m1 = 0.f, r1 = 1.f;
  auto load_row = [&](int row) {
    if (row < n) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * TPR + gl) * V;
        if (p.dh) cd[c].load(p.dh, row, col, d);
        if (pre) {
          cu[c].load(p.du, row, col, d);
          ch[c].load(p.h_in, row, col, d);
        }
        if (need_z) cz[c].load(p.z, row, col, d);
      }
      if (post) m0 = p.stats[row], r0 = p.stats[(size_t)n + row];
      if (pre) m1 = p.stats[2 * (size_t)n + row], r1 = p.stats[3 * (size_t)n + row];
    }
  };
  load_row(blockIdx.x * G + grp);
  for (int base = blockIdx.x * G; base < n; base += stride) {
    const int row = base + grp;
    const bool live = row < n;
    float D[C][V], t[C][V], xh[C][V];
    const float ra = r0, rb = r1, ma = m0, mb = m1;
    K z[C];
#pragma unroll
    for (int c = 0; c < C; ++c) z[c] = cz[c];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < V; ++j)
        D[c][j] = live && K::in((c * TPR + gl) * V, j, d) ? cd[c].get(j) : 0.f;  // 0 without dh
    if (pre) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float wv[V];
        load_columns<TAIL>(p.pre.w, (c * TPR + gl) * V, d, wv);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const bool in = live && K::in((c * TPR + gl) * V, j, d);
          const float g = in ? cu[c].get(j) : 0.f;
          xh[c][j] = in ? (ch[c].get(j) - mb) * rb : 0.f;
          S[0][c][j] = fmaf(g, xh[c][j], S[0][c][j]);
          S[1][c][j] += g;
          t[c][j] = g * wv[j];
          s[0] += t[c][j];
          s[1] = fmaf(t[c][j], xh[c][j], s[1]);
        }
      }
      row_sum(s);
      const float q1 = pre == kLayer ? s[0] * inv_d : 0.f, q2 = s[1] * inv_d;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < V; ++j)  // (past the row's end these stay out of every sum and store)
          D[c][j] = fmaf(rb, t[c][j] - q1 - xh[c][j] * q2, D[c][j]);
    }
    // the next row, under the rest of this one (asked for earlier, its registers do not
    // fit beside the first norm's)
    load_row(row + stride);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (live) {
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = p.scale * D[c][j];
        K::template store<kNt>(p.dx, row, (c * TPR + gl) * V, d, o);
      }
    // the block's side: t = gate D (w)
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * TPR + gl) * V;
      float gt[V], wv[V];
#pragma unroll
      for (int j = 0; j < V; ++j) gt[j] = wv[j] = 1.f;
      if (p.gate) load_columns<TAIL>(p.gate, col, d, gt);
      if (post) load_columns<TAIL>(p.post.w, col, d, wv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const bool in = live && K::in(col, j, d);
        const float Dj = in ? D[c][j] : 0.f;
        xh[c][j] = in ? (z[c].get(j) - ma) * ra : 0.f;
        S[2][c][j] = fmaf(Dj, xh[c][j], S[2][c][j]);
        S[3][c][j] += Dj;
        t[c][j] = Dj * gt[j] * wv[j];
        s[0] += t[c][j];
        s[1] = fmaf(t[c][j], xh[c][j], s[1]);
      }
    }
    float q1 = 0.f, q2 = 0.f;
    if (post) {
      row_sum(s);
      q1 = post == kLayer ? s[0] * inv_d : 0.f;
      q2 = s[1] * inv_d;
    }
    if (live) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = post ? ra * (t[c][j] - q1 - xh[c][j] * q2) : t[c][j];
        K::template store<kNt>(p.dz, row, (c * TPR + gl) * V, d, o);
      }
    }
  }
  if constexpr (TPR < 64)
#pragma unroll
    for (int off = TPR; off < 64; off *= 2)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < V; ++j) S[i][c][j] += __shfl_xor(S[i][c][j], off);
  const int wg = threadIdx.x / TW;
  const bool mine = (int)threadIdx.x % TW < TPR;  // (below 64 threads a row: the wave's first group)
#pragma unroll
  for (int half = WG / 2; half > 0; half /= 2) {
#pragma unroll
    for (int two = 0; two < 4; two += 2) {  // two sums at a time
      auto each = [&](int at, auto fn) {
        if (mine)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
              for (int j = 0; j < V; j += 4) fn(i, c, j, at * COLS + (c * TPR + gl) * V + j);
      };
      if (wg >= half && wg < 2 * half)
        each(wg - half, [&](int i, int c, int j, int at) {
          const float *v = &S[two + i][c][j];
          *(f32x4 *)&s_col[i][at] = f32x4{v[0], v[1], v[2], v[3]};
        });
      __syncthreads();
      if (wg < half)
        each(wg, [&](int i, int c, int j, int at) {
          const f32x4 q = *(const f32x4 *)&s_col[i][at];
#pragma unroll
          for (int y = 0; y < 4; ++y) S[two + i][c][j + y] += q[y];
        });
      __syncthreads();
    }
  }
  if (wg == 0 && mine)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)
        store_columns<TAIL>(p.part + ((size_t)blockIdx.x * 4 + i) * d, (c * TPR + gl) * V, d, S[i][c]);
}

// The parameters' gradients from P partial rows [P][4][d], in a fixed order: a
// block takes 16 columns of the four sums, 64 slabs of the rows by four threads
// of four columns each, then the slabs' sums in order.
__global__ __launch_bounds__(1024) void block_norm_sum_kernel(BlockNormParams p, int P, float *dgate, float *dpost_w,
                                                              float *dpost_b, float *dpre_w, float *dpre_b) {
  __shared__ __attribute__((aligned(16))) float s_p[64][64];
  __shared__ float s_q[4][64];
  __shared__ float s_s[4][16];
  const int d = p.d, tid = threadIdx.x, slab = tid >> 4, i = (tid >> 2) & 3, c4 = (tid & 3) * 4;
  const int base = blockIdx.x * 16, left = d - base - c4;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int b = slab; b < P; b += 64) {
    const float *q = p.part + ((size_t)b * 4 + i) * d + base + c4;
    if (left >= 4) {
      v += *(const f32x4_any *)q;
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j)
        if (j < left) v[j] += q[j];
    }
  }
  *(f32x4 *)&s_p[slab][i * 16 + c4] = v;
  __syncthreads();
  if (tid < 256) {
    float a = 0.f;
    for (int j = 0; j < 16; ++j) a += s_p[(tid >> 6) * 16 + j][tid & 63];
    s_q[tid >> 6][tid & 63] = a;
  }
  __syncthreads();
  if (tid < 64) s_s[tid >> 4][tid & 15] = s_q[0][tid] + s_q[1][tid] + s_q[2][tid] + s_q[3][tid];
  __syncthreads();
  const int c = base + tid;
  if (tid >= 16 || c >= d) return;
  const float S1 = s_s[0][tid], S2 = s_s[1][tid], S3 = s_s[2][tid], S4 = s_s[3][tid];
  if (p.pre.kind) {
    if (dpre_w) dpre_w[c] = S1;
    if (dpre_b) dpre_b[c] = S2;
  }
  const float gt = p.gate ? p.gate[c] : 1.f;
  if (p.post.kind) {
    if (dpost_w) dpost_w[c] = gt * S3;
    if (dpost_b) dpost_b[c] = gt * S4;
    if (dgate) dgate[c] = fmaf(p.post.w[c], S3, p.post.b ? p.post.b[c] * S4 : 0.f);
  } else if (dgate) {
    dgate[c] = S3;
  }
}

constexpr int kRowThreads = 2048;  // threads per CU of the forward pass

int grad_blocks(int rows) { return rows < 256 ? rows : 256; }

template <bool BF, bool TAIL>
hipError_t launch_fwd(const BlockNormParams &p, hipStream_t st) {
  return with_layout<BF, TAIL>(p.d, [&](auto cc, auto tt) {
    constexpr int C = decltype(cc)::value, TPR = decltype(tt)::value;
    constexpr int NT = TPR > 256 ? TPR : 256, G = NT / TPR;
    const int want = (p.n + G - 1) / G, cap = 256 * kRowThreads / NT;
    block_norm_kernel<BF, TAIL, C, TPR><<<want < cap ? want : cap, NT, 0, st>>>(p);
    return hipGetLastError();
  });
}

template <bool BF, bool TAIL>
hipError_t launch_grad(const BlockNormParams &p, int &P, hipStream_t st) {
  return with_layout<BF, TAIL>(p.d, [&](auto cc, auto tt) {
    constexpr int C = decltype(cc)::value, TPR = decltype(tt)::value;
    constexpr int G = kGradThreads / TPR;
    P = grad_blocks((p.n + G - 1) / G);
    if (P > 0) block_norm_grad_kernel<BF, TAIL, C, TPR><<<P, kGradThreads, 0, st>>>(p);
    return hipGetLastError();
  });
}

NormRef ref(const BlockNorm &a) { return NormRef{a.kind, a.eps, a.weight, a.bias}; }

}  // namespace

size_t block_norm_grad_bytes(int n, int d) { return (size_t)grad_blocks(n) * 4 * d * sizeof(float); }

hipError_t launch_block_norm(const BlockNormArgs &a, hipStream_t st) {
  if (a.n == 0) return hipSuccess;
  BlockNormParams p{};
  p.x = a.x;
  p.z = a.z;
  p.scale = a.scale;
  p.gate = a.gate;
  p.post = ref(a.post);
  p.pre = ref(a.pre);
  p.h = a.h;
  p.u = a.u;
  p.stats = a.stats;
  p.n = a.n;
  p.d = a.d;
  if (a.bf16) return launch_fwd<true, false>(p, st);
  if (a.d % 4 == 0) return launch_fwd<false, false>(p, st);
  return launch_fwd<false, true>(p, st);
}

hipError_t launch_block_norm_grad(const BlockNormArgs &a, hipStream_t st) {
  BlockNormParams p{};
  p.dh = a.dh;
  p.du = a.du;
  p.z = a.z;
  p.h_in = a.h;
  p.scale = a.scale;
  p.gate = a.gate;
  p.post = ref(a.post);
  p.pre = ref(a.pre);
  p.stats = a.stats;
  p.dx = a.dx;
  p.dz = a.dz;
  p.part = a.part;
  p.n = a.n;
  p.d = a.d;
  int P = 0;
  const hipError_t e = a.bf16 ? launch_grad<true, false>(p, P, st)
                              : (a.d % 4 == 0 ? launch_grad<false, false>(p, P, st) : launch_grad<false, true>(p, P, st));
  if (e != hipSuccess) return e;
  if (!a.dgate && !a.dpost_w && !a.dpost_b && !a.dpre_w && !a.dpre_b) return hipSuccess;
  block_norm_sum_kernel<<<(a.d + 15) / 16, 1024, 0, st>>>(p, P, a.dgate, a.dpost_w, a.dpost_b, a.dpre_w, a.dpre_b);
  return hipGetLastError();
}

}  // namespace moe
