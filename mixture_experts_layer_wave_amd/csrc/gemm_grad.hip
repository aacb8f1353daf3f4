// Grouped bf16 products of the expert FFN's gradient (gemm_grad.h has the
// formulas).
//
//   DH   dh0 = dy W2            rows x d_ff, K = d       (and the epilogue's dg, du, w h)
//   DX   da  = dg W1 + du W3    rows x d,    K = 2 d_ff  (two ranges of d_ff)
//   DW13 dW1 = dg^T a, dW3 = du^T a   d_ff x d, K = the pile's rows
//   DW2  dW2 = dy^T (w h)             d x d_ff, K = the pile's rows
//
// In the forward products both operands are contiguous along K.  Here the
// weights of DH and DX and both operands of the weight gradients are
// contiguous along the output's columns or rows instead: their tiles lie in
// LDS as they do in memory, K row by K row, and the MFMA fragments (eight
// consecutive K of one column per lane) are read with ds_read_b64_tr_b16,
// which transposes a 4 x 16 block of 16-bit values among 16 lanes.  No
// operand is ever transposed in memory.
//
// Block: 8 waves arranged 2 x 4, tile BM x BN, K steps of 64 through two LDS
// stages filled by direct-to-LDS copies, MFMA 32x32x16, f32 accumulators,
// the K loop rotated by one slice against its barriers as in the forward
// GEMM (gemm_big.hip).  Loads past a buffer's record count return zero:
// that fills ragged rows, columns and the K tail.
#include <atomic>

#include "common.h"
#include "gemm_common.h"
#include "gemm_grad.h"
#include "kernels.h"
#include "kmajor.h"

namespace moe {
namespace {

using namespace gemm;

constexpr int kBK = 64;

enum Mode { DH, DX, DW13, DW2 };

struct GradParams {
  const uint16_t *a0, *a1;  // DH dy; DX dg, du; DW13 dg, du; DW2 dy
  const uint16_t *b0, *b1;  // DH W2; DX W1, W3; DW13 a; DW2 w h
  uint32_t src_bytes;       // bytes of the gathered matrix (dy or a)
  const int32_t *perm;      // gather of dy / a, or NULL
  const int32_t *offsets;
  const int32_t *slot;
  int n_slots;
  int E, R, d, f;
  int n_mt, n_nt;           // tiles along the output's rows (weight gradients) and columns
  void *c0, *c1;            // DX da; DW13 dW1, dW3; DW2 dW2
  // DH epilogue
  const uint16_t *g, *u;
  uint16_t *dg, *du, *hs;
  float *part;
  const int32_t *inv;
  const float *topk_w;
  int k;
};

__device__ __forceinline__ void lgkm_wait0() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
}

// Combine weight of pile row r of token t: that of the pair whose row it is.
__device__ __forceinline__ float pair_weight(const int32_t *inv, const float *w, int k, int t, int r) {
  float v = 0.f;
  for (int j = 0; j < k; ++j)
    if (inv[(size_t)t * k + j] == r) v = w[(size_t)t * k + j];
  return v;
}

// DH epilogue.  Two runs of four columns of a row, held by lanes l and
// l + 32, are exchanged so that a lane has eight consecutive columns: g and u
// come and dg, du, w h go as 16-B pieces.  dh0, h and the products stay
// float32; dg, du and w h are rounded once to bf16, the type of the MFMA that
// reads them next.  The row sums of dh0 h over this wave's columns go to
// part[plane][row].
template <int TM, int TN, int WM, int WN>
__device__ __forceinline__ void store_dh(const f32x16 (&acc)[TM][TN], const GradParams &p,
                                         const float (&wrow)[TM], int row0, int rows, int n0, int nt,
                                         int wm, int wn) {
  const int lane = __lane_id(), lr = lane & 31, lg = lane >> 5;
  const int N = p.f;
  const size_t base = (size_t)row0 * N;
  const uint32_t bytes = (uint32_t)rows * (uint32_t)N * 2u;
  const __amdgpu_buffer_rsrc_t rg = rsrc(p.g + base, bytes), ru = rsrc(p.u + base, bytes);
  const __amdgpu_buffer_rsrc_t rdg = rsrc(p.dg + base, bytes), rdu = rsrc(p.du + base, bytes),
                               rhs = rsrc(p.hs + base, bytes);
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) {
    const int r = wm * WM + tm * 32 + lr;
    uint32_t off[TN][2];
    u32x4 gq[TN][2], uq[TN][2];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = n0 + wn * WN + j * 32 + 16 * h + lg * 8;
        off[j][h] = (r < rows && col < N) ? ((uint32_t)r * (uint32_t)N + (uint32_t)col) * 2u : kOOB;
        gq[j][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rg, off[j][h], 0, 0));
        uq[j][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ru, off[j][h], 0, 0));
      }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float dh[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto sw = __builtin_amdgcn_permlane32_swap(
              __float_as_uint(acc[tm][j][8 * h + i]), __float_as_uint(acc[tm][j][8 * h + 4 + i]), false,
              false);
          dh[i] = __uint_as_float(sw[0]);
          dh[4 + i] = __uint_as_float(sw[1]);
        }
        u32x4 odg, odu, ohs;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float dgv[2], duv[2], hv[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float g = __uint_as_float(b ? gq[j][h][q] & 0xffff0000u : gq[j][h][q] << 16);
            const float u = __uint_as_float(b ? uq[j][h][q] & 0xffff0000u : uq[j][h][q] << 16);
            const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
            const float a = g * s;  // silu(g)
            const float d0 = dh[2 * q + b];
            sum = fmaf(d0, a * u, sum);
            const float dw = d0 * wrow[tm];
            duv[b] = dw * a;
            dgv[b] = dw * u * fmaf(a, 1.0f - s, s);  // silu'(g) = s + g s (1 - s)
            hv[b] = wrow[tm] * (a * u);
          }
          odg[q] = pack_bf16x2(dgv[0], dgv[1]);
          odu[q] = pack_bf16x2(duv[0], duv[1]);
          ohs[q] = pack_bf16x2(hv[0], hv[1]);
        }
        __builtin_amdgcn_raw_buffer_store_b128(odg, rdg, off[j][h], 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(odu, rdu, off[j][h], 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(ohs, rhs, off[j][h], 0, 0);
      }
    sum += __shfl_xor(sum, 32, 64);
    if (p.part && lg == 0 && r < rows) p.part[(size_t)(nt * (kNW / 2) + wn) * p.R + row0 + r] = sum;
  }
}

template <Mode MODE, bool GATHER, int BM, int BN>
__global__ __launch_bounds__(kNT, 1) void grad_gemm_kernel(GradParams p) {
  constexpr bool WEIGHT = MODE == DW13 || MODE == DW2;  // A is K-major too
  constexpr int WM = BM / 2, WN = BN / (kNW / 2), TM = WM / 32, TN = WN / 32;
  constexpr int A_BYTES = BM * kBK * 2, B_BYTES = BN * kBK * 2, STAGE = A_BYTES + B_BYTES;
  constexpr int A_RUNS = A_BYTES / 1024 / kNW, B_RUNS = B_BYTES / 1024 / kNW;
  constexpr int SLICES = kBK / 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ TileSlot s_t;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = MODE == DH || MODE == DW2 ? p.f : p.d;  // output columns

  // ---- block -> tile ------------------------------------------------------
  int e, nt, m0, rows;  // output rows m0 .. m0 + rows (pile rows, or weight rows of the expert)
  int nk;               // K steps
  int kcount;           // K of one range
  bool second = false;  // DW13: the tile is dW3's
  int pile0 = 0;        // weight gradients: the pile's first row
  if constexpr (!WEIGHT) {
    if (wave == 0) map_block<BM, false, true>(p.offsets, p.E, p.n_nt, 1, lane, &s_t, 1, 4);
    __syncthreads();
    e = s_t.e;
    if (e < 0) return;
    nt = s_t.nt;
    m0 = s_t.row0;
    rows = s_t.rows;
    kcount = MODE == DH ? p.d : p.f;
    nk = (kcount + kBK - 1) / kBK * (MODE == DX ? 2 : 1);
  } else {
    // Every XCD (block b runs on XCD b mod 8) takes an eighth of each
    // expert's tiles, so that all have the same share of large and small
    // piles; within it, groups of eight row tiles column by column.
    const int T = p.n_mt * p.n_nt, per = (T + 7) / 8;
    const int slot = blockIdx.x >> 3;
    e = slot / per;
    const int tile = (blockIdx.x & 7) * per + slot % per;
    if (tile >= T) return;
    constexpr int RG = 8;
    const int grp = tile / (RG * p.n_nt), within = tile - grp * RG * p.n_nt;
    const int gr = min(RG, p.n_mt - grp * RG);
    nt = within / gr;
    int mt = grp * RG + within % gr;
    const int M = MODE == DW13 ? p.f : p.d;
    if (MODE == DW13 && mt >= p.n_mt / 2) {
      second = true;
      mt -= p.n_mt / 2;
    }
    m0 = mt * BM;
    rows = min(BM, M - m0);
    pile0 = p.offsets[e];
    kcount = p.offsets[e + 1] - pile0;
    nk = (kcount + kBK - 1) / kBK;
  }
  const int n0 = nt * BN;

  // ---- operands -------------------------------------------------------------
  const int lda = WEIGHT ? (MODE == DW13 ? p.f : p.d) : kcount;  // A's row pitch
  const int ldb = N;
  constexpr bool A_GATHER = GATHER && (MODE == DH || MODE == DW2);
  constexpr bool B_GATHER = GATHER && MODE == DW13;
  // A pile's rows start at m0 (row products) or pile0; gathered matrices are
  // addressed from their start.
  const size_t a_first = A_GATHER ? 0 : (size_t)(WEIGHT ? pile0 : m0) * lda;
  const uint32_t a_bytes = A_GATHER ? p.src_bytes : (uint32_t)(WEIGHT ? kcount : rows) * (uint32_t)lda * 2u;
  const uint16_t *a_base = (MODE == DW13 && second ? p.a1 : p.a0) + a_first;
  const __amdgpu_buffer_rsrc_t ra0 = rsrc(a_base, a_bytes);
  const __amdgpu_buffer_rsrc_t ra1 = MODE == DX ? rsrc(p.a1 + a_first, a_bytes) : ra0;
  size_t b_first;
  uint32_t b_bytes;
  if constexpr (!WEIGHT) {
    b_first = (size_t)phys_slot(p.slot, p.n_slots, e) * p.d * p.f;
    b_bytes = (uint32_t)p.d * (uint32_t)p.f * 2u;
  } else {
    b_first = B_GATHER ? 0 : (size_t)pile0 * ldb;
    b_bytes = B_GATHER ? p.src_bytes : (uint32_t)kcount * (uint32_t)ldb * 2u;
  }
  const __amdgpu_buffer_rsrc_t rb0 = rsrc(p.b0 + b_first, b_bytes);
  const __amdgpu_buffer_rsrc_t rb1 = MODE == DX ? rsrc(p.b1 + b_first, b_bytes) : rb0;

  // ---- per-lane copy offsets --------------------------------------------------
  // K-major tile of W columns: run q fills 1024 / (2 W) rows; lane i of run
  // kNW j + wave has row kr + j KROWS, stored chunk i % (W / 8).
  constexpr int A_CPR = BM / 8, B_CPR = BN / 8;             // chunks per K-major row
  constexpr int A_RPR = 64 / A_CPR, B_RPR = 64 / B_CPR;     // rows per run
  const int b_kr = wave * B_RPR + lane / B_CPR;
  const int b_col = n0 + (((lane % B_CPR) ^ kmaj_key<BN>(b_kr)) << 3);
  const uint32_t b_pen = b_col < N ? 0u : kOOB;
  const int a_kr = wave * A_RPR + lane / A_CPR;
  const int a_col = WEIGHT ? m0 + (((lane % A_CPR) ^ kmaj_key<BM>(a_kr)) << 3) : 0;
  const uint32_t a_pen = WEIGHT && a_col >= lda ? kOOB : 0u;
  static_assert((kNW * A_RPR) % 4 == 0 && (kNW * B_RPR) % 4 == 0, "a lane's key is the same in every run");
  // Row-major A tile (rows of 64 K, 128 B): as in the forward GEMM.
  const int c = dma_chunk<kBK * 2>(wave, lane);
  const int a_r = wave * 8 + lane / 8;
  uint32_t a_off[!WEIGHT ? A_RUNS : 1];
  if constexpr (!WEIGHT) {
    int src[A_RUNS];
#pragma unroll
    for (int j = 0; j < A_RUNS; ++j) {
      const int r = a_r + j * 64;
      src[j] = A_GATHER ? p.perm[m0 + min(r, rows - 1)] : r;
    }
#pragma unroll
    for (int j = 0; j < A_RUNS; ++j)
      a_off[j] = a_r + j * 64 < rows ? ((uint32_t)src[j] * (uint32_t)lda + (uint32_t)c * 8u) * 2u : kOOB;
  }
  // Gathered K-major operand: the token of each of this lane's K rows of the
  // next step, loaded one step ahead of the copies that use it.
  constexpr int K_RUNS = A_GATHER ? A_RUNS : B_RUNS;
  const int g_kr = A_GATHER ? a_kr : b_kr;
  constexpr int G_ROWS = kNW * (A_GATHER ? A_RPR : B_RPR);
  int tok[WEIGHT && GATHER ? K_RUNS : 1];
  auto load_tokens = [&](int kt) {
    if constexpr (WEIGHT && GATHER)
#pragma unroll
      for (int j = 0; j < K_RUNS; ++j)
        tok[j] = p.perm[pile0 + min(kt * kBK + g_kr + j * G_ROWS, kcount - 1)];
  };

  // Copies of K step kt into LDS stage `stage`; a step past the end copies zeros.
  const int nk_range = MODE == DX ? nk / 2 : nk;
  auto issue = [&](int kt, int stage) {
    const bool sec = MODE == DX && kt >= nk_range;
    const int k0 = (sec ? kt - nk_range : kt) * kBK;
    uint8_t *sa = smem + stage * STAGE, *sb = sa + A_BYTES;
    if constexpr (!WEIGHT) {
      const uint32_t pen = k0 + c * 8 < kcount ? 0u : kOOB;
#pragma unroll
      for (int j = 0; j < A_RUNS; ++j)
        dma16(sec ? ra1 : ra0, sa + (kNW * j + wave) * 1024, (a_off[j] + (uint32_t)k0 * 2u) | pen);
    } else {
#pragma unroll
      for (int j = 0; j < A_RUNS; ++j) {
        const int kr = k0 + a_kr + j * kNW * A_RPR;
        const uint32_t row = A_GATHER ? (uint32_t)tok[j] : (uint32_t)kr;
        const uint32_t pen = kr < kcount ? a_pen : kOOB;
        dma16(ra0, sa + (kNW * j + wave) * 1024, ((row * (uint32_t)lda + (uint32_t)a_col) * 2u) | pen);
      }
    }
#pragma unroll
    for (int j = 0; j < B_RUNS; ++j) {
      const int kr = k0 + b_kr + j * kNW * B_RPR;
      const uint32_t row = B_GATHER ? (uint32_t)tok[j] : (uint32_t)kr;
      const uint32_t pen = kr < kcount ? b_pen : kOOB;
      dma16(sec ? rb1 : rb0, sb + (kNW * j + wave) * 1024, ((row * (uint32_t)ldb + (uint32_t)b_col) * 2u) | pen);
    }
    load_tokens(kt + 1);
  };

  const int wm = wave / (kNW / 2), wn = wave % (kNW / 2);
  const int lr = lane & 31, lg = lane >> 5;
  f32x16 acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

  // Combine weights of this lane's rows (DH), looked up before the K loop.
  float wrow[TM];
  if constexpr (MODE == DH) {
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      wrow[tm] = 1.f;
      const int r = wm * WM + tm * 32 + lr;
      if (GATHER && r < rows) wrow[tm] = pair_weight(p.inv, p.topk_w, p.k, p.perm[m0 + r], m0 + r);
    }
  }

  int a_lane[WEIGHT ? TM : 1], b_lane[TN];
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) b_lane[tn] = kmaj_lane<BN>(wn * WN + tn * 32, lane);
  if constexpr (WEIGHT)
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) a_lane[tm] = kmaj_lane<BM>(wm * WM + tm * 32, lane);

  auto read_frags = [&](auto actc, const uint8_t *sa, int kk, bf16x8 *af, bf16x8 *bfr) {
    constexpr int ACT = decltype(actc)::value;
    const uint8_t *sb = sa + A_BYTES;
#pragma unroll
    for (int tm = 0; tm < ACT; ++tm) {
      if constexpr (WEIGHT)
        af[tm] = kmaj_frag<BM>(sa, a_lane[tm], kk);
      else
        af[tm] = *(const bf16x8 *)(sa + swz<kBK * 2>(wm * WM + tm * 32 + lr, kk * 2 + lg));
    }
    if constexpr (ACT > 0) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) bfr[tn] = kmaj_frag<BN>(sb, b_lane[tn], kk);
    }
  };
  auto mfmas = [&](auto actc, const bf16x8 *af, const bf16x8 *bfr) {
    constexpr int ACT = decltype(actc)::value;
#pragma unroll
    for (int tm = 0; tm < ACT; ++tm)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn)
        acc[tm][tn] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bfr[tn], af[tm], acc[tm][tn], 0, 0, 0);
  };

  auto kloop = [&](auto actc) {
    constexpr int ACT = decltype(actc)::value;
    constexpr int NF = ACT > 0 ? ACT * (WEIGHT ? 2 : 1) + TN * 2 : 0;  // LDS reads per slice
    constexpr int NM = ACT * TN;                                       // MFMAs per slice
    constexpr int RPM = NM > 0 ? (NF + NM - 1) / NM : 1;               // reads per MFMA
    wait_vmcnt<0>();
    __syncthreads();
    bf16x8 a0[TM], b0[TN], a1[TM], b1[TN];
    read_frags(actc, smem, 0, a0, b0);
    issue(1, 1);
    __builtin_amdgcn_sched_barrier(0);
    auto slices = [&](int st) {
      const uint8_t *sa = smem + st * STAGE;
#pragma unroll
      for (int kk = 0; kk + 1 < SLICES; ++kk) {
        bf16x8 *ac = (kk & 1) ? a1 : a0, *bc = (kk & 1) ? b1 : b0;
        bf16x8 *an = (kk & 1) ? a0 : a1, *bn = (kk & 1) ? b0 : b1;
        read_frags(actc, sa, kk + 1, an, bn);
        mfmas(actc, ac, bc);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (i * RPM < NF) __builtin_amdgcn_sched_group_barrier(0x100, RPM, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int kt = 0; kt + 1 < nk; ++kt) {
      const int st = kt & 1;
      slices(st);
      // This stage's copies have landed and the last slice's fragments are
      // in registers on every wave before anyone copies into it again.
      wait_vmcnt<0>();
      lgkm_wait0();
      __syncthreads();
      read_frags(actc, smem + (st ^ 1) * STAGE, 0, a0, b0);
      mfmas(actc, a1, b1);
#pragma unroll
      for (int i = 0; i < NF; ++i) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
      for (int i = 0; i < NM; ++i) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_barrier(0);
      issue(kt + 2, st);
    }
    slices((nk - 1) & 1);
    mfmas(actc, a1, b1);
  };
  if (nk > 0) {  // (an empty pile's weight gradients are zeros)
    load_tokens(0);
    issue(0, 0);
    const int act = __builtin_amdgcn_readfirstlane(min(TM, max(0, (rows - wm * WM + 31) / 32)));
    static_assert(TM == 2 || TM == 4, "row groups per wave");
    if (act == TM) {
      kloop(std::integral_constant<int, TM>{});
    } else if (act == 0) {
      kloop(std::integral_constant<int, 0>{});
    } else if (act == 1) {
      kloop(std::integral_constant<int, 1>{});
    } else if constexpr (TM == 4) {
      if (act == 2)
        kloop(std::integral_constant<int, 2>{});
      else
        kloop(std::integral_constant<int, 3>{});
    }
    wait_vmcnt<0>();
  }

  // ---- epilogue ---------------------------------------------------------------
  if constexpr (MODE == DH) {
    store_dh<TM, TN, WM, WN>(acc, p, wrow, m0, rows, n0, nt, wm, wn);
  } else {
    // da: the tile's pile rows; weight gradients: rows m0 .. of expert e
    uint16_t *out = (uint16_t *)(MODE == DW13 && second ? p.c1 : p.c0) +
                    (WEIGHT ? (size_t)e * p.d * p.f : (size_t)0) + (size_t)m0 * N;
    store_bf16_regs<TM, TN, WM, WN>(acc, rsrc(out, (uint32_t)rows * (uint32_t)N * 2u), N, rows, n0, wm, wn);
  }
}

template <Mode MODE, bool GATHER, int BM, int BN>
hipError_t launch(const GradParams &p, int blocks, hipStream_t st) {
  constexpr int lds = 2 * (BM + BN) * kBK * 2;
  auto kern = grad_gemm_kernel<MODE, GATHER, BM, BN>;
  static std::atomic<uint64_t> allowed{0};  // devices on which LDS above 64 KB is allowed
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    err = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (err != hipSuccess) return err;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  kern<<<blocks, kNT, lds, st>>>(p);
  return hipGetLastError();
}

template <Mode MODE, int BM, int BN>
hipError_t run(GradParams p, hipStream_t st) {
  const int N = MODE == DH || MODE == DW2 ? p.f : p.d;
  p.n_nt = (N + BN - 1) / BN;
  int blocks;
  if constexpr (MODE == DW13 || MODE == DW2) {
    const int M = MODE == DW13 ? p.f : p.d;
    p.n_mt = (M + BM - 1) / BM * (MODE == DW13 ? 2 : 1);
    blocks = p.E * 8 * ((p.n_mt * p.n_nt + 7) / 8);
  } else {
    blocks = ((p.R + BM - 1) / BM + (p.E < p.R ? p.E : p.R)) * p.n_nt;
  }
  if constexpr (MODE != DX)
    if (p.perm) return launch<MODE, true, BM, BN>(p, blocks, st);
  return launch<MODE, false, BM, BN>(p, blocks, st);
}

}  // namespace

int grad_planes_bf16(int d_ff) { return (d_ff + 255) / 256 * (kNW / 2); }

hipError_t launch_grad_bf16(const FfnGradArgs &a, const FfnGradWs &w, hipStream_t st) {
  GradParams b{};
  b.offsets = a.offsets;
  b.slot = a.slot;
  b.n_slots = a.n_slots;
  b.E = a.E;
  b.R = a.R;
  b.d = a.d;
  b.f = a.d_ff;
  b.src_bytes = (uint32_t)((size_t)(a.perm ? a.n : a.R) * a.d * 2);

  GradParams p = b;
  p.a0 = (const uint16_t *)a.dy;
  p.b0 = (const uint16_t *)a.w2;
  p.perm = a.perm;
  p.inv = a.inv;
  p.topk_w = a.topk_w;
  p.k = a.k;
  p.g = (const uint16_t *)a.g;
  p.u = (const uint16_t *)a.u;
  p.dg = (uint16_t *)w.dg;
  p.du = (uint16_t *)w.du;
  p.hs = (uint16_t *)w.hs;
  p.part = a.perm ? w.part : nullptr;
  hipError_t e = run<DH, 256, 256>(p, st);
  if (e != hipSuccess) return e;

  p = b;
  p.a0 = (const uint16_t *)w.dg;
  p.a1 = (const uint16_t *)w.du;
  p.b0 = (const uint16_t *)a.w1;
  p.b1 = (const uint16_t *)a.w3;
  p.c0 = a.da;
  e = run<DX, 256, 256>(p, st);
  if (e != hipSuccess) return e;

  p = b;
  p.a0 = (const uint16_t *)w.dg;
  p.a1 = (const uint16_t *)w.du;
  p.b0 = (const uint16_t *)a.a;
  p.perm = a.perm;
  p.c0 = a.dw1;
  p.c1 = a.dw3;
  e = run<DW13, 256, 256>(p, st);
  if (e != hipSuccess) return e;

  p = b;
  p.a0 = (const uint16_t *)a.dy;
  p.b0 = (const uint16_t *)w.hs;
  p.perm = a.perm;
  p.c0 = a.dw2;
  return run<DW2, 256, 256>(p, st);
}

}  // namespace moe
