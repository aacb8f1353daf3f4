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
#include "route_dev.h"

namespace moe {
namespace {

using namespace gemm;

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
  // DX with few blocks: K in `splits` ranges, range s of every tile to the
  // float32 plane dx_part[s][R][d]; the planes are added later, in order.
  int splits;
  float *dx_part;
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

// Epilogues.  An accumulator holds runs of four columns of 32 rows; stored
// straight from registers a wave's instruction would touch 32 bytes of each
// of 32 rows.  Instead a wave passes 32 rows x 64 columns at a time through
// its own piece of LDS (float32, rows 272 bytes apart) and goes on with whole
// 128-byte lines: 8 lanes a row, eight consecutive columns each, 8 rows per
// instruction.
constexpr int kEpiPitch = 68;                      // floats per row
constexpr int kEpiWave = 32 * kEpiPitch * 4;       // bytes per wave

// Rows 32 tm .. and columns 64 jj .. of the wave's tile into its LDS piece.
template <int TM, int TN>
__device__ __forceinline__ void epi_put(const f32x16 (&acc)[TM][TN], int tm, int jj, float *piece) {
  const int lane = __lane_id(), lr = lane & 31, lg = lane >> 5;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *(f32x4 *)(piece + lr * kEpiPitch + j * 32 + g * 8 + lg * 4) =
          f32x4{acc[tm][2 * jj + j][g * 4], acc[tm][2 * jj + j][g * 4 + 1], acc[tm][2 * jj + j][g * 4 + 2],
                acc[tm][2 * jj + j][g * 4 + 3]};
}
// Eight columns of row 8 i + lane / 8 of the piece.
__device__ __forceinline__ void epi_get(const float *piece, int i, float (&v)[8]) {
  const int lane = __lane_id();
  const float *p = piece + (8 * i + (lane >> 3)) * kEpiPitch + (lane & 7) * 8;
  const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}

// bf16 rows [0, rows) of a tile in ro (row pitch N), each value rounded once.
// AUX: cache policy of the stores; 2 is the non-temporal hint, for the weight
// gradients, which nothing here reads again.
template <int TM, int TN, int WM, int WN, int AUX>
__device__ __forceinline__ void store_lines(const f32x16 (&acc)[TM][TN], __amdgpu_buffer_rsrc_t ro, int N,
                                            int rows, int n0, int wm, int wn, float *piece) {
  const int lane = __lane_id();
#pragma unroll
  for (int tm = 0; tm < TM; ++tm)
#pragma unroll
    for (int jj = 0; jj < TN / 2; ++jj) {
      epi_put<TM, TN>(acc, tm, jj, piece);
      const int col = n0 + wn * WN + jj * 64 + (lane & 7) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = wm * WM + tm * 32 + 8 * i + (lane >> 3);
        float v[8];
        epi_get(piece, i, v);
        const u32x4 o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7])};
        const uint32_t off =
            (r < rows && col < N) ? ((uint32_t)r * (uint32_t)N + (uint32_t)col) * 2u : kOOB;
        __builtin_amdgcn_raw_buffer_store_b128(o, ro, off, 0, AUX);
      }
    }
}

// float32 rows [0, rows) of a tile in ro (row pitch N floats).
template <int TM, int TN, int WM, int WN>
__device__ __forceinline__ void store_lines_f32(const f32x16 (&acc)[TM][TN], __amdgpu_buffer_rsrc_t ro, int N,
                                                int rows, int n0, int wm, int wn, float *piece) {
  const int lane = __lane_id();
#pragma unroll
  for (int tm = 0; tm < TM; ++tm)
#pragma unroll
    for (int jj = 0; jj < TN / 2; ++jj) {
      epi_put<TM, TN>(acc, tm, jj, piece);
      const int col = n0 + wn * WN + jj * 64 + (lane & 7) * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = wm * WM + tm * 32 + 8 * i + (lane >> 3);
        float v[8];
        epi_get(piece, i, v);
        const uint32_t off =
            (r < rows && col < N) ? ((uint32_t)r * (uint32_t)N + (uint32_t)col) * 4u : kOOB;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(u32x4, f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]}), ro,
              off + 16u * h, 0, 0);
      }
    }
}

// DH: g and u come and dg, du, w h go as such lines.  dh0, h and the products
// stay float32; dg, du and w h are rounded once to bf16, the type of the MFMA
// that reads them next.  The row sums of dh0 h over 64 columns go to
// part[column / 64][row].  s_w: combine weights of the tile's rows.
template <int TM, int TN, int WM, int WN>
__device__ __forceinline__ void store_dh(const f32x16 (&acc)[TM][TN], const GradParams &p, const float *s_w,
                                         int row0, int rows, int n0, int wm, int wn, float *piece) {
  const int lane = __lane_id();
  const int N = p.f;
  const size_t base = (size_t)row0 * N;
  const uint32_t bytes = (uint32_t)rows * (uint32_t)N * 2u;
  const __amdgpu_buffer_rsrc_t rg = rsrc(p.g + base, bytes), ru = rsrc(p.u + base, bytes);
  const __amdgpu_buffer_rsrc_t rdg = rsrc(p.dg + base, bytes), rdu = rsrc(p.du + base, bytes),
                               rhs = rsrc(p.hs + base, bytes);
#pragma unroll
  for (int tm = 0; tm < TM; ++tm)
#pragma unroll
    for (int jj = 0; jj < TN / 2; ++jj) {
      const int c0 = n0 + wn * WN + jj * 64, col = c0 + (lane & 7) * 8;
      uint32_t off[4];
      u32x4 gq[4], uq[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = wm * WM + tm * 32 + 8 * i + (lane >> 3);
        off[i] = (r < rows && col < N) ? ((uint32_t)r * (uint32_t)N + (uint32_t)col) * 2u : kOOB;
        gq[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rg, off[i], 0, 0));
        uq[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ru, off[i], 0, 0));
      }
      epi_put<TM, TN>(acc, tm, jj, piece);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = wm * WM + tm * 32 + 8 * i + (lane >> 3);
        const float wr = s_w[r];
        float dh[8], sum = 0.f;
        epi_get(piece, i, dh);
        u32x4 odg, odu, ohs;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float dgv[2], duv[2], hv[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float g = __uint_as_float(b ? gq[i][q] & 0xffff0000u : gq[i][q] << 16);
            const float u = __uint_as_float(b ? uq[i][q] & 0xffff0000u : uq[i][q] << 16);
            const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
            const float a = g * s;  // silu(g)
            const float d0 = dh[2 * q + b];
            sum = fmaf(d0, a * u, sum);
            const float dw = d0 * wr;
            duv[b] = dw * a;
            dgv[b] = dw * u * fmaf(a, 1.0f - s, s);  // silu'(g) = s + g s (1 - s)
            hv[b] = wr * (a * u);
          }
          odg[q] = pack_bf16x2(dgv[0], dgv[1]);
          odu[q] = pack_bf16x2(duv[0], duv[1]);
          ohs[q] = pack_bf16x2(hv[0], hv[1]);
        }
        __builtin_amdgcn_raw_buffer_store_b128(odg, rdg, off[i], 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(odu, rdu, off[i], 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(ohs, rhs, off[i], 0, 0);
        sum = group_sum(sum, 8);
        if (p.part && (lane & 7) == 0 && r < rows && c0 < N)
          p.part[(size_t)(c0 / 64) * p.R + row0 + r] = sum;
      }
    }
}

// A set of tiles: BM x BN of the products over pile rows and of the weight
// gradients, waves per block, K step, waves per SIMD asked of the register
// allocator, and the blocks per CU that da's split K aims at.
template <int RBM_, int RBN_, int WBM_, int WBN_, int NW_, int BK_, int OCC_, int HOLD_>
struct Cfg {
  static constexpr int RBM = RBM_, RBN = RBN_, WBM = WBM_, WBN = WBN_, NW = NW_, BK = BK_, OCC = OCC_;
  static constexpr int HOLD = HOLD_;
  static constexpr int NT = NW * 64;
  static constexpr int max(int a, int b) { return a > b ? a : b; }
  // stages, or the epilogue's pieces (and the rows' combine weights)
  static constexpr int EPI = NW * kEpiWave + RBM * 4;
  static constexpr int ROW_LDS = max(2 * (RBM + RBN) * BK * 2, EPI);
  static constexpr int WEIGHT_LDS = max(2 * (WBM + WBN) * BK * 2, EPI);
};

// One block's tile; `block` counts from the product's first block.
template <Mode MODE, bool GATHER, int BM, int BN, int NW, int BK>
__device__ __forceinline__ void grad_tile(const GradParams &p, int block, uint8_t *smem, TileSlot &s_t) {
  constexpr bool WEIGHT = MODE == DW13 || MODE == DW2;  // A is K-major too
  constexpr int WM = BM / 2, WN = BN / (NW / 2), TM = WM / 32, TN = WN / 32;
  constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE = A_BYTES + B_BYTES;
  constexpr int A_RUNS = A_BYTES / 1024 / NW, B_RUNS = B_BYTES / 1024 / NW;
  constexpr int SLICES = BK / 16;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = MODE == DH || MODE == DW2 ? p.f : p.d;  // output columns

  // ---- block -> tile ------------------------------------------------------
  int e, nt, m0, rows;  // output rows m0 .. m0 + rows (pile rows, or weight rows of the expert)
  int nk;               // K steps
  int kcount;           // K of one range
  int kt0 = 0;          // first step of this block's K range (DX)
  int split = 0;
  bool second = false;  // DW13: the tile is dW3's
  int pile0 = 0;        // weight gradients: the pile's first row
  if constexpr (!WEIGHT) {
    const int S = MODE == DX ? p.splits : 1;
    if (wave == 0) map_block<BM, false, true>(p.offsets, p.E, p.n_nt, S, lane, &s_t, S, 4);
    __syncthreads();
    e = s_t.e;
    if (e < 0) return;
    nt = s_t.nt;
    m0 = s_t.row0;
    rows = s_t.rows;
    kcount = MODE == DH ? p.d : p.f;
    nk = (kcount + BK - 1) / BK * (MODE == DX ? 2 : 1);
    if (MODE == DX && S > 1) {
      split = s_t.split;
      kt0 = (int)((long long)split * nk / S);
      nk = (int)((long long)(split + 1) * nk / S) - kt0;
    }
  } else {
    // Every XCD (block b runs on XCD b mod 8) takes an eighth of each
    // expert's tiles, so that all have the same share of large and small
    // piles; within it, groups of eight row tiles column by column.
    const int T = p.n_mt * p.n_nt, per = (T + 7) / 8;
    const int slot = block >> 3;
    e = slot / per;
    const int tile = (block & 7) * per + slot % per;
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
    nk = (kcount + BK - 1) / BK;
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
  // NW j + wave has row kr + j KROWS, stored chunk i % (W / 8).
  constexpr int A_CPR = WEIGHT ? BM / 8 : 8, B_CPR = BN / 8;  // chunks per K-major row
  constexpr int A_RPR = 64 / A_CPR, B_RPR = 64 / B_CPR;     // rows per run
  const int b_kr = wave * B_RPR + lane / B_CPR;
  const int b_col = n0 + (((lane % B_CPR) ^ kmaj_key<BN>(b_kr)) << 3);
  const uint32_t b_pen = b_col < N ? 0u : kOOB;
  const int a_kr = wave * A_RPR + lane / A_CPR;
  int a_col = 0;
  if constexpr (WEIGHT) a_col = m0 + (((lane % A_CPR) ^ kmaj_key<BM>(a_kr)) << 3);
  const uint32_t a_pen = WEIGHT && a_col >= lda ? kOOB : 0u;
  static_assert((NW * A_RPR) % 4 == 0 && (NW * B_RPR) % 4 == 0, "a lane's key is the same in every run");
  // Row-major A tile: as in the forward GEMM.
  const int c = dma_chunk<BK * 2>(wave, lane);
  constexpr int RPR = 1024 / (BK * 2), RUN_ROWS = NW * RPR;  // rows of a run, and of all waves' runs
  const int a_r = wave * RPR + lane / (BK / 8);
  uint32_t a_off[!WEIGHT ? A_RUNS : 1];
  if constexpr (!WEIGHT) {
    int src[A_RUNS];
#pragma unroll
    for (int j = 0; j < A_RUNS; ++j) {
      const int r = a_r + j * RUN_ROWS;
      src[j] = A_GATHER ? p.perm[m0 + min(r, rows - 1)] : r;
    }
#pragma unroll
    for (int j = 0; j < A_RUNS; ++j)
      a_off[j] = a_r + j * RUN_ROWS < rows ? ((uint32_t)src[j] * (uint32_t)lda + (uint32_t)c * 8u) * 2u : kOOB;
  }
  // Gathered K-major operand: the token of each of this lane's K rows of the
  // next step, loaded one step ahead of the copies that use it.
  constexpr int K_RUNS = A_GATHER ? A_RUNS : B_RUNS;
  const int g_kr = A_GATHER ? a_kr : b_kr;
  constexpr int G_ROWS = NW * (A_GATHER ? A_RPR : B_RPR);
  int tok[WEIGHT && GATHER ? K_RUNS : 1];
  auto load_tokens = [&](int kt) {
    if constexpr (WEIGHT && GATHER)
#pragma unroll
      for (int j = 0; j < K_RUNS; ++j)
        tok[j] = p.perm[pile0 + min(kt * BK + g_kr + j * G_ROWS, kcount - 1)];
  };

  // Copies of K step kt into LDS stage `stage` (a step past the end is copied
  // and not used, or copies zeros).
  const int nk_range = (kcount + BK - 1) / BK;
  auto issue = [&](int kt, int stage) {
    const bool sec = MODE == DX && kt0 + kt >= nk_range;
    const int k0 = (kt0 + kt - (sec ? nk_range : 0)) * BK;
    uint8_t *sa = smem + stage * STAGE, *sb = sa + A_BYTES;
    if constexpr (!WEIGHT) {
      const uint32_t pen = k0 + c * 8 < kcount ? 0u : kOOB;
#pragma unroll
      for (int j = 0; j < A_RUNS; ++j)
        dma16(sec ? ra1 : ra0, sa + (NW * j + wave) * 1024, (a_off[j] + (uint32_t)k0 * 2u) | pen);
    } else {
#pragma unroll
      for (int j = 0; j < A_RUNS; ++j) {
        const int kr = k0 + a_kr + j * NW * A_RPR;
        const uint32_t row = A_GATHER ? (uint32_t)tok[j] : (uint32_t)kr;
        const uint32_t pen = kr < kcount ? a_pen : kOOB;
        dma16(ra0, sa + (NW * j + wave) * 1024, ((row * (uint32_t)lda + (uint32_t)a_col) * 2u) | pen);
      }
    }
#pragma unroll
    for (int j = 0; j < B_RUNS; ++j) {
      const int kr = k0 + b_kr + j * NW * B_RPR;
      const uint32_t row = B_GATHER ? (uint32_t)tok[j] : (uint32_t)kr;
      const uint32_t pen = kr < kcount ? b_pen : kOOB;
      dma16(sec ? rb1 : rb0, sb + (NW * j + wave) * 1024, ((row * (uint32_t)ldb + (uint32_t)b_col) * 2u) | pen);
    }
    load_tokens(kt + 1);
  };

  const int wm = wave / (NW / 2), wn = wave % (NW / 2);
  const int lr = lane & 31, lg = lane >> 5;
  f32x16 acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

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
        af[tm] = *(const bf16x8 *)(sa + swz<BK * 2>(wm * WM + tm * 32 + lr, kk * 2 + lg));
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
    static_assert(TM >= 2 && TM <= 5, "row groups per wave");
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
    } else if constexpr (TM == 5) {
      if (act == 2)
        kloop(std::integral_constant<int, 2>{});
      else if (act == 3)
        kloop(std::integral_constant<int, 3>{});
      else
        kloop(std::integral_constant<int, 4>{});
    }
    wait_vmcnt<0>();
  }

  // ---- epilogue ---------------------------------------------------------------
  __syncthreads();  // every wave is done with the stages
  float *piece = (float *)(smem + wave * kEpiWave);
  if constexpr (MODE == DH) {
    float *s_w = (float *)(smem + NW * kEpiWave);
    for (int r = tid; r < BM; r += NW * 64)
      s_w[r] = GATHER && r < rows ? pair_weight(p.inv, p.topk_w, p.k, p.perm[m0 + r], m0 + r) : 1.f;
    __syncthreads();
    store_dh<TM, TN, WM, WN>(acc, p, s_w, m0, rows, n0, wm, wn, piece);
  } else if (MODE == DX && p.splits > 1) {
    float *out = p.dx_part + ((size_t)split * p.R + m0) * N;
    store_lines_f32<TM, TN, WM, WN>(acc, rsrc(out, (uint32_t)rows * (uint32_t)N * 4u), N, rows, n0, wm, wn,
                                    piece);
  } else {
    // da: the tile's pile rows; weight gradients: rows m0 .. of expert e
    uint16_t *out = (uint16_t *)(MODE == DW13 && second ? p.c1 : p.c0) +
                    (WEIGHT ? (size_t)e * p.d * p.f : (size_t)0) + (size_t)m0 * N;
    store_lines<TM, TN, WM, WN, WEIGHT ? 2 : 0>(acc, rsrc(out, (uint32_t)rows * (uint32_t)N * 2u), N, rows, n0,
                                                wm, wn, piece);
  }
}

// dg, du, w h: everything else waits for them.
template <bool GATHER, typename C>
__global__ __launch_bounds__(C::NT, C::OCC) void grad_dh_kernel(GradParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ TileSlot s_t;
  grad_tile<DH, GATHER, C::RBM, C::RBN, C::NW, C::BK>(p, blockIdx.x, smem, s_t);
}

// The products that follow, in one grid: da's blocks (the longest) first,
// then dW1 and dW3, then dW2, so that a product's last, half-empty round of
// blocks is filled by the next product's.
struct RestParams {
  GradParams dx, dw13, dw2;
  int end_dx, end_dw13, end_dw2;  // block ranges, multiples of 8
};

template <bool GATHER, typename C>
__global__ __launch_bounds__(C::NT, C::OCC) void grad_rest_kernel(RestParams q) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ TileSlot s_t;
  const int b = blockIdx.x;
  if (b < q.end_dx)
    grad_tile<DX, false, C::RBM, C::RBN, C::NW, C::BK>(q.dx, b, smem, s_t);
  else if (b < q.end_dw13)
    grad_tile<DW13, GATHER, C::WBM, C::WBN, C::NW, C::BK>(q.dw13, b - q.end_dx, smem, s_t);
  else
    grad_tile<DW2, GATHER, C::WBM, C::WBN, C::NW, C::BK>(q.dw2, b - q.end_dw13, smem, s_t);
}

// Dynamic LDS above 64 KB must be allowed once per device and kernel.
template <typename Kern>
hipError_t allow_lds(Kern kern, int lds, std::atomic<uint64_t> &done) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(done.load(std::memory_order_acquire) & bit)) {
    err = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (err != hipSuccess) return err;
    done.fetch_or(bit, std::memory_order_release);
  }
  return hipSuccess;
}

int tiles(int v, int b) { return (v + b - 1) / b; }

// Row tiles of the piles at most (one ragged tile per pile), and blocks of a
// weight gradient (E experts, each an eighth of its tiles per XCD).
int row_tiles(int R, int E, int bm) { return tiles(R, bm) + (E < R ? E : R); }
int weight_blocks(const GradParams &p) { return p.E * 8 * tiles(p.n_mt * p.n_nt, 8); }

// K ranges of da's product: its K is 2 d_ff, so with few row tiles its blocks
// would outlast everything that runs beside them.  With fewer blocks than
// HOLD per CU, K is split until there are as many, each range 512 deep at
// least (Switch-shaped, 8 tokens: 165 -> 71 us; 4096 tokens: 347 -> 311).
template <typename C>
int dx_splits(int R, int E, int d, int f) {
  const int blocks = row_tiles(R, E, C::RBM) * tiles(d, C::RBN), hold = 256 * C::HOLD;
  int S = blocks < hold ? hold / blocks : 1;
  if (S > 2 * f / 512) S = 2 * f / 512;
  return S < 1 ? 1 : S;
}

template <bool GATHER, typename C>
hipError_t launch_both(GradParams dh, RestParams q, hipStream_t st) {
  auto k1 = grad_dh_kernel<GATHER, C>;
  auto k2 = grad_rest_kernel<GATHER, C>;
  constexpr int rest_lds = C::ROW_LDS > C::WEIGHT_LDS ? C::ROW_LDS : C::WEIGHT_LDS;
  static std::atomic<uint64_t> allowed1{0}, allowed2{0};
  hipError_t err = allow_lds(k1, C::ROW_LDS, allowed1);
  if (err == hipSuccess) err = allow_lds(k2, rest_lds, allowed2);
  if (err != hipSuccess) return err;
  const int f = dh.f, d = dh.d;
  dh.n_nt = tiles(f, C::RBN);
  q.dx.n_nt = tiles(d, C::RBN);
  q.dw13.n_mt = 2 * tiles(f, C::WBM);
  q.dw13.n_nt = tiles(d, C::WBN);
  q.dw2.n_mt = tiles(d, C::WBM);
  q.dw2.n_nt = tiles(f, C::WBN);
  const int rt = row_tiles(dh.R, dh.E, C::RBM);
  k1<<<rt * dh.n_nt, C::NT, C::ROW_LDS, st>>>(dh);
  q.end_dx = tiles(rt * q.dx.n_nt * q.dx.splits, 8) * 8;
  q.end_dw13 = q.end_dx + weight_blocks(q.dw13);
  q.end_dw2 = q.end_dw13 + weight_blocks(q.dw2);
  k2<<<q.end_dw2, C::NT, rest_lds, st>>>(q);
  return hipGetLastError();
}

}  // namespace

namespace {

// One block of 8 waves per CU; or four blocks of 4 waves, which overlap each
// other's first loads and last stores but move 1.6 times the bytes through L2
// per product.
using Big = Cfg<320, 256, 256, 256, 8, 64, 1, 1>;
using Small = Cfg<128, 128, 128, 128, 4, 32, 4, 2>;

// Small tiles where blocks are short, few, or mostly padding (measured, Big
// against Small, us):
//   at most 128 rows per expert: 128 experts, d = d_ff = 2880, 256 tokens top-4
//     2838 against 2154, 4096 tokens Zipf-skewed 4237 against 3642 (uniform
//     3843 against 4039); at 256 rows (8 experts, 1024 x 4096) 199 against 234
//   the dh product under half a round of the CUs: 1 expert, 2048 x 8192, 500
//     tokens 168 against 155; 1024 tokens (160 blocks) 268 against 260
//   padding: d = 264, d_ff = 520, 8000 tokens 116 against 88.  Without padding
//     Small takes 1.2 times as long (Mixtral-shaped 11.7 against 14.1 ms).
bool use_small(const FfnGradArgs &a) {
  auto area = [&](int b) { return (double)(tiles(a.d, b) * b) * (tiles(a.d_ff, b) * b); };
  return a.R <= 128ll * a.E || row_tiles(a.R, a.E, Big::RBM) * tiles(a.d_ff, Big::RBN) < 128 ||
         1.2 * area(128) < area(256);
}

}  // namespace

GradPlan grad_plan_bf16(const FfnGradArgs &a) {
  GradPlan p{};
  p.dw_planes = tiles(a.d_ff, 64);
  p.dx_splits = use_small(a) ? dx_splits<Small>(a.R, a.E, a.d, a.d_ff) : dx_splits<Big>(a.R, a.E, a.d, a.d_ff);
  return p;
}

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
  b.splits = 1;

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

  RestParams q{b, b, b, 0, 0, 0};
  q.dx.a0 = q.dw13.a0 = (const uint16_t *)w.dg;
  q.dx.a1 = q.dw13.a1 = (const uint16_t *)w.du;
  q.dx.b0 = (const uint16_t *)a.w1;
  q.dx.b1 = (const uint16_t *)a.w3;
  q.dx.c0 = a.da;
  q.dx.splits = w.plan.dx_splits;
  q.dx.dx_part = w.dx_part;
  q.dw13.b0 = (const uint16_t *)a.a;
  q.dw13.perm = q.dw2.perm = a.perm;
  q.dw13.c0 = a.dw1;
  q.dw13.c1 = a.dw3;
  q.dw2.a0 = (const uint16_t *)a.dy;
  q.dw2.b0 = (const uint16_t *)w.hs;
  q.dw2.c0 = a.dw2;
  if (use_small(a))
    return a.perm ? launch_both<true, Small>(p, q, st) : launch_both<false, Small>(p, q, st);
  return a.perm ? launch_both<true, Big>(p, q, st) : launch_both<false, Big>(p, q, st);
}

}  // namespace moe
