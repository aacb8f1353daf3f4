// Grouped bf16 products of the expert FFN's gradient (gemm_grad.h has the
// formulas).
//
//   DH  dh0 = dy W2            rows x d_ff, K = d       (and the epilogue's dg, du, w h)
//   DX  da  = dg W1 + du W3    rows x d,    K = 2 d_ff  (two ranges of d_ff)
//   weight gradients  dW1 = dg^T a, dW3 = du^T a, dW2 = dy^T (w h),  K = the pile's rows
//
// In the forward products both operands are contiguous along K.  Here the
// weights of DH and DX and both operands of the weight gradients are
// contiguous along the output's columns or rows instead: their tiles lie in
// LDS as they do in memory, K row by K row, and the MFMA fragments (eight
// consecutive K of one column per lane) are read with ds_read_b64_tr_b16,
// which transposes a 4 x 16 block of 16-bit values among 16 lanes.  No
// operand is ever transposed in memory.
//
// Block: 8 waves arranged 2 x 4 (or 4 waves 2 x 2), K steps of 64 (32) through
// two LDS stages filled by direct-to-LDS copies, MFMA 32x32x16, f32
// accumulators, the K loop rotated by one slice against its barriers as in
// the forward GEMM (gemm_big.hip).  Loads past a buffer's record count return zero:
// that fills ragged rows, columns and the K tail.
//
// Measured (medians of profiled launches), 8 experts of 4096 x 14336 and 16384
// rows (11.5 Tflop): dh 2116 us, the rest 9106 us; within it da's blocks run at
// 1240 TFLOP/s and the weight tiles' loops at 1090 to 1200, where the power
// limit sets the clock (a large library product: 1222).  8 experts of 1024 x
// 4096, 4096 rows: 81 and 251 us (the whole pass 305 back to back).  128 experts
// of 2880 x 2880, 16384 skewed rows: 663 and 2896 us for 13 GB of weights,
// gradients and activations.
#include <atomic>
#include <type_traits>

#include "common.h"
#include "gemm_common.h"
#include "gemm_grad.h"
#include "kernels.h"
#include "kmajor.h"
#include "route_dev.h"

namespace moe {
namespace {

using namespace gemm;

enum Mode { DH, DX };

// The products over pile rows.
struct RowParams {
  const uint16_t *a0, *a1;  // DH dy; DX dg, du
  const uint16_t *b0, *b1;  // DH W2; DX W1, W3
  uint32_t src_bytes;       // bytes of the gathered matrix (dy)
  const int32_t *perm;      // gather of dy, or NULL
  const int32_t *offsets;
  const int32_t *slot;
  int n_slots;
  int E, R, d, f;
  int n_nt;                 // column tiles
  uint16_t *c;              // DX: da
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

// The weight gradients: dW1 = dg^T a and dW3 = du^T a (f x d), dW2 = dy^T hs
// (d x f), all sums over a pile's rows of a pile matrix (dg, du, hs: [R][f])
// and a gathered one (a, dy: d wide).
struct WeightParams {
  const uint16_t *pile[3], *src[3];  // dW1, dW3, dW2: pile matrix and gathered matrix
  uint16_t *out[3];
  uint32_t src_bytes;
  const int32_t *perm, *offsets;
  int E, d, f;
  int ft, dt;                        // tiles along f and d
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

// DH: g and u come and dg, du, w h go as such lines.  ALONE (one block per
// CU): g and u of a piece of the tile are on their way while the piece before
// it is worked on, the first one's before the barrier that frees the stages,
// and the stores carry the non-temporal hint (Mixtral-shaped, 8 experts, 4096
// x 14336, 16384 rows: 2240 -> 2133 us); blocks that share a CU overlap each
// other and keep the registers.  dh0, h and the products stay float32; dg, du
// and w h are rounded once to bf16, the type of the MFMA that reads them next:
// the gradients are then off by 2.3e-3 of themselves (root mean square, against
// 64 bits), where their own rounding to bf16 alone is 1.7e-3.
// The row sums of dh0 h over 64 columns go to part[column / 64][row].  s_w:
// combine weights of the tile's rows.
template <int TM, int TN, int WM, int WN, bool ALONE>
__device__ __forceinline__ void store_dh(const f32x16 (&acc)[TM][TN], const RowParams &p, const float *s_w,
                                         int row0, int rows, int n0, int wm, int wn, float *piece) {
  constexpr int NP = TM * (TN / 2);  // pieces of 32 rows x 64 columns
  const int lane = __lane_id();
  const int N = p.f;
  const size_t base = (size_t)row0 * N;
  const uint32_t bytes = (uint32_t)rows * (uint32_t)N * 2u;
  const __amdgpu_buffer_rsrc_t rg = rsrc(p.g + base, bytes), ru = rsrc(p.u + base, bytes);
  const __amdgpu_buffer_rsrc_t rdg = rsrc(p.dg + base, bytes), rdu = rsrc(p.du + base, bytes),
                               rhs = rsrc(p.hs + base, bytes);
  auto row_of = [&](int q, int i) { return wm * WM + q / (TN / 2) * 32 + 8 * i + (lane >> 3); };
  auto offset = [&](int q, int i) {
    const int r = row_of(q, i), col = n0 + wn * WN + q % (TN / 2) * 64 + (lane & 7) * 8;
    return (r < rows && col < N) ? ((uint32_t)r * (uint32_t)N + (uint32_t)col) * 2u : kOOB;
  };
  constexpr int NB = ALONE ? 2 : 1, AUX = ALONE ? 2 : 0;
  u32x4 gq[NB][4], uq[NB][4];
  auto load = [&](int q) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t off = offset(q, i);
      gq[q % NB][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rg, off, 0, 0));
      uq[q % NB][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ru, off, 0, 0));
    }
  };
  load(0);
  lds_barrier();  // every wave is done with the stages
#pragma unroll
  for (int q = 0; q < NP; ++q) {
    if (ALONE && q + 1 < NP) load(q + 1);
    if (!ALONE && q > 0) load(q);
    if constexpr (ALONE) __builtin_amdgcn_sched_barrier(0);
    epi_put<TM, TN>(acc, q / (TN / 2), q % (TN / 2), piece);
    const int c0 = n0 + wn * WN + q % (TN / 2) * 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row_of(q, i);
      const uint32_t off = offset(q, i);
      const float wr = s_w[r];
      float dh[8], sum = 0.f;
      epi_get(piece, i, dh);
      u32x4 odg, odu, ohs;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float dgv[2], duv[2], hv[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t gb = gq[q % NB][i][x], ub = uq[q % NB][i][x];
          const float g = __uint_as_float(b ? gb & 0xffff0000u : gb << 16);
          const float u = __uint_as_float(b ? ub & 0xffff0000u : ub << 16);
          const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
          const float a = g * s;  // silu(g)
          const float d0 = dh[2 * x + b];
          sum = fmaf(d0, a * u, sum);
          const float dw = d0 * wr;
          duv[b] = dw * a;
          dgv[b] = dw * u * fmaf(a, 1.0f - s, s);  // silu'(g) = s + g s (1 - s)
          hv[b] = wr * (a * u);
        }
        odg[x] = pack_bf16x2(dgv[0], dgv[1]);
        odu[x] = pack_bf16x2(duv[0], duv[1]);
        ohs[x] = pack_bf16x2(hv[0], hv[1]);
      }
      __builtin_amdgcn_raw_buffer_store_b128(odg, rdg, off, 0, AUX);
      __builtin_amdgcn_raw_buffer_store_b128(odu, rdu, off, 0, AUX);
      __builtin_amdgcn_raw_buffer_store_b128(ohs, rhs, off, 0, AUX);
      sum = group_sum(sum, 8);
      if (p.part && (lane & 7) == 0 && r < rows && c0 < N)
        p.part[(size_t)(c0 / 64) * p.R + row0 + r] = sum;
    }
  }
}

// A set of tiles: BM x BN of the products over pile rows, WB x WB of the
// weight gradients, waves per block, K step, waves per SIMD asked of the
// register allocator, and the blocks per CU that da's split K aims at.
template <int RBM_, int RBN_, int WB_, int NW_, int BK_, int OCC_, int HOLD_>
struct Cfg {
  static constexpr int RBM = RBM_, RBN = RBN_, WB = WB_, NW = NW_, BK = BK_, OCC = OCC_, HOLD = HOLD_;
  static constexpr int NT = NW * 64;
  static constexpr int max(int a, int b) { return a > b ? a : b; }
  // stages, or the epilogue's pieces
  static constexpr int EPI = NW * kEpiWave;
  static constexpr int ROW_LDS = max(2 * (RBM + RBN) * BK * 2, EPI);
  static constexpr int WEIGHT_LDS = max(4 * WB * BK * 2, EPI);
};

// fn(integral_constant<ACT>) for act = 0 .. TM, the number of this wave's
// 32-row groups that hold rows.
template <int TM, typename F>
__device__ __forceinline__ void by_act(int act, F fn) {
  static_assert(TM >= 2 && TM <= 5, "row groups per wave");
  if (act == TM) {
    fn(std::integral_constant<int, TM>{});
  } else if (act == 0) {
    fn(std::integral_constant<int, 0>{});
  } else if (act == 1) {
    fn(std::integral_constant<int, 1>{});
  } else if constexpr (TM >= 3) {
    if (act == 2) {
      fn(std::integral_constant<int, 2>{});
    } else if constexpr (TM >= 4) {
      if (act == 3) {
        fn(std::integral_constant<int, 3>{});
      } else if constexpr (TM >= 5) {
        fn(std::integral_constant<int, 4>{});
      }
    }
  }
}

// The K loop over nk > 0 steps, of which step 0's copies have been issued:
// issue(kt, stage) copies a step, read_frags reads a slice's fragments (READS
// LDS reads with ACT row groups), mfmas multiplies them.  Rotated by one slice
// against its barriers: the last slice's products run after the barrier that
// publishes the next stage, over that stage's first reads.
template <int ACT, int TM, int TN, int SLICES, int READS, typename Issue, typename Read, typename Mul>
__device__ __forceinline__ void k_loop(const uint8_t *smem, int stage_bytes, int nk, Issue issue, Read read_frags,
                                       Mul mfmas) {
  constexpr std::integral_constant<int, ACT> actc{};
  constexpr int NF = ACT > 0 ? READS : 0, NM = ACT * TN;    // LDS reads and MFMAs per slice
  constexpr int RPM = NM > 0 ? (NF + NM - 1) / NM : 1;      // reads per MFMA
  wait_vmcnt<0>();
  __syncthreads();
  bf16x8 a0[TM], b0[TN], a1[TM], b1[TN];
  read_frags(actc, smem, 0, a0, b0);
  issue(1, 1);
  __builtin_amdgcn_sched_barrier(0);
  auto slices = [&](int st) {
    const uint8_t *sa = smem + st * stage_bytes;
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
    // This stage's copies have landed and the last slice's fragments are in
    // registers on every wave before anyone copies into it again.
    wait_vmcnt<0>();
    lgkm_wait0();
    __syncthreads();
    read_frags(actc, smem + (st ^ 1) * stage_bytes, 0, a0, b0);
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
}

// One block's tile of DH or DX; `block` counts from the product's first block.
// s_w (DH): room for the combine weights of the tile's rows.
template <Mode MODE, bool GATHER, int BM, int BN, int NW, int BK>
__device__ __forceinline__ void row_tile(const RowParams &p, int block, uint8_t *smem, TileSlot &s_t,
                                         float *s_w = nullptr) {
  constexpr int WM = BM / 2, WN = BN / (NW / 2), TM = WM / 32, TN = WN / 32;
  constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE = A_BYTES + B_BYTES;
  constexpr int A_RUNS = A_BYTES / 1024 / NW, B_RUNS = B_BYTES / 1024 / NW;
  constexpr int SLICES = BK / 16;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = MODE == DH ? p.f : p.d;  // output columns

  // ---- block -> tile ------------------------------------------------------
  const int S = MODE == DX ? p.splits : 1;
  if (wave == 0) map_block<BM, false, true>(p.offsets, p.E, p.n_nt, S, lane, &s_t, S, 4, block);
  __syncthreads();
  const int e = s_t.e;
  if (e < 0) return;
  const int m0 = s_t.row0, rows = s_t.rows, n0 = s_t.nt * BN;
  const int kcount = MODE == DH ? p.d : p.f;  // K of one range
  int nk = (kcount + BK - 1) / BK * (MODE == DX ? 2 : 1);
  int kt0 = 0, split = 0;  // first step of this block's K range
  if (MODE == DX && S > 1) {
    split = s_t.split;
    kt0 = (int)((long long)split * nk / S);
    nk = (int)((long long)(split + 1) * nk / S) - kt0;
  }

  // ---- operands -------------------------------------------------------------
  constexpr bool A_GATHER = GATHER && MODE == DH;
  const size_t a_first = A_GATHER ? 0 : (size_t)m0 * kcount;
  const uint32_t a_bytes = A_GATHER ? p.src_bytes : (uint32_t)rows * (uint32_t)kcount * 2u;
  const __amdgpu_buffer_rsrc_t ra0 = rsrc(p.a0 + a_first, a_bytes);
  const __amdgpu_buffer_rsrc_t ra1 = MODE == DX ? rsrc(p.a1 + a_first, a_bytes) : ra0;
  const size_t b_first = (size_t)phys_slot(p.slot, p.n_slots, e) * p.d * p.f;
  const uint32_t b_bytes = (uint32_t)p.d * (uint32_t)p.f * 2u;
  const __amdgpu_buffer_rsrc_t rb0 = rsrc(p.b0 + b_first, b_bytes);
  const __amdgpu_buffer_rsrc_t rb1 = MODE == DX ? rsrc(p.b1 + b_first, b_bytes) : rb0;

  // ---- per-lane copy offsets --------------------------------------------------
  // K-major tile of W columns: run q fills 1024 / (2 W) rows; lane i of run
  // NW j + wave has row kr + j NW RPR, stored chunk i % (W / 8).
  constexpr int B_CPR = BN / 8, B_RPR = 64 / B_CPR;  // chunks per row, rows per run
  const int b_kr = wave * B_RPR + lane / B_CPR;
  const int b_col = n0 + (((lane % B_CPR) ^ kmaj_key<BN>(b_kr)) << 3);
  const uint32_t b_off = b_col < N ? ((uint32_t)b_kr * (uint32_t)N + (uint32_t)b_col) * 2u : kOOB;
  static_assert((NW * B_RPR) % 4 == 0, "a lane's key is the same in every run");
  // Row-major A tile: as in the forward GEMM.
  const int c = dma_chunk<BK * 2>(wave, lane);
  constexpr int RPR = 1024 / (BK * 2), RUN_ROWS = NW * RPR;  // rows of a run, and of all waves' runs
  const int a_r = wave * RPR + lane / (BK / 8);
  uint32_t a_off[A_RUNS];
  int src[A_RUNS];
#pragma unroll
  for (int j = 0; j < A_RUNS; ++j) {
    const int r = a_r + j * RUN_ROWS;
    src[j] = A_GATHER ? p.perm[m0 + min(r, rows - 1)] : r;
  }
#pragma unroll
  for (int j = 0; j < A_RUNS; ++j)
    a_off[j] = a_r + j * RUN_ROWS < rows ? ((uint32_t)src[j] * (uint32_t)kcount + (uint32_t)c * 8u) * 2u : kOOB;

  // Copies of K step kt into LDS stage `stage` (a step past the end is copied
  // and not used, or copies zeros).
  const int nk_range = (kcount + BK - 1) / BK;
  auto issue = [&](int kt, int stage) {
    const bool sec = MODE == DX && kt0 + kt >= nk_range;
    const int k0 = (kt0 + kt - (sec ? nk_range : 0)) * BK;
    uint8_t *sa = smem + stage * STAGE, *sb = sa + A_BYTES;
    const uint32_t pen = k0 + c * 8 < kcount ? 0u : kOOB;
#pragma unroll
    for (int j = 0; j < A_RUNS; ++j)
      dma16(sec ? ra1 : ra0, sa + (NW * j + wave) * 1024, (a_off[j] + (uint32_t)k0 * 2u) | pen);
#pragma unroll
    for (int j = 0; j < B_RUNS; ++j)  // (rows past K are past the buffer's end)
      dma16(sec ? rb1 : rb0, sb + (NW * j + wave) * 1024, b_off + (uint32_t)(k0 + j * NW * B_RPR) * ((uint32_t)N * 2u));
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

  int b_lane[TN];
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) b_lane[tn] = kmaj_lane<BN>(wn * WN + tn * 32, lane);

  auto read_frags = [&](auto actc, const uint8_t *sa, int kk, bf16x8 *af, bf16x8 *bfr) {
    constexpr int ACT = decltype(actc)::value;
    const uint8_t *sb = sa + A_BYTES;
#pragma unroll
    for (int tm = 0; tm < ACT; ++tm)
      af[tm] = *(const bf16x8 *)(sa + swz<BK * 2>(wm * WM + tm * 32 + lr, kk * 2 + lg));
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
    k_loop<ACT, TM, TN, SLICES, ACT + TN * 2>(smem, STAGE, nk, issue, read_frags, mfmas);
  };
  issue(0, 0);
  if constexpr (MODE == DH)  // the rows' combine weights, looked up under the first copies
    for (int r = tid; r < BM; r += NW * 64)
      s_w[r] = GATHER && r < rows ? pair_weight(p.inv, p.topk_w, p.k, p.perm[m0 + r], m0 + r) : 1.f;
  by_act<TM>(__builtin_amdgcn_readfirstlane(min(TM, max(0, (rows - wm * WM + 31) / 32))), kloop);
  wait_vmcnt<0>();

  // ---- epilogue ---------------------------------------------------------------
  float *piece = (float *)(smem + wave * kEpiWave);
  if constexpr (MODE == DH) {
    store_dh<TM, TN, WM, WN, NW == 8>(acc, p, s_w, m0, rows, n0, wm, wn, piece);
  } else {
    __syncthreads();  // every wave is done with the stages
    if (S > 1) {
      float *out = p.dx_part + ((size_t)split * p.R + m0) * N;
      store_lines_f32<TM, TN, WM, WN>(acc, rsrc(out, (uint32_t)rows * (uint32_t)N * 4u), N, rows, n0, wm, wn,
                                      piece);
    } else {
      uint16_t *out = p.c + (size_t)m0 * N;
      store_lines<TM, TN, WM, WN, 0>(acc, rsrc(out, (uint32_t)rows * (uint32_t)N * 2u), N, rows, n0, wm, wn,
                                     piece);
    }
  }
}

// ---- weight gradients ----------------------------------------------------------
// A tile is a 256 (128) column range of the pile matrix against one of the
// gathered matrix; dW1 and dW3 have the pile matrix's columns as their rows,
// dW2 the gathered one's, which is a choice of LDS regions, so one loop takes
// all three.
struct WeightTile {
  int e, which;       // 0 dW1, 1 dW3, 2 dW2
  int f0, d0;
  int pile0, kcount;  // the pile's rows
};

// The block's tile (false: none).  Every XCD (block b runs on XCD b mod 8)
// takes an eighth of each expert's tiles of dW1 and dW3, then of dW2, so that
// all have the same share of large and small piles; within an eighth, groups
// of eight row tiles column by column (dW2, whose row operand is the gathered
// one: four, 8 experts of 4096 x 14336 1% faster than with eight).
template <int B>
__device__ __forceinline__ bool weight_place(const WeightParams &p, int block, WeightTile &t) {
  const int T13 = 2 * p.ft * p.dt, T2 = p.ft * p.dt;
  const int per13 = (T13 + 7) / 8, per2 = (T2 + 7) / 8;
  int i = block >> 3;
  const bool w2 = i >= p.E * per13;
  if (w2) i -= p.E * per13;
  const int per = w2 ? per2 : per13, T = w2 ? T2 : T13;
  const int n_mt = w2 ? p.dt : 2 * p.ft, n_nt = w2 ? p.ft : p.dt;
  t.e = i / per;
  const int tile = (block & 7) * per + i % per;
  if (tile >= T) return false;
  const int RG = w2 ? 4 : 8;
  const int grp = tile / (RG * n_nt), within = tile - grp * RG * n_nt;
  const int gr = min(RG, n_mt - grp * RG);
  const int nt = within / gr;
  int mt = grp * RG + within % gr;
  t.which = w2 ? 2 : (mt >= p.ft ? 1 : 0);
  if (!w2 && mt >= p.ft) mt -= p.ft;
  t.f0 = (w2 ? nt : mt) * B;
  t.d0 = (w2 ? mt : nt) * B;
  t.pile0 = p.offsets[t.e];
  t.kcount = p.offsets[t.e + 1] - t.pile0;
  return true;
}

// `block` counts from the first of the weight gradients' blocks.  (Blocks that
// stay and take tiles from a queue per XCD, the next tile's first copies
// under this one's stores, were no faster on any of the measured shapes.)
template <bool GATHER, int B, int NW, int BK>
__device__ __forceinline__ void weight_tile(const WeightParams &p, int block, uint8_t *smem) {
  constexpr int WM = B / 2, WN = B / (NW / 2), TM = WM / 32, TN = WN / 32;
  constexpr int REGION = B * BK * 2, STAGE = 2 * REGION, RUNS = REGION / 1024 / NW, SLICES = BK / 16;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  WeightTile t;
  if (!weight_place<B>(p, block, t)) return;
  const bool w2 = t.which == 2;
  const int M = w2 ? p.d : p.f, N = w2 ? p.f : p.d, m0 = w2 ? t.d0 : t.f0, n0 = w2 ? t.f0 : t.d0;
  const int rows = min(B, M - m0), nk = (t.kcount + BK - 1) / BK;

  // Lane i of run NW j + wave of a region has K row kr + j KROWS, stored chunk
  // i % CPR.
  constexpr int CPR = B / 8, RPR = 64 / CPR, KROWS = NW * RPR;
  const int kr = wave * RPR + lane / CPR;
  const int chunk = ((lane % CPR) ^ kmaj_key<B>(kr)) << 3;
  static_assert(KROWS % 4 == 0, "a lane's key is the same in every run");

  // The token of each of this lane's K rows of the step to come, loaded one
  // step ahead of the copies that use it.
  int tok[RUNS];
  auto load_tokens = [&](int kt) {
    if constexpr (GATHER)
#pragma unroll
      for (int j = 0; j < RUNS; ++j)
        tok[j] = p.perm[t.pile0 + min(kt * BK + kr + j * KROWS, t.kcount - 1)];
  };
  // The tile's two operands and this lane's columns of them.
  const __amdgpu_buffer_rsrc_t rp =
      rsrc(p.pile[t.which] + (size_t)t.pile0 * p.f, (uint32_t)t.kcount * (uint32_t)p.f * 2u);
  const __amdgpu_buffer_rsrc_t rs = rsrc(p.src[t.which] + (GATHER ? (size_t)0 : (size_t)t.pile0 * p.d),
                                         GATHER ? p.src_bytes : (uint32_t)t.kcount * (uint32_t)p.d * 2u);
  const uint32_t foff = t.f0 + chunk < p.f ? ((uint32_t)kr * (uint32_t)p.f + (uint32_t)(t.f0 + chunk)) * 2u : kOOB;
  const uint32_t soff = t.d0 + chunk < p.d ? (GATHER ? (uint32_t)(t.d0 + chunk) * 2u
                                                     : ((uint32_t)kr * (uint32_t)p.d + (uint32_t)(t.d0 + chunk)) * 2u)
                                           : kOOB;
  // Copies of K step kt into LDS stage `stage`: the pile matrix's columns, then
  // the gathered one's.  Rows past the pile copy zeros: in order they are past
  // the buffer's end, gathered ones are sent there.  What an address owes to
  // the step and the run is the same for all lanes and added from a scalar.
  auto issue = [&](int kt, int stage) {
    uint8_t *s0 = smem + stage * STAGE;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const uint32_t k = (uint32_t)(kt * BK + j * KROWS);
      dma16(rp, s0 + (NW * j + wave) * 1024, foff + k * ((uint32_t)p.f * 2u));
      uint32_t off;
      if constexpr (GATHER)
        off = (int)k + kr < t.kcount ? (uint32_t)tok[j] * ((uint32_t)p.d * 2u) + soff : kOOB;
      else
        off = soff + k * ((uint32_t)p.d * 2u);
      dma16(rs, s0 + REGION + (NW * j + wave) * 1024, off);
    }
    load_tokens(kt + 1);
  };

  const int wm = wave / (NW / 2), wn = wave % (NW / 2);
  const int a_reg = w2 ? REGION : 0, b_reg = REGION - a_reg;
  int a_lane[TM], b_lane[TN];
#pragma unroll
  for (int tm = 0; tm < TM; ++tm) a_lane[tm] = a_reg + kmaj_lane<B>(wm * WM + tm * 32, lane);
#pragma unroll
  for (int tn = 0; tn < TN; ++tn) b_lane[tn] = b_reg + kmaj_lane<B>(wn * WN + tn * 32, lane);
  f32x16 acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
  auto read_frags = [&](auto actc, const uint8_t *st, int kk, bf16x8 *af, bf16x8 *bfr) {
    constexpr int ACT = decltype(actc)::value;
#pragma unroll
    for (int tm = 0; tm < ACT; ++tm) af[tm] = kmaj_frag<B>(st, a_lane[tm], kk);
    if constexpr (ACT > 0) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) bfr[tn] = kmaj_frag<B>(st, b_lane[tn], kk);
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
    k_loop<ACT, TM, TN, SLICES, ACT * 2 + TN * 2>(smem, STAGE, nk, issue, read_frags, mfmas);
  };
  if (nk > 0) {  // (an empty pile's weight gradients are zeros)
    load_tokens(0);
    issue(0, 0);
    by_act<TM>(__builtin_amdgcn_readfirstlane(min(TM, max(0, (rows - wm * WM + 31) / 32))), kloop);
    wait_vmcnt<0>();
  }
  __syncthreads();  // every wave is done with the stages
  uint16_t *out = p.out[t.which] + ((size_t)t.e * M + m0) * N;
  store_lines<TM, TN, WM, WN, 2>(acc, rsrc(out, (uint32_t)rows * (uint32_t)N * 2u), N, rows, n0, wm, wn,
                                 (float *)(smem + wave * kEpiWave));
}

// dg, du, w h: everything else waits for them.
template <bool GATHER, typename C>
__global__ __launch_bounds__(C::NT, C::OCC) void grad_dh_kernel(RowParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ TileSlot s_t;
  __shared__ float s_w[C::RBM];
  row_tile<DH, GATHER, C::RBM, C::RBN, C::NW, C::BK>(p, blockIdx.x, smem, s_t, s_w);
}

// The products that follow, in one grid: da's blocks (the longest) first, then
// the weight gradients', which fill the CUs that da's last, half-empty round
// of blocks leaves.
struct RestParams {
  RowParams dx;
  WeightParams dw;
  int end_dx;  // a multiple of 8 blocks
};

template <bool GATHER, typename C>
__global__ __launch_bounds__(C::NT, C::OCC) void grad_rest_kernel(RestParams q) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ TileSlot s_t;
  const int b = blockIdx.x;
  if (b < q.end_dx)
    row_tile<DX, false, C::RBM, C::RBN, C::NW, C::BK>(q.dx, b, smem, s_t);
  else
    weight_tile<GATHER, C::WB, C::NW, C::BK>(q.dw, b - q.end_dx, smem);
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

// Row tiles of the piles at most (one ragged tile per pile).
int row_tiles(int R, int E, int bm) { return tiles(R, bm) + (E < R ? E : R); }

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
hipError_t launch_both(RowParams dh, RestParams q, hipStream_t st) {
  auto k1 = grad_dh_kernel<GATHER, C>;
  auto k2 = grad_rest_kernel<GATHER, C>;
  constexpr int rest_lds = C::ROW_LDS > C::WEIGHT_LDS ? C::ROW_LDS : C::WEIGHT_LDS;
  static std::atomic<uint64_t> allowed1{0}, allowed2{0};
  hipError_t err = allow_lds(k1, C::ROW_LDS, allowed1);
  if (err == hipSuccess) err = allow_lds(k2, rest_lds, allowed2);
  if (err != hipSuccess) return err;
  const int rt = row_tiles(dh.R, dh.E, C::RBM);
  dh.n_nt = tiles(dh.f, C::RBN);
  k1<<<rt * dh.n_nt, C::NT, C::ROW_LDS, st>>>(dh);
  q.dx.n_nt = tiles(dh.d, C::RBN);
  q.end_dx = tiles(rt * q.dx.n_nt * q.dx.splits, 8) * 8;
  q.dw.ft = tiles(dh.f, C::WB);
  q.dw.dt = tiles(dh.d, C::WB);
  const int per_xcd = dh.E * (tiles(2 * q.dw.ft * q.dw.dt, 8) + tiles(q.dw.ft * q.dw.dt, 8));
  k2<<<q.end_dx + 8 * per_xcd, C::NT, rest_lds, st>>>(q);
  return hipGetLastError();
}

}  // namespace

namespace {

// One block of 8 waves per CU; or four blocks of 4 waves, which overlap each
// other's first loads and last stores but move 1.6 times the bytes through L2
// per product.
using Big = Cfg<320, 256, 256, 8, 64, 1, 1>;
using Small = Cfg<128, 128, 128, 4, 32, 4, 2>;

// Small tiles where blocks are short, few, or mostly padding (measured, Big
// against Small, us):
//   at most 144 rows per expert.  The piles' own sizes decide, which the host
//     does not know: with even piles Big is ahead from about 110 rows on, with
//     Zipf-skewed ones Small up to 250 and more.  At 144 either mistake costs
//     about as much:
//       128 experts, 2880 x 2880: even, 64 rows 3160 against 2890, 112 rows 3540
//         against 3600, 144 4050 against 4260, 208 4700 against 4960; skewed, 64
//         rows 2910 against 2560, 144 4290 against 3880, 208 5180 against 4910
//       64 experts, 2048 x 4096: even, 64 rows 1650 against 1580, 112 rows 1820
//         against 1920, 144 2030 against 2240; skewed, 144 rows 2160 against
//         1940, 256 3000 against 2790
//       128 experts, 2048 x 768: even, 80 rows 718 against 643, 112 rows 755
//         against 752, 144 823 against 857; skewed, 144 rows 842 against 774, 208
//         1041 against 959
//       8 experts, 1024 x 4096: even, 256 rows 206 against 233
//   the dh product under half a round of the CUs: 1 expert, 2048 x 8192, 500
//     tokens 168 against 154; 1024 tokens (160 blocks) 260 against 253
//   padding: d = 264, d_ff = 520, 8000 tokens 135 against 91.  Without padding
//     Small takes 1.2 times as long (8 experts, 4096 x 14336, 16384 rows: 11.7
//     against 14.1 ms).
bool use_small(const FfnGradArgs &a) {
  auto area = [&](int b) { return (double)(tiles(a.d, b) * b) * (tiles(a.d_ff, b) * b); };
  return a.R <= 144ll * a.E || row_tiles(a.R, a.E, Big::RBM) * tiles(a.d_ff, Big::RBN) < 128 ||
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
  RowParams p{};
  p.offsets = a.offsets;
  p.slot = a.slot;
  p.n_slots = a.n_slots;
  p.E = a.E;
  p.R = a.R;
  p.d = a.d;
  p.f = a.d_ff;
  p.src_bytes = (uint32_t)((size_t)(a.perm ? a.n : a.R) * a.d * 2);
  p.splits = 1;

  RestParams q{p, {}, 0};
  q.dx.a0 = (const uint16_t *)w.dg;
  q.dx.a1 = (const uint16_t *)w.du;
  q.dx.b0 = (const uint16_t *)a.w1;
  q.dx.b1 = (const uint16_t *)a.w3;
  q.dx.c = (uint16_t *)a.da;
  q.dx.splits = w.plan.dx_splits;
  q.dx.dx_part = w.dx_part;
  const void *pile[3] = {w.dg, w.du, w.hs}, *src[3] = {a.a, a.a, a.dy};
  void *out[3] = {a.dw1, a.dw3, a.dw2};
  for (int i = 0; i < 3; ++i) {
    q.dw.pile[i] = (const uint16_t *)pile[i];
    q.dw.src[i] = (const uint16_t *)src[i];
    q.dw.out[i] = (uint16_t *)out[i];
  }
  q.dw.src_bytes = p.src_bytes;
  q.dw.perm = a.perm;
  q.dw.offsets = a.offsets;
  q.dw.E = a.E;
  q.dw.d = a.d;
  q.dw.f = a.d_ff;

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
  if (use_small(a))
    return a.perm ? launch_both<true, Small>(p, q, st) : launch_both<false, Small>(p, q, st);
  return a.perm ? launch_both<true, Big>(p, q, st) : launch_both<false, Big>(p, q, st);
}

}  // namespace moe
