// Product with an MXFP4 matrix (moe_mxfp4_linear): y = x W^T + bias, x in bf16 or
// MXFP4.
//
// Few rows (linear_rows_kernel) are bound by reading W: the weight rows go straight
// into the matrix cores (wave_stream.h).  A workgroup takes an equal run of output
// columns in tiles of at most 16; its waves share out the tiles and, where there are
// fewer tiles than waves, a tile's K steps, whose sums meet in LDS.  One row, 4096 ->
// 14336, takes 8.9 us, 31 MB at 3.5 TB/s (at a large copy's rate 6.0); 2880 -> 2880 5.1,
// near a launch.  8 waves: with 16 the one row took 9.1 and 12 rows 17.9 instead of 11.9,
// as their exchange buffers left no room for the rows.
// Many rows (linear_gemm_kernel) are a GEMM, from 17 on, where the rows' second group of 16
// would read W again (us, rows kernel / GEMM): 4096 -> 14336 16 rows 19.9 / 21.6, 17 30.6 /
// 21.7, 32 37.7 / 22.7; MXFP4 rows with their encoding 16 13.2 / 17.2, 17 15.6 / 17.4, 32 18.5 /
// 17.6.  Narrow matrices would be better off later: 2880 -> 2880 16 rows 8.0 / 12.2, 17
// 11.7 / 12.4, 32 14.3 / 12.9, 1024 -> 4096 17 rows 6.3 / 11.9, 32 6.6 / 12.2.
#include <algorithm>
#include <atomic>

#include "common.h"
#include "gemm_common.h"
#include "kernels.h"
#include "wave_stream.h"

namespace moe {
namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kRows = 16;  // the M of the MFMA
// x lies in LDS where it fits, else its pieces come from memory with each chunk (12 rows
// of 4096 11.9 us, 16 rows 20.0).
constexpr int kRowsLds = 160 * 1024 - kWaves * kExchange;
constexpr int kRowsMany = 16;  // rows above which the GEMM takes over (see above)
constexpr int kLargeTiles = 150;  // 256 x 256 tiles from which they are taken
constexpr int kBlocks = 256;       // blocks of one round: the device's CUs
constexpr int kSplitSteps = 11;    // K steps that a plane has at least
constexpr int kShort = 48;         // K steps up to which three groups share a tile (see LinearPlan)

struct LinearParams {
  const uint8_t *x, *xs, *w, *ws;
  const float *bias;
  void *y;
  int n, d, m, out_bf16;
  int G;  // workgroups of one group of 16 rows
};

__device__ __forceinline__ void put(const LinearParams &p, int t, int c, float v) {
  if (p.bias) v += p.bias[c];
  const size_t at = (size_t)t * p.m + c;
  if (p.out_bf16)
    ((uint16_t *)p.y)[at] = (uint16_t)f32_to_bf16_bits(v);
  else
    ((float *)p.y)[at] = v;
}

// XL: the rows of x fit LDS.
template <int WT, bool XL, bool NARROW, int PC>
__global__ __launch_bounds__(kThreads) void linear_rows_kernel(LinearParams p) {
  using F = Form<WT>;
  constexpr int NF = F::kActBytes / 16, RC = kRowChunk<WT>, SL = (RC - 16) / 16;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_x[];
  __shared__ __attribute__((aligned(16))) uint8_t s_ex[kWaves][kExchange];  // later the waves' sums
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = blockIdx.x % p.G, t0 = blockIdx.x / p.G * kRows, rows = min(kRows, p.n - t0);
  const int d = p.d, m = p.m;
  const int c_lo = (int)((long long)m * part / p.G), c_hi = (int)((long long)m * (part + 1) / p.G);
  const int cols = c_hi - c_lo, tiles = (cols + 15) / 16;
  int KS = kWaves;  // waves on one tile
  while (KS > 1 && tiles > kWaves / KS) KS >>= 1;
  const int mine = wave / KS, step = kWaves / KS, kp = wave % KS;  // this wave's tiles: mine, mine + step, ..
  const int C = (F::blocks(d) + kChunkBlocks - 1) / kChunkBlocks, k_lo = C * kp / KS, k_hi = C * (kp + 1) / KS;
  const int segs = tiles > mine ? (tiles - mine + step - 1) / step : 0;
  const size_t xb = WT == kMx4 ? (size_t)d / 2 : (size_t)d * 2;
  auto col = [&](int tile) { return c_lo + (int)((long long)cols * tile / max(tiles, 1)); };
  const int tok = min(r, rows - 1);
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  // (KS > 1: a wave has one tile at most, and its part k_lo .. k_hi - 1 of the chunks)
  stream<WT, PC, NARROW>(
      C, d, s_ex[wave],
      [&](int i, Segment &w) {
        if (i >= segs || k_lo == k_hi) return false;
        const int tile = mine + i * step, c = col(tile);
        rows_of_one<WT>(w, p.w, p.ws, c, col(tile + 1) - c, d);
        w.first = k_lo;
        w.count = k_hi - k_lo;
        return true;
      },
      [&] {  // the first weights are on their way
        if constexpr (XL) {
          for (int i = tid / SL; i < rows * C; i += kThreads / SL) {
            const int c = i / rows, t = i - c * rows;
            stage_row_chunk<WT>(s_x + i * RC, p.x + (t0 + t) * xb, c, d, tid % SL);
          }
          lds_barrier();
        }
      },
      [&](int, int &c, int &left) {
        c = k_lo;
        left = k_hi - k_lo;
      },
      [&](int, int c, int b, u32x4 (&a)[NF], uint32_t &as) {
        if constexpr (XL) {
          const uint8_t *px = s_x + (c * rows + tok) * RC + b * F::kActBytes;
#pragma unroll
          for (int q = 0; q < NF; ++q) a[q] = *(const u32x4 *)(px + q * 16);
        } else {
          load_block<WT>(p.x + (t0 + tok) * xb, c * kChunkBlocks + b, d, a);
        }
        if constexpr (WT == kMx4) as = p.xs[(size_t)(t0 + tok) * (d / 32) + min(c * kChunkBlocks + b, d / 32 - 1)];
      },
      [&](int i, f32x4 v) {
        if (KS > 1) {
          sum = v;
          return;
        }
        const int tile = mine + i * step, c = col(tile), cnt = col(tile + 1) - c;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r < cnt && 4 * g + q < rows) put(p, t0 + 4 * g + q, c + r, v[q]);
      });
  if (KS == 1) return;
  *(f32x4 *)(s_ex[wave] + lane * 16) = sum;
  __syncthreads();
  if (kp == 0 && segs > 0) {
    const int c = col(mine), cnt = col(mine + 1) - c;
    for (int j = 1; j < KS; ++j) sum += *(const f32x4 *)(s_ex[wave + j] + lane * 16);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (r < cnt && 4 * g + q < rows) put(p, t0 + 4 * g + q, c + r, sum[q]);
  }
}

template <int WT, bool XL, bool NARROW, int PC>
hipError_t launch_rows(const LinearParams &p, hipStream_t st) {
  auto kern = linear_rows_kernel<WT, XL, NARROW, PC>;
  int lds = 0;
  if constexpr (XL) {
    lds = std::min(kRows, p.n) * ((Form<WT>::blocks(p.d) + kChunkBlocks - 1) / kChunkBlocks) * kRowChunk<WT>;
    // The LDS limit is raised once per device (a per-device kernel attribute).
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load(std::memory_order_acquire) & bit)) {
      err = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, kRowsLds);
      if (err != hipSuccess) return err;
      attr_done.fetch_or(bit, std::memory_order_release);
    }
  }
  kern<<<p.G * ((p.n + kRows - 1) / kRows), kThreads, lds, st>>>(p);
  return hipGetLastError();
}

template <int WT>
bool rows_fit(int n, int d) {
  return (long long)std::min(kRows, n) * ((Form<WT>::blocks(d) + kChunkBlocks - 1) / kChunkBlocks) * kRowChunk<WT> <=
         kRowsLds;
}

// ---- many rows --------------------------------------------------------------------
// y = x W^T with x's rows as the second and W's as the first operand of 32 x 32 MFMAs.
// A block takes BM rows of x by BN rows of W through two LDS stages filled by direct
// copies, 16-byte chunks swizzled by row.  A step is 128 bytes of a row of x, in four
// slices:
//   bf16 rows (MX = false): 64 elements.  Lane half h of a wave converts W's block h of
//     the step (v_cvt_scalef32_pk_bf16_fp4), whose elements 8 s .. are slice s's, and
//     takes x's elements 32 h + 8 s .. to match.  W's codes of a step are 32 bytes a row;
//     they come four steps at a time, a quarter of the rows with each step: copies of
//     whole 128 bytes (32 at a time 8192 x 4096 -> 14336 took 831 us, so 821).  The scale
//     is one byte a lane and step, straight from memory.
//   MXFP4 rows: 256 elements, both operands in their stored form on the scaled MFMA.
//     A step's scales are eight bytes a row, laid out step by step by a kernel in front
//     (as stored they start at any byte); slice s of lane half h takes byte 4 h + s.
// With 256 x 256 tiles a block takes several, one behind the other, and the next one's
// first copies are under way during the stores (8192 x 4096 -> 14336 829 -> 809 us, MXFP4
// rows with their encoding 294 -> 286).
// What bounds it: 8192 x 4096 -> 14336 takes 801 to 821 us (1.17 to 1.20 PFLOP/s) with bf16
// rows, where a large bf16 product of the vendor's library takes 738 and a loop of MFMAs on registers
// reaches 2.28; with MXFP4 rows 260 us (3.7 PFLOP/s; 283 to 285 with their encoding), of
// which the scales take 5, the stores about 50, and the loop runs at 4.7 of 9.5 PFLOP/s: its
// LDS traffic, 267 KB a step at 128 bytes a clock, takes as long as its products.  Neither a
// third and fourth stage, nor four waves of 128 x 128 (a third fewer LDS reads), nor the
// rotation below changed the loop's rate.
struct GemmParams {
  const uint8_t *a, *b;      // [n] rows of rb bytes, [m] rows of d / 2
  const uint8_t *as, *bs;    // MX: [steps][np], [steps][mp] x 8 scales; else bs [m][d / 32]
  const float *bias;
  void *y;                   // [n][m], or with splits > 1 the planes [splits][n][mp4]
  int n, m, d, rb, steps, np, mp, out_bf16;
  int rt, ct;                // row and column tiles
  int splits, per;           // K splits, steps of each
};

typedef u32x4 u32x4_any2 __attribute__((aligned(2)));

// Eight columns of a row of y from element `at` on, of which `left` are inside the row.
__device__ __forceinline__ void store_columns8(char *y, size_t at, int left, bool half, const float (&o)[8]) {
  if (left >= 8) {
    if (half) {
      *(u32x4_any2 *)((uint16_t *)y + at) = u32x4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                                                  pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
    } else {
      *(f32x4_any *)((float *)y + at) = f32x4{o[0], o[1], o[2], o[3]};
      *(f32x4_any *)((float *)y + at + 4) = f32x4{o[4], o[5], o[6], o[7]};
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (e < left) {
      if (half)
        ((uint16_t *)y)[at + e] = (uint16_t)f32_to_bf16_bits(o[e]);
      else
        ((float *)y)[at + e] = o[e];
    }
}

constexpr int kRowGroup = 4;  // row tiles that blocks running together share

// b a + c of 64 MXFP4 elements, byte S of each scale.
template <int S>
__device__ __forceinline__ f32x16 scaled(v8i b, v8i a, f32x16 c, uint32_t bs, uint32_t as) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 4, 4, S, (int)bs, S, (int)as);
}

template <bool MX, int BM, int BN, int NW, int KG, bool MANY>
struct GemmTile {
  static constexpr int WN_ = NW / 2, WM = BM / 2, WN = BN / WN_, TM = WM / 32, TN = WN / 32;
  // a stage: x's rows, and with MX W's rows and the scales; else W's rows lie four steps
  // at a time in two buffers of their own behind the two stages
  static constexpr int A = BM * 128, B = BN * 128, S = MX ? (BM + BN) * 8 : 0;
  static constexpr int STAGE = A + (MX ? B + S : 0), W = 2 * STAGE;
  // the epilogue's pieces of 32 x 64, a wave each: over the stages; with MANY in what the
  // next tile's first copies leave free: with MX stage 1, else stage 1 and W's buffer 1.
  // Rows 16 bytes apart from each other's banks: by their pitch, or where there is no
  // room for that by a swizzle.
  static constexpr int PITCH = MX ? 272 : 256, PIECE = 32 * PITCH, PIECES = NW * PIECE;
  static constexpr int ALL = 2 * STAGE + (MX ? 0 : 2 * B), LDS = KG * ALL;
  static_assert(WN % 64 == 0 && (!MANY ? PIECES <= ALL : MX ? PIECES <= STAGE : PIECES / 2 <= A && PIECES / 2 <= B),
                "the pieces fit");
  __device__ static int at(int row, int chunk) { return row * PITCH + ((MX ? chunk : chunk ^ (row & 15)) << 4); }
  static_assert(A / 1024 % NW == 0 && B / 1024 % NW == 0, "whole copies a wave");
};

// KG: groups of NW waves in a block, each with stages of its own and every KG-th part of
// the block's K range; the groups' products meet in LDS in front of the stores.
template <bool MX, int BM, int BN, int NW, int KG, bool MANY>
__global__ __launch_bounds__(NW * KG * 64, 1) void linear_gemm_kernel(GemmParams p) {
  using T = GemmTile<MX, BM, BN, NW, KG, MANY>;
  static_assert(KG == 1 || !MANY, "groups: a tile a block");
  using namespace gemm;
  extern __shared__ __attribute__((aligned(16))) uint8_t all_smem[];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lg = lane >> 5;
  const int id = __builtin_amdgcn_readfirstlane(tid >> 6), wave = id % NW, group = id / NW;
  uint8_t *smem = all_smem + group * T::ALL;
  // Block -> tile: an eighth of the list to each XCD; groups of kRowGroup row tiles,
  // column tile by column tile within a group.
  const int total = p.rt * p.ct * p.splits, xcd = blockIdx.x & 7, stride = gridDim.x >> 3;
  int base = 0, slot = blockIdx.x >> 3;
  for (int x = 0; x < xcd; ++x) base += (total - x + 7) >> 3;
  const int slots = (total - xcd + 7) >> 3;
  if (slot >= slots) return;

  // Copies: run q of wave w is the 1 KB of rows 8 (NW q + w) .. + 7, lane l's chunk l % 8.
  const uint32_t wb = (uint32_t)p.d / 2;  // bytes of a row of W
  const int crow = wave * 8 + (lane >> 3), chunk = (lane & 7) ^ swz_key<128>(crow);
  static_assert(NW * 8 % 16 == 0, "the swizzle key repeats every 16 rows");
  static_assert(T::B / 4096 % NW == 0, "whole copies of a quarter of W's rows a wave");
  const uint32_t off0 = (uint32_t)crow * (uint32_t)p.rb + chunk * 16, rstep = (uint32_t)(NW * 8) * (uint32_t)p.rb;
  const int wm = wave / T::WN_, wn = wave % T::WN_;
  // not MX: this lane's scales, of the blocks 2 kt + lg
  const int KB = p.d / 32;
  const uint8_t *sp[T::TN];
  uint8_t sc[T::TN];
  int split, row0, col0, rows, cols, k_lo, k_hi;  // the tile whose copies are issued
  __amdgpu_buffer_rsrc_t ra, rbw;
  auto open = [&] {
    const int item = base + min(slot, slots - 1), L = item / p.splits;
    split = item % p.splits;
    const int grp = L / (kRowGroup * p.ct), within = L - grp * kRowGroup * p.ct;
    const int gr = min(kRowGroup, p.rt - grp * kRowGroup);
    row0 = (grp * kRowGroup + within % gr) * BM;
    col0 = within / gr * BN;
    rows = min(BM, p.n - row0);
    cols = min(BN, p.m - col0);
    k_lo = (split * KG + group) * p.per;
    k_hi = slot < slots ? min(p.steps, k_lo + p.per) : 0;  // (behind the last tile: nothing)
    ra = rsrc(p.a + (size_t)row0 * p.rb, (uint32_t)rows * (uint32_t)p.rb);
    rbw = rsrc(p.b + (size_t)col0 * wb, (uint32_t)cols * wb);
    if constexpr (!MX)
#pragma unroll
      for (int j = 0; j < T::TN; ++j)
        sp[j] = p.bs + (size_t)(col0 + min(wn * T::WN + j * 32 + lr, cols - 1)) * KB;
  };
  auto issue = [&](int kt, int st) {
    uint8_t *sa = smem + st * T::STAGE;
    const uint32_t k = (uint32_t)kt * 128u;
    const uint32_t out = (kt < k_hi && (int)k + chunk * 16 < p.rb) ? 0u : kOOB;
    // (rows past the tile lie past the buffer's record count: zeros)
    const uint32_t at = (off0 + k) | out;
#pragma unroll
    for (int q = 0; q < T::A / 1024 / NW; ++q) dma16(ra, sa + (NW * q + wave) * 1024, at + q * rstep);
    if constexpr (MX) {
#pragma unroll
      for (int q = 0; q < T::B / 1024 / NW; ++q) dma16(rbw, sa + T::A + (NW * q + wave) * 1024, at + q * rstep);
    }
    if constexpr (MX) {
      static_assert(BM * 8 / 256 % NW == 0 && BN * 8 / 256 % NW == 0, "whole copies of scales a wave");
      const size_t kc = (size_t)min(kt, p.steps - 1);
#pragma unroll
      for (int q = 0; q < BM * 8 / 256 / NW; ++q)
        dma4(rsrc(p.as + (kc * p.np + row0) * 8, BM * 8), sa + T::A + T::B + (NW * q + wave) * 256,
             (NW * q + wave) * 256 + lane * 4);
#pragma unroll
      for (int q = 0; q < BN * 8 / 256 / NW; ++q)
        dma4(rsrc(p.bs + (kc * p.mp + col0) * 8, BN * 8), sa + T::A + T::B + BM * 8 + (NW * q + wave) * 256,
             (NW * q + wave) * 256 + lane * 4);
    }
  };

  // not MX: a quarter of W's rows, four steps of them from step kt on
  auto issue_w = [&](int kt, int quarter, int buf) {
    const uint32_t k = (uint32_t)kt * 32u + chunk * 16;
    const uint32_t at = (uint32_t)(quarter * (BN / 4) + crow) * wb + k;
#pragma unroll
    for (int q = 0; q < T::B / 4096 / NW; ++q)
      dma16(rbw, smem + T::W + buf * T::B + quarter * (T::B / 4) + (NW * q + wave) * 1024,
            (kt < k_hi && k < wb) ? at + (uint32_t)(NW * 8 * q) * wb : kOOB);
  };
  auto load_scales = [&](int kt) {
    if constexpr (!MX)
#pragma unroll
      for (int j = 0; j < T::TN; ++j) sc[j] = sp[j][min(2 * kt + lg, KB - 1)];
  };
  f32x16 acc[T::TM][T::TN];

  // The loop is rotated by one slice against its barriers: behind the barrier that
  // publishes a step a wave reads slice 0 of it and then multiplies the last slice of
  // the step before, so that no wave stands at a barrier with nothing to multiply.
  u32x4 a0[T::TM], b0[T::TN], a1[T::TM], b1[T::TN];
  uint32_t as[T::TM], bs[T::TN], an[T::TM], bn[T::TN];  // MX: this step's scales, the next one's
  u32x4 codes[T::TN];                                // not MX: this step's codes
  float scale[T::TN];
  const int lw = swz<128>(wn * T::WN + lr, lg);  // (rows 32 apart have the same swizzle)
  auto read_step = [&](const uint8_t *sa, int i) {  // the tile's step i
    if constexpr (MX) {
      const uint8_t *sb = sa + T::A;
      const uint8_t *pa = sb + T::B + ((wm * T::WM + lr) * 8 + lg * 4);
      const uint8_t *pb = sb + T::B + ((BM + wn * T::WN + lr) * 8 + lg * 4);
#pragma unroll
      for (int i = 0; i < T::TM; ++i) an[i] = *(const uint32_t *)(pa + i * 32 * 8);
#pragma unroll
      for (int j = 0; j < T::TN; ++j) bn[j] = *(const uint32_t *)(pb + j * 32 * 8);
    } else {
      const uint8_t *sb = smem + T::W + ((i >> 2) & 1) * T::B + (lw ^ ((2 * (i & 3)) << 4));
#pragma unroll
      for (int j = 0; j < T::TN; ++j) codes[j] = *(const u32x4 *)(sb + j * 32 * 128);
    }
  };
  auto begin_step = [&] {
    if constexpr (MX) {
#pragma unroll
      for (int i = 0; i < T::TM; ++i) as[i] = an[i];
#pragma unroll
      for (int j = 0; j < T::TN; ++j) bs[j] = bn[j];
    }
  };
  auto convert = [&](int s, u32x4 *bf) {
    if constexpr (!MX)
#pragma unroll
      for (int j = 0; j < T::TN; ++j)
        bf[j] = u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j][s], scale[j], 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j][s], scale[j], 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j][s], scale[j], 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[j][s], scale[j], 3))};
  };
  const int la = swz<128>(wm * T::WM + lr, MX ? lg : 4 * lg), lb = T::A + lw;
  auto read_slice = [&](const uint8_t *sa, int s, u32x4 *af, u32x4 *bf) {
    const int flip = (MX ? 2 * s : s) << 4;  // from slice 0's chunk to slice s's
    const uint8_t *pa = sa + (la ^ flip), *pb = sa + (lb ^ flip);
#pragma unroll
    for (int i = 0; i < T::TM; ++i) af[i] = *(const u32x4 *)(pa + i * 32 * 128);
    if constexpr (MX)
#pragma unroll
      for (int j = 0; j < T::TN; ++j) bf[j] = *(const u32x4 *)(pb + j * 32 * 128);
  };
  auto multiply_slice = [&](int s, const u32x4 *af, const u32x4 *bf) {
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
      for (int j = 0; j < T::TN; ++j) {
        if constexpr (MX) {
          const v8i bv = {(int)bf[j].x, (int)bf[j].y, (int)bf[j].z, (int)bf[j].w, 0, 0, 0, 0};
          const v8i av = {(int)af[i].x, (int)af[i].y, (int)af[i].z, (int)af[i].w, 0, 0, 0, 0};
          acc[i][j] = s == 0   ? scaled<0>(bv, av, acc[i][j], bs[j], as[i])
                      : s == 1 ? scaled<1>(bv, av, acc[i][j], bs[j], as[i])
                      : s == 2 ? scaled<2>(bv, av, acc[i][j], bs[j], as[i])
                               : scaled<3>(bv, av, acc[i][j], bs[j], as[i]);
        } else {
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, bf[j]),
                                                              __builtin_bit_cast(bf16x8, af[i]), acc[i][j], 0, 0, 0);
        }
      }
  };
  constexpr int NM = T::TM * T::TN, NR = MX ? T::TM + T::TN : T::TM;  // products and reads of a slice
  // Slices 0 .. 2 of a step: each reads the next one's operands while it multiplies.
  auto slices = [&](const uint8_t *sa) {
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      u32x4 *ac = s & 1 ? a1 : a0, *bc = s & 1 ? b1 : b0, *ax = s & 1 ? a0 : a1, *bx = s & 1 ? b0 : b1;
      read_slice(sa, s + 1, ax, bx);
      convert(s + 1, bx);
      multiply_slice(s, ac, bc);
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i < NR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto take_scales = [&](int kt) {
    if constexpr (!MX)
#pragma unroll
      for (int j = 0; j < T::TN; ++j) scale[j] = e8m0_to_f32(2 * kt + lg < KB ? sc[j] : 127u);
  };
  // MANY: a block's tiles, one behind the other; the first copies of the next one are
  // issued in front of the epilogue's stores.
  constexpr int LPR = 8, RPI = 8, J = T::WN / 64;  // lanes a row, rows an instruction, pieces of the epilogue
  constexpr int kStores = J * T::TM * (32 / RPI);  // instructions of a wave's 16-byte stores, at least
  auto start = [&] {  // a tile's first copies
    issue(k_lo, 0);
    if constexpr (!MX)
#pragma unroll
      for (int q = 0; q < 4; ++q) issue_w(k_lo, q, 0);
    load_scales(k_lo);
  };
  // What is loaded behind the barrier in front of step i: the next step, and a quarter of
  // the next four steps' rows of W, whose buffer is free since step i - i % 4.
  auto more = [&](int i) {
    issue(k_lo + i + 1, (i + 1) & 1);
    if constexpr (!MX) issue_w(k_lo + (i & ~3) + 4, i & 3, ((i >> 2) + 1) & 1);
    load_scales(k_lo + i + 1);
  };
  open();
  start();
  bool counted = false;  // kStores or more stores of this wave lie behind its copies
  for (;;) {
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
      for (int j = 0; j < T::TN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    if (counted)
      wait_vmcnt<kStores>();
    else
      wait_vmcnt<0>();
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();  // (no fence: it would wait for the stores)
    asm volatile("" ::: "memory");
    take_scales(k_lo);
    read_step(smem, 0);
    read_slice(smem, 0, a0, b0);
    more(0);
    begin_step();
    convert(0, b0);
    __builtin_amdgcn_sched_barrier(0);
    const int steps = KG == 1 ? k_hi - k_lo : p.per;  // (groups meet at barriers: as many steps each)
    for (int i = 0; i + 1 < steps; ++i) {
      slices(smem + (i & 1) * T::STAGE);
      // the next step's copies are there, and every wave has the last of this one
      wait_vmcnt<0>();
      __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // lgkmcnt(0)
      __syncthreads();
      const uint8_t *sa = smem + ((i + 1) & 1) * T::STAGE;
      read_step(sa, i + 1);
      read_slice(sa, 0, a0, b0);
      multiply_slice(3, a1, b1);
      __builtin_amdgcn_sched_group_barrier(0x100, NR + (MX ? T::TM + T::TN : T::TN), 0);
      __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
      __builtin_amdgcn_sched_barrier(0);
      take_scales(k_lo + i + 1);
      more(i + 1);
      begin_step();
      convert(0, b0);
    }
    slices(smem + ((steps - 1) & 1) * T::STAGE);
    multiply_slice(3, a1, b1);
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<0>();  // (the copies past the end, which nobody reads)
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
    __syncthreads();
    const int er0 = row0, erows = rows;
    const bool whole = rows == BM && cols == BN, plane = p.splits > 1, half = p.out_bf16 && !plane;
    const int pitch = plane ? (p.m + 7) / 8 * 8 : p.m, width = plane ? pitch : p.m;
    char *out = (char *)p.y + (plane ? (size_t)split * p.n * pitch * 4 : 0);
    // (the lane is read afresh, so that nothing of the epilogue stays live in the loop)
    int el = __lane_id();
    asm volatile("" : "+v"(el));
    const int cl = el % LPR * 8, c = col0 + wn * T::WN + cl;
    const __amdgpu_buffer_rsrc_t rbias = rsrc(p.bias, p.bias && !plane ? (uint32_t)p.m * 4 : 0);
    float bv[J][8];
#pragma unroll
    for (int e = 0; e < 8 * J; ++e)
      bv[e / 8][e % 8] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(rbias, (uint32_t)(c + e / 8 * 64 + e % 8) * 4, 0, 0));
    // (no branch before the products are stored: they would sink behind it, and their
    // operands stay in registers)
    if constexpr (MANY) {
      slot += stride;
      open();
      start();
      // The next tile waits for these copies by counting the stores behind them, so no
      // store may move in front of one: neither in the IR nor in the schedule.
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
    // Epilogue: 32 rows at a time through the wave's own piece of LDS, so that stores
    // take whole rows of it, eight columns a lane (y's rows start at any element).
    uint8_t *piece = smem + (!MANY                 ? wave * T::PIECE
                             : MX || wave < NW / 2 ? T::STAGE + wave * T::PIECE
                                                   : T::W + T::B + (wave - NW / 2) * T::PIECE);
#pragma unroll
    for (int part = 0; part < T::TM * J; ++part) {
      const int i = part / J, jj = part % J;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16 &v = acc[i][2 * jj + j];
          *(f32x4 *)(piece + T::at(el % 32, j * 8 + q * 2 + el / 32)) =
              f32x4{v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]};
        }
      const int r0 = wm * T::WM + i * 32;
      if constexpr (KG > 1) lds_barrier();
#pragma unroll
      for (int v = 0; v < 32 / RPI; ++v) {
        if (KG > 1 && v % KG != group) continue;
        const int r = v * RPI + el / LPR;
        f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = x0;
        const uint8_t *from = piece - group * T::ALL;
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          x0 += *(const f32x4 *)(from + k * T::ALL + T::at(r, cl / 4));
          x1 += *(const f32x4 *)(from + k * T::ALL + T::at(r, cl / 4 + 1));
        }
        if (r0 + r < erows) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = x0[e] + bv[jj][e], o[4 + e] = x1[e] + bv[jj][4 + e];
          store_columns8(out, (size_t)(er0 + r0 + r) * pitch + c + jj * 64, width - c - jj * 64, half, o);
        }
      }
      // the pieces are read before the next rows go there
      if constexpr (KG > 1)
        lds_barrier();
      else
        __builtin_amdgcn_wave_barrier();
    }
    if (!MANY || slot >= slots) break;
    counted = whole;
  }
  if constexpr (MANY) wait_vmcnt<0>();  // (no copy into LDS outlives its block)
}

// y = bias + the planes' sum, in plane order: blocks of 8 x 256 columns of a row.
__global__ __launch_bounds__(256) void linear_sum_kernel(const float *__restrict__ part, int splits, int n, int m, int mp,
                                                         const float *__restrict__ bias, char *__restrict__ y,
                                                         int out_bf16) {
  const size_t plane = (size_t)n * mp;
  const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= m) return;
  float bv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bv[e] = bias && c + e < m ? bias[c + e] : 0.f;
  for (int r = blockIdx.y; r < n; r += gridDim.y) {
    const float *p = part + (size_t)r * mp + c;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    for (int s = 0; s < splits; ++s) {
      a += *(const f32x4 *)(p + s * plane);
      b += *(const f32x4 *)(p + s * plane + 4);
    }
    float o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = a[e] + bv[e], o[4 + e] = b[e] + bv[4 + e];
    store_columns8(y, (size_t)r * m + c, m - c, out_bf16, o);
  }
}

// Scales [rows][KB] of two matrices as [steps][padded rows][8], a step's even blocks
// before its odd ones, 127 (one) where there are none.
__global__ __launch_bounds__(256) void linear_scales_kernel(const uint8_t *__restrict__ xs, uint2 *__restrict__ xo, int n,
                                                            int np, const uint8_t *__restrict__ ws,
                                                            uint2 *__restrict__ wo, int m, int mp, int KB, int steps) {
  const int per = (np + mp), total = per * steps;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    // (steps of a row next to each other: the reads are consecutive)
    const int kt = i % steps, rr = i / steps;
    const bool first = rr < np;
    const int row = first ? rr : rr - np;
    const bool in = row < (first ? n : m);
    const uint8_t *s = (first ? xs : ws) + (size_t)row * KB + kt * 8;
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo |= (in && kt * 8 + 2 * j < KB ? s[2 * j] : 127u) << (8 * j);
      hi |= (in && kt * 8 + 2 * j + 1 < KB ? s[2 * j + 1] : 127u) << (8 * j);
    }
    (first ? xo : wo)[(size_t)kt * (first ? np : mp) + row] = uint2{lo, hi};
  }
}

// How a product is run: by rows (streamed weights) or by a GEMM.  (Times of MXFP4 rows are
// with their encoding in front.)
//   256 x 256 tiles where there are enough of them to fill most of the device (bf16 and
//     MXFP4 rows, us, smaller tiles / these: 128 tiles 70 / 91 and 31.5 / 36.5, 160 tiles
//     118 / 93 and 43.0 / 39.3, 192 tiles 121 / 104 and 48.3 / 44.7).
//   MXFP4 rows: two K groups a block, on 64 x 128 tiles while there is a CU for each and
//     128 x 128 tiles then (us, one group of 128 x 128 with K in planes / two groups of
//     64 / of 128: 333 x 2880 -> 5001 20.9 / 16.8 / 17.5, 512 x 4096 -> 4096 26.8 / 17.7 /
//     19.0, 1024 x 4096 -> 4096 32.5 / 27.9 / 21.2); with more tiles than CUs one group
//     (300 x 4096 -> 14336 26.1 / 38.6 / 30.2).
//   bf16 rows: the same idea pays less, as a block's W needs more LDS: two groups of
//     128 x 128 where they are one round of blocks (1024 x 4096 -> 4096 49.3 -> 45.1),
//     three of 64 x 128 where those are and K is short (333 x 2880 -> 5001 25.3 -> 23.5,
//     300 x 2048 -> 6000 22.8 -> 20.4, 200 x 2880 -> 8192 26.1 -> 22.1, but 512 x 4096 -> 4096
//     34.4 -> 36.9; between 48 and 64 steps the border could lie higher: 500 x 3584 -> 4096
//     30.7 -> 28.5); else one group of 128 x 128 and K in planes while that gives more blocks
//     and a plane has kSplitSteps (no planes / 22 / 11 / 6 steps at least: 17 x 4096 -> 4096
//     37.5 / 23.4 / 15.8 / 14.0, 65 x 4096 -> 14336 51 / 33.1 / 26.4 / 26.3, 300 x 8192 -> 2048
//     98 / 33.3 / 27.8 / 27.7, 200 x 2048 -> 2048 21.7 / 21.4 / 16.9 / 15.7).
struct LinearPlan {
  bool rows;
  int bm, bn, groups, splits, per, steps, rb, np, mp;
  size_t xs, ws, part, total;  // workspace: scales step by step; planes
};

LinearPlan plan_linear(int n, int d, int m, bool mx) {
  LinearPlan P{};
  P.rows = n <= kRowsMany;
  if (P.rows) return P;
  auto tiles = [&](int bm, int bn) { return (long long)((n + bm - 1) / bm) * ((m + bn - 1) / bn); };
  P.rb = mx ? d / 2 : d * 2;
  P.steps = (P.rb + 127) / 128;
  P.splits = 1;
  P.bm = P.bn = 256;
  P.groups = 1;
  const long long t64 = tiles(64, 128), t128 = tiles(128, 128);
  auto one_round = [&](long long t) { return t > kBlocks / 2 && t <= kBlocks; };
  if (tiles(256, 256) < kLargeTiles) {
    P.bn = 128;
    if (mx ? t64 <= kBlocks : one_round(t64) && P.steps <= kShort) {
      P.bm = 64;
      P.groups = mx ? 2 : 3;
    } else {
      P.bm = 128;
      P.groups = (mx ? t128 <= kBlocks : one_round(t128)) ? 2 : 1;
      if (!mx && P.groups == 1)
        while (P.splits < 8 && t128 * P.splits * 2 <= 2 * kBlocks && P.steps / (P.splits * 2) >= kSplitSteps)
          P.splits *= 2;
    }
  }
  P.per = (P.steps + P.splits * P.groups - 1) / (P.splits * P.groups);
  P.splits = (P.steps + P.per * P.groups - 1) / (P.per * P.groups);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  P.np = (n + 255) / 256 * 256;
  P.mp = (m + 255) / 256 * 256;
  if (mx) {
    P.xs = take((size_t)P.steps * P.np * 8);
    P.ws = take((size_t)P.steps * P.mp * 8);
  }
  P.part = take(P.splits > 1 ? (size_t)P.splits * n * ((m + 7) / 8 * 8) * 4 : 0);
  P.total = o;
  return P;
}

template <bool MX, int BM, int BN, int NW, int KG>
hipError_t launch_gemm(const GemmParams &p, hipStream_t st) {
  constexpr bool MANY = BM == 256;  // a block a CU, which takes several tiles
  using T = GemmTile<MX, BM, BN, NW, KG, MANY>;
  auto kern = linear_gemm_kernel<MX, BM, BN, NW, KG, MANY>;
  if (T::LDS > 64 * 1024) {
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load(std::memory_order_acquire) & bit)) {
      err = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);
      if (err != hipSuccess) return err;
      attr_done.fetch_or(bit, std::memory_order_release);
    }
  }
  const int total = p.rt * p.ct * p.splits;
  const int blocks = (total + 7) / 8 * 8, most = MANY ? std::max(8, cu_count() / 8 * 8) : blocks;
  kern<<<std::min(blocks, most), NW * KG * 64, T::LDS, st>>>(p);
  return hipGetLastError();
}

template <bool MX>
hipError_t launch_many(const LinearArgs &a, hipStream_t st) {
  const LinearPlan P = plan_linear(a.n, a.d, a.m, MX);
  char *ws = (char *)a.ws;
  GemmParams p{};
  p.a = (const uint8_t *)a.x;
  p.bias = a.bias;
  p.n = a.n;
  p.m = a.m;
  p.rb = P.rb;
  p.steps = P.steps;
  p.np = P.np;
  p.mp = P.mp;
  p.out_bf16 = a.out_bf16;
  p.rt = (a.n + P.bm - 1) / P.bm;
  p.ct = (a.m + P.bn - 1) / P.bn;
  p.splits = P.splits;
  p.per = P.per;
  p.y = P.splits > 1 ? (void *)(ws + P.part) : a.y;
  p.b = a.w;
  p.d = a.d;
  hipError_t e = hipSuccess;
  if (MX) {
    p.as = (uint8_t *)ws + P.xs;
    p.bs = (uint8_t *)ws + P.ws;
    const long long total = (long long)(P.np + P.mp) * P.steps;
    linear_scales_kernel<<<(int)std::min<long long>((total + 255) / 256, 2048), 256, 0, st>>>(
        a.x_s, (uint2 *)(ws + P.xs), a.n, P.np, a.w_s, (uint2 *)(ws + P.ws), a.m, P.mp, a.d / 32, P.steps);
    e = hipGetLastError();
  } else {
    p.bs = a.w_s;
  }
  if (e != hipSuccess) return e;
  e = P.bm == 256     ? launch_gemm<MX, 256, 256, 8, 1>(p, st)
      : P.bm == 64    ? launch_gemm<MX, 64, 128, 2, MX ? 2 : 3>(p, st)
      : P.groups == 2 ? launch_gemm<MX, 128, 128, 4, 2>(p, st)
                      : launch_gemm<MX, 128, 128, 4, 1>(p, st);
  if (e != hipSuccess || P.splits == 1) return e;
  const int mp = (a.m + 7) / 8 * 8;
  linear_sum_kernel<<<dim3((mp / 8 + 255) / 256, std::min(a.n, 32768)), 256, 0, st>>>(
      (const float *)(ws + P.part), P.splits, a.n, a.m, mp, a.bias, (char *)a.y, a.out_bf16);
  return hipGetLastError();
}

}  // namespace

size_t mxfp4_linear_bytes(int n, int d, int m, bool x_mx4) { return plan_linear(n, d, m, x_mx4).total; }

hipError_t launch_mxfp4_linear(const LinearArgs &a, hipStream_t st) {
  if (!plan_linear(a.n, a.d, a.m, a.x_mx4).rows) return a.x_mx4 ? launch_many<true>(a, st) : launch_many<false>(a, st);
  LinearParams p{};
  p.x = (const uint8_t *)a.x;
  p.xs = a.x_s;
  p.w = a.w;
  p.ws = a.w_s;
  p.bias = a.bias;
  p.y = a.y;
  p.n = a.n;
  p.d = a.d;
  p.m = a.m;
  p.out_bf16 = a.out_bf16;
  p.G = std::min(cu_count(), a.m);
  if (a.x_mx4) {
    if (a.d < 128) return launch_rows<kMx4, true, true, 2>(p, st);
    return rows_fit<kMx4>(a.n, a.d) ? launch_rows<kMx4, true, false, 2>(p, st) : launch_rows<kMx4, false, false, 2>(p, st);
  }
  if (a.d < 128) return launch_rows<kMx, true, true, 2>(p, st);
  return rows_fit<kMx>(a.n, a.d) ? launch_rows<kMx, true, false, 2>(p, st) : launch_rows<kMx, false, false, 2>(p, st);
}

}  // namespace moe
