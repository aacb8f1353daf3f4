// The whole layer for at most 16 tokens in two kernels (moe_forward_few).
//
//   z = x Wg^T + b, top-k and weights as in the router,
//   y[t] = sum_j w_tj (silu(x_t W1_e) (x_t W3_e)) W2_e,  e = idx[t][j]
//
// With a few tokens the layer is bound by reading the chosen experts' weights
// once, and by the launches, barriers and round trips between the steps that
// depend on each other.  few_router_kernel takes the logits (one workgroup per
// expert).  few_layer_kernel does the rest: every workgroup takes the top-k of
// all tokens by itself (cheaper than a launch), then its part of the up
// projections, and once all parts are done, its part of the outputs.
//
// The parts are tickets from one counter: 0 .. G-1 are the up parts, G .. 2G-1
// the output parts.  A workgroup takes a ticket, does it and takes the next; an
// output part waits until all G up parts are done.  A ticket is only ever taken
// by a running workgroup, up parts never wait, and a workgroup does its tickets
// in order, so when an output part waits, every up part is done or in the hands
// of a running workgroup that does not wait: the wait ends however few of the
// workgroups are resident and whatever else runs on the GPU (two calls at once
// among it).  What a part computes depends on its ticket alone, so results do
// not depend on who takes it.
//
// The products (wave_stream.h) take the tokens as the 16 rows of a 16 x 16 MFMA and 16
// weight rows as its columns.  Up: a tile is 8 rows of W1 and the same 8 of W3, over all
// of K, so gate and value meet in one wave; a part is an equal run of the chosen experts'
// hidden columns, whose tiles its waves take in turn.  Output: a part is an equal run of
// output columns over all chosen experts, its waves equal runs of (expert, chunk of K);
// each wave adds an expert's product to its tokens' sums where its run of the expert
// ends, and the waves' sums meet in LDS in a fixed order.  The hidden is multiplied by
// its combine weight before its one rounding, so that the output needs no pass of its
// own.  It is handed over through memory by write-through stores and counters; with a
// release fence a workgroup the hand-over took 15 us.
//
// What bounds it: reading the chosen experts, and about 17 us around that: two launches,
// the logits (4.6 us), the top-k, the hand-over.  d = d_ff = 2880, 128 MXFP4 experts, k = 4
// (us; a copy's rate takes 10, 20, 38, 73 and 129 for the weights alone): 1 token 29, 2 39, 4 61,
// 8 98, 16 170, against 32, 46, 65, 95 and 145 in the steps of moe_forward: the streaming
// here reaches 4.5 TB/s, and 5.2 with the products left out.  d = 4096, d_ff = 14336,
// k = 2, 8 MXFP4 experts: 1 token 45 (moe_forward 106), 8 143 (334), 16, whose rows do not
// fit LDS, 306 (337); 8 bf16 experts: 120 (184), 16 530 (567); d = 1024, d_ff = 4096, 8
// bf16 experts, k = 1: 24 (46) and 49 (64).
// 8 waves with two chunks in flight each: four cost 3% at 1 token and 2% at 8.
#include <algorithm>
#include <atomic>

#include "common.h"
#include "kernels.h"
#include "route_dev.h"
#include "wave_stream.h"

namespace moe {
namespace {

constexpr int kT = kFewMaxTokens;  // 16: the M of the MFMA
constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kInFlight = 2;  // chunks of weights in flight a wave
constexpr int kFewLds = 160 * 1024;
// Tries of a waiting output part (each at least a microsecond): seconds, where a
// call takes microseconds.  Past it the part writes NaN.
constexpr int kMaxTries = 1 << 23;
// Parts done are counted in kDone counters (part i in counter i mod kDone), each on a
// line of its own: 256 additions to one address, with the waiting workgroups reading
// it, took 4 us.
constexpr int kQueue = 8;  // segments a wave has loaded ahead of those it finished, at most kInFlight + 1
static_assert(kInFlight < kQueue, "segments ahead");
constexpr int kDone = 8, kCountInts = 64;

struct FewLds {
  int x;      // the tokens' row chunks, later a round's hidden
  int cap;    // row chunks that fit there
  int ex;     // the waves' exchange buffers
  int idx, w, mask, aidx, act, slot, pre, pile, row, queue, misc, total;
};

struct FewParams {
  const void *x;
  const float *logits;
  const uint8_t *w1, *w3, *w2, *s1, *s3, *s2;
  const int32_t *slot;
  int n_slots;
  int n, d, E, k, f;
  int renorm, out_bf16;
  void *h;         // [n k][f], bf16 or f32
  void *y;
  int32_t *idx;    // [n][k] or NULL
  float *w;
  int *count;      // kCounts counters a line apart: tickets, then parts done in kDone pieces
  int G;
  FewLds lds;
};

// XL: the tokens' rows fit LDS.
template <int WT, int PER, bool XL, bool NARROW, int PC>
__global__ __launch_bounds__(kThreads) void few_layer_kernel(FewParams p) {
  using F = Form<WT>;
  constexpr int NF = F::kActBytes / 16, RC = kRowChunk<WT>;
  constexpr int SL = (RC - 16) / 16;  // lanes of a row chunk
  constexpr int kStage = 4;  // loads of the hidden a wave has in flight
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  const FewLds &L = p.lds;
  int *s_idx = (int *)(smem + L.idx), *s_mask = (int *)(smem + L.mask), *s_act = (int *)(smem + L.act);
  int *s_slot = (int *)(smem + L.slot), *s_pre = (int *)(smem + L.pre);
  float *s_w = (float *)(smem + L.w);
  uint16_t *s_aidx = (uint16_t *)(smem + L.aidx), *s_pile = (uint16_t *)(smem + L.pile);
  int *s_misc = (int *)(smem + L.misc);  // active experts, ticket, whether the wait ended, tiles taken
  int *s_queue = (int *)(smem + L.queue), *s_row = (int *)(smem + L.row);
  uint8_t *s_x = smem + L.x, *xbuf = smem + L.ex + (threadIdx.x >> 6) * kExchange;
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = p.n, k = p.k, E = p.E, d = p.d, f = p.f, R = n * k, G = p.G;
  const size_t xrow = (size_t)d * (F::f32 ? 4 : 2), hrow = (size_t)f * (F::f32 ? 4 : 2);
  const int Cd = (F::blocks(d) + kChunkBlocks - 1) / kChunkBlocks, Cf = (F::blocks(f) + kChunkBlocks - 1) / kChunkBlocks;

  auto take = [&]() {
    return __hip_atomic_fetch_add(p.count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  int first = 0;
  if (tid == 0) first = take();
  for (int e = tid; e < E; e += kThreads) s_mask[e] = 0;
  // The top-k, and the tokens' rows into LDS: by the waves without a token where there
  // are enough of them, else by all behind their tokens.
  const int TG = topk_group(E), busy = (n * TG + 63) / 64, from = XL && busy <= kWaves / 2 ? busy : 0;
  if (from == 0 || wave < from)
    for (int t0 = 0; t0 < n; t0 += kThreads / TG)
      topk_token_t<PER>(p.logits, 1, 0, t0 + tid / TG, n, E, k, p.renorm, s_idx, s_w, nullptr, nullptr);
  if (XL && (from == 0 || wave >= from)) {
    const int pieces = Cd * SL;  // of a row
    for (int i = tid - from * 64; i < pieces; i += kThreads - from * 64)
      for (int t0 = 0; t0 < n; t0 += 4) {
        u32x4 q[4];
#pragma unroll
        for (int v = 0; v < 4; ++v)
          q[v] = row_chunk_piece<WT>((const uint8_t *)p.x + min(t0 + v, n - 1) * xrow, i / SL, d, i % SL);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (t0 + v < n) *(u32x4 *)(s_x + (i / SL * n + t0 + v) * RC + i % SL * 16) = q[v];
      }
  }
  if (tid == 0) {
    s_misc[1] = first;
    s_misc[3] = 0;
  }
  __syncthreads();
  // ---- who takes which expert ------------------------------------------------
  for (int q = tid; q < R; q += kThreads) atomicOr(&s_mask[s_idx[q]], 1 << (q / k));
  __syncthreads();
  if (wave == 0) {
    int a = 0, m0 = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
      const int e = e0 + lane, m = e < E ? __popc(s_mask[e]) : 0;
      const uint64_t bits = __ballot(m != 0);
      const int incl = wave_incl_scan(m);
      if (m) {
        const int at = a + __popcll(bits & ((1ull << lane) - 1));
        s_aidx[e] = (uint16_t)at;
        s_act[at] = e;
        s_slot[at] = phys_slot(p.slot, p.n_slots, e);
        s_pre[at] = m0 + incl - m;
      }
      a += __popcll(bits);
      m0 += __builtin_amdgcn_readlane(incl, 63);
    }
    if (lane == 0) {
      s_misc[0] = a;
      s_pre[a] = m0;
    }
  }
  __syncthreads();
  for (int q = tid; q < R; q += kThreads) {
    const int e = s_idx[q], t = q / k, a = s_aidx[e], j = __popc(s_mask[e] & ((1 << t) - 1));
    s_pile[a * kT + j] = (uint16_t)q;
    s_row[s_pre[a] + j] = a << 16 | q;  // pile rows in order: expert and pair
  }
  __syncthreads();
  const int A = uniform(s_misc[0]);
  int ticket = uniform(s_misc[1]);

  if (ticket == 0 && p.idx)
    for (int q = tid; q < R; q += kThreads) p.idx[q] = s_idx[q];
  if (ticket == 0 && p.w)
    for (int q = tid; q < R; q += kThreads) p.w[q] = s_w[q];

  int *queue = s_queue + wave * (4 * kQueue);  // the segments loaded ahead
  // (a block's tickets ascend, so no up part follows an output part, whose
  // staging overwrites the tokens' rows)
  for (int turn = 0; ticket < 2 * G && turn < 2 * G; ++turn) {
    if (ticket < G) {
      // ---- up: hidden columns [u0, u1) of the chosen experts' A f -----------
      const long long U = (long long)A * f;
      const int u0 = (int)(U * ticket / G), cols = (int)(U * (ticket + 1) / G) - u0;
      // Tiles of at most 8 columns, a tile for every wave at least; the waves take them
      // in turn (the older waves of a SIMD run ahead of the younger).  A tile has a
      // segment for each expert it meets.
      const int tiles = max((cols + 7) / 8, min(cols, kWaves));
      int lu = 0, lu_to = 0;  // what is left of the tile to load
      const size_t rb = F::row_bytes(d);
      const int tok = min(r, n - 1);  // (rows past the last token: any)
      stream<WT, PC, NARROW>(
          Cd, d, xbuf,
          [&](int i, Segment &w) {
            if (lu == lu_to) {
              int t = 0;
              if (lane == 0) t = atomicAdd(&s_misc[3], 1);
              t = uniform(t);
              if (t >= tiles) return false;
              lu = u0 + (int)((long long)cols * t / tiles);
              lu_to = u0 + (int)((long long)cols * (t + 1) / tiles);
            }
            const int a = lu / f, c = lu - a * f, cnt = min(lu_to - lu, f - c);
            if (lane == 0) *(i32x4 *)(queue + 4 * (i % kQueue)) = i32x4{a, c, cnt, 0};
            w.first = 0;
            w.count = Cd;
            lu += cnt;
            const size_t wr = (size_t)uniform(s_slot[a]) * f + c;
            w.row[0] = p.w1 + wr * rb;
            w.row[1] = p.w3 + wr * rb;
            w.scale[0] = F::mx ? p.s1 + wr * (d / 32) : nullptr;
            w.scale[1] = F::mx ? p.s3 + wr * (d / 32) : nullptr;
            w.cnt[0] = w.cnt[1] = cnt;
            return true;
          },
          [] {},
          [&](int, int &c, int &left) {
            c = 0;
            left = Cd;
          },
          [&](int, int c, int b, u32x4 (&a)[NF], uint32_t &) {
            if constexpr (XL) {
              const uint8_t *px = s_x + (c * n + tok) * RC + b * F::kActBytes;
#pragma unroll
              for (int q = 0; q < NF; ++q) a[q] = *(const u32x4 *)(px + q * 16);
            } else {
              load_block<WT>((const uint8_t *)p.x + tok * xrow, c * kChunkBlocks + b, d, a);
            }
          },
          [&](int i, f32x4 v) {
            const i32x4 at = *(const i32x4 *)(queue + 4 * (i % kQueue));
            const int a = at[0], c = at[1], cnt = at[2];
            const int mask = s_mask[s_act[a]];
            // lane (r, g): token 4 g + i, column c + r (r < 8: gate, r + 8: value)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = __shfl_xor(v[i], 8, 64);
              const int t = 4 * g + i;
              if (r < cnt && r < 8 && ((mask >> t) & 1)) {
                const int q = s_pile[a * kT + __popc(mask & ((1 << t) - 1))];
                const float hv = s_w[q] * (silu(v[i]) * u);
                if constexpr (F::f32)
                  __hip_atomic_store((float *)p.h + (size_t)q * f + c + r, hv, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_AGENT);
                else
                  __hip_atomic_store((uint16_t *)p.h + (size_t)q * f + c + r, (uint16_t)f32_to_bf16_bits(hv),
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
              }
            }
          });
      // (all workgroups that run have their first ticket by now: the next one is taken
      // here, under the other waves' work)
      int next = 0;
      if (tid == 0) next = take();
      // The hidden's stores write through to the memory that all XCDs share (atomic
      // stores of agent scope); waited for, they are there before the count is.  An
      // agent-scope release fence would write back the whole L2 besides: with one per
      // workgroup the last of 256 came 15 us after the first.
      __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
      lds_barrier();
      if (tid == 0) {
        __hip_atomic_fetch_add(p.count + (1 + ticket % kDone) * kCountInts, 1, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        s_misc[1] = next;
        s_misc[3] = 0;
      }
      lds_barrier();
      ticket = uniform(s_misc[1]);
      continue;
    }
    // ---- output columns [c_lo, c_hi) ------------------------------------------
    // The chosen experts' (expert, chunk of K) pairs in order, in rounds whose hidden
    // fits LDS; every wave takes an equal run of a round.  Pair (a, c) has m = popc(mask)
    // row chunks, pre[a] Cf + m c of them before it.
    const int part = ticket - G;
    const int c_lo = (int)((long long)d * part / G), c_hi = (int)((long long)d * (part + 1) / G);
    bool waited = false;
    struct Round {
      int a, c, w0;     // its first expert and chunk, row chunks before them
      int a_to, c_to;   // behind its last
      int lo, hi;       // this wave's run, in chunks from the first expert's chunk 0 on
    };
    auto next_round = [&](Round &q) {  // false behind the last
      q.a = q.a_to;
      q.c = q.c_to;
      if (q.a == A) return false;
      const int pre = s_pre[q.a];
      q.w0 = uniform(pre * Cf + (s_pre[q.a + 1] - pre) * q.c);
      // the experts that fit whole, then chunks of the next
      for (;;) {
        const bool fits = q.a_to + lane < A && s_pre[min(q.a_to + lane, A - 1) + 1] * Cf - q.w0 <= L.cap;
        const int add = __popcll(__ballot(fits));
        q.a_to += add;
        if (add < 64) break;
      }
      q.c_to = 0;
      if (q.a_to < A) {
        const int at = s_pre[q.a_to], m = s_pre[q.a_to + 1] - at;
        q.c_to = uniform((L.cap + q.w0 - at * Cf) / m);
      }
      const int total = (q.a_to - q.a) * Cf + q.c_to - q.c;
      q.lo = q.c + (int)((long long)total * wave / kWaves);
      q.hi = q.c + (int)((long long)total * (wave + 1) / kWaves);
      return true;
    };
    if (c_lo < c_hi)
      for (int c0 = c_lo; c0 < c_hi; c0 += 16) {
        const int cnt = min(16, c_hi - c0);
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        Round lr{0, 0, 0, 0, 0, 0, 0}, ur = lr;  // the round that is loaded, the one in LDS
        int l_at = 0, l_a = 0, l_round = -1, u_round = -1;
        // The next round's hidden into LDS (all waves together).
        auto enter = [&] {
          next_round(ur);
          ++u_round;
          if (!waited) {
            waited = true;
            if (wave == 0) {
              // lane i: the parts i, i + kDone, .. of G
              const int all = lane < kDone ? (G - lane + kDone - 1) / kDone : 0;
              int tries = 0, done = 0;
              do {
                if (lane < kDone)
                  done = __hip_atomic_load(p.count + (1 + lane) * kCountInts, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
              } while (__any(done < all) && ++tries < kMaxTries);
              __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
              if (lane == 0) s_misc[2] = tries < kMaxTries;
            }
          }
          lds_barrier();  // also: the round before is done with its hidden
          // Half a pile row to a wave at a time, kStage loads in flight; 64 / SL chunks a load.
          const int r_lo = s_pre[ur.a], r_hi = ur.c_to ? s_pre[ur.a_to + 1] : s_pre[ur.a_to];
          for (int v = wave; v < 2 * (r_hi - r_lo); v += kWaves) {
            const int row = uniform(r_lo + (v >> 1)), pair = uniform(s_row[row]), a = pair >> 16, q = pair & 0xffff;
            const int pre = uniform(s_pre[a]), m = uniform(s_pre[a + 1]) - pre;
            int ca = a == ur.a ? ur.c : 0, cb = a == ur.a_to ? ur.c_to : Cf;
            const int mid = (ca + cb) >> 1;
            (v & 1 ? ca : cb) = mid;
            const uint8_t *src = (const uint8_t *)p.h + q * hrow;
            // (row chunks are counted first: all of a pile's, in bytes, do not fit 31 bits)
            const int to = pre * Cf + (row - pre) - ur.w0;
            uint8_t *dst = s_x + lane % SL * 16;
            for (int c = ca + lane / SL; c < cb; c += kStage * (64 / SL)) {
              u32x4 w[kStage];
#pragma unroll
              for (int i = 0; i < kStage; ++i)
                if (c + i * (64 / SL) < cb) w[i] = row_chunk_piece<WT>(src, c + i * (64 / SL), f, lane % SL);
#pragma unroll
              for (int i = 0; i < kStage; ++i)
                if (c + i * (64 / SL) < cb) *(u32x4 *)(dst + (to + m * (c + i * (64 / SL))) * RC) = w[i];
            }
          }
          lds_barrier();
        };
        int at = 0, m = 0, e_mask = 0;  // the segment's: the lane's first row chunk, rows, tokens
        stream<WT, PC, NARROW>(
            Cf, f, xbuf,
            [&](int i, Segment &w) {
              while (l_at == lr.hi) {
                if (!next_round(lr)) return false;
                ++l_round;
                l_a = lr.a + lr.lo / Cf;
                l_at = lr.lo;
              }
              const int c = l_at - (l_a - lr.a) * Cf;
              w.first = c;
              w.count = min(lr.hi - l_at, Cf - c);
              if (lane == 0) *(i32x4 *)(queue + 4 * (i % kQueue)) = i32x4{l_a, c, w.count, l_round};
              rows_of_one<WT>(w, p.w2, p.s2, (size_t)uniform(s_slot[l_a]) * d + c0, cnt, f);
              l_at += w.count;
              if (c + w.count == Cf) ++l_a;
              return true;
            },
            enter,
            [&](int i, int &c, int &left) {
              const i32x4 s = *(const i32x4 *)(queue + 4 * (i % kQueue));
              const int a = uniform(s[0]), round = uniform(s[3]);
              c = uniform(s[1]);
              left = uniform(s[2]);
              while (u_round < round) enter();
              const int pre = s_pre[a];
              m = uniform(s_pre[a + 1] - pre);
              e_mask = s_mask[s_act[a]];
              at = pre * Cf - ur.w0 + min(__popc(e_mask & ((1 << r) - 1)), m - 1);
            },
            [&](int, int c, int b, u32x4 (&a)[NF], uint32_t &) {
              const uint8_t *ph = s_x + (at + m * c) * RC + b * F::kActBytes;
#pragma unroll
              for (int q = 0; q < NF; ++q) a[q] = *(const u32x4 *)(ph + q * 16);
            },
            [&](int, f32x4 v) {  // only the expert's own tokens: 0 times a NaN weight is NaN
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if ((e_mask >> (4 * g + q)) & 1) sum[q] += v[q];
            });
        while (ur.a_to < A) enter();  // (rounds in which this wave has nothing)
        if (tid == 0 && c0 + 16 >= c_hi) s_misc[1] = take();
        *(f32x4 *)(xbuf + lane * 16) = sum;
        lds_barrier();
        if (wave < 4) {  // wave i: token 4 g + i
          float v = 0.f;
#pragma unroll
          for (int j = 0; j < kWaves; ++j) v += *(const float *)(smem + L.ex + j * kExchange + lane * 16 + wave * 4);
          if (!s_misc[2]) v = __builtin_nanf("");
          const int t = 4 * g + wave;
          if (t < n && r < cnt) {
            const size_t at = (size_t)t * d + c0 + r;
            if (p.out_bf16)
              ((uint16_t *)p.y)[at] = (uint16_t)f32_to_bf16_bits(v);
            else
              ((float *)p.y)[at] = v;
          }
        }
        lds_barrier();
      }
    else if (tid == 0)
      s_misc[1] = take();
    lds_barrier();
    ticket = uniform(s_misc[1]);
    lds_barrier();  // (read before the next ticket is written)
  }
}

constexpr int kRouterThreads = 512;

// logits[t][e] = x_t . wg_e + bias_e, one workgroup per expert; the first also
// clears the next kernel's counters.  N >= n tokens: the loads of all of them are
// in flight together, rows past the last one as the last (waited for one by one,
// 8 tokens of 2880 took 5.4 us and 16 of 1024 5.5).  Rows of bf16 in 16-byte pieces.
template <bool BF, int N>
__global__ __launch_bounds__(kRouterThreads) void few_router_kernel(const void *__restrict__ x, const void *__restrict__ wg,
                                                         const float *__restrict__ bias, int n, int d, int E,
                                                         float *__restrict__ logits, int *__restrict__ count) {
  __shared__ float s_sum[kRouterThreads / 64][N];
  const int e = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (e == 0 && tid <= kDone) count[tid * kCountInts] = 0;
  float acc[N] = {};
  if constexpr (BF) {
    const u32x4 *wr = (const u32x4 *)((const uint16_t *)wg + (size_t)e * d);
    for (int c = tid; c < d / 8; c += kRouterThreads) {
      const u32x4 w = wr[c];
      u32x4 v[N];
#pragma unroll
      for (int t = 0; t < N; ++t) v[t] = ((const u32x4 *)((const uint16_t *)x + (size_t)min(t, n - 1) * d))[c];
#pragma unroll
      for (int t = 0; t < N; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[t] = fmaf(__uint_as_float(w[i] << 16), __uint_as_float(v[t][i] << 16), acc[t]);
          acc[t] = fmaf(__uint_as_float(w[i] & 0xffff0000u), __uint_as_float(v[t][i] & 0xffff0000u), acc[t]);
        }
    }
  } else {
    const float *wr = (const float *)wg + (size_t)e * d;
    for (int c = tid; c < d; c += kRouterThreads) {
      const float w = wr[c];
      float v[N];
#pragma unroll
      for (int t = 0; t < N; ++t) v[t] = ((const float *)x)[(size_t)min(t, n - 1) * d + c];
#pragma unroll
      for (int t = 0; t < N; ++t) acc[t] = fmaf(w, v[t], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const float v = group_sum(acc[t], 64);
    if (lane == 0) s_sum[wave][t] = v;
  }
  __syncthreads();
  if (tid < n) {
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < kRouterThreads / 64; ++j) v += s_sum[j][tid];
    logits[(size_t)tid * E + e] = bias ? v + bias[e] : v;
  }
}

template <bool BF>
void launch_router(const FewArgs &a, float *logits, int *count, hipStream_t st) {
  auto kern = a.n == 1   ? few_router_kernel<BF, 1>
              : a.n <= 4 ? few_router_kernel<BF, 4>
              : a.n <= 8 ? few_router_kernel<BF, 8>
                         : few_router_kernel<BF, kT>;
  kern<<<a.E, kRouterThreads, 0, st>>>(a.x, a.wg, a.bias, a.n, a.d, a.E, logits, count);
}

int up16(int v) { return (v + 15) / 16 * 16; }

struct FewPlan {
  size_t logits, count, h, total;  // workspace
};

FewPlan plan_of(int n, int E, int k, int d_ff, bool f32) {
  FewPlan P{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  P.logits = 0;
  P.count = up((size_t)n * E * 4);
  P.h = P.count + up((1 + kDone) * kCountInts * sizeof(int));
  P.total = P.h + up((size_t)n * k * d_ff * (f32 ? 4 : 2));
  return P;
}

template <int WT>
int chunks_of(int K) {
  return (Form<WT>::blocks(K) + kChunkBlocks - 1) / kChunkBlocks;
}

// LDS of a launch: the tables, and in what is left the activations.
template <int WT>
FewLds lds_of(const FewParams &p) {
  FewLds L{};
  const int R = p.n * p.k, A = std::min(R, p.E);
  int o = 0;
  auto put = [&](int bytes) {
    const int at = o;
    o += up16(bytes);
    return at;
  };
  L.ex = put(kWaves * kExchange);
  L.idx = put(R * 4);
  L.w = put(R * 4);
  L.mask = put(p.E * 4);
  L.aidx = put(p.E * 2);
  L.act = put(A * 4);
  L.slot = put(A * 4);
  L.pre = put((A + 1) * 4);
  L.pile = put(A * kT * 2);
  L.row = put(R * 4);
  L.queue = put(kWaves * 4 * kQueue * 4);
  L.misc = put(16);
  // the rest: the tokens' rows, later a round's hidden (16 row chunks at least)
  L.x = o;
  L.cap = (kFewLds - o) / kRowChunk<WT>;
  L.total = o + (int)std::min<long long>(L.cap, (long long)p.n * std::max<long long>(chunks_of<WT>(p.d), (long long)p.k * chunks_of<WT>(p.f))) * kRowChunk<WT>;
  return L;
}

template <int WT, int PER, bool XL, bool NARROW, int PC>
hipError_t launch(FewParams &p, hipStream_t st) {
  auto kern = few_layer_kernel<WT, PER, XL, NARROW, PC>;
  p.lds = lds_of<WT>(p);
  const FewLds &L = p.lds;
  if (L.total > kFewLds) return hipErrorInvalidValue;
  if (L.total > 64 * 1024) {
    // The LDS limit is raised once per device (a per-device kernel attribute).
    static std::atomic<uint64_t> attr_done{0};
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(attr_done.load(std::memory_order_acquire) & bit)) {
      err = hipFuncSetAttribute((const void *)kern, hipFuncAttributeMaxDynamicSharedMemorySize, kFewLds);
      if (err != hipSuccess) return err;
      attr_done.fetch_or(bit, std::memory_order_release);
    }
  }
  kern<<<p.G, kThreads, L.total, st>>>(p);
  return hipGetLastError();
}

}  // namespace

size_t forward_few_bytes(int n, int E, int k, int d_ff, bool f32) { return plan_of(n, E, k, d_ff, f32).total; }

hipError_t launch_forward_few(const FewArgs &a, hipStream_t st) {
  const bool f32 = a.w_dtype == 0;
  const FewPlan P = plan_of(a.n, a.E, a.k, a.d_ff, f32);
  char *base = (char *)a.ws;
  FewParams p{};
  p.x = a.x;
  p.logits = (float *)(base + P.logits);
  p.count = (int *)(base + P.count);
  p.h = base + P.h;
  p.w1 = (const uint8_t *)a.w1;
  p.w3 = (const uint8_t *)a.w3;
  p.w2 = (const uint8_t *)a.w2;
  p.s1 = a.s1;
  p.s3 = a.s3;
  p.s2 = a.s2;
  p.slot = a.slot;
  p.n_slots = a.n_slots;
  p.n = a.n;
  p.d = a.d;
  p.E = a.E;
  p.k = a.k;
  p.f = a.d_ff;
  p.renorm = a.renorm;
  p.out_bf16 = a.out_bf16;
  p.y = a.y;
  p.idx = a.idx;
  p.w = a.w;
  p.G = cu_count();
  float *logits = (float *)(base + P.logits);
  if (f32)
    launch_router<false>(a, logits, p.count, st);
  else
    launch_router<true>(a, logits, p.count, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const bool few = topk_per(a.E) == 2;
  auto rows_fit = [&](auto form) {
    constexpr int WT = decltype(form)::value;
    return (long long)p.n * chunks_of<WT>(p.d) <= lds_of<WT>(p).cap;
  };
  if (a.w_dtype == 2) {
    const bool fit = rows_fit(std::integral_constant<int, kMx>{});
    if (std::min(a.d, a.d_ff) < 128)
      return fit ? launch<kMx, 16, true, true, kInFlight>(p, st) : launch<kMx, 16, false, true, kInFlight>(p, st);
    if (!fit) return launch<kMx, 16, false, false, kInFlight>(p, st);
    return few ? launch<kMx, 2, true, false, kInFlight>(p, st) : launch<kMx, 16, true, false, kInFlight>(p, st);
  }
  if (a.w_dtype == 1) {
    if (!rows_fit(std::integral_constant<int, kBf>{})) return launch<kBf, 16, false, false, kInFlight>(p, st);
    return few ? launch<kBf, 2, true, false, kInFlight>(p, st) : launch<kBf, 16, true, false, kInFlight>(p, st);
  }
  if (a.d % 4 || a.d_ff % 4)
    return rows_fit(std::integral_constant<int, kF4Tail>{}) ? launch<kF4Tail, 16, true, false, 1>(p, st)
                                                            : launch<kF4Tail, 16, false, false, 1>(p, st);
  return rows_fit(std::integral_constant<int, kF4>{}) ? launch<kF4, 16, true, false, kInFlight>(p, st)
                                                      : launch<kF4, 16, false, false, kInFlight>(p, st);
}

}  // namespace moe
