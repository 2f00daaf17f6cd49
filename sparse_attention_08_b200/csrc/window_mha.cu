// window_mha.cu -- attention of a prompt in the MHA form of MLA over a sliding
// window and a few first tokens that stay visible, on sm_100a.
//
//   out[t,h,:] = sum_{s in V_t} softmax_s(scale q[t,h,:] . k[s,h,:]) v[s,h,:]
//   lse[t,h]   = log sum_{s in V_t} exp(scale q[t,h,:] . k[s,h,:])
//
// with V_t = { s <= p : s > p - window or s < sinks } for the query at
// position p (every head with its own 192-d key and 128-d value).
//
// A persistent grid of one CTA per SM.  A work item is a pair of 128-query
// tiles of one sequence and head; it walks the 128-key tiles that hold a key some row
// of the pair sees (the first tokens' tiles, then the window's).  The two
// query tiles have their own score and output accumulators in TMEM and an MMA
// warp each, so the softmax of one runs under the products of the other:
//
//   ... P V (tile 0, j)  S (tile 0, j+1)  P V (tile 1, j)  S (tile 1, j+1) ...
//
//  warp 0      TMA: queries, then keys and values as 16 KB boxes (128 rows x 64
//              columns) through one ring of eight; a key tile is three boxes,
//              a value tile two, and a box is reloaded as soon as both query
//              tiles are done with it;
//  warps 1, 2  MMA issuers, one per query tile: S = Q K^T (12 MMAs, M128 N128
//              K16), O += P V (8 MMAs, P read from TMEM, V MN-major from shared
//              memory);
//  warps 4..11 a warpgroup per query tile, a thread one row: P over the
//              scores' own columns.  The running maximum of the tile before
//              serves as the exponentials' reference; only where a row's weights
//              over it add up to more than 2^32 is the tile's maximum taken
//              first and O rescaled.
// TMEM: S (and P) at columns 0 and 128, O at 256 and 384.
//
// Two bounds lie close together: a step's 40 MMAs take 2560 cycles, its exponentials
// (2 x 128 x 128 at 16 a cycle) 2050.  What a step takes is the turn's way around:
// twice (P V 550, keys' wait 165, S 940, hand-over 380), 4030 cycles, under which a
// softmax of 1850 is hidden.  Measured at L = 4096, 128 heads: causal 622 us
// (1.10 PFLOP/s, the tensor cores' share 0.65), window 1024 with four first tokens
// 364 us (0.83), where an item's ends cost about 2 steps (the read-out, and
// keys that come late since the ring holds 1.6 key tiles).
//
// Tried: the first 96 keys' weights handed over by themselves (2 % slower: its vote,
// store and barrier cost more than the 380 cycles of products it hides), the turn
// given back before the last S MMAs (5-10 % slower), the first tokens' tile cut to
// the MMAs it needs (even), a part of the exponentials on the FMA pipe as a polynomial
// (1545 -> 1445 cycles for one softmax alone, 2500 -> 2400-2700 for two at once).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

using paged::all_wait;
using paged::tma_load_3d;
using paged::uniform;

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kDv = 128;
constexpr uint32_t kBox = 128 * 128;                   // 128 rows of 64 columns: 16 KB
constexpr int kRing = 8;
constexpr uint32_t kOffQ = 0;                          // two tiles of three boxes
constexpr uint32_t kOffRing = 6 * kBox;
constexpr uint32_t kOffBar = kOffRing + kRing * kBox;
// barriers: full[4] (units), empty[8] (boxes), q_full[2], q_empty[2], s_full[2], p_full[2],
// o_full[2], turn[2], drain
constexpr uint32_t kNumBars = 4 + kRing + 12 + 1;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr uint32_t kIdescS = instr_desc(kFmtBF16, kFmtBF16, 0, 0, kBM, kBN);
constexpr uint32_t kIdescPV = instr_desc(kFmtBF16, kFmtBF16, 0, 1, kBM, kDv);
constexpr uint32_t kIdescPV64 = instr_desc(kFmtBF16, kFmtBF16, 0, 1, kBM, 64);
// A row's weights are 2^(score - reference).  P is bf16 and O fp32, with 8-bit
// exponents both, so any reference within a factor of 2^32 or so of the row's largest
// weight serves: it starts at 0 and is moved, to the tile's maximum, only when a
// tile's weights add up to more than kMost, or the first ones that a row sees to less
// than kLeast.  (Values of up to 2^70 times 2^32 and a sum over 2^24 keys stay finite; weights down
// to 2^-94 of the first stay above the smallest normal number.)  Starting from the
// first tile's maximum cost that tile twice, and a limit of 2^8 every other tile
// of a row that began with a few keys of its window.
constexpr float kMost = 4294967296.f;         // 2^32
constexpr float kLeast = 2.3283064e-10f;      // 2^-32

static_assert(kSmem <= 232448, "shared memory budget");

struct Params {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t total_k;
  int B, H;
  int max_len_q;
  int pairs;                // query-tile pairs per sequence slot
  int window, sinks;        // window 0: no limit
  int items, rounds;        // rounds: items per CTA
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  DevErr err;
};

// One work item: query rows [q0, q0 + rows) of sequence b, head h.
struct Item {
  int b, h, q0, rows, tiles;   // tiles: query tiles, 1 or 2 (0: nothing here)
  int cq, ck, len_k, off;      // query i of the sequence sits at position off + i
  int a, w0;                   // key tiles: the first a, then from w0 on
  int n;                       // steps; one key tile each, but for
  int pair;                    // 1: the last step, with query tile 0 on tile w0 - 1, 1 on the next
  __device__ __forceinline__ int key_tile(int i, int t) const {
    return pair != 0 && i == n - 1 && t == 0 ? w0 - 1 : i < a ? i : w0 + (i - a);
  }
  __device__ __forceinline__ bool split(int i) const { return pair != 0 && i == n - 1; }
};

// What query tile t (rows of one accumulator) sees of key tile j.
struct Rows {
  int p0, p1, lo;              // positions of its rows, first key of its first row's window
  __device__ __forceinline__ Rows(const Params& P, const Item& x, int t) {
    p0 = x.off + x.q0 + t * kBM;
    p1 = x.off + x.q0 + min(x.rows, (t + 1) * kBM) - 1;
    lo = P.window > 0 ? max(0, p0 - P.window + 1) : 0;
  }
  __device__ __forceinline__ bool any(const Params& P, int j) const {
    return j * kBN <= p1 && (j * kBN + kBN > lo || j * kBN < P.sinks);
  }
  __device__ __forceinline__ bool all(const Params& P, int j) const {
    return j * kBN + kBN - 1 <= p0 &&
           (P.window == 0 || j * kBN > p1 - P.window || j * kBN + kBN <= P.sinks);
  }
};

// A CTA's n-th item.  Every other round of the grid goes backwards: the items' work
// repeats with the heads, and in one direction a CTA would keep meeting the long ones
// (causal, L = 4096, 128 heads: the busiest CTA has 1.23 times the mean, this way 1.07).
__device__ __forceinline__ Item item_of(const Params& P, int n) {
  Item x;
  const uint32_t c = (n & 1) != 0 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  uint32_t i = static_cast<uint32_t>(n) * gridDim.x + c;
  const bool none = i >= static_cast<uint32_t>(P.items);   // (the last round's rest, or past it)
  if (none) i = 0;
  // the query tiles of a head are neighbours: they share its keys in L2; the
  // last ones, which may have the most keys, go first
  const uint32_t bh = i / static_cast<uint32_t>(P.pairs);
  x.b = static_cast<int>(bh / static_cast<uint32_t>(P.H));
  x.h = static_cast<int>(bh) - x.b * P.H;
  x.q0 = (P.pairs - 1 - static_cast<int>(i - bh * P.pairs)) * (2 * kBM);
  x.cq = __ldg(P.cu_q + x.b);
  x.ck = __ldg(P.cu_k + x.b);
  const int len_q = __ldg(P.cu_q + x.b + 1) - x.cq;
  x.len_k = __ldg(P.cu_k + x.b + 1) - x.ck;
  x.off = x.len_k - len_q;
  x.rows = min(2 * kBM, min(len_q, P.max_len_q) - x.q0);
  if (none) x.rows = 0;
  x.tiles = x.rows <= 0 || x.off < 0 ? 0 : (x.rows > kBM ? 2 : 1);
  const int p0 = x.off + x.q0, p1 = p0 + x.rows - 1;
  const int lo = P.window > 0 ? max(0, p0 - P.window + 1) : 0;
  x.a = (min(P.sinks, lo) + kBN - 1) / kBN;
  x.w0 = max(lo / kBN, x.a);
  x.n = x.a + p1 / kBN + 1 - x.w0;
  // A window's first key tile is query tile 0's alone, its last one query tile 1's:
  // they make one step, the last.  (One after the other they left a query tile idle at
  // each end, and the next item's keys came late: the ring held the other's last
  // tiles.  L = 4096, 128 heads: window 128 176 -> 163 us, 1024 368 -> 364.)
  x.pair = x.tiles == 2 && !Rows(P, x, 1).any(P, x.w0) && !Rows(P, x, 0).any(P, p1 / kBN) ? 1 : 0;
  if (x.pair != 0) {
    ++x.w0;
    --x.n;
  }
  return x;
}

// Bits [lo, hi) of a 32-bit word.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  const uint32_t below = hi == 32 ? 0xFFFFFFFFu : (1u << hi) - 1u;
  const uint32_t skip = lo == 32 ? 0xFFFFFFFFu : (1u << lo) - 1u;
  return below & ~skip;
}

__global__ void __launch_bounds__(kThreads, 1)
    window_mha_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto full = [&](uint32_t unit) { return bar0 + 8u * (unit & 3); };
  auto empty = [&](uint32_t box) { return bar0 + 8u * (4 + (box & (kRing - 1))); };
  auto q_full = [&](int t) { return bar0 + 8u * (4 + kRing + t); };
  auto q_empty = [&](int t) { return bar0 + 8u * (6 + kRing + t); };
  auto s_full = [&](int t) { return bar0 + 8u * (8 + kRing + t); };
  auto p_full = [&](int t) { return bar0 + 8u * (10 + kRing + t); };
  auto o_full = [&](int t) { return bar0 + 8u * (12 + kRing + t); };
  auto turn = [&](int t) { return bar0 + 8u * (14 + kRing + t); };
  const uint32_t drain = bar0 + 8u * (16 + kRing);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) mbar_init(full(i), 1);
    for (int i = 0; i < kRing; ++i) mbar_init(empty(i), 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(q_empty(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 4);
      mbar_init(o_full(t), 1);
      mbar_init(turn(t), 1);
    }
    mbar_init(drain, 2);
    fence_barrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA
    uint32_t box = 0, unit = 0, nq0 = 0, nq1 = 0;
    bool ok = true;
    // one unit (a step's key or value tile, or two of them): its boxes, announced on its barrier
    auto load = [&](const CUtensorMap* m, int each, int h, int row, int second) {
      const int boxes = second < 0 ? each : 2 * each;
#pragma unroll 1
      for (int c = 0; ok && c < boxes; ++c, ++box) {
        ok = all_wait(empty(box), ((box / kRing) & 1) ^ 1, P.err);
        if (!ok) break;
        if (lane == 0) {
          if (c == 0) mbar_arrive_expect_tx(full(unit), static_cast<uint32_t>(boxes) * kBox);
          tma_load_3d(sbase + kOffRing + (box & (kRing - 1)) * kBox, m,
                      64 * (c < each ? c : c - each), h, c < each ? row : second, full(unit));
        }
        __syncwarp();
      }
      if (ok) ++unit;
    };
#pragma unroll 1
    for (int it = 0; ok && it < P.rounds; ++it) {
      const Item x = item_of(P, it);
      // more queries than keys (there is no such sequence), or than the call allows
      if (lane == 0 && x.rows > 0 &&
          (x.off < 0 || __ldg(P.cu_q + x.b + 1) - x.cq > P.max_len_q))
        raise_error(P.err, kErrBounds);
      if (x.tiles == 0) continue;
      auto queries = [&](int t) {
        ok = ok && all_wait(q_empty(t), ((t ? nq1 : nq0) & 1) ^ 1, P.err);
        if (!ok) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full(t), 3 * kBox);
#pragma unroll 1
          for (int c = 0; c < 3; ++c)
            tma_load_3d(sbase + kOffQ + (3 * t + c) * kBox, &tq, 64 * c, x.h, x.cq + x.q0 + t * kBM,
                        q_full(t));
        }
        __syncwarp();
        if (t) ++nq1; else ++nq0;
      };
      queries(0);
#pragma unroll 1
      for (int j = 0; ok && j < x.n; ++j) {
        const int row = x.ck + x.key_tile(j, 0) * kBN;
        const int second = x.split(j) ? x.ck + x.key_tile(j, 1) * kBN : -1;
        load(&tk, 3, x.h, row, second);
        // (query tile 1 is done with the item before later than tile 0)
        if (j == 0 && x.tiles > 1) queries(1);
        load(&tv, 2, x.h, row, second);
      }
    }
    // Let the copies in flight land before the memory goes: this warp may have asked
    // for its last unit when the ones that wait for it give up.  (After a failure of
    // its own, a unit may also have been asked for in part.)
    if (lane == 0) {
      if (nq0 > 0) mbar_wait_drain(q_full(0), (nq0 - 1) & 1, P.err);
      if (nq1 > 0) mbar_wait_drain(q_full(1), (nq1 - 1) & 1, P.err);
      for (uint32_t u = unit > 3 ? unit - 3 : 0; u <= unit; ++u)
        if (u < unit || (!ok && box > 0)) mbar_wait_drain(full(u), (u / 4) & 1, P.err);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA
    // Warp 1 issues for query tile 0, warp 2 for tile 1, in turns: P V of one
    // key tile and S of the next, then the other query tile's.  The turns keep
    // the two tiles half a step apart, so that one's softmax runs under the
    // other's products (left to themselves the two fall into step: both softmaxes
    // at once, then all the products: 5500 against 4000 cycles).  A single issuer
    // for both tiles loses about 800 cycles a step to its own waits.
    const int t = static_cast<int>(uniform(warp - 1));
    const uint32_t sc = tmem + 128u * t, oc = tmem + kColO + 128u * t;
    const uint64_t dQ = smem_desc(sbase + kOffQ + 3 * t * kBox, 16, 1024, kSwizzle128B);
    const uint64_t dR = smem_desc(sbase + kOffRing, 16, 1024, kSwizzle128B);
    // a value tile: two boxes of 64 dims, MN-major
    const uint64_t dV = smem_desc(sbase + kOffRing, kBox, 1024, kSwizzle128B);
    uint32_t box = 0, unit = 0, ns = 0, nq = 0, turns = 0;
    bool ok = true;
    // The next item is looked up while this one's first softmax runs: at an item's
    // end the lookup (loads, divisions, code not in the cache) cost 3000 cycles.
    Item nx = item_of(P, 0);
#pragma unroll 1
    for (int it = 0; ok && it < P.rounds;) {
      const Item x = nx;
      ++it;
      if (x.tiles == 0) {
        nx = item_of(P, it);
        continue;
      }
      const Rows mine(P, x, t), other(P, x, t ^ 1);
      auto needs = [&](int u, int i) -> bool {
        return u < x.tiles && (u == t ? mine : other).any(P, x.key_tile(i, u));
      };
      int last = x.n - 1;         // the tile's last key tile
      while (t < x.tiles && last > 0 && !needs(t, last)) --last;
      if (t < x.tiles) {
        ok = all_wait(q_full(t), nq & 1, P.err);
        ++nq;
      }
      uint32_t more = 0;          // 1: O holds something
      // (i = -1: only the scores of the first key tile)
#pragma unroll 1
      for (int i = -1; ok && i < x.n; ++i) {
        const bool pv = i >= 0 && needs(t, i), sn = i + 1 < x.n && needs(t, i + 1);
        // (a step in which the other query tile has no weights to wait for is no turn)
        const bool both = pv && needs(t ^ 1, i);
        // the step's value boxes, the next one's key boxes; in a split step the query
        // tile's own ones, and after them or before them the other's
        const uint32_t vs = i >= 0 && x.split(i) ? 2 : 0, ks = x.split(i + 1) ? 3 : 0;
        const uint32_t v0 = box, k0 = box + (i >= 0 ? 2 + vs : 0);
        const uint32_t vb = uniform(v0 + vs * t), kb = uniform(k0 + ks * t);
        // Values and the turn first: the weights then meet an issuer with no other wait
        // left (each one costs it 200 cycles, there or not; the weights before the turn:
        // causal 653 against 640 us).  The next keys after the product: they come
        // half a step later, when the other query tile has let go of the boxes (waited for
        // first: 654 against 622).  The issuing lane waits for them alone (640 -> 630; all
        // waits by that lane: 688).
        if (i >= 0) {
          ok = all_wait(full(unit), (unit / 4) & 1, P.err);
          if (!ok) break;
          ++unit;
          // value rows past the sequence are another's (or unwritten memory):
          // their weights are 0, and so must they be (0 * NaN is not)
          const int rem = x.len_k - x.key_tile(i, t) * kBN;
          if (pv && rem < kBN && x.ck + x.len_k < P.total_k) {
#pragma unroll 1
            for (int e = rem * 8 + lane; e < kBN * 8; e += 32) {
              const uint32_t o = (e >> 3) * 128 + (e & 7) * 16;
              *reinterpret_cast<uint4*>(smem + kOffRing + (vb & (kRing - 1)) * kBox + o) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(smem + kOffRing + ((vb + 1) & (kRing - 1)) * kBox + o) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (both) {
          ok = all_wait(turn(t), (turns & 1) ^ (t == 0 ? 1u : 0u), P.err);
          if (!ok) break;
          ++turns;
        }
        if (pv) {
          ok = all_wait(p_full(t), ns & 1, P.err);
          if (!ok) break;
          ++ns;
        }
        tc_fence_after();
        bool lost = false;
        if (elect_one()) {
          if (pv) {
            const uint64_t b0 = dV + (((vb & (kRing - 1)) * kBox) >> 4);
            if ((vb & (kRing - 1)) != kRing - 1) {
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk)
                mma_f16_ts(oc, sc + 8u * kk, b0 + ((kk * 2048) >> 4), kIdescPV, kk > 0 ? 1u : more);
            } else {
              // one value tile in eight wraps around the ring's end: its two
              // boxes are not neighbours, and take an MMA each
#pragma unroll 1
              for (int kk = 0; kk < kBN / 16; ++kk) {
                mma_f16_ts(oc, sc + 8u * kk, b0 + ((kk * 2048) >> 4), kIdescPV64, kk > 0 ? 1u : more);
                mma_f16_ts(oc + 64u, sc + 8u * kk, dV + ((kk * 2048) >> 4), kIdescPV64, kk > 0 ? 1u : more);
              }
            }
            if (i == last) mma_commit(o_full(t));
            mma_commit(empty(vb));
            mma_commit(empty(vb + 1));
          }
          bool there = true;
          if (i + 1 < x.n) {
            there = paged::one_wait(full(unit), (unit / 4) & 1, P.err);
            tc_fence_after();
          }
          lost = !there;
          if (sn && there) {
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              const uint64_t b = dR + ((((kb + c) & (kRing - 1)) * kBox) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f16(sc, dQ + ((c * kBox + kk * 32) >> 4), b + ((kk * 32) >> 4), kIdescS,
                        (c | kk) != 0 ? 1u : 0u);
            }
            mma_commit(s_full(t));
            if (i + 1 == last) mma_commit(q_empty(t));
            mma_commit(empty(kb));
            mma_commit(empty(kb + 1));
            mma_commit(empty(kb + 2));
          }
        }
        __syncwarp();
        if (i + 1 < x.n) {
          ++unit;
          ok = !__any_sync(0xffffffffu, lost);
          if (!ok) break;
        }
        if (pv) more = 1;
        // boxes that this query tile has no use for
        if (i >= 0 && !pv && lane < 2) mbar_arrive(empty(vb + lane));
        if (i + 1 < x.n && !sn && lane < 3) mbar_arrive(empty(kb + lane));
        if (lane < vs) mbar_arrive(empty(v0 + vs * (1 - t) + lane));
        if (lane < ks) mbar_arrive(empty(k0 + ks * (1 - t) + lane));
        if (both && lane == 0) mbar_arrive(turn(t ^ 1));
        box = k0 + (i + 1 < x.n ? 3 + ks : 0);
        if (i < 0) nx = item_of(P, it);
      }
    }
    mma_commit_warp(drain);
    if (lane == 0) mbar_wait_drain(drain, 0, P.err);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    // A warpgroup per query tile, a thread one row.  (Two warpgroups a tile, half a
    // row each, came out even: 1550 against 1700 cycles for the weights, and two
    // barriers between the halves.)
    const int t = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t sc = tmem + lane_base + 128u * t;          // scores, then P
    const uint32_t oc = tmem + lane_base + kColO + 128u * t;
    uint32_t ns = 0, no = 0;
    bool ok = true;
    Item nx = item_of(P, 0);
#pragma unroll 1
    for (int it = 0; ok && it < P.rounds;) {
      const Item x = nx;
      ++it;
      if (t >= x.tiles) {
        nx = item_of(P, it);
        continue;
      }
      const Rows rr(P, x, t);
      const bool row_ok = t * kBM + r < x.rows;
      const int i = x.q0 + (row_ok ? t * kBM + r : x.rows - 1);   // local query index
      const int p = x.off + i;
      const int first = P.window > 0 ? max(0, p - P.window + 1) : 0;
      float m = 0.f;              // the row's reference
      // sums of the weights, and of the weights as rounded to bf16 for the product:
      // O is divided by the latter, so that its weights add up to one exactly (a
      // row that sees one key, or all but one from afar, gets that key's value)
      float2 l = make_float2(0.f, 0.f), lr = l;
#pragma unroll 1
      for (int k = 0; k < x.n; ++k) {
        const int j = x.key_tile(k, t);
        if (!rr.any(P, j)) continue;
        ok = all_wait(s_full(t), ns & 1, P.err);
        if (!ok) break;
        ++ns;
        tc_fence_after();
        uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
        const bool whole = rr.all(P, j);
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int s0 = j * kBN + 32 * c;
            see[c] = bit_range(first - s0, p + 1 - s0) | bit_range(0, min(P.sinks, p + 1) - s0);
          }
        }
        uint32_t pk[64];
        float2 sum, sumr;
        // the weights over the reference m: 32 columns at a time, the next ones
        // arriving under this one's arithmetic
        auto weigh = [&]() {
          const float2 s2 = make_float2(P.scale_log2, P.scale_log2), n2 = make_float2(-m, -m);
          sum = sumr = make_float2(0.f, 0.f);
          auto part = [&](int c, uint32_t (&v)[32]) {
            // (a warp's rows cross few of a tile's quarters: 445 cycles for a masked one)
            if (!whole && __any_sync(0xffffffffu, see[c] != ~0u)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((see[c] >> e) & 1u)) v[e] = 0xff800000u;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])),
                                          s2, n2);
              const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
              sum = __fadd2_rn(sum, w);
              const uint32_t b = pack_bf16x2(w.x, w.y);
              sumr = __fadd2_rn(sumr, make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)));
              pk[16 * c + e] = b;
            }
          };
          uint32_t va[32], vb[32];
          tmem_ld_32x32b_x32(sc, va);
          tmem_wait_ld();
          tmem_ld_32x32b_x32(sc + 32u, vb);
          part(0, va);
          tmem_wait_ld();
          tmem_ld_32x32b_x32(sc + 64u, va);
          part(1, vb);
          tmem_wait_ld();
          tmem_ld_32x32b_x32(sc + 96u, vb);
          part(2, va);
          tmem_wait_ld();
          part(3, vb);
        };
        weigh();
        const float all = sum.x + sum.y;
        const bool fresh = l.x + l.y == 0.f;          // the row has no weight yet
        if (__any_sync(0xffffffffu, all > kMost || (all < kLeast && fresh &&
                                                    (see[0] | see[1] | see[2] | see[3]) != 0u))) {
          // the tile's maximum first
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(sc + 32u * c, v);
            tmem_wait_ld();
            const uint32_t bits = c == 0 ? see[0] : c == 1 ? see[1] : c == 2 ? see[2] : see[3];
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((bits >> e) & 1u) mx = fmaxf(mx, __uint_as_float(v[e]));
          }
          mx *= P.scale_log2;
          // up, or for a row without a weight yet also down
          float al = 1.f;
          if (mx > m || (fresh && mx > -INFINITY)) {
            al = fresh ? 0.f : fast_exp2(m - mx);
            m = mx;
            l = __fmul2_rn(l, make_float2(al, al));
            lr = __fmul2_rn(lr, make_float2(al, al));
          }
          // O is complete up to the tile before: its product was issued before
          // these scores'
          if (k > 0 && __any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(oc + 32u * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
              tmem_st_32x32b_x32(oc + 32u * c, o);
            }
          }
          weigh();
        }
        l = __fadd2_rn(l, sum);
        lr = __fadd2_rn(lr, sumr);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = pk[32 * c + e];
          tmem_st_32x32b_x32(sc + 32u * c, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t));
      }
      if (!ok) break;
      // ---------------------------------------------------------- read-out
      const int64_t row = static_cast<int64_t>(x.cq + i) * P.H + x.h;
      nx = item_of(P, it);        // (under the last product)
      ok = all_wait(o_full(t), no & 1, P.err);
      if (!ok) break;
      ++no;
      tc_fence_after();
      const float total = l.x + l.y, rounded = lr.x + lr.y;
      const float inv = rounded == 0.f ? 0.f : 1.f / rounded;
      // Eight lanes trade their rows' 16-byte pieces, so that a store covers whole
      // lines (a row's neighbour lies H * 256 bytes away: with a lane per row every
      // store touched 32 lines, 4500 cycles for the tile).
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        uint32_t u[8][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(oc + 64u * half + 32u * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e)
            u[4 * c + e / 4][e & 3] =
                pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) {
          const bool up = (lane & d) != 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (j & d) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? u[j][e] : u[j | d][e], d);
              if (up) u[j][e] = got; else u[j | d][e] = got;
            }
          }
        }
        // u[j]: piece lane % 8 of row j of the eight
        const int r0 = t * kBM + (warp & 3) * 32 + (lane & ~7);
        __nv_bfloat16* dst = P.out + (static_cast<int64_t>(x.cq + x.q0 + r0) * P.H + x.h) * kDv +
                             64 * half + 8 * (lane & 7);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r0 + j < x.rows)
            *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(j) * P.H * kDv) =
                make_uint4(u[j][0], u[j][1], u[j][2], u[j][3]);
      }
      if (row_ok && P.lse)
        P.lse[row] = total == 0.f ? -INFINITY : (m + log2f(total)) * 0.69314718055994531f;
      // the next item's first product over O waits for this warp's P, which
      // comes after these reads
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_window_mha(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const WindowMhaArgs& a, DevErr err, cudaStream_t s) {
  Params P;
  P.cu_q = a.cu_q;
  P.cu_k = a.cu_k;
  P.total_k = a.total_k;
  P.B = a.B;
  P.H = a.H;
  P.max_len_q = a.max_len_q;
  P.pairs = (a.max_len_q + 2 * kBM - 1) / (2 * kBM);
  P.window = a.window;
  P.sinks = a.sinks;
  P.items = a.B * a.H * P.pairs;     // (below 2^30: the caller checks)
  P.scale_log2 = a.sm_scale * 1.4426950408889634f;
  P.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  P.err = err;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(window_mha_kernel, static_cast<int>(kSmem), allowed);
  if (e != cudaSuccess) return e;
  const int grid = P.items < a.num_sms ? P.items : a.num_sms;
  P.rounds = (P.items + grid - 1) / grid;
  window_mha_kernel<<<grid, kThreads, kSmem, s>>>(tq, tk, tv, P);
  return cudaGetLastError();
}

}  // namespace dsa
