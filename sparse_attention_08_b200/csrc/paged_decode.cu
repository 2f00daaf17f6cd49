// paged_decode.cu -- attention of one new token per sequence over a paged
// latent cache, in the MQA mode of MLA, on sm_100a.
//
// What it computes (b a sequence, h a head, x[s] the 576-d latent of entry s,
// its first 512 dims the value, V_b the entries the newest token sees):
//
//   out[b,h,:] = sum_{s in V_b} softmax_s(scale q[b,h,:] . x[s]) x[s, 0:512]
//   lse[b,h]   = log sum_{s in V_b} exp(scale q[b,h,:] . x[s])
//
// One CTA works on up to 64 heads and a run of 64-key tiles.  The products are
// formed with the KEYS (and then the value dims) as the MMA's rows and the heads
// as its columns:
//
//   S^T [64 keys x 64 heads]      = X [64 x 576] Q^T         36 MMAs, M64 N64 K16
//   O^T [4 x 128 dims x 64 heads] += X[:, 0:512]^T P^T       16 MMAs, M128 N64 K16
//
// With the heads as rows the second product would be M = 64 too, at twice the
// time (an M = 64 MMA costs what an M = 128 one does).  The latents are read
// from shared memory as they lie: rows of 64-column chunks are K-major for S^T
// and, transposed, MN-major for O^T; P^T (a key's 64 heads in 128 bytes) is
// written as an MN-major operand.
//
// The softmax needs no maximum over the lanes on the common path: any
// reference m[h] within 2^32 of the row's maximum serves (P is bf16 and O fp32,
// both with an 8-bit exponent), so a tile only votes whether a key's weights
// over the references exceed that; then the columns' maxima are reduced and
// O^T and the sums are rescaled.
//
// Shared memory: the heads' queries (72 KB) and two tiles (72 KB each, nine
// chunks in five parts with their own empty barriers).  P^T overwrites the RoPE
// chunk of its tile, which the values do not need.  A part is reloaded as soon as
// its product is done.  The two tiles are half a cycle apart: the softmax of one
// and the reload of its latents run under the products of the other.  Two
// issuers, one for the S^T products and one for the O^T products, so that neither
// waits behind the other.
//
// What bounds it, on 64 sequences of 4K-128K: with up to 64 heads the cache's one
// read (16 heads 780 us, 6.5 TB/s; 64 heads 876 us, 5.8 TB/s); with 128 the tensor
// cores, whose products take 2600 cycles a tile as issued (S^T 1650, M = 64 at 46
// cycles each; O^T 950): 1.50 ms, 815 TFLOP/s.  One tile of 128 keys at a time (M =
// 128 for S^T) needs only 3300 tensor cycles per 128 keys, but idles through its
// softmax and reload: 5900 cycles in all, 1.54 ms with 128 heads and 967 us with 64.
//
// The sequences' tiles stand in one line that is cut into equal pieces, one
// per CTA (times the head groups, which read the same keys at the same time, so
// the second finds them in L2).  A sequence inside one piece is finished there; the
// parts of a split one go to the workspace and combine_kernel joins them in
// the order of the pieces, so the result does not depend on timing.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

using namespace paged;

constexpr int kTile = 64;                             // keys per tile
constexpr int kHeads = 64;                            // heads per CTA (MMA N)
constexpr int kDv = 512;
constexpr uint32_t kChunkBytes = kTile * 128;         // one 64-column chunk of a tile: 8 KB
constexpr uint32_t kTileBytes = kChunks * kChunkBytes;
constexpr uint32_t kQChunk = kHeads * 128;            // 8 KB
constexpr uint32_t kOffX = 0;                         // two tiles
constexpr uint32_t kOffP = 8 * kChunkBytes;           // in a tile: P^T over the RoPE chunk
constexpr uint32_t kOffQ = kOffX + 2 * kTileBytes;
constexpr uint32_t kOffBar = kOffQ + kChunks * kQChunk;
constexpr int kParts = 5;                             // chunk pairs 0..3, the RoPE chunk
// barriers: per tile slot full[3] (parts 0 and 1, parts 2 and 3, part 4), empty[5], s_full, p_full;
// then q_full, q_empty, o_full, o_empty, refs, pv_done, drain
constexpr uint32_t kSlotBars = 3 + kParts + 2;
constexpr uint32_t kNumBars = 2 * kSlotBars + 7;
constexpr int kLoaders = 2;                           // loading warps: warp i brings in parts i, i + 2, i + 4
constexpr int kIssueS = kLoaders, kIssueO = kLoaders + 1;
constexpr int kSoft = 16;                             // softmax warps: eight per tile slot
constexpr int kSoftThreads = 32 * kSoft, kGroupThreads = kSoftThreads / 2;
constexpr int kWarps = kLoaders + 2 + kSoft;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;         // TMEM slot, plan scratch
constexpr uint32_t kOffRef = (kOffMisc + 16 + (kWarps + 4) * 4 + 127) / 128 * 128;   // -m[64], alpha[64]
constexpr uint32_t kOffRed = kOffRef + 2 * kHeads * 4;        // [2][8][64]
constexpr uint32_t kSmem = kOffRed + 16 * kHeads * 4 + 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;                         // + 64 * (dims / 128)
constexpr uint32_t kColS = 256;                       // lanes 0-15 of each 32 for slot 0, 16-31 for slot 1
constexpr uint32_t kIdescS = instr_desc(kFmtBF16, kFmtBF16, 0, 0, kTile, kHeads);
constexpr uint32_t kIdescO = instr_desc(kFmtBF16, kFmtBF16, 1, 1, 128, kHeads);
constexpr float kMost = 4294967296.f;                 // 2^32: largest sum of weights over the references
constexpr float kNoRef = -1e30f;                      // no score yet: any finite one is above
constexpr float kLn2 = 0.69314718055994531f;

static_assert(kSmem <= 232448, "shared memory budget");

struct Params {
  Cache c;
  int H, groups, pieces;
  float scale_log2;
  __nv_bfloat16* out;   // [B, H, 512]
  float* lse;           // [B, H], nullable
  int32_t* plan;        // workspace: [B] first tile of each sequence, [B] tiles per piece
  float4* ml;           // workspace: [2 * pieces * groups][64] reference, sums
  float* part;          // workspace: [2 * pieces * groups][64][512] unnormalised O
  DevErr err;
};

__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tq,
                        const __grid_constant__ CUtensorMap tx, const Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto full = [&](uint32_t slot, int part) { return bar0 + 8u * (slot * kSlotBars + part / 2); };
  auto empty = [&](uint32_t slot, int part) { return bar0 + 8u * (slot * kSlotBars + 3 + part); };
  auto s_full = [&](uint32_t slot) { return bar0 + 8u * (slot * kSlotBars + 3 + kParts); };
  auto p_full = [&](uint32_t slot) { return bar0 + 8u * (slot * kSlotBars + 4 + kParts); };
  const uint32_t q_full = bar0 + 8u * (2 * kSlotBars), q_empty = q_full + 8;
  const uint32_t o_full = q_full + 16, o_empty = q_full + 24;
  const uint32_t refs = q_full + 32, pv_done = q_full + 40, drain = q_full + 48;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc);
  volatile uint32_t* version = tmem_slot + 1;       // counts the changes of the references
  int* scratch = reinterpret_cast<int*>(smem + kOffMisc + 16);
  float* ref = reinterpret_cast<float*>(smem + kOffRef);
  float* alpha = ref + kHeads;
  float* red = reinterpret_cast<float*>(smem + kOffRed);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int g = blockIdx.x % P.groups;
  const int piece = blockIdx.x / P.groups;
  const int heads = min(kHeads, P.H - g * kHeads);

  if (threadIdx.x == 0) {
    for (uint32_t u = 0; u < 2; ++u) {
      mbar_init(full(u, 0), 2);
      mbar_init(full(u, 2), 2);
      mbar_init(full(u, 4), 1);
      for (int i = 0; i < kParts; ++i) mbar_init(empty(u, i), 1);
      mbar_init(s_full(u), 1);
      mbar_init(p_full(u), kSoft / 2);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_full, 1);
    mbar_init(o_empty, kSoft);
    mbar_init(refs, kSoft / 2);
    mbar_init(pv_done, 1);
    mbar_init(drain, 2);
    *version = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tx);
  }
  if (warp == kIssueS) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), kTmemCols);
    tmem_relinquish();
  }
  // query rows past the last head stay zero (their columns are never stored)
  if (heads < kHeads)
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < kChunks * kQChunk / 16; i += kThreads)
      reinterpret_cast<uint4*>(smem + kOffQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  tc_fence_before();
  const Start start = find_start<kTile, true>(P.c, piece, P.pieces, 1, kWarps, scratch, P.err);
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  grid_release();
  if (blockIdx.x == 0 && threadIdx.x == 0) P.plan[P.c.B] = start.per;
  Walk<kTile> w(P.c, start, 1);

  if (warp < kLoaders) {
    // ------------------------------------------------------------ loads
    // Lane i brings in box i of each of the warp's parts of a tile.
    uint32_t n = 0;               // tiles so far: tile n uses slot n % 2
    bool ok = true;
    int seg = 0, stop = 0;        // segments so far, parts of tile n that were asked for
    auto ahead = [&](int i) {
      Box x;
      x.on = false;
      if (i < w.i1) {
        x = box_of(P.c, w.k, w.b, w.k.tile(i), lane, P.err);
        if (warp == 1) prefetch_box(P.c, x);
      }
      return x;
    };
#pragma unroll 1
    for (; ok && w.next(seg == 0); ++seg) {
      // Page ids and an L2 prefetch two tiles ahead, looked up when a tile has been
      // asked for (before that, a segment's first loads wait for three lookups:
      // 48 sequences, window 4096, 64 heads: 66.8 against 64.1 us).
      Box x = box_of(P.c, w.k, w.b, w.k.tile(w.i0), lane, P.err), nx;
#pragma unroll 1
      for (int i = w.i0; i < w.i1; ++i, ++n) {
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, x.on)) *
                               static_cast<uint32_t>(P.c.box) * 128;
        const uint32_t slot = n & 1;
        const uint32_t dst = sbase + kOffX + slot * kTileBytes +
                             static_cast<uint32_t>(lane * P.c.box) * 128;
#pragma unroll 1
        for (int c = warp; c < kParts; c += kLoaders) {
          ok = all_wait(empty(slot, c), ((n >> 1) & 1) ^ 1, P.err);
          if (!ok) {
            stop = c;
            break;
          }
          const uint32_t cols = c < 4 ? 2u : 1u;
          if (lane == 0) mbar_arrive_expect_tx(full(slot, c), bytes * cols);
          __syncwarp();
          if (x.on)
#pragma unroll 1
            for (uint32_t u = 0; u < cols; ++u)
              tma_load_3d(dst + (2 * c + u) * kChunkBytes, &tx, 64 * (2 * c + u), x.row, x.page,
                          full(slot, c));
        }
        if (!ok) break;
        if (i == w.i0) x = ahead(i + 1); else x = nx;
        nx = ahead(i + 2);
      }
      if (!ok) break;
    }
    // Let the copies in flight land before the memory goes: this warp may have asked
    // for its last tile when the ones that wait for it give up.
    if (lane == 0) {
#pragma unroll 1
      for (uint32_t u = 0; u < 2; ++u)
#pragma unroll 1
        for (int c = warp; c < kParts; c += kLoaders) {
          // tiles asked for in slot u: those before n, and n itself up to part `stop`
          const uint32_t asked = (n + 1 - u) / 2 + ((n & 1) == u && c < stop ? 1 : 0);
          if (asked > 0) mbar_wait_drain(full(u, c), (asked - 1) & 1, P.err);
        }
    }
    __syncwarp();
  } else if (warp == kIssueS) {
    // ------------------------------------------------------------ S^T products
    // The whole warp walks the tiles and one elected lane issues each run of
    // MMAs: every operand stays warp-uniform.  (Issued from a one-lane branch an
    // MMA took about 90 cycles to issue, twice its own time.)
    const uint64_t dX = smem_desc(sbase + kOffX, 16, 1024, kSwizzle128B);
    const uint64_t dQ = smem_desc(sbase + kOffQ, 16, 1024, kSwizzle128B);
    uint32_t n = 0;
    bool ok = true;
#pragma unroll 1
    for (int seg = 0; ok && w.next(seg == 0); ++seg) {
      // this warp also brings the queries, while the loaders start on the tiles
      if (seg > 0) ok = all_wait(q_empty, (seg - 1) & 1, P.err);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full, kChunks * static_cast<uint32_t>(heads) * 128);
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c)
          tma_load_2d(sbase + kOffQ + c * kQChunk, &tq, 64 * c, w.b * P.H + g * kHeads, q_full);
      }
      __syncwarp();
      ok = all_wait(q_full, seg & 1, P.err);
      // (after a failure, let the copies land before the memory goes)
      if (!ok && lane == 0) mbar_wait_drain(q_full, seg & 1, P.err);
#pragma unroll 1
      for (int i = w.i0; ok && i < w.i1; ++i, ++n) {
        const uint32_t slot = uniform(n & 1), ph = (n >> 1) & 1;
        const uint64_t a = dX + ((slot * kTileBytes) >> 4);
        const uint32_t d = tmem + kColS + (slot << 20);           // lane offset 16 for slot 1
        // (the slot's last scores have been read: its latents could only be
        // replaced after the product that their weights went into)
        ok = ok && all_wait(full(slot, 0), ph, P.err);
        if (!ok) break;
        tc_fence_after();
        // The issuing lane waits for the other parts alone: with a wait and a vote of
        // the warp between the runs 64 sequences of 4K-128K took 1548 us (128 heads;
        // 64: 900, 16: 800), so 1499 (876, 784).
        bool lost = false;
        if (elect_one()) {
          auto run = [&](int c) {
#pragma unroll
            for (int kk = 0; kk < 16; ++kk)
              mma_f16(d, a + (((c + kk / 4) * kChunkBytes + (kk % 4) * 32) >> 4),
                      dQ + (((c + kk / 4) * kQChunk + (kk % 4) * 32) >> 4), kIdescS,
                      c + kk > 0 ? 1u : 0u);
          };
          run(0);
          lost = !one_wait(full(slot, 2), ph, P.err);
          tc_fence_after();
          if (!lost) run(4);
          lost = lost || !one_wait(full(slot, 4), ph, P.err);
          tc_fence_after();
          if (!lost)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16(d, a + ((8 * kChunkBytes + kk * 32) >> 4), dQ + ((8 * kQChunk + kk * 32) >> 4),
                      kIdescS, 1u);
          mma_commit(s_full(slot));
          if (i + 1 == w.i1) mma_commit(q_empty);
        }
        ok = !__any_sync(0xffffffffu, lost);
      }
    }
    mma_commit_warp(drain);
    if (lane == 0) mbar_wait_drain(drain, 0, P.err);
    __syncwarp();
  } else if (warp == kIssueO) {
    // ------------------------------------------------------------ O^T products
    const uint64_t dX = smem_desc(sbase + kOffX, kChunkBytes, 1024, kSwizzle128B);
    const uint64_t dP = smem_desc(sbase + kOffX + kOffP, kChunkBytes, 1024, kSwizzle128B);
    uint32_t n = 0;
    bool ok = true;
#pragma unroll 1
    for (int seg = 0; ok && w.next(seg == 0); ++seg) {
      // the last segment's O^T must have been read out
      if (seg > 0) ok = all_wait(o_empty, (seg - 1) & 1, P.err);
#pragma unroll 1
      for (int i = w.i0; ok && i < w.i1; ++i, ++n) {
        const uint32_t slot = uniform(n & 1);
        ok = all_wait(p_full(slot), (n >> 1) & 1, P.err);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t a = dX + ((slot * kTileBytes) >> 4), b = dP + ((slot * kTileBytes) >> 4);
          const uint32_t more = i > w.i0 ? 1u : 0u;
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_f16(tmem + kColO + 64u * mt, a + ((mt * 2 * kChunkBytes + kk * 2048) >> 4),
                      b + ((kk * 2048) >> 4), kIdescO, kk > 0 ? 1u : more);
            mma_commit(empty(slot, mt));
          }
          mma_commit(empty(slot, 4));
          mma_commit(pv_done);
          if (i + 1 == w.i1) mma_commit(o_full);
        }
        __syncwarp();
      }
    }
    mma_commit_warp(drain);
    if (lane == 0) mbar_wait_drain(drain, 0, P.err);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // Eight warps per tile slot, two per TMEM sub-partition: a warp has 16 of
    // the tile's keys and 32 of the heads, a thread two keys and eight heads
    // (lane t: keys t/4 and t/4 + 8, heads 8i + 2(t%4) + {0,1}).
    const int grp = (warp - kLoaders - 2) >> 3;       // the slot
    const int half = ((warp - kLoaders - 2) >> 2) & 1;
    const int sp = warp & 3;                          // TMEM sub-partition
    const int tid = threadIdx.x - 32 * (kLoaders + 2);        // 0..511
    const int gtid = tid & (kGroupThreads - 1);       // in the group
    const int ra = sp * 16 + lane / 4, rb = ra + 8;   // keys in the tile
    const int hq = 32 * half + 2 * (lane & 3);        // heads hq + 8i + {0,1}
    const uint32_t scores = tmem + kColS + 32u * half + (static_cast<uint32_t>(sp * 32 + 16 * grp) << 16);
    uint8_t* tile = smem + kOffX + grp * kTileBytes;
    const float2 sc = make_float2(P.scale_log2, P.scale_log2);
    const uint32_t gbar = 1 + grp;
    uint32_t n = 0;
    bool ok = true;
#pragma unroll 1
    for (int seg = 0; w.next(seg == 0); ++seg) {
      // Sums of the weights, and of the weights as rounded to bf16 for the product
      // (O^T is divided by the latter, so that its weights add up to one exactly),
      // and the references they are over.
      float2 l[4], lr[4], rr[4];
      uint32_t seen_version = 0;
      bool mine = false;          // a tile of this segment was this group's
#pragma unroll
      for (int e = 0; e < 4; ++e) l[e] = lr[e] = rr[e] = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int i = w.i0; i < w.i1; ++i, ++n) {
        if (static_cast<int>(n & 1) != grp || !ok) continue;
        const int s0 = w.k.tile(i) * kTile;
        const bool sa = w.k.key(s0 + ra), sb = w.k.key(s0 + rb);
        // the tile before has settled the references
        bool bad = n > 0 && !all_wait(refs, (n - 1) & 1, P.err);
        bad = bad || !all_wait(s_full(grp), (n >> 1) & 1, P.err);
        float2 ya[4], yb[4];      // scores, then over the references, then weights
        auto load = [&]() {
          uint32_t v[16];
          tmem_ld_16x256b_x4(scores, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ya[e] = sa ? make_float2(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]))
                       : make_float2(-INFINITY, -INFINITY);
            yb[e] = sb ? make_float2(__uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]))
                       : make_float2(-INFINITY, -INFINITY);
          }
        };
        // takes over the references in shared memory, and brings the sums to them
        auto adopt = [&]() {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 m = *reinterpret_cast<const float2*>(ref + hq + 8 * e);
            if (mine) {
              const float2 f = make_float2(fast_exp2(m.x - rr[e].x), fast_exp2(m.y - rr[e].y));
              l[e] = __fmul2_rn(l[e], f);
              lr[e] = __fmul2_rn(lr[e], f);
            }
            rr[e] = m;
          }
          seen_version = *version;
          mine = true;
        };
        auto weigh = [&]() -> float {
          float2 all = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ya[e] = __ffma2_rn(ya[e], sc, rr[e]);
            yb[e] = __ffma2_rn(yb[e], sc, rr[e]);
            ya[e] = make_float2(fast_exp2(ya[e].x), fast_exp2(ya[e].y));
            yb[e] = make_float2(fast_exp2(yb[e].x), fast_exp2(yb[e].y));
            all = __fadd2_rn(all, __fadd2_rn(ya[e], yb[e]));
          }
          return all.x + all.y;
        };
        bool over = false;
        if (!bad) {
          tc_fence_after();
          load();
          if (i > w.i0) {
            if (!mine || *version != seen_version) adopt();
            // (a weight above it makes the sum so; so does a NaN, which must not hide
            // one from the vote)
            over = !(weigh() <= kMost);
          }
        }
        // one vote for the group; it also takes its warps out together when a
        // wait of one of them gave up
        if (named_bar_or(gbar, kGroupThreads, bad || over) || i == w.i0) {
          if (named_bar_or(gbar, kGroupThreads, bad)) {
            ok = false;
            continue;                         // (on to the segment's end, where all meet)
          }
          // new references: the columns' maxima over the tile
          if (i > w.i0) load();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 m = make_float2(fmaxf(ya[e].x, yb[e].x) * P.scale_log2,
                                   fmaxf(ya[e].y, yb[e].y) * P.scale_log2);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, d));
              m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, d));
            }
            if (lane < 4) *reinterpret_cast<float2*>(red + sp * kHeads + hq + 8 * e) = m;
          }
          named_bar_sync(gbar, kGroupThreads);
          if (gtid < kHeads) {
            const float old = i > w.i0 ? -ref[gtid] : kNoRef;
            const float top = fmaxf(fmaxf(red[gtid], red[kHeads + gtid]),
                                    fmaxf(red[2 * kHeads + gtid], red[3 * kHeads + gtid]));
            const float now = fmaxf(old, top);
            alpha[gtid] = fast_exp2(old - now);
            ref[gtid] = -now;
            if (gtid == 0) *version = *version + 1;
          }
          named_bar_sync(gbar, kGroupThreads);
          if (i > w.i0) {
            // O^T up to the tile before, in the new measure
            bad = !all_wait(pv_done, (n - 1) & 1, P.err);
            if (named_bar_or(gbar, kGroupThreads, bad)) {
              ok = false;
              continue;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 8 * half; c < 8 * half + 8; ++c) {
              uint32_t o[16];
              const uint32_t at = tmem + kColO + 16u * c + (static_cast<uint32_t>(sp * 32) << 16);
              tmem_ld_x16(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha[(16 * c + e) & (kHeads - 1)]);
              tmem_st_x16(at, o);
            }
            tmem_wait_st();
          }
          adopt();
          weigh();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(refs);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[e] = __fadd2_rn(l[e], __fadd2_rn(ya[e], yb[e]));
          const uint32_t at = ((4 * half + e) ^ (lane / 4)) * 16 + 4 * (lane & 3);
          const uint32_t pa = pack_bf16x2(ya[e].x, ya[e].y), pb = pack_bf16x2(yb[e].x, yb[e].y);
          *reinterpret_cast<uint32_t*>(tile + kOffP + ra * 128 + at) = pa;
          *reinterpret_cast<uint32_t*>(tile + kOffP + rb * 128 + at) = pb;
          lr[e] = __fadd2_rn(lr[e], __fadd2_rn(make_float2(__uint_as_float(pa << 16), __uint_as_float(pa & 0xFFFF0000u)),
                                               make_float2(__uint_as_float(pb << 16), __uint_as_float(pb & 0xFFFF0000u))));
        }
        // an unseen row of the tile holds whatever its memory held: its
        // weight is 0, and so must its value be (0 * NaN is not)
        const int row = gtid >> 2;
        if (!w.k.key(s0 + row)) {
#pragma unroll 1
          for (int c = 2 * (gtid & 3); c < 2 * (gtid & 3) + 2; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<uint4*>(tile + c * kChunkBytes + row * 128 + (j ^ (row & 7)) * 16) =
                  make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(grp));
      }
      // ---------------------------------------------------------- read-out
      // All sixteen warps: the sums of both groups, in the last references.
      bool bad = !ok || !all_wait(o_full, seg & 1, P.err);
      if (named_bar_or(3, kSoftThreads, bad)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float4 t = make_float4(l[e].x, l[e].y, lr[e].x, lr[e].y);
        if (mine) {
          const float2 m = *reinterpret_cast<const float2*>(ref + hq + 8 * e);
          const float2 f = make_float2(fast_exp2(m.x - rr[e].x), fast_exp2(m.y - rr[e].y));
          t = make_float4(t.x * f.x, t.y * f.y, t.z * f.x, t.w * f.y);
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          t.x += __shfl_xor_sync(0xffffffffu, t.x, d);
          t.y += __shfl_xor_sync(0xffffffffu, t.y, d);
          t.z += __shfl_xor_sync(0xffffffffu, t.z, d);
          t.w += __shfl_xor_sync(0xffffffffu, t.w, d);
        }
        if (lane < 4) {
          float* to = red + (4 * grp + sp) * kHeads + hq + 8 * e;
          *reinterpret_cast<float2*>(to) = make_float2(t.x, t.y);
          *reinterpret_cast<float2*>(to + 8 * kHeads) = make_float2(t.z, t.w);
        }
      }
      named_bar_sync(3, kSoftThreads);
      const int tiles = max(w.k.n, 1);
      const bool whole = w.i0 == 0 && w.i1 == tiles;
      const int64_t slot = (static_cast<int64_t>(piece) * 2 + (seg == 0 ? 0 : 1)) * P.groups + g;
      if (tid < heads) {
        float sum = 0.f, sumr = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          sum += red[e * kHeads + tid];
          sumr += red[(8 + e) * kHeads + tid];
        }
        const int64_t at = static_cast<int64_t>(w.b) * P.H + g * kHeads + tid;
        if (whole) {
          if (P.lse) P.lse[at] = sum == 0.f ? -INFINITY : (log2f(sum) - ref[tid]) * kLn2;
        } else {
          P.ml[slot * kHeads + tid] = make_float4(-ref[tid], sum, sumr, 0.f);
        }
        alpha[tid] = sumr == 0.f ? 0.f : 1.f / sumr;
      }
      if (w.i0 == 0 && g == 0 && tid == 0)
        P.plan[w.b] = piece * start.per + start.left - w.left - (w.i1 - w.i0);
      named_bar_sync(3, kSoftThreads);
      const int h0 = 16 * (tid >> 7);                 // a warp's 16 heads of O^T's 128 lanes
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t o[16];
        tmem_ld_x16(tmem + kColO + 64u * mt + h0 + (static_cast<uint32_t>(sp * 32) << 16), o);
        tmem_wait_ld();
        if (whole) {
          // lanes hold neighbouring dims: pairs of lanes swap so that each
          // stores two dims of one head
          const int d = mt * 128 + sp * 32 + (lane & ~1);
          __nv_bfloat16* dst = P.out + (static_cast<int64_t>(w.b) * P.H + g * kHeads + h0) * kDv + d;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 iv = *reinterpret_cast<const float2*>(alpha + h0 + e);
            const float a = __uint_as_float(o[e]) * iv.x, b = __uint_as_float(o[e + 1]) * iv.y;
            const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : b, 1);
            const int h = e + (lane & 1);
            if (h0 + h < heads)
              *reinterpret_cast<uint32_t*>(dst + h * kDv) =
                  (lane & 1) ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
          }
        } else {
          float* dst = P.part + (slot * kHeads + h0) * kDv + mt * 128 + sp * 32 + lane;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (h0 + e < heads) dst[e * kDv] = __uint_as_float(o[e]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
      // the references and sums are read above; the next segment rewrites them
      named_bar_sync(3, kSoftThreads);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kIssueS) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the sequences that were split: with the parts'
// references m_i and M their maximum, out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// One CTA per (head, sequence), a thread four value dims of every kJoin-th part.
// Every warp works out all the weights for itself (a lane has every 32nd part):
// one round of loads, and no barrier before the parts' own loads.
constexpr int kMaxParts = 160;
template <int kJoin>
__global__ void __launch_bounds__(128 * kJoin) combine_kernel(Params P) {
  __shared__ float4 sums[kJoin > 1 ? kJoin - 1 : 1][128];
  const int h = blockIdx.x;
  const int b = blockIdx.y + gridDim.y * blockIdx.z;
  if (b >= P.c.B) return;
  grid_wait();
  const int per = P.plan[P.c.B];
  const int t0 = P.plan[b];
  const int n = max(seen_of<kTile>(P.c, seq_len(P.c, b)).n, 1);
  // (after a launch that gave up on a wait the plan may hold anything)
  if (per < 1 || t0 < 0 || static_cast<int64_t>(t0) + n > static_cast<int64_t>(per) * P.pieces) return;
  const int r0 = t0 / per, r1 = (t0 + n - 1) / per;
  if (r0 == r1) return;
  const int parts = r1 - r0 + 1;
  const int lane = threadIdx.x % 32, k = threadIdx.x / 128, d = threadIdx.x % 128;
  const int g = h / kHeads, hh = h % kHeads;
  auto slot = [&](int i) {
    return ((static_cast<int64_t>(r0 + i) * 2 + (i == 0 && t0 > r0 * per ? 1 : 0)) * P.groups + g) *
               kHeads + hh;
  };
  float4 x[kMaxParts / 32];
  float top = -INFINITY;
#pragma unroll
  for (int u = 0; u < kMaxParts / 32; ++u) {
    x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane + 32 * u < parts) x[u] = P.ml[slot(lane + 32 * u)];
  }
#pragma unroll
  for (int u = 0; u < kMaxParts / 32; ++u)
    if (x[u].y != 0.f) top = fmaxf(top, x[u].x);      // a part without a weight has no reference
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, e));
  float l = 0.f, lr = 0.f;
#pragma unroll
  for (int u = 0; u < kMaxParts / 32; ++u) {
    const float f = x[u].y != 0.f ? exp2f(x[u].x - top) : 0.f;
    l += f * x[u].y;
    lr += f * x[u].z;
    x[u].x = f;
  }
#pragma unroll
  for (int e = 16; e > 0; e >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, e);
    lr += __shfl_xor_sync(0xffffffffu, lr, e);
  }
  // thread group k adds up every kJoin-th part; the groups' sums are then added
  // in their order
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int i, float w) {
    const float4 y = *reinterpret_cast<const float4*>(P.part + slot(i) * kDv + 4 * d);
    const float f = __shfl_sync(0xffffffffu, w, i & 31);
    o.x += f * y.x;
    o.y += f * y.y;
    o.z += f * y.z;
    o.w += f * y.w;
  };
#pragma unroll 4
  for (int i = k; i < min(32, parts); i += kJoin) add(i, x[0].x);
  if (parts > 32) {
#pragma unroll
    for (int u = 1; u < kMaxParts / 32; ++u)
#pragma unroll kJoin > 1 ? 4 : 1
      for (int i = 32 * u + k; i < min(32 * u + 32, parts); i += kJoin) add(i, x[u].x);
  }
  if (kJoin > 1) {
    if (k > 0) sums[k - 1][d] = o;
    __syncthreads();
    if (k > 0) return;
#pragma unroll
    for (int j = 0; j < kJoin - 1; ++j) {
      const float4 y = sums[j][d];
      o.x += y.x;
      o.y += y.y;
      o.z += y.z;
      o.w += y.w;
    }
  }
  const float inv = lr == 0.f ? 0.f : 1.f / lr;
  const int64_t row = static_cast<int64_t>(b) * P.H + h;
  *reinterpret_cast<uint2*>(P.out + row * kDv + 4 * d) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (d == 0 && P.lse) P.lse[row] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

constexpr int kMaxCtas = 148;

int groups_of(int H) { return (H + kHeads - 1) / kHeads; }

// Pieces the tile line is cut into: one CTA per SM over all head groups, and
// no more than there can be tiles.
int pieces_of(int B, int H, int max_len_k) {
  const int64_t each = (max_len_k + kTile - 1) / kTile;
  const int64_t tiles = static_cast<int64_t>(B) * (each > 0 ? each : 1);
  const int64_t most = kMaxCtas / groups_of(H);
  return static_cast<int>(tiles < most ? tiles : most);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t paged_decode_workspace_bytes(int B, int H, int max_len_k) {
  const size_t slots = static_cast<size_t>(2) * pieces_of(B, H, max_len_k) * groups_of(H);
  return up256((static_cast<size_t>(B) + 1) * 4) + slots * kHeads * (16 + kDv * 4);
}

cudaError_t launch_paged_decode(const CUtensorMap& tq, const CUtensorMap& tx,
                                const PagedDecodeArgs& a, DevErr err, cudaStream_t s) {
  Params P;
  P.c = a.cache;
  P.H = a.H;
  P.groups = groups_of(a.H);
  P.pieces = pieces_of(a.cache.B, a.H, a.max_len_k);
  P.scale_log2 = a.sm_scale * 1.4426950408889634f;
  P.out = static_cast<__nv_bfloat16*>(a.out);
  P.lse = a.lse;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  P.plan = reinterpret_cast<int32_t*>(ws);
  ws += up256((static_cast<size_t>(a.cache.B) + 1) * 4);
  P.ml = reinterpret_cast<float4*>(ws);
  ws += static_cast<size_t>(2) * P.pieces * P.groups * kHeads * 16;
  P.part = reinterpret_cast<float*>(ws);
  P.err = err;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(paged_decode_kernel, static_cast<int>(kSmem), allowed);
  if (e != cudaSuccess) return e;
  paged_decode_kernel<<<static_cast<unsigned>(P.pieces * P.groups), kThreads, kSmem, s>>>(tq, tx, P);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.max_len_k <= kTile) return cudaSuccess;     // one tile per sequence: nothing is split
  const unsigned y = a.cache.B < 65535 ? static_cast<unsigned>(a.cache.B) : 65535u;
  const unsigned z = (static_cast<unsigned>(a.cache.B) + y - 1) / y;
  // With few sequences each is cut into many parts, which four thread groups
  // share (one of 131072 entries, 74 parts: 29 -> 13 us); with many, a sequence
  // has two or three and the larger CTAs only cost (48 sequences: 10 against 20 us).
  // Eight groups where every CTA has an SM to itself (one sequence, both kernels: 16
  // heads 53.2 -> 50.9 us, 128 heads 69.4 -> 68.2; 16 sequences of 64 heads 45 -> 55).
  const dim3 grid(static_cast<unsigned>(a.H), y, z);
  if (static_cast<int64_t>(a.cache.B) * a.H <= kMaxCtas)
    return launch_after(combine_kernel<8>, grid, 1024, 0, s, P);
  return a.cache.B * 4 < P.pieces ? launch_after(combine_kernel<4>, grid, 512, 0, s, P)
                                  : launch_after(combine_kernel<1>, grid, 128, 0, s, P);
}

}  // namespace dsa
