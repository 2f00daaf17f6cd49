// paged_mass.cu -- the attention weight that each entry of a paged latent
// cache gets from a sequence's newest token, summed over the heads and added
// to a running total, on sm_100a.
//
//   mass_out[b,s] = mass_in[b,s] + sum_h exp(scale q[b,h,:] . x[s] - lse[b,h])
//
// for the entries s the token sees, and mass_in[b,s] for the others below the
// sequence's length (x[s] the cached 576-d latent; lse from the attention call).
//
// The scores are formed with the keys as the MMA's 128 rows and the heads as its
// columns, S^T [128 x N] = X Q^T with N = H up to 128 heads in one CTA: a thread
// of the read-out then owns one key and sums its heads in registers, so no sum
// crosses a lane, every total is written by one thread, and the result does not
// depend on timing.  More than 128 heads are done in launches of 128, each adding
// to the one before.
//
// A latent is used once, so the kernel is a stream: 64-column chunks of the
// tiles (16 KB) go through a ring of as many stages as the queries leave room for
// (5 beside 128 heads), and two score buffers in TMEM let the read-out of one
// tile overlap the products of the next.  One read of the cache (1152 bytes an
// entry) bounds it: the 36 MMAs of a tile take 2300 cycles at N = 128, its bytes
// about 6300 of an SM's share of the memory.  16 sequences of 4K-128K (1.18 GB), 128
// heads: 198-222 us, 5.3-6.0 TB/s.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

using namespace paged;

constexpr int kTile = 128;                             // keys per tile (MMA M)
constexpr uint32_t kChunkBytes = kTile * 128;          // one 64-column chunk of a tile: 16 KB
constexpr int kMaxStages = 12;
constexpr uint32_t kOffBar = 0;                       // full[12], empty[12], q_full, q_empty, s_full[2], s_empty[2], drain
constexpr uint32_t kNumBars = 2 * kMaxStages + 7;
constexpr uint32_t kOffMisc = kNumBars * 8;           // TMEM slot, plan scratch
constexpr uint32_t kOffLse = (kOffMisc + 96 + 127) / 128 * 128;   // [2][128]: -lse
constexpr uint32_t kOffQ = (kOffLse + 2 * 128 * 4 + 1023) / 1024 * 1024;
constexpr int kWarps = 8;                             // 2 load, MMA, idle, 4 read-out
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kSmemMax = 232448 - 1024;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  Cache c;
  int H, h0, heads;       // all heads; the launch's first and count
  int n_mma;              // MMA N: heads
  int stages, pieces;
  float scale;
  const float* lse;       // [B, H]
  const float* in;        // nullable
  float* out;
  int64_t ld;
  DevErr err;
};

__host__ __device__ constexpr uint32_t q_bytes(int heads) { return static_cast<uint32_t>(kChunks) * heads * 128; }

__global__ void __launch_bounds__(kThreads, 1)
    paged_mass_kernel(const __grid_constant__ CUtensorMap tq,
                      const __grid_constant__ CUtensorMap tx, const Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + kOffBar;
  auto full = [&](int i) { return bar0 + 8u * i; };
  auto empty = [&](int i) { return bar0 + 8u * (kMaxStages + i); };
  const uint32_t q_full = bar0 + 8u * (2 * kMaxStages), q_empty = q_full + 8;
  auto s_full = [&](uint32_t i) { return q_full + 16 + 8u * i; };
  auto s_empty = [&](uint32_t i) { return q_full + 32 + 8u * i; };
  const uint32_t drain = q_full + 48;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffMisc);
  int* scratch = reinterpret_cast<int*>(smem + kOffMisc + 16);
  const uint32_t off_x = (kOffQ + q_bytes(P.heads) + 1023) / 1024 * 1024;

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < P.stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(s_empty(i), 4);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tx);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  const Start start = find_start<kTile, false>(P.c, blockIdx.x, P.pieces, 0, kWarps, scratch, P.err);
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  Walk<kTile> w(P.c, start, 0);

  if (warp < 2) {
    // ------------------------------------------------------------ loads
    // The two warps take every other chunk of the stream.
    uint32_t t = 0;               // chunks of the stream so far
    bool ok = true;
    int seg = 0;
#pragma unroll 1
    for (; ok && w.next(seg == 0); ++seg) {
      if (warp == 0) {
        if (seg > 0) ok = all_wait(q_empty, (seg - 1) & 1, P.err);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, q_bytes(P.heads));
#pragma unroll 1
          for (int c = 0; c < kChunks; ++c)
            tma_load_2d(sbase + kOffQ + c * P.heads * 128, &tq, 64 * c, w.b * P.H + P.h0, q_full);
        }
      }
      Box x = box_of(P.c, w.k, w.b, w.k.tile(w.i0), lane, P.err);
#pragma unroll 1
      for (int i = w.i0; ok && i < w.i1; ++i) {
        Box nx;
        nx.on = false;
        if (i + 1 < w.i1) {
          nx = box_of(P.c, w.k, w.b, w.k.tile(i + 1), lane, P.err);
          if (warp == 1) prefetch_box(P.c, nx);
        }
        const uint32_t bytes =
            __popc(__ballot_sync(0xffffffffu, x.on)) * static_cast<uint32_t>(P.c.box) * 128;
        const uint32_t at = static_cast<uint32_t>(lane * P.c.box) * 128;
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c, ++t) {
          if ((t & 1) != static_cast<uint32_t>(warp)) continue;
          const uint32_t st = t % P.stages;
          ok = all_wait(empty(st), ((t / P.stages) & 1) ^ 1, P.err);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(full(st), bytes);
          __syncwarp();
          if (x.on)
            tma_load_3d(sbase + off_x + st * kChunkBytes + at, &tx, 64 * c, x.row, x.page, full(st));
        }
        x = nx;
      }
    }
    // Let the copies in flight land before the memory goes (these warps may have
    // asked for their last chunk when the ones that wait for it give up): every stage's
    // newest phase completes, or the wait's limit passes.
    if (lane == 0) {
      if (warp == 0 && seg > 0) mbar_wait_drain(q_full, (seg - 1) & 1, P.err);
#pragma unroll 1
      for (uint32_t u = t > static_cast<uint32_t>(P.stages) ? t - P.stages : 0; u < t; ++u)
        if ((u & 1) == static_cast<uint32_t>(warp))
          mbar_wait_drain(full(u % P.stages), (u / P.stages) & 1, P.err);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA
    const uint32_t idesc = instr_desc(kFmtBF16, kFmtBF16, 0, 0, 128, 0) |
                           (static_cast<uint32_t>(P.n_mma >> 3) << 17);
    const uint64_t dX = smem_desc(sbase + off_x, 16, 1024, kSwizzle128B);
    const uint64_t dQ = smem_desc(sbase + kOffQ, 16, 1024, kSwizzle128B);
    uint32_t t = 0, n = 0, st = 0, ph = 0;
    bool ok = true;
#pragma unroll 1
    for (int seg = 0; ok && w.next(seg == 0); ++seg) {
      ok = all_wait(q_full, seg & 1, P.err);
#pragma unroll 1
      for (int i = w.i0; ok && i < w.i1; ++i, ++n) {
        ok = all_wait(s_empty(n & 1), ((n >> 1) & 1) ^ 1, P.err);
#pragma unroll 1
        for (int c = 0; ok && c < kChunks; ++c, ++t) {
          ok = all_wait(full(st), ph, P.err);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a = dX + ((st * kChunkBytes) >> 4);
            const uint64_t b = dQ + ((c * P.heads * 128) >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16(tmem + 128u * (n & 1), a + ((kk * 32) >> 4), b + ((kk * 32) >> 4), idesc,
                      c + kk > 0 ? 1u : 0u);
            mma_commit(empty(st));
            if (c == kChunks - 1) {
              mma_commit(s_full(n & 1));
              if (i + 1 == w.i1) mma_commit(q_empty);
            }
          }
          __syncwarp();
          if (++st == static_cast<uint32_t>(P.stages)) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
    mma_commit_warp(drain);
    if (lane == 0) mbar_wait_drain(drain, 0, P.err);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ read-out
    const int sp = warp & 3;
    const int r = sp * 32 + lane;
    const int tid = threadIdx.x - 128;
    const uint32_t lane_base = static_cast<uint32_t>(sp * 32) << 16;
    float* ml = reinterpret_cast<float*>(smem + kOffLse);
    uint32_t n = 0;
    bool ok = true;
#pragma unroll 1
    for (int seg = 0; w.next(seg == 0); ++seg) {
      // this segment's -lse, in a buffer that the segment before last used
      float* lse = ml + (seg & 1) * 128;
      if (tid < P.heads)
        lse[tid] = -__ldg(P.lse + static_cast<int64_t>(w.b) * P.H + P.h0 + tid);
      // the barrier also takes the four warps out together when a wait gave up
      if (named_bar_or(1, 128, !ok)) {
        ok = false;
        break;
      }
#pragma unroll 1
      for (int i = w.i0; ok && i < w.i1; ++i, ++n) {
        const int s = w.k.tile(i) * kTile + r;
        const int64_t at = static_cast<int64_t>(w.b) * P.ld + s;
        float total = 0.f;
        if (P.in && s < w.k.len) total = P.in[at];
        ok = all_wait(s_full(n & 1), (n >> 1) & 1, P.err);
        if (!ok) break;
        tc_fence_after();
        float2 sum = make_float2(0.f, 0.f), sum2 = sum;
        // The change to base 2 comes after the difference, so that no error grows with the
        // scores' size: with scale and lse changed before, a head's
        // weights at an lse of 290 were all off by 8e-6 alike.
        const float2 sc = make_float2(P.scale, P.scale), to2 = make_float2(kLog2e, kLog2e);
#pragma unroll 1
        for (int h = 0; h < P.n_mma; h += 16) {
          uint32_t v[16];
          tmem_ld_x16(tmem + lane_base + 128u * (n & 1) + h, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 m = *reinterpret_cast<const float4*>(lse + h + e);
            const float2 y = __fmul2_rn(__ffma2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                                   sc, make_float2(m.x, m.y)), to2);
            const float2 z = __fmul2_rn(__ffma2_rn(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                                   sc, make_float2(m.z, m.w)), to2);
            sum = __fadd2_rn(sum, make_float2(fast_exp2(y.x), fast_exp2(y.y)));
            sum2 = __fadd2_rn(sum2, make_float2(fast_exp2(z.x), fast_exp2(z.y)));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty(n & 1));
        if (s < w.k.len)
          P.out[at] = w.k.key(s) ? total + ((sum.x + sum.y) + (sum2.x + sum2.y)) : total;
      }
    }
    // The entries between the first tokens' tiles and the window's, which no
    // tile above covers, keep their totals (without a window there are none).  The
    // sequences are spread over the grid's read-out warps, a sequence over several where
    // these are more.  (With every CTA looking at every sequence 2048 of 100-700 entries, 16
    // heads, took 921 us with a window of 64 and 378 without, so 110 and 180; 16 of
    // 4K-128K, 128 heads, window 4096: 37.8, so 24.4.)
    if (P.in != P.out && P.c.window > 0) {
      constexpr int kPer = 8;           // loads in flight per lane
      const int warps = static_cast<int>(gridDim.x) * 4, me = static_cast<int>(blockIdx.x) * 4 + sp;
      const int split = max(1, warps / P.c.B), step = warps / split;
#pragma unroll 1
      for (int b = me < step * split ? me / split : P.c.B; b < P.c.B; b += step) {
        const Seen<kTile> k = seen_of<kTile>(P.c, seq_len(P.c, b));
        const int64_t row = static_cast<int64_t>(b) * P.ld;
        const int end = k.w0 * kTile;
#pragma unroll 1
        for (int s = k.a * kTile + me % split * (32 * kPer) + lane; s < end; s += split * (32 * kPer)) {
          float v[kPer];
#pragma unroll
          for (int u = 0; u < kPer; ++u)
            v[u] = P.in && s + 32 * u < end ? P.in[row + s + 32 * u] : 0.f;
#pragma unroll
          for (int u = 0; u < kPer; ++u)
            if (s + 32 * u < end) P.out[row + s + 32 * u] = v[u];
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace

cudaError_t launch_paged_mass(const CUtensorMap* tq, int launches, const CUtensorMap& tx,
                              const PagedMassArgs& a, const DevErr* err, cudaStream_t s) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(paged_mass_kernel, 232448, allowed);
  if (e != cudaSuccess) return e;
  for (int i = 0; i < launches; ++i) {
    Params P;
    P.c = a.cache;
    P.H = a.H;
    P.h0 = 128 * i;
    P.heads = a.H - P.h0 < 128 ? a.H - P.h0 : 128;
    P.n_mma = P.heads;
    const uint32_t off_x = (kOffQ + q_bytes(P.heads) + 1023) / 1024 * 1024;
    const int room = static_cast<int>((kSmemMax - off_x) / kChunkBytes);
    P.stages = room < kMaxStages ? room : kMaxStages;
    const int64_t each = (a.max_len_k + kTile - 1) / kTile;
    const int64_t tiles = static_cast<int64_t>(a.cache.B) * (each > 0 ? each : 1);
    P.pieces = static_cast<int>(tiles < a.num_sms ? tiles : a.num_sms);
    P.scale = a.sm_scale;
    P.lse = a.lse;
    P.in = i == 0 ? a.in : a.out;
    P.out = a.out;
    P.ld = a.ld;
    P.err = err[i];
    const uint32_t smem = 1024 + off_x + static_cast<uint32_t>(P.stages) * kChunkBytes;
    paged_mass_kernel<<<static_cast<unsigned>(P.pieces), kThreads, smem, s>>>(tq[i], tx, P);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace dsa
