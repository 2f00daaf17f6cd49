// cache_evict.cu -- cuts the sequences of a paged latent cache down to a
// budget of entries by a running total per entry, on sm_100a.
//
// A sequence of at most `budget` entries keeps them all.  A longer one keeps
// its first `sinks`, its last `recent`, and the budget - sinks - recent
// entries between them with the largest totals (ties to the lower position).
// The kept entries' latents move, in their order, to the pages of a new block
// table; their positions, totals and the new lengths are written out.
//
// Two launches:
//  * select_kernel: one CTA of 1024 threads per sequence, or a cluster of eight
//    for long ones, each CTA with its stretch of the row as order-preserving
//    32-bit keys in shared memory, read once.  Three histogram passes (11, 11
//    and 10 bits from the top; the CTAs read one another's histograms through
//    distributed shared memory) find the key T of the last entry kept and how
//    many entries equal to it are kept.  Lanes own contiguous stretches, so
//    prefixes over lanes, warps and CTAs give every kept entry its slot in
//    position order, ties to the lower position included.  A chain of
//    barriers and shared-memory atomics bounds it, not the row's bytes: 12 us
//    for a row of 131072 (reading it 3.5, a histogram pass 2, the slots and the
//    writes 3.5), of which its bytes at the memory's rate are 0.1 us.
//  * move_kernel: a warp moves four latents at a time, nine 16-byte loads in
//    flight per lane; bound by the memory (2304 bytes per kept entry): 65536
//    entries in about 27 us, 5.6 TB/s.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

namespace cg = cooperative_groups;
using namespace paged;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kClusterC = 8;
constexpr int kAhead = 16;                // loads in flight per thread while a row is read
constexpr int kOneCta = 8192;            // rows of at most this many entries take one CTA

struct Params {
  Cache c;
  const float* mass;
  int64_t ld_mass;
  int budget, sinks, recent;
  int wseg;               // entries per warp, a multiple of 32
  int32_t* idx;           // [B, budget]
  int32_t* new_lens;      // [B]
  float* new_mass;        // [B, ld_new], nullable
  int64_t ld_new;
  const int32_t* new_table;
  int64_t new_ld;
  DevErr err;
};

// Larger totals map to larger keys; -0 equals +0, every NaN is above all numbers.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0xFFFFFFFFu;
  if ((u << 1) == 0) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Sum of the lanes below this one.
__device__ __forceinline__ uint32_t sum_before(uint32_t v) {
  uint32_t inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, inc, d);
    if (static_cast<int>(threadIdx.x % 32) >= d) inc += x;
  }
  return inc - v;
}

// Where a warp's entry i lies in shared memory: a word of padding per 32, so
// that lanes with stretches of their own do not meet in a bank.
__device__ __forceinline__ int slot_of(int i) { return i + (i >> 5); }

template <int C>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const Params P) {
  extern __shared__ uint32_t keys[];     // [kWarps][slot_of(wseg)]
  __shared__ uint32_t hist[3][kBins];    // a buffer per pass: the other CTAs may still read the last
  __shared__ alignas(8) uint32_t group[3][kBins / 32];
  __shared__ uint32_t wgt[kWarps], weq[kWarps];
  __shared__ uint32_t found[3];          // the pass's bin, the rank left inside it, whether that is all of it
  __shared__ alignas(8) uint32_t xch[2]; // this CTA's entries above T, equal to T
  const int rank = C == 1 ? 0 : static_cast<int>(cg::this_cluster().block_rank());
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  grid_wait();
  grid_release();
  // Lengths and totals by plain loads: the kernel before on the stream may have written
  // them while this one was already here, which a load through the read-only path
  // (__ldg) would rule out, and only plain ones are kept behind the wait.
  const int raw = P.c.lens[b];
  const int n = min(max(raw, 0), P.c.cap);
  const float* row = P.mass + static_cast<int64_t>(b) * P.ld_mass;
  int32_t* idx = P.idx + static_cast<int64_t>(b) * P.budget;
  float* nm = P.new_mass ? P.new_mass + static_cast<int64_t>(b) * P.ld_new : nullptr;
  const int kept = min(n, P.budget);
  auto sync_all = [&]() {
    if (C == 1) __syncthreads(); else cg::this_cluster().sync();
  };
  auto remote = [&](uint32_t* p, int q) -> const uint32_t* {
    return C == 1 ? p : cg::this_cluster().map_shared_rank(p, (rank + q) % C);
  };
  if (rank == 0 && tid == 0) {
    P.new_lens[b] = kept;
    if (raw < 0 || raw > P.c.cap) raise_error(P.err, kErrBounds);
  }
  const bool cut = n > P.budget;
  // what is kept whatever the totals say, and the padding behind it
  const int head = cut ? P.sinks : kept;
  const int tail = cut ? P.budget - P.recent : kept;
  for (int j = rank * kThreads + tid; j < P.budget; j += C * kThreads) {
    if (j >= head && j < tail) continue;
    const int s = j < head ? j : (cut ? n - P.budget + j : -1);
    idx[j] = s;
    if (nm) nm[j] = s >= 0 ? row[s] : 0.f;
  }
  const int room = P.budget - P.sinks - P.recent;
  if (!cut || room <= 0) return;         // the whole cluster alike

  // this warp's stretch of the entries in between
  const int lo = P.sinks, m = n - P.sinks - P.recent;
  const int w0 = (rank * kWarps + warp) * P.wseg;
  const int len = min(max(m - w0, 0), P.wseg);
  uint32_t* mine = keys + warp * slot_of(P.wseg);
  const float* src = row + lo + w0;
  for (int i = tid; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  // the row is read once, and counted by its top 11 bits as it arrives
#pragma unroll 1
  for (int i = lane; i < len; i += 32 * kAhead) {
    float x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = i + 32 * u < len ? src[i + 32 * u] : 0.f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i + 32 * u < len) {
        const uint32_t k = order_key(x[u]);
        mine[slot_of(i + 32 * u)] = k;
        atomicAdd(&hist[0][k >> 21], 1u);
      }
    }
  }

  // keep every key above T and the first `want` equal ones
  uint32_t want = static_cast<uint32_t>(room), prefix = 0, T = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int up = pass == 1 ? 21 : 10;      // where the bits above the digit start
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    uint32_t* h = hist[pass];
    uint32_t* gr = group[pass];
    if (pass > 0) {
#pragma unroll 4
      for (int i = lane; i < len; i += 32) {
        const uint32_t k = mine[slot_of(i)];
        if ((k >> up) == prefix) atomicAdd(h + ((k >> shift) & mask), 1u);
      }
    }
    __syncthreads();
    // The bin of the want-th largest, in two steps from the top: the bins in 64
    // groups of 32, then the 32 bins of the group that holds it.  Both steps
    // read the other CTAs' counts once, 64 and 32 words each, instead of all
    // their 2048 (which took 2 us a pass).
    {
      const uint32_t v0 = __reduce_add_sync(0xffffffffu, h[64 * warp + lane]);
      const uint32_t v1 = __reduce_add_sync(0xffffffffu, h[64 * warp + 32 + lane]);
      if (lane == 0) *reinterpret_cast<uint2*>(gr + 2 * warp) = make_uint2(v0, v1);
    }
    sync_all();
    if (warp == 0) {
      // lane l: groups 63 - 2l and 62 - 2l, summed over the cluster
      uint32_t c0 = 0, c1 = 0;
#pragma unroll
      for (int q = 0; q < C; ++q) {
        const uint2 x = *reinterpret_cast<const uint2*>(remote(gr, q) + 62 - 2 * lane);
        c0 += x.y;
        c1 += x.x;
      }
      uint32_t before = sum_before(c0 + c1);
      uint32_t g = 0, left = 0;
      const bool here = before < want && want <= before + c0 + c1;
      if (here) {
        const bool second = want > before + c0;
        g = 63 - 2 * lane - (second ? 1 : 0);
        left = want - before - (second ? c0 : 0);
      }
      const int who = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      g = __shfl_sync(0xffffffffu, g, who);
      left = __shfl_sync(0xffffffffu, left, who);
      // lane l: bin 32 g + 31 - l
      uint32_t c = 0;
#pragma unroll
      for (int q = 0; q < C; ++q) c += remote(h, q)[32 * g + 31 - lane];
      before = sum_before(c);
      if (before < left && left <= before + c) {
        found[0] = 32 * g + 31 - lane;
        found[1] = left - before;
        found[2] = left - before == c ? 1u : 0u;      // every key of the bin is kept
      }
    }
    __syncthreads();
    prefix = (prefix << (pass == 2 ? 10 : 11)) | found[0];
    want = found[1];
    if (found[2] != 0u) {
      // No need to look inside the bin: the cut lies below it.  (The usual end, after
      // two passes of three.  The smallest key, -inf's, is 2^23 - 1: no bin starts at 0.)
      T = (prefix << shift) - 1u;
      want = 0;
      break;
    }
    T = prefix;
  }

  // Each lane owns a stretch of the warp's entries, so that slots follow from
  // one prefix over lanes, warps and CTAs.
  const int each = P.wseg / 32;
  const int i0 = lane * each, i1 = min(i0 + each, len);
  uint32_t above = 0, level = 0;         // its entries above T and equal to it (at most 32)
#pragma unroll 4
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = mine[slot_of(i)];
    above |= (k > T ? 1u : 0u) << (i - i0);
    level |= (k == T ? 1u : 0u) << (i - i0);
  }
  const uint32_t gt = __popc(above), eq = __popc(level);
  uint32_t bg = sum_before(gt), be = sum_before(eq);
  if (lane == 31) {
    wgt[warp] = bg + gt;
    weq[warp] = be + eq;
  }
  __syncthreads();
  bg += __reduce_add_sync(0xffffffffu, lane < warp ? wgt[lane] : 0u);
  be += __reduce_add_sync(0xffffffffu, lane < warp ? weq[lane] : 0u);
  if constexpr (C > 1) {
    if (tid == kThreads - 1) {
      xch[0] = bg + gt;
      xch[1] = be + eq;
    }
    sync_all();
#pragma unroll
    for (int q = 0; q < C; ++q) {
      const uint2 o = *reinterpret_cast<const uint2*>(cg::this_cluster().map_shared_rank(xch, q));
      if (q < rank) {
        bg += o.x;
        be += o.y;
      }
    }
    cg::this_cluster().barrier_arrive();
  }
#pragma unroll 1
  for (uint32_t left = above | level; left != 0; left &= left - 1) {
    const int u = __ffs(left) - 1;
    const bool over = (above >> u) & 1u;
    if (over || be < want) {
      const int s = lo + w0 + i0 + u;
      const int64_t j = P.sinks + static_cast<int64_t>(bg) + min(be, want);
      idx[j] = s;
      // the total itself, from its key unless that stands for several
      if (nm) {
        const uint32_t k = mine[slot_of(i0 + u)];
        nm[j] = k == 0xFFFFFFFFu || k == 0x80000000u ? row[s] : key_value(k);
      }
    }
    if (over) ++bg; else ++be;
  }
  // nobody's shared memory goes away while another CTA may still read it
  if constexpr (C > 1) cg::this_cluster().barrier_wait();
}

// Four kept latents per warp: 288 pieces of 16 bytes, nine per lane.
constexpr int kMoveRows = 4;
__global__ void __launch_bounds__(256, 4) move_kernel(Params P, uint8_t* pool, int groups) {
  const int lane = threadIdx.x % 32;
  const int64_t all = static_cast<int64_t>(groups) * P.c.B;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 8;
  // (the tables are not written under this kernel: it starts when the choice has passed its own wait)
  grid_release();
  grid_wait();
  for (int64_t t = blockIdx.x * 8ll + threadIdx.x / 32; t < all; t += stride) {
    const int b = static_cast<int>(t / groups);
    const int j = static_cast<int>(t % groups) * kMoveRows + lane;
    // lanes 0..3: where row j comes from and goes to (-1: nothing to move)
    int64_t from = -1, to = -1;
    if (lane < kMoveRows && j < P.budget) {
      const int s = P.idx[static_cast<int64_t>(b) * P.budget + j];
      if (s >= 0) {
        const int ps = page_of(P.c, s), pd = page_of(P.c, j);
        const int a = __ldg(P.c.table + static_cast<int64_t>(b) * P.c.table_ld + ps);
        const int d = __ldg(P.new_table + static_cast<int64_t>(b) * P.new_ld + pd);
        if (a < 0 || a >= P.c.n_pages || d < 0 || d >= P.c.n_pages) {
          raise_error(P.err, kErrBounds);
        } else {
          from = (a * P.c.page_stride + static_cast<int64_t>(s - ps * P.c.page) * 576) * 2;
          to = (d * P.c.page_stride + static_cast<int64_t>(j - pd * P.c.page) * 576) * 2;
        }
      }
    }
    uint4 v[9];
#pragma unroll
    for (int u = 0; u < 9; ++u) {
      const int p = lane + 32 * u, r = p / 72;
      const int64_t f = __shfl_sync(0xffffffffu, from, r);
      if (f >= 0) v[u] = *reinterpret_cast<const uint4*>(pool + f + (p - r * 72) * 16);
    }
#pragma unroll
    for (int u = 0; u < 9; ++u) {
      const int p = lane + 32 * u, r = p / 72;
      const int64_t d = __shfl_sync(0xffffffffu, to, r);
      if (d >= 0) *reinterpret_cast<uint4*>(pool + d + (p - r * 72) * 16) = v[u];
    }
  }
}

template <int C>
cudaError_t launch_select(const Params& P, size_t smem, cudaStream_t s) {
  // (the most that rows of up to 262144 entries take)
  constexpr int kMostSmem = kWarps * (262144 / (kClusterC * kWarps) / 32 * 33) * 4;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(select_kernel<C>, kMostSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(P.c.B) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  // (its start under the end of the kernel before: two calls in a row 16.4 -> 14.5 us
  // for one row of 131072; the attention kernels gain nothing by it, and the decode
  // lost 4 % where two CTAs read the same keys)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel<C>, P);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictArgs& a, DevErr err, cudaStream_t s) {
  Params P;
  P.c = a.cache;
  P.mass = a.mass;
  P.ld_mass = a.ld_mass;
  P.budget = a.budget;
  P.sinks = a.sinks;
  P.recent = a.recent;
  P.idx = a.idx;
  P.new_lens = a.new_lens;
  P.new_mass = a.new_mass;
  P.ld_new = a.ld_new;
  P.new_table = a.new_table;
  P.new_ld = a.new_ld;
  P.err = err;
  const int C = P.c.cap <= kOneCta ? 1 : kClusterC;
  const int warps = C * kWarps;
  P.wseg = ((P.c.cap + warps - 1) / warps + 31) / 32 * 32;
  static_assert(262144 / (kClusterC * kWarps) <= 1024 && kOneCta / kWarps <= 1024,
                "at most 32 entries per lane");
  const size_t smem = static_cast<size_t>(kWarps) * (P.wseg + P.wseg / 32) * 4;
  cudaError_t e = C == 1 ? launch_select<1>(P, smem, s) : launch_select<kClusterC>(P, smem, s);
  if (e != cudaSuccess) return e;
  const int most_kept = a.budget < P.c.cap ? a.budget : P.c.cap;
  const int groups = (most_kept + kMoveRows - 1) / kMoveRows;
  if (groups == 0) return cudaSuccess;
  const int64_t ctas = (static_cast<int64_t>(groups) * P.c.B + 7) / 8;
  const int64_t most = static_cast<int64_t>(a.num_sms) * 16;
  return launch_after(move_kernel, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), 256, 0,
                      s, P, const_cast<uint8_t*>(P.c.pool), groups);
}

}  // namespace dsa
