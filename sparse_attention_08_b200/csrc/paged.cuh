// paged.cuh -- what the kernels over a paged latent cache share: which keys a
// sequence's newest token sees, how those tiles are dealt out to the CTAs, and
// the loads of one tile through the block table.
//
// A cache is a pool of pages of `page` latent rows; row s of sequence b is row
// s % page of pool page table[b, s / page].  The newest token of a sequence of
// n entries sees all of them, or (window > 0) the entries s >= n - window and
// s < sinks.  Keys are worked on in tiles of kTile positions; the tiles that
// hold a seen key are numbered 0 .. n_tiles-1 within the sequence.
#pragma once

#include "ptx.cuh"

namespace dsa {
namespace paged {

constexpr int kChunks = 9;                      // 64-column chunks of a 576-d row

struct Cache {
  const int32_t* table;    // [B, table_ld]
  const int32_t* lens;     // [B]
  const uint8_t* pool;
  int64_t page_stride;     // elements
  int64_t table_ld;
  int B;
  int page;                // rows per page, a multiple of 16
  uint64_t page_inv;       // 2^43 / page, rounded up: s / page = (s * page_inv) >> 43 for s < 2^24
  int box;                 // rows per TMA box: a power of two that divides page, at most a tile
  int n_pages;             // pages in the pool
  int cap;                 // longest sequence the call allows
  int window, sinks;
};

// The page of its sequence that holds entry s.
__device__ __forceinline__ int page_of(const Cache& c, int s) {
  return static_cast<int>((static_cast<uint64_t>(s) * c.page_inv) >> 43);
}

// The length of sequence b, kept inside [0, cap].
__device__ __forceinline__ int seq_len(const Cache& c, int b) {
  return min(max(__ldg(c.lens + b), 0), c.cap);
}

// The tiles of a sequence that hold a seen key: the first `a` tiles (the
// first tokens), then tiles from `w0` on (the window).
template <int kTile>
struct Seen {
  int len, lo, ns;   // seen: s < ns or lo <= s < len
  int a, w0, n;
  __device__ __forceinline__ int tile(int i) const { return i < a ? i : w0 + (i - a); }
  __device__ __forceinline__ bool key(int s) const { return s < ns || (s >= lo && s < len); }
  // any seen key in [s, s + rows)?
  __device__ __forceinline__ bool any(int s, int rows) const {
    return s < ns || (s < len && s + rows > lo);
  }
};

template <int kTile>
__device__ __forceinline__ Seen<kTile> seen_of(const Cache& c, int len) {
  Seen<kTile> k;
  k.len = len;
  k.lo = c.window > 0 ? max(0, len - c.window) : 0;
  k.ns = min(c.sinks, k.lo);
  k.a = (k.ns + kTile - 1) / kTile;
  k.w0 = max(k.lo / kTile, k.a);
  k.n = k.a + (len + kTile - 1) / kTile - k.w0;
  return k;
}

// A warp's wait in which every lane polls: the verdict needs no broadcast,
// which shortens the wake-up by about 100 cycles against warp_wait.  The waiting
// loop is out of line to keep the roles' loops short, and looks at the launch's
// error word and the clock only every 1024 polls: the load of the word takes as
// long as a dozen polls, during which a finished phase goes unseen.
static __device__ __noinline__ bool wait_loop(uint32_t bar, uint32_t parity, unsigned* word,
                                              unsigned gen, uint64_t limit_ns) {
  DevErr e;
  e.word = word;
  e.gen = gen;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 1023u) == 0) {
      if (launch_failed(e)) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) {
        raise_error(e, kErrTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool all_wait(uint32_t bar, uint32_t parity, const DevErr& e) {
  const bool ok = mbar_try_wait(bar, parity) || wait_loop(bar, parity, e.word, e.gen, e.limit_ns);
  return __all_sync(0xffffffffu, ok);
}

// The same by one lane alone, inside the branch that issues MMAs.
__device__ __forceinline__ bool one_wait(uint32_t bar, uint32_t parity, const DevErr& e) {
  return mbar_try_wait(bar, parity) || wait_loop(bar, parity, e.word, e.gen, e.limit_ns);
}

// A value that all lanes hold alike, in a form the compiler knows to be so: MMA
// operands made from it stay in uniform registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Sum over the warp, the same in every lane.
__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The tiles of all sequences in one line, cut into `ranges` pieces of `per`
// tiles (the last ones shorter or empty).  min_tiles = 1 gives a sequence
// without a seen key one (empty) tile, so that somebody writes its output.
struct Start {
  int b;         // sequence of the piece's first tile (B: the piece is empty)
  int skip;      // its tiles that belong to earlier pieces
  int per;       // tiles per piece
  int left;      // this one's
};

// kWhole: up to two tiles more per piece are taken if every piece then lies
// in one sequence, which ends with shorter pieces: a piece's second sequence starts
// like the first (queries, a pipeline to fill, a part to write), at the price of
// about two tiles (decode, 64 heads, 48 sequences, window 1000: 38.6 -> 34.2 us).
//
// Called by every thread of the CTA (nwarps whole warps), which it brings together;
// scratch: nwarps + 3 ints.
constexpr int kFewSeqs = 128;
template <int kTile, bool kWhole>
__device__ __forceinline__ Start find_start(const Cache& c, int range, int ranges, int min_tiles,
                                            int nwarps, int* scratch, const DevErr& err) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto tiles_of = [&](int b) { return max(seen_of<kTile>(c, seq_len(c, b)).n, min_tiles); };
  Start s;
  if (c.B <= kFewSeqs) {
    // A few sequences: every warp works it all out for itself, four sequences a
    // lane, with one round of loads and no barrier but the last.
    int n[kFewSeqs / 32], sum = 0;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kFewSeqs / 32; ++e) {
      const int b = 32 * e + lane;
      n[e] = b < c.B ? tiles_of(b) : 0;
      if (b < c.B) {
        const int raw = __ldg(c.lens + b);
        bad |= raw < 0 || raw > c.cap;
      }
      sum += n[e];
    }
    if (bad && range == 0 && warp == 0) raise_error(err, kErrBounds);
    const int total = warp_sum(sum);
    s.per = max(1, (total + ranges - 1) / ranges);
    int more = -1;
    if (kWhole && s.per > 1 && c.B < ranges) {
#pragma unroll 1
      for (int e = 0; more < 0 && e < 3; ++e) {
        const uint32_t per = s.per + e;
        uint32_t need = 0;
#pragma unroll
        for (int u = 0; u < kFewSeqs / 32; ++u) need += (n[u] + per - 1) / per;
        if (warp_sum(need) <= ranges) more = e;
      }
      if (more > 0) s.per += more;
    }
    // the line that is cut: tiles, or with whole sequences pieces
    const bool whole = more >= 0;
    const int at = whole ? range : min(static_cast<int64_t>(range) * s.per, static_cast<int64_t>(total));
    s.b = c.B;
    s.skip = 0;
    s.left = s.per;
    int first = 0;
#pragma unroll
    for (int e = 0; e < kFewSeqs / 32; ++e) {
      if (32 * e >= c.B || s.b < c.B) continue;
      const int own = whole ? static_cast<int>((n[e] + s.per - 1) / static_cast<uint32_t>(s.per)) : n[e];
      int end = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, end, d);
        if (lane >= d) end += v;
      }
      end += first;
      const uint32_t here = __ballot_sync(0xffffffffu, at >= end - own && at < end);
      if (here != 0) {
        const int who = __ffs(here) - 1;
        const int into = __shfl_sync(0xffffffffu, at - (end - own), who);
        s.b = 32 * e + who;
        s.skip = whole ? into * s.per : into;
        if (whole) s.left = min(s.per, __shfl_sync(0xffffffffu, n[e], who) - s.skip);
      }
      first = __shfl_sync(0xffffffffu, end, 31);
    }
    __syncthreads();
    return s;
  }
  // Warp w adds up sequences [w, w+1) * B / nwarps; the warp whose stretch holds
  // the piece's first tile then finds its sequence with a scan.
  const int each = ((c.B + nwarps - 1) / nwarps + 31) / 32 * 32;
  const int b0 = min(c.B, warp * each), b1 = min(c.B, b0 + each);
  int sum = 0;
  bool bad = false;
#pragma unroll 1
  for (int b = b0 + lane; b < b1; b += 32) {
    const int raw = __ldg(c.lens + b);
    bad |= raw < 0 || raw > c.cap;
    sum += tiles_of(b);
  }
  if (bad && range == 0) raise_error(err, kErrBounds);
  sum = warp_sum(sum);
  if (lane == 0) scratch[warp] = sum;
  if (threadIdx.x == 0) scratch[nwarps] = c.B;
  __syncthreads();
  int total = 0, before = 0;
#pragma unroll 1
  for (int w = 0; w < nwarps; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  s.per = s.left = max(1, (total + ranges - 1) / ranges);
  const int first = min(static_cast<int64_t>(range) * s.per, static_cast<int64_t>(total));
  if (first < total && first >= before && first < before + sum) {
#pragma unroll 1
    for (int b = b0; b < b1; b += 32) {
      const int n = b + lane < b1 ? tiles_of(b + lane) : 0;
      int inc = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += v;
      }
      const int end = before + inc;
      if (first >= end - n && first < end) {
        scratch[nwarps] = b + lane;
        scratch[nwarps + 1] = first - (end - n);
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
      if (before > first) break;
    }
  }
  __syncthreads();
  s.b = scratch[nwarps];
  s.skip = scratch[nwarps + 1];
  return s;
}

// Walks the tiles of one piece, segment by segment (a segment: the piece's
// share of one sequence).  Every role of a CTA walks the same way.
template <int kTile>
struct Walk {
  const Cache& c;
  int b, i0, i1, left, min_tiles;
  Seen<kTile> k;
  __device__ __forceinline__ Walk(const Cache& cache, const Start& s, int min_t)
      : c(cache), b(s.b), i0(s.skip), i1(0), left(s.left), min_tiles(min_t) {}
  // Moves to the next segment: sequence b, its tiles [i0, i1).
  __device__ __forceinline__ bool next(bool first) {
    if (!first) {
      ++b;
      i0 = 0;
    }
#pragma unroll 1
    for (; left > 0 && b < c.B; ++b) {
      k = seen_of<kTile>(c, seq_len(c, b));
      const int n = max(k.n, min_tiles);
      if (n > i0) {
        i1 = min(n, i0 + left);
        left -= i1 - i0;
        return true;
      }
      i0 = 0;
    }
    return false;
  }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y,
                                            int32_t z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// What a lane of the loading warp brings in of one tile: box `lane` of the
// tile's kTile / box boxes, if it holds a seen key.
struct Box {
  bool on;
  int32_t page, row;
};

// Pulls a box's rows, which lie one after the other, into L2 ahead of its
// loads: from there the tile's copies take half as long as from DRAM.
__device__ __forceinline__ void prefetch_box(const Cache& c, const Box& x) {
  if (x.on && x.page >= 0 && x.page < c.n_pages)
    prefetch_l2_bulk(c.pool + (static_cast<int64_t>(x.page) * c.page_stride + static_cast<int64_t>(x.row) * 576) * 2,
                     static_cast<uint32_t>(c.box) * 1152u);
}

template <int kTile>
__device__ __forceinline__ Box box_of(const Cache& c, const Seen<kTile>& k, int b, int tile, int lane,
                                      const DevErr& err) {
  Box x;
  const int s = tile * kTile + lane * c.box;
  x.on = lane * c.box < kTile && k.any(s, c.box);
  x.page = 0;
  x.row = 0;
  if (x.on) {
    const int j = page_of(c, s);
    x.page = __ldg(c.table + static_cast<int64_t>(b) * c.table_ld + j);
    x.row = s - j * c.page;
    // an id outside the pool reads zeros (the copy's own bounds check)
    if (x.page < 0 || x.page >= c.n_pages) raise_error(err, kErrBounds);
  }
  return x;
}

// 16 lanes x 256 bits, repeated 4 times along the columns (32 columns): with t
// the thread in the warp, registers 4i, 4i+1 hold lane addr.lane + t/4, columns
// 8i + 2(t%4) + {0,1}; registers 4i+2, 4i+3 lane addr.lane + t/4 + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 32 lanes x 32 bits, 16 consecutive columns (thread t <-> lane addr.lane + t).
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

}  // namespace paged
}  // namespace dsa
