// How the attention kernels over the paged cache share their work.
//
// An item is one unit's block of query rows.  Its work is the tiles of cache
// rows its last row can see.  Heads keep very different numbers of rows
// after eviction, so the items' tiles are laid end to end on one line and every
// CTA takes an equal piece of it, crossing items where it must (a fixed number of
// splits per head would wait for the longest head).  Beginning an item takes time of
// its own (its queries, its result), so on the line an item is `pad` places longer than
// its tiles, and a CTA that crosses into one has that much less to do.  Lengths live on the device;
// every CTA adds them up itself.  A CTA's part of an item that it does not cover
// whole is a partial result; a CTA has at most two, of its first and its last
// item, in slots 2 cta and 2 cta + 1.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.cuh"

namespace kvzip {

struct AttnShape {
  const int32_t* q_lens;
  int n_q, G;
  int block;       // query rows of one item; row r of a unit is token r / G, head r % G
  int blocks;      // items per unit
  int tile;        // cache rows of one tile
  int pad;         // places on the line before an item's first tile
};

struct AttnItem {
  int64_t u;
  int len;         // rows the unit holds
  int m;           // its new tokens
  int row0, rows;  // query rows [row0, row0 + rows)
  int vis;         // cache rows the item's last query row sees
  int n_tiles;
  int span;        // places on the line
};

// Cache rows that token i sees (may be negative: none).
__device__ __forceinline__ int seen_rows(const AttnItem& it, int i) { return it.len - it.m + i + 1; }

__device__ __forceinline__ AttnItem attn_item(const CacheArgs& c, const AttnShape& s, int64_t w) {
  AttnItem it;
  it.u = static_cast<uint32_t>(w) / static_cast<uint32_t>(s.blocks);   // w < 2^31
  const int b = static_cast<int>(w - it.u * s.blocks);
  it.len = held_to(__ldcg(c.lens + it.u), cache_cap(c), c.status);
  it.m = s.q_lens ? held_to(__ldcg(s.q_lens + it.u), s.n_q, c.status) : s.n_q;
  it.row0 = b * s.block;
  it.rows = min(s.block, it.m * s.G - it.row0);
  it.vis = 0;
  if (it.rows > 0) it.vis = max(0, seen_rows(it, (it.row0 + it.rows - 1) / s.G));
  it.n_tiles = (it.vis + s.tile - 1) / s.tile;
  it.span = it.n_tiles > 0 ? it.n_tiles + s.pad : 0;
  return it;
}

// An item as the thread that counted its tiles hands it to the block.
struct LineSpot {
  int64_t item, at;      // the item and its first place
  AttnItem info;
};

// The line as the THREADS threads of a block see it; `sums` (THREADS / 32 entries) and
// `spot` are shared scratch.  Up to THREADS items are loaded once, one per thread, and
// a spot costs one barrier; more are walked again for every question.
template <int THREADS>
struct Line {
  const CacheArgs& c;
  const AttnShape& s;
  int64_t items;
  int64_t* sums;
  LineSpot* spot;
  int64_t all;         // places of all items
  int64_t mine_end;    // items <= THREADS: places up to and with item threadIdx.x
  AttnItem mine;

  __device__ Line(const CacheArgs& c_, const AttnShape& s_, int64_t items_, int64_t* sums_,
                  LineSpot* spot_)
      : c(c_), s(s_), items(items_), sums(sums_), spot(spot_), all(0), mine_end(0) {
    int64_t v = 0;
    if (items <= THREADS) {
      if (threadIdx.x < items) {
        mine = attn_item(c, s, threadIdx.x);
        v = mine.span;
      }
      mine_end = scan(v, &all);
    } else {
      for (int64_t i = threadIdx.x; i < items; i += THREADS) v += attn_item(c, s, i).span;
      scan(v, &all);
    }
  }

  // Inclusive prefix sum over the block's threads, and the total.  Two calls need a
  // barrier between them.
  __device__ int64_t scan(int64_t v, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, v, k);
      if (lane >= k) v += o;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    int64_t t = 0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) {
      if (k < warp) v += sums[k];
      t += sums[k];
    }
    *total = t;
    return v;
  }

  // The spot of place p (0 <= p < all); one use per block.
  __device__ LineSpot find(int64_t p) {
    if (items <= THREADS) {
      if (threadIdx.x < items && mine_end - mine.span <= p && p < mine_end)
        *spot = LineSpot{static_cast<int64_t>(threadIdx.x), mine_end - mine.span, mine};
    } else {
      int64_t base = 0;
      for (int64_t i0 = 0; i0 < items; i0 += THREADS) {
        const int64_t i = i0 + threadIdx.x;
        AttnItem it;
        it.span = 0;
        if (i < items) it = attn_item(c, s, i);
        int64_t sum;
        __syncthreads();
        const int64_t end = base + scan(it.span, &sum);
        if (end - it.span <= p && p < end) *spot = LineSpot{i, end - it.span, it};
        base += sum;
        if (base > p) break;      // the same for every thread
      }
    }
    __syncthreads();
    return *spot;
  }

  // The spot of item w; one use per block.
  __device__ LineSpot of_item(int64_t w) {
    if (items <= THREADS) {
      if (threadIdx.x == w) *spot = LineSpot{w, mine_end - mine.span, mine};
    } else {
      int64_t v = 0, sum;
      for (int64_t i = threadIdx.x; i < w; i += THREADS) v += attn_item(c, s, i).span;
      __syncthreads();
      scan(v, &sum);
      if (threadIdx.x == 0) *spot = LineSpot{w, sum, attn_item(c, s, w)};
    }
    __syncthreads();
    return *spot;
  }
};

// The tiles [t0, t1) of an item that begins at place `at` within places [p, p1); false
// if there are none.
__device__ __forceinline__ bool line_tiles(const AttnItem& it, const AttnShape& s, int64_t at,
                                           int64_t p, int64_t p1, int& t0, int& t1) {
  const int64_t first = at + s.pad;
  t0 = static_cast<int>(max(p - first, static_cast<int64_t>(0)));
  t1 = static_cast<int>(max(min(p1 - first, static_cast<int64_t>(it.n_tiles)), static_cast<int64_t>(0)));
  return t0 < t1;
}

// CTAs of the line: no more than there are places, so that no piece is empty and every
// CTA between those with an item's first and last tile has tiles of it, and a slot.
__device__ __forceinline__ int64_t line_ctas(int64_t all, int64_t grid) {
  return all < grid ? all : grid;
}
// a / b for a, b >= 0: 32-bit division where it will do (a 64-bit one is a few
// hundred instructions, which show in a decoding step).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Piece of the line that CTA i of n takes: [line_cut(i), line_cut(i + 1)).
__device__ __forceinline__ int64_t line_cut(int64_t all, int64_t i, int64_t n) {
  return quotient(all * i, n);
}
// Slot of CTA i's part of the item whose first tile is at place `first`.
__device__ __forceinline__ int64_t line_slot(int64_t all, int64_t i, int64_t n, int64_t first) {
  return 2 * i + (line_cut(all, i, n) >= first ? 0 : 1);
}
// The CTA that takes place p.
__device__ __forceinline__ int64_t line_cta(int64_t all, int64_t p, int64_t n) {
  int64_t i = quotient(p * n, all);
  while (i + 1 < n && line_cut(all, i + 1, n) <= p) ++i;
  while (i > 0 && line_cut(all, i, n) > p) --i;
  return i;
}

}  // namespace kvzip
