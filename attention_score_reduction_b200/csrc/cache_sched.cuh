// How the attention kernels over the paged cache share their work.
//
// An item is one unit's block of query rows.  Its work is the tiles of cache
// rows its last row can see.  Heads keep very different numbers of rows
// after eviction, so the items' tiles are laid end to end on one line and every
// CTA takes an equal piece of it, crossing items where it must (a fixed number of
// splits per head would wait for the longest head).  Lengths live on the device;
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
};

struct AttnItem {
  int64_t u;
  int len;         // rows the unit holds
  int m;           // its new tokens
  int row0, rows;  // query rows [row0, row0 + rows)
  int vis;         // cache rows the item's last query row sees
  int n_tiles;
};

// Cache rows that token i sees (may be negative: none).
__device__ __forceinline__ int seen_rows(const AttnItem& it, int i) { return it.len - it.m + i + 1; }

__device__ __forceinline__ AttnItem attn_item(const CacheArgs& c, const AttnShape& s, int64_t w) {
  AttnItem it;
  it.u = w / s.blocks;
  const int b = static_cast<int>(w - it.u * s.blocks);
  it.len = held_to(c.lens[it.u], cache_cap(c), c.status);
  it.m = s.q_lens ? held_to(s.q_lens[it.u], s.n_q, c.status) : s.n_q;
  it.row0 = b * s.block;
  it.rows = min(s.block, it.m * s.G - it.row0);
  it.vis = 0;
  if (it.rows > 0) it.vis = max(0, seen_rows(it, (it.row0 + it.rows - 1) / s.G));
  it.n_tiles = (it.vis + s.tile - 1) / s.tile;
  return it;
}

// Sum of v over the block (THREADS threads, all of them); scratch: THREADS / 32 entries.
template <int THREADS>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* scratch) {
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t t = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) t += scratch[i];
  return t;
}

// Tiles of all items, and of the items before item w.
struct LineTotals {
  int64_t all, before;
};
template <int THREADS>
__device__ __forceinline__ LineTotals line_totals(const CacheArgs& c, const AttnShape& s,
                                                  int64_t items, int64_t w, int64_t* scratch) {
  int64_t all = 0, before = 0;
  for (int64_t i = threadIdx.x; i < items; i += THREADS) {
    const int t = attn_item(c, s, i).n_tiles;
    all += t;
    if (i < w) before += t;
  }
  LineTotals r;
  r.all = block_sum<THREADS>(all, scratch);
  r.before = block_sum<THREADS>(before, scratch);
  return r;
}

// The item that holds tile p of the line (0 <= p < all) and its first tile's place.
template <int THREADS>
__device__ __forceinline__ void line_find(const CacheArgs& c, const AttnShape& s, int64_t items,
                                          int64_t p, int64_t* item, int64_t* item_at,
                                          int64_t* scratch, int64_t* found) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t base = 0;
  for (int64_t i0 = 0; i0 < items; i0 += THREADS) {
    const int64_t i = i0 + threadIdx.x;
    const int t = i < items ? attn_item(c, s, i).n_tiles : 0;
    int64_t inc = t;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, inc, w);
      if (lane >= w) inc += o;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    int64_t off = base;
    int64_t sum = 0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) {
      if (k < warp) off += scratch[k];
      sum += scratch[k];
    }
    if (t > 0 && off + inc - t <= p && p < off + inc) {
      found[0] = i;
      found[1] = off + inc - t;
    }
    base += sum;
    if (base > p) break;      // the same for every thread
  }
  __syncthreads();
  *item = found[0];
  *item_at = found[1];
  __syncthreads();
}

// CTAs with work: no more than there are tiles, so that every one's piece holds
// at least one tile and every slot between an item's first and last CTA is written.
__device__ __forceinline__ int64_t line_ctas(int64_t all, int64_t grid) {
  return all < grid ? all : grid;
}
// Piece of the line that CTA i of n takes: [line_cut(i), line_cut(i + 1)).
__device__ __forceinline__ int64_t line_cut(int64_t all, int64_t i, int64_t n) {
  return all * i / n;
}
// Slot of CTA i's part of the item whose tiles begin at `before` on the line.
__device__ __forceinline__ int64_t line_slot(int64_t all, int64_t i, int64_t n, int64_t before) {
  return 2 * i + (line_cut(all, i, n) >= before ? 0 : 1);
}
// The CTA that takes tile p.
__device__ __forceinline__ int64_t line_cta(int64_t all, int64_t p, int64_t n) {
  int64_t i = p * n / all;
  while (i + 1 < n && line_cut(all, i + 1, n) <= p) ++i;
  while (i > 0 && line_cut(all, i, n) > p) --i;
  return i;
}

}  // namespace kvzip
