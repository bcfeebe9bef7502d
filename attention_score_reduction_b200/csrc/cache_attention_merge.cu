// Joins the partial results of attention over the paged cache, and sizes the
// workspace they live in.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "cache_attention.cuh"
#include "kvzip_internal.h"
#include "sm100_ptx.cuh"

namespace kvzip {

namespace {

constexpr int kMergeThreads = 256;
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kWarpSplits = 8;      // up to this many parts a warp joins a row alone

// One row's elements as a warp holds them: lane * 4 + 128 i.
template <int D>
struct RowPart {
  float4 v[D / 128];
};

template <int D>
__device__ __forceinline__ void add_part(RowPart<D>& acc, const float* o, float f) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < D / 128; ++i) {
    const float4 x = __ldcg(reinterpret_cast<const float4*>(o) + lane + 32 * i);
    acc.v[i].x = fmaf(x.x, f, acc.v[i].x);
    acc.v[i].y = fmaf(x.y, f, acc.v[i].y);
    acc.v[i].z = fmaf(x.z, f, acc.v[i].z);
    acc.v[i].w = fmaf(x.w, f, acc.v[i].w);
  }
}

// Elements e .. e + 3 of an output row: x / L.
__device__ __forceinline__ void put4(const CacheAttnArgs& a, const AttnShape& s, const AttnItem& it,
                                     int row, int e, float4 x, float L) {
  const int r = it.row0 + row, tok = r / s.G, g = r - tok * s.G;
  if (!out_in_bounds(a, it, tok, g)) return;
  const int64_t at = it.u * a.o_unit + g * a.o_head + tok * a.o_row + e;
  const float inv = attn_inverse(L, seen_rows(it, tok) <= 0);
  x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  if (a.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = x;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}
template <int D>
__device__ __forceinline__ void put_row(const CacheAttnArgs& a, const AttnShape& s,
                                        const AttnItem& it, int row, const RowPart<D>& acc, float L) {
#pragma unroll
  for (int i = 0; i < D / 128; ++i) put4(a, s, it, row, 4 * (threadIdx.x & 31) + 128 * i, acc.v[i], L);
}

// Which item a block joins does not depend on the results, so it is found before
// the wait for the grid that computes them.  Blocks are one per item, or (many
// items: few of them are split) one per cut between two CTAs, of which the first
// inside an item serves it.
struct Split {
  AttnItem it;
  int64_t c0, slot0;      // the first CTA with a part of the item, and its slot
  int parts;              // 0: not split, or another block's

  // slot of part i: later CTAs begin with the item
  __device__ __forceinline__ int64_t slot(int i) const { return i == 0 ? slot0 : 2 * (c0 + i); }
};
__device__ __forceinline__ Split find_split(const CacheAttnArgs& a, const AttnShape& shape,
                                            int64_t items, int ctas, int by_item) {
  __shared__ int64_t scratch[kMergeWarps];
  __shared__ LineSpot spot_s;
  bool split = false;
  Line<kMergeThreads> t(a.c, shape, items, scratch, &spot_s);
  const int64_t n = line_ctas(t.all, ctas);
  LineSpot spot;
  spot.at = 0;
  spot.info.span = 0;
  if (by_item) {
    spot = t.of_item(blockIdx.x);
    split = spot.info.span > 0;
  } else if (blockIdx.x + 1 < n) {
    const int64_t cut = line_cut(t.all, blockIdx.x + 1, n);
    spot = t.find(cut);
    // the first cut among the item's tiles
    split = spot.at + shape.pad < cut && line_cut(t.all, blockIdx.x, n) <= spot.at + shape.pad;
  }
  Split r;
  r.it = spot.info;
  r.c0 = r.slot0 = 0;
  r.parts = 0;
  if (split) {
    const int64_t first = spot.at + shape.pad;
    r.c0 = line_cta(t.all, first, n);
    r.slot0 = line_slot(t.all, r.c0, n, first);
    r.parts = static_cast<int>(line_cta(t.all, first + r.it.n_tiles - 1, n) - r.c0) + 1;
    if (r.parts < 2) r.parts = 0;
    if (r.parts > 0 && !(slot_in_bounds(shape, r.slot0, ctas, 0) &&
                         slot_in_bounds(shape, r.slot(r.parts - 1), ctas, r.it.rows - 1)))
      r.parts = 0;
  }
  return r;
}

// Items that see nothing: zeros.
template <int D>
__device__ __forceinline__ void put_zeros(const CacheAttnArgs& a, const AttnShape& shape,
                                          int64_t items) {
  const RowPart<D> zero = {};
  for (int64_t z = blockIdx.x; z < items; z += gridDim.x) {
    const AttnItem iz = attn_item(a.c, shape, z);
    if (iz.n_tiles == 0)
      for (int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); row < iz.rows;
           row += gridDim.y * kMergeWarps)
        put_row<D>(a, shape, iz, row, zero, 0.f);
  }
}

// Parts of the few-rows kernel: a slot's o is [row][D].  Items with few parts give a row
// to each warp; with many (one token: dozens) the warps of a block share a row's parts,
// so that their loads are in flight together.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    cache_attn_merge(const CacheAttnArgs a, const AttnShape shape, int64_t items, int ctas,
                     int by_item, const float2* ml, const float* o) {
  __shared__ RowPart<D> acc_s[kMergeWarps][32];
  __shared__ float l_s[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Split sp = find_split(a, shape, items, ctas, by_item);
  const AttnItem& it = sp.it;
  begin_after_previous();                // the partial results are complete and visible

  if (sp.parts > 0) {
    const int parts = sp.parts;
    auto part = [&](int i) { return sp.slot(i) * shape.block; };
    if (parts <= kWarpSplits) {
      for (int row = blockIdx.y * kMergeWarps + warp; row < it.rows; row += gridDim.y * kMergeWarps) {
        const float2 x = lane < parts ? __ldcg(ml + part(lane) + row) : make_float2(-INFINITY, 0.f);
        float M = x.x;
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) M = fmax_nan(M, __shfl_xor_sync(0xffffffffu, M, k));
        const float f = exp2f(x.x - (M == -INFINITY ? 0.f : M));
        float L = lane < parts ? x.y * f : 0.f;
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) L += __shfl_xor_sync(0xffffffffu, L, k);
        RowPart<D> acc = {};
#pragma unroll 4
        for (int i = 0; i < parts; ++i)
          add_part<D>(acc, o + (part(i) + row) * D, __shfl_sync(0xffffffffu, f, i));
        put_row<D>(a, shape, it, row, acc, L);
      }
    } else {
      for (int row = blockIdx.y; row < it.rows; row += gridDim.y) {
        // this warp's first parts are requested before the maximum is known
        constexpr int AHEAD = 3;
        RowPart<D> x[AHEAD];
        float2 xl[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          const int i = warp + k * kMergeWarps;
          if (i < parts) {
            const int64_t slot = part(i) + row;
            xl[k] = __ldcg(ml + slot);
#pragma unroll
            for (int e = 0; e < D / 128; ++e)
              x[k].v[e] = __ldcg(reinterpret_cast<const float4*>(o + slot * D) + lane + 32 * e);
          } else {
            xl[k] = make_float2(-INFINITY, 0.f);
            x[k] = {};
          }
        }
        float M = -INFINITY;
        for (int i = lane; i < parts; i += 32) M = fmax_nan(M, __ldcg(ml + part(i) + row).x);
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) M = fmax_nan(M, __shfl_xor_sync(0xffffffffu, M, k));
        const float sub = M == -INFINITY ? 0.f : M;
        RowPart<D> acc = {};
        float L = 0.f;
        auto add = [&](const RowPart<D>& p, float2 v) {
          const float f = exp2f(v.x - sub);
          L = fmaf(v.y, f, L);
#pragma unroll
          for (int e = 0; e < D / 128; ++e) {
            acc.v[e].x = fmaf(p.v[e].x, f, acc.v[e].x);
            acc.v[e].y = fmaf(p.v[e].y, f, acc.v[e].y);
            acc.v[e].z = fmaf(p.v[e].z, f, acc.v[e].z);
            acc.v[e].w = fmaf(p.v[e].w, f, acc.v[e].w);
          }
        };
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) add(x[k], xl[k]);
        for (int i = warp + AHEAD * kMergeWarps; i < parts; i += kMergeWarps) {
          const int64_t slot = part(i) + row;
          RowPart<D> y;
#pragma unroll
          for (int e = 0; e < D / 128; ++e)
            y.v[e] = __ldcg(reinterpret_cast<const float4*>(o + slot * D) + lane + 32 * e);
          add(y, __ldcg(ml + slot));
        }
        acc_s[warp][lane] = acc;
        if (lane == 0) l_s[warp] = L;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int k = 1; k < kMergeWarps; ++k) {
            const RowPart<D> x = acc_s[k][lane];
#pragma unroll
            for (int i = 0; i < D / 128; ++i) {
              acc.v[i].x += x.v[i].x;
              acc.v[i].y += x.v[i].y;
              acc.v[i].z += x.v[i].z;
              acc.v[i].w += x.v[i].w;
            }
            L += l_s[k];
          }
          put_row<D>(a, shape, it, row, acc, L);
        }
        __syncthreads();
      }
    }
  }
  put_zeros<D>(a, shape, items);
}

// Parts of the tensor-memory kernel: a slot's o is [D / 4][block] of four elements, as its
// threads (a query row each) can store it with whole lines; a warp joins 32 rows of four
// elements, all its loads whole lines too.  One pass over the parts, eight at a time, with
// a running maximum (a question of 33 tokens, 18 parts of 165 rows: 44 us in all; eight
// elements and four parts at a time 46).
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    cache_attn_merge_cols(const CacheAttnArgs a, const AttnShape shape, int64_t items, int ctas,
                          int by_item, const float2* ml,
                          const float4* o) {
  constexpr int AHEAD = 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Split sp = find_split(a, shape, items, ctas, by_item);
  const AttnItem& it = sp.it;
  begin_after_previous();                // the partial results are complete and visible

  const int tasks = sp.parts > 0 ? ((it.rows + 31) / 32) * (D / 4) : 0;
  for (int task = blockIdx.y * kMergeWarps + warp; task < tasks; task += gridDim.y * kMergeWarps) {
    const int chunk = task % (D / 4), row = task / (D / 4) * 32 + lane;   // elements 4 chunk ..
    if (row >= it.rows) continue;
    float M = -INFINITY, L = 0.f;
    float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < sp.parts; i0 += AHEAD) {
      float2 x[AHEAD];
      float4 p[AHEAD];
      float top = M;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        x[k] = make_float2(-INFINITY, 0.f);
        p[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + k < sp.parts) {
          const int64_t s = sp.slot(i0 + k);
          x[k] = __ldcg(ml + s * shape.block + row);
          p[k] = __ldcg(o + (s * (D / 4) + chunk) * shape.block + row);
        }
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) top = fmax_nan(top, x[k].x);
      const float sub = top == -INFINITY ? 0.f : top;
      const float f = exp2f(M - sub);
      M = top;
      L *= f;
      u = make_float4(u.x * f, u.y * f, u.z * f, u.w * f);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float w = exp2f(x[k].x - sub);
        L = fmaf(x[k].y, w, L);
        u.x = fmaf(p[k].x, w, u.x);
        u.y = fmaf(p[k].y, w, u.y);
        u.z = fmaf(p[k].z, w, u.z);
        u.w = fmaf(p[k].w, w, u.w);
      }
    }
    put4(a, shape, it, row, 4 * chunk, u, L);
  }
  put_zeros<D>(a, shape, items);
}

}  // namespace

cudaError_t launch_attn_merge(const CacheAttnArgs& a, const AttnShape& shape, int64_t items,
                              int ctas, bool cols, const float2* ml, const float* o,
                              cudaStream_t st) {
  // y: blocks that share an item's rows.  Few-rows parts: a row a block where an item is
  // likely to have many parts, else eight; otherwise eight tasks of 32 rows x 4 elements.
  const int by_item = items <= ctas;
  const int64_t x = by_item ? items : ctas;
  const int64_t rows = std::min<int64_t>(shape.block, static_cast<int64_t>(shape.n_q) * shape.G);
  int64_t y = cols ? (rows + 31) / 32 * (a.c.d / 4) / kMergeWarps
                   : (ctas > kWarpSplits * items ? rows : (rows + kMergeWarps - 1) / kMergeWarps);
  // (a block finds its item first, which costs as much as joining a few parts: one per cut,
  // of which most have little to do, comes in fours; 300 us for four questions, 313 in
  // sixteens)
  y = std::max<int64_t>(1, std::min<int64_t>(y, 148 * (cols && !by_item ? 4 : 8) / x));
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
  if (cols) {
    const float4* o4 = reinterpret_cast<const float4*>(o);
    return a.c.d == 128 ? launch_after(cache_attn_merge_cols<128>, grid, kMergeThreads, 0, st, a, shape, items, ctas,
                                       by_item, ml, o4)
                        : launch_after(cache_attn_merge_cols<256>, grid, kMergeThreads, 0, st, a, shape, items, ctas,
                                       by_item, ml, o4);
  }
  return a.c.d == 128 ? launch_after(cache_attn_merge<128>, grid, kMergeThreads, 0, st, a, shape, items, ctas,
                                       by_item, ml, o)
                      : launch_after(cache_attn_merge<256>, grid, kMergeThreads, 0, st, a, shape, items, ctas,
                                       by_item, ml, o);
}

cudaError_t bounds_flag_cache_attention_merge(unsigned int* out) { return take_bounds_flag(out); }

// Few query rows a unit go to the mma.sync kernel, 16 at a time, which each time read the
// cache again (from L2, mostly); many to the tensor-memory kernel, whose tiles hold 128 and
// which unpacks quantised pages first.  Measured, rows kernel against the other, us, 284K
// rows in 8 heads:  bf16 d = 128: 32 rows 42 / 45, 48 75 / 55;  d = 256: 32 108 / 72;
// fp8 d = 128: 32 35 / 65, 64 57 / 70, 96 82 / 67;  d = 256: 32 66 / 83, 48 102 / 96;
// int4 d = 128: 64 56 / 65, 96 109 / 86;  d = 256: 32 83 / 95, 48 113 / 89.
static bool few_rows(int64_t rows, int d, int format) {
  return rows <= (d == 128 ? 32 : 16) * (format == kFmtBf16 ? 1 : 2);
}

size_t cache_attn_ws_bytes(int G, int n_q, int d, int format) {
  if (!few_rows(static_cast<int64_t>(n_q) * G, d, format)) return attn_ws_bytes(kTcCtas, tc_block(d), d);
  const int block = rows_block(static_cast<int64_t>(n_q) * G);
  return attn_ws_bytes(rows_ctas(format, d, block), block, d);
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t s, int* launches) {
  return few_rows(static_cast<int64_t>(a.n_q) * a.G, a.c.d, a.c.format)
             ? launch_cache_attn_rows(a, s, launches)
             : launch_cache_attn_tc(a, s, launches);
}

}  // namespace kvzip
