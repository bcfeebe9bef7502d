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
    const float4 x = reinterpret_cast<const float4*>(o)[lane + 32 * i];
    acc.v[i].x = fmaf(x.x, f, acc.v[i].x);
    acc.v[i].y = fmaf(x.y, f, acc.v[i].y);
    acc.v[i].z = fmaf(x.z, f, acc.v[i].z);
    acc.v[i].w = fmaf(x.w, f, acc.v[i].w);
  }
}

// out row = acc / L (0 where L is 0), four elements a lane.
template <int D>
__device__ __forceinline__ void put_row(const CacheAttnArgs& a, const AttnShape& s,
                                        const AttnItem& it, int row, const RowPart<D>& acc, float L) {
  const int lane = threadIdx.x & 31;
  const int r = it.row0 + row, tok = r / s.G, g = r - tok * s.G;
  const int64_t at = it.u * a.o_unit + g * a.o_head + tok * a.o_row + 4 * lane;
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : NAN);
#pragma unroll
  for (int i = 0; i < D / 128; ++i) {
    float4 x = acc.v[i];
    x = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                 : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (a.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + 128 * i) = x;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + 128 * i) =
          make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  }
}

// Which item a block joins does not depend on the results, so it is found before
// the wait for the grid that computes them.  Blocks are one per item, or (many
// items: few of them are split) one per cut between two CTAs, of which the first
// inside an item serves it.  Items with few parts (a long chunk: two or three)
// give a row to each warp; with many (one token: dozens) the warps of a block
// share a row's parts, so that their loads are in flight together.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    cache_attn_merge(const CacheAttnArgs a, const AttnShape shape, int64_t items, int ctas,
                     int by_item, const float2* __restrict__ ml, const float* __restrict__ o) {
  __shared__ int64_t scratch[kMergeWarps];
  __shared__ LineSpot spot_s;
  __shared__ RowPart<D> acc_s[kMergeWarps][32];
  __shared__ float l_s[kMergeWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool split = false;
  int64_t c0 = 0, c1 = 0;                // CTAs with a part of the item, inclusive
  Line<kMergeThreads> t(a.c, shape, items, scratch, &spot_s);
  const int64_t n = line_ctas(t.all, ctas);
  LineSpot spot;
  if (by_item) {
    spot = t.of_item(blockIdx.x);
    split = spot.info.n_tiles > 0;
  } else if (blockIdx.x + 1 < n) {
    const int64_t cut = line_cut(t.all, blockIdx.x + 1, n);
    spot = t.find(cut);
    // the first cut inside the item
    split = spot.at < cut && line_cut(t.all, blockIdx.x, n) <= spot.at;
  }
  const int64_t before = spot.at;
  const AttnItem it = spot.info;
  if (split) {
    c0 = line_cta(t.all, before, n);
    c1 = line_cta(t.all, before + it.n_tiles - 1, n);
    split = c0 != c1;
  }
  cudaGridDependencySynchronize();       // the partial results are complete and visible

  if (split) {
    const int parts = static_cast<int>(c1 - c0) + 1;
    const int64_t slot0 = line_slot(t.all, c0, n, before);     // later CTAs begin with the item
    auto part = [&](int i) { return (i == 0 ? slot0 : 2 * (c0 + i)) * shape.block; };
    if (parts <= kWarpSplits) {
      for (int row = blockIdx.y * kMergeWarps + warp; row < it.rows; row += gridDim.y * kMergeWarps) {
        const float2 x = lane < parts ? ml[part(lane) + row] : make_float2(-INFINITY, 0.f);
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
            xl[k] = ml[slot];
#pragma unroll
            for (int e = 0; e < D / 128; ++e)
              x[k].v[e] = reinterpret_cast<const float4*>(o + slot * D)[lane + 32 * e];
          } else {
            xl[k] = make_float2(-INFINITY, 0.f);
            x[k] = {};
          }
        }
        float M = -INFINITY;
        for (int i = lane; i < parts; i += 32) M = fmax_nan(M, ml[part(i) + row].x);
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
            y.v[e] = reinterpret_cast<const float4*>(o + slot * D)[lane + 32 * e];
          add(y, ml[slot]);
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
  // items that see nothing: zeros
  const RowPart<D> zero = {};
  for (int64_t z = blockIdx.x; z < items; z += gridDim.x) {
    const AttnItem iz = attn_item(a.c, shape, z);
    if (iz.n_tiles == 0)
      for (int row = blockIdx.y * kMergeWarps + warp; row < iz.rows; row += gridDim.y * kMergeWarps)
        put_row<D>(a, shape, iz, row, zero, 0.f);
  }
}

}  // namespace

cudaError_t launch_attn_merge(const CacheAttnArgs& a, const AttnShape& shape, int64_t items,
                              int ctas, const float2* ml, const float* o, cudaStream_t st) {
  // y: blocks that share an item's rows, a row or eight at a time
  const int by_item = items <= ctas;
  const int64_t x = by_item ? items : ctas;
  const int64_t y = by_item ? std::min<int64_t>(shape.block, std::max<int64_t>(1, 148 * 8 / x))
                            : 148 * 8 / x;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(y));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // overlaps the launch latency
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return a.c.d == 128 ? cudaLaunchKernelEx(&cfg, cache_attn_merge<128>, a, shape, items, ctas,
                                           by_item, ml, o)
                      : cudaLaunchKernelEx(&cfg, cache_attn_merge<256>, a, shape, items, ctas,
                                           by_item, ml, o);
}

// Up to 16 query rows a unit go to the mma.sync kernel, which reads the cache once
// for them; beyond, the tensor-memory kernel, whose tiles hold 128.
static bool few_rows(int n_q, int G) { return static_cast<int64_t>(n_q) * G <= 16; }

size_t cache_attn_ws_bytes(int G, int n_q, int d, int format) {
  if (!few_rows(n_q, G)) return attn_ws_bytes(kTcCtas, tc_block(d), d);
  const int block = rows_block(static_cast<int64_t>(n_q) * G);
  return attn_ws_bytes(rows_ctas(format, d, block), block, d);
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t s, int* launches) {
  return few_rows(a.n_q, a.G) ? launch_cache_attn_rows(a, s, launches)
                              : launch_cache_attn_tc(a, s, launches);
}

}  // namespace kvzip
