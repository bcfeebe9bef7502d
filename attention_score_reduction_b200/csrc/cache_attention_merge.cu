// Joins the partial results of attention over the paged cache, and sizes the
// workspace they live in.
#include <cuda_runtime.h>

#include <cstdint>

#include "cache_attention.cuh"
#include "kvzip_internal.h"

namespace kvzip {

namespace {

constexpr int kMergeThreads = 256;

// Block (item, y) merges rows y, y + gridDim.y, ... of the item.  The threads
// are D / 4 columns of four elements by 1024 / D groups of splits, so the loads of
// a row's splits are in flight together; groups meet in shared memory.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    cache_attn_merge(const CacheAttnArgs a, const AttnShape shape, int64_t items, int ctas,
                     const float2* __restrict__ ml, const float* __restrict__ o) {
  constexpr int COLS = D / 4, GROUPS = kMergeThreads / COLS;
  __shared__ int64_t scratch[kMergeThreads / 32];
  __shared__ float4 acc_s[GROUPS][COLS];
  __shared__ float l_s[GROUPS];
  cudaGridDependencySynchronize();       // the partial results are complete and visible
  const int64_t w = blockIdx.x;
  const AttnItem it = attn_item(a.c, shape, w);
  if (it.rows <= 0 || static_cast<int>(blockIdx.y) >= it.rows) return;
  const int n_tiles = it.n_tiles;
  int64_t c0 = 0, c1 = 0;                // CTAs with a part of the item, inclusive
  int64_t slot0 = 0;                     // slot of c0's part; later CTAs begin with the item
  if (n_tiles > 0) {
    const LineTotals t = line_totals<kMergeThreads>(a.c, shape, items, w, scratch);
    const int64_t n = line_ctas(t.all, ctas);
    c0 = line_cta(t.all, t.before, n);
    c1 = line_cta(t.all, t.before + n_tiles - 1, n);
    if (c0 == c1) return;                // one CTA wrote the output itself
    slot0 = line_slot(t.all, c0, n, t.before);
  }
  const int col = threadIdx.x % COLS, grp = threadIdx.x / COLS;
  for (int row = blockIdx.y; row < it.rows; row += gridDim.y) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (n_tiles > 0) {
      float M = -INFINITY;
      for (int64_t c = c0; c <= c1; ++c) M = fmaxf(M, ml[(c == c0 ? slot0 : 2 * c) * shape.block + row].x);
      const float sub = M == -INFINITY ? 0.f : M;
#pragma unroll 4
      for (int64_t c = c0 + grp; c <= c1; c += GROUPS) {
        const int64_t slot = (c == c0 ? slot0 : 2 * c) * shape.block + row;
        const float2 v = ml[slot];
        const float f = exp2f(v.x - sub);
        const float4 x = reinterpret_cast<const float4*>(o + slot * D)[col];
        l = fmaf(v.y, f, l);
        acc.x = fmaf(x.x, f, acc.x);
        acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z);
        acc.w = fmaf(x.w, f, acc.w);
      }
    }
    acc_s[grp][col] = acc;
    if (col == 0) l_s[grp] = l;
    __syncthreads();
    if (threadIdx.x < D / 8) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      float L = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const float4 x = acc_s[g][2 * threadIdx.x], y = acc_s[g][2 * threadIdx.x + 1];
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
        L += l_s[g];
      }
      const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : NAN);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = L == 0.f ? 0.f : v[k] * inv;
      attn_store8(a, shape, it, row, 8 * threadIdx.x, v);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_attn_merge(const CacheAttnArgs& a, const AttnShape& shape, int64_t items,
                              int ctas, const float2* ml, const float* o, cudaStream_t st) {
  // enough blocks to fill the machine, rows of an item shared by several
  int64_t y = (148 * 8 + items - 1) / items;
  if (y > shape.block) y = shape.block;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items), static_cast<unsigned>(y));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // overlaps the launch latency
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return a.c.d == 128
             ? cudaLaunchKernelEx(&cfg, cache_attn_merge<128>, a, shape, items, ctas, ml, o)
             : cudaLaunchKernelEx(&cfg, cache_attn_merge<256>, a, shape, items, ctas, ml, o);
}

// Up to 16 query rows a unit go to the mma.sync kernel, which reads the cache once
// for them; beyond, the tensor-memory kernel, whose tiles hold 128.
static bool few_rows(int n_q, int G) { return static_cast<int64_t>(n_q) * G <= 16; }

size_t cache_attn_ws_bytes(int64_t units, int G, int n_q, int d, int format) {
  (void)units;
  return few_rows(n_q, G)
             ? attn_ws_bytes(rows_ctas(format, d), rows_block(static_cast<int64_t>(n_q) * G), d)
             : attn_ws_bytes(kTcCtas, tc_block(d), d);
}

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t s, int* launches) {
  return few_rows(a.n_q, a.G) ? launch_cache_attn_rows(a, s, launches)
                              : launch_cache_attn_tc(a, s, launches);
}

}  // namespace kvzip
