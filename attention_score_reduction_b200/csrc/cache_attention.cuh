// Shared by the attention kernels over the paged cache: storing output rows and
// merging the partial results of items that several CTAs worked on.
#pragma once
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cache_sched.cuh"

namespace kvzip {

// What a row's sum is multiplied by: 1 / L.  L = 0 where it sees nothing, which gives zeros,
// or only logits of -infinity, which have no softmax: NaN.
__device__ __forceinline__ float attn_inverse(float L, bool blind) {
  return L > 0.f ? 1.f / L : (L == 0.f && blind ? 0.f : NAN);
}

// Query head g of token tok of an item has an output row.
__device__ __forceinline__ bool out_in_bounds(const CacheAttnArgs& a, const AttnItem& it, int tok, int g) {
  return in_bounds(it.u >= 0 && it.u < a.c.units && tok >= 0 && tok < a.n_q && tok < it.m && g >= 0 && g < a.G);
}
// Row `row` of a slot is one of the workspace's: two slots a CTA of `block` rows each.
__device__ __forceinline__ bool slot_in_bounds(const AttnShape& s, int64_t slot, int ctas, int row) {
  return in_bounds(slot >= 0 && slot < 2 * static_cast<int64_t>(ctas) && row >= 0 && row < s.block);
}

// Eight consecutive elements of query row `row` of an item.
__device__ __forceinline__ void attn_store8(const CacheAttnArgs& a, const AttnShape& s,
                                            const AttnItem& it, int row, int e,
                                            const float (&v)[8]) {
  const int r = it.row0 + row, tok = r / s.G, g = r - tok * s.G;
  if (!out_in_bounds(a, it, tok, g)) return;
  const int64_t at = it.u * a.o_unit + g * a.o_head + tok * a.o_row + e;
  if (a.out_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  }
}

inline AttnShape attn_shape(const int32_t* q_lens, int n_q, int G, int block, int tile, int pad) {
  const int64_t rows = static_cast<int64_t>(n_q) * G;
  return AttnShape{q_lens, n_q, G, block, static_cast<int>((rows + block - 1) / block), tile,
                   pad};
}

// Workspace: (m, l) of two slots per CTA, then their o rows.
inline size_t attn_ml_bytes(int ctas, int block) {
  return (2 * static_cast<size_t>(ctas) * block * sizeof(float2) + 255) / 256 * 256;
}
inline size_t attn_ws_bytes(int ctas, int block, int d) {
  return attn_ml_bytes(ctas, block) + 2 * static_cast<size_t>(ctas) * block * d * sizeof(float);
}

// out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the CTAs of each item
// that no CTA covered whole; zeros for items (and rows) that see nothing.  A
// slot holds shape.block rows of (m, l), m in the log2 domain, and of o: [block][d], or
// (cols) [d / 4][block][4].
cudaError_t launch_attn_merge(const CacheAttnArgs& a, const AttnShape& shape, int64_t items,
                              int ctas, bool cols, const float2* ml, const float* o,
                              cudaStream_t st);

// Few query rows a unit: mma.sync, straight from global memory.
int rows_ctas(int format, int d, int block);
int rows_block(int64_t rows);      // query rows of an item, for `rows` rows a unit
cudaError_t launch_cache_attn_rows(const CacheAttnArgs& a, cudaStream_t s, int* launches);

// Many: tcgen05, one CTA per SM.
constexpr int kTcCtas = 148;
int tc_block(int d);
cudaError_t launch_cache_attn_tc(const CacheAttnArgs& a, cudaStream_t s, int* launches);

}  // namespace kvzip
