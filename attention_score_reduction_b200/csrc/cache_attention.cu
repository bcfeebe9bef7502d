// Attention of new tokens over the paged cache, for few query rows a unit.
//
// For unit u with len rows, m new tokens (already written: they are its last m
// rows) and G query heads, query row (i, g) sees rows j < len - m + i + 1:
//   out = sum_j softmax_j(scale q.k_j) v_j,  zeros where nothing is seen.
// With a handful of query rows (decoding: G of them) every cache byte is used
// once, so the kernel is bound by HBM.  Each warp walks batches of rows of its
// CTA's piece of the work line with K and V going from global memory straight to
// the registers of mma.sync fragments, no shared memory in between:
//   logits  S = Q K^T       M = 16 query rows, N = 8 cache rows, K = 16 elements
//   output  O^T += V^T P^T  M = 16 elements, N = 8 query rows, K = 16 cache rows
// The order of the elements inside a product is free as long as both operands
// agree, so a lane's share of a K row is 16 consecutive bytes (B fragment: lane
// group `quad` = cache row, lane in quad = 16-byte piece), and its share of V is
// 16 consecutive bytes of four rows (A fragment: `quad` = piece, lane in quad =
// rows): every load is a whole sector of a row, and pairs of V rows are
// interleaved with byte permutes.  The accumulator fragment of S is the B
// fragment of P^T as it stands.  The next batch's K is requested as soon as this
// batch's logits are formed, the next V as soon as the output is, so that a few
// KB per warp are always in flight.
//
// Quantised formats multiply the codes themselves, as fp16 (exact for e4m3 and
// for 0..15), and fold the rows' parameters into logits and weights:
//   x_j = c (s_j S_j + z_j sum(q)),     out = sum_j (p_j s_j) code_j + sum_j p_j z_j.
// Q goes to fp16 scaled by a power of two per row (a bf16 value is exact in fp16
// down to 2^-32 of the row's largest).  The weights p_j s_j are formed relative
// to their own running maximum, as fp16: rounded by at most 2^-11 of a weight,
// an eighth of the rounding of a bf16 output.  bf16 caches take the weights as
// two bf16 parts (about 16 bits).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "cache_attention.cuh"
#include "cache_sched.cuh"
#include "kvzip_internal.h"

namespace kvzip {

namespace {

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int FMT>
__device__ __forceinline__ void mma_fmt(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FMT == kFmtBf16) mma_bf16(d, a0, a1, a2, a3, b0, b1);
  else mma_f16(d, a0, a1, a2, a3, b0, b1);
}

constexpr int kRowsTile = 64;     // cache rows of a tile: two or four batches, one per warp

template <int FMT, int D>
struct RowsCfg {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int RB = CacheRow<FMT, D>::BYTES;
  static constexpr int BR = FMT == kFmtBf16 ? 16 : 32;   // cache rows of one batch
  static constexpr int NJ = BR / 8;                       // 8-row tiles of the logits
  static constexpr int KC = RB / 64;                      // 16-byte pieces of a K row per lane
  static constexpr int KS = D / 16;                       // k-steps of the logits; m-tiles of the output
};

// Everything a warp carries through its batches of one item.
template <int FMT, int D, int NT>
struct RowsState {
  float m[NT], l[NT], mo[NT], oz[NT];
  float o[NT][D / 16][4];
};

// NT: 8-row groups of query rows in an item (1 or 2).
template <int FMT, int D, int NT>
__global__ void __launch_bounds__(RowsCfg<FMT, D>::THREADS)
    cache_attn_rows(const CacheAttnArgs a, const AttnShape shape, int64_t items, float c,
                    float2* __restrict__ ml_out, float* __restrict__ o_out) {
  using Cfg = RowsCfg<FMT, D>;
  constexpr int WARPS = Cfg::WARPS, THREADS = Cfg::THREADS, RB = Cfg::RB, BR = Cfg::BR;
  constexpr int NJ = Cfg::NJ, KC = Cfg::KC, KS = Cfg::KS, RQ = 8 * NT;
  constexpr bool QUANT = FMT != kFmtBf16;
  __shared__ int64_t scratch[WARPS];
  __shared__ int64_t found[2];
  __shared__ float xm[WARPS][RQ], xl[WARPS][RQ];
  __shared__ float xo[WARPS / 2][RQ][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, qp = lane & 3;
  const int64_t cta = blockIdx.x;

  cudaTriggerProgrammaticLaunchCompletion();   // the merge may be launched; it waits for this grid
  Line<THREADS> line(a.c, shape, items, scratch, found);
  const int64_t all = line.all;
  const int64_t n_cta = line_ctas(all, gridDim.x);
  if (cta >= n_cta) return;
  const int64_t p0 = line_cut(all, cta, n_cta), p1 = line_cut(all, cta + 1, n_cta);
  int64_t w, w_at;
  line.find(p0, &w, &w_at);

  for (int64_t p = p0; p < p1; ++w) {
    const AttnItem it = attn_item(a.c, shape, w);
    const int n_tiles = it.n_tiles;
    const int64_t at = w_at;
    w_at += n_tiles;
    if (n_tiles == 0) continue;
    const int t0 = static_cast<int>(p - at);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(n_tiles), p1 - at));
    p = at + t1;
    const int r_end = min(t1 * kRowsTile, it.vis);

    // ---- query fragments and per-row limits (rows quad and quad + 8 of the item)
    uint32_t qa[KS][2 * NT];
    float cq[NT], qsum[NT];
    int lim[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = it.row0 + quad + 8 * t;
      const bool live = quad + 8 * t < it.rows;
      const int tok = row / shape.G;
      lim[t] = live ? seen_rows(it, tok) : 0;
      const uint16_t* qr = static_cast<const uint16_t*>(a.q) + it.u * a.q_unit +
                           (row - tok * shape.G) * a.q_head + tok * a.q_row;
      float f = 1.f;
      if constexpr (QUANT) {
        // the row's largest magnitude, then a power of two that lifts it to [2^14, 2^15)
        uint32_t top = 0;
        if (live) {
          const uint4* q4 = reinterpret_cast<const uint4*>(qr) + qp * (D / 32);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint4 v = q4[i];
            const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              top = max(top, max((ws[k] << 16) & 0x7fff0000u, ws[k] & 0x7fff0000u));
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = static_cast<int>(top >> 23) - 127;       // -127 for zeros and subnormals
        f = __uint_as_float(static_cast<uint32_t>(min(max(127 + 14 - e, 1), 254)) << 23);
      }
      cq[t] = QUANT ? c / f : c;
      float sum = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t w0 = 0, w1 = 0;      // the pairs of fragment columns 2 qp and 2 qp + 8
        if (live) {
          if constexpr (FMT == kFmtInt4) {
            // word ks / 2 of the lane's pieces: elements e0..e7; (e0, e4), (e1, e5) then (e2, e6), (e3, e7)
            const int el = 128 * (ks / 8) + 32 * qp + 8 * ((ks % 8) / 2) + 2 * (ks & 1);
            w0 = qr[el] | (static_cast<uint32_t>(qr[el + 4]) << 16);
            w1 = qr[el + 1] | (static_cast<uint32_t>(qr[el + 5]) << 16);
          } else {
            const int el = FMT == kFmtBf16 ? 32 * (ks / 2) + 8 * qp + 4 * (ks & 1)
                                           : 64 * (ks / 4) + 16 * qp + 4 * (ks & 3);
            const uint2 v = *reinterpret_cast<const uint2*>(qr + el);
            w0 = v.x;
            w1 = v.y;
          }
          if constexpr (QUANT) {
            const float f0 = bf16_lo(w0) * f, f1 = bf16_hi(w0) * f;
            const float f2 = bf16_lo(w1) * f, f3 = bf16_hi(w1) * f;
            sum += (f0 + f1) + (f2 + f3);
            w0 = pack_f16x2(f0, f1);
            w1 = pack_f16x2(f2, f3);
          }
        }
        qa[ks][2 * t] = w0;
        qa[ks][2 * t + 1] = w1;
      }
      if constexpr (FMT == kFmtInt4) {
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      }
      qsum[t] = sum;
    }

    RowsState<FMT, D, NT> st;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      st.m[t] = st.mo[t] = -INFINITY;
      st.l[t] = st.oz[t] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[t][k][e] = 0.f;
    }

    // ---- batches of this warp: rows r0 + (warp + WARPS n) * BR
    const int r_first = t0 * kRowsTile + warp * BR;
    int64_t base[BR / 16];               // pool row of each 16-row group of the batch, or -1
    auto find = [&](int r) {
#pragma unroll
      for (int g = 0; g < BR / 16; ++g)
        base[g] = r + 16 * g < r_end ? cache_slot(a.c, it.u, r + 16 * g) : -1;
    };
    uint4 kreg[NJ][KC];
    uint4 vreg[BR / 4][RB / 128 > 0 ? RB / 128 : 1];
    uint2 kpar[QUANT ? NJ : 1], vpar[QUANT ? NJ : 1];
    const uint8_t* kp = static_cast<const uint8_t*>(a.c.k_pages);
    const uint8_t* vp = static_cast<const uint8_t*>(a.c.v_pages);
    auto load_k = [&](int r) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t b = base[j / 2];
        const bool ok = b >= 0 && r + 8 * j + quad < r_end;
        const uint8_t* src = kp + (b + 8 * (j & 1) + quad) * RB + 16 * qp;
#pragma unroll
        for (int k = 0; k < KC; ++k)
          kreg[j][k] = ok ? ldg_stream16(src + 64 * k) : make_uint4(0, 0, 0, 0);
        if constexpr (QUANT) {
          const int64_t pr = b + 8 * (j & 1) + 2 * qp;
          kpar[j] = b >= 0 ? ldg_stream8(a.c.k_params + pr) : make_uint2(0, 0);
        }
      }
    };
    // rows of this lane's V registers: group g = 16 g + {0, 1, 8, 9} + 2 qp
    auto load_v = [&](int r) {
#pragma unroll
      for (int g = 0; g < BR / 16; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int dr = 2 * qp + (i & 1) + 8 * (i >> 1);
          const bool ok = base[g] >= 0 && r + 16 * g + dr < r_end;
          const uint8_t* src = vp + (base[g] + dr) * RB;
          if constexpr (RB >= 128) {
#pragma unroll
            for (int h = 0; h < RB / 128; ++h)
              vreg[4 * g + i][h] =
                  ok ? ldg_stream16(src + 128 * h + 16 * quad) : make_uint4(0, 0, 0, 0);
          } else {
            const uint2 v = ok ? ldg_stream8(src + 8 * quad) : make_uint2(0, 0);
            vreg[4 * g + i][0].x = v.x;
            vreg[4 * g + i][0].y = v.y;
          }
        }
      if constexpr (QUANT) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int64_t pr = base[j / 2] + 8 * (j & 1) + 2 * qp;
          vpar[j] = base[j / 2] >= 0 ? ldg_stream8(a.c.v_params + pr) : make_uint2(0, 0);
        }
      }
    };
    if (r_first < r_end) {
      find(r_first);
      load_k(r_first);
      load_v(r_first);
    }
    for (int r = r_first; r < r_end; r += WARPS * BR) {
      const int rn = r + WARPS * BR;
      // ---- logits
      float s[NJ][4];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const uint32_t ws[4] = {kreg[j][k].x, kreg[j][k].y, kreg[j][k].z, kreg[j][k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (FMT == kFmtBf16) {
              if (i & 1) continue;
              const int ks = 2 * k + i / 2;
              mma_bf16(s[j], qa[ks][0], NT > 1 ? qa[ks][2 * NT - 2] : 0u, qa[ks][1],
                       NT > 1 ? qa[ks][2 * NT - 1] : 0u, ws[i], ws[i + 1]);
            } else if constexpr (FMT == kFmtFp8) {
              const int ks = 4 * k + i;
              mma_f16(s[j], qa[ks][0], NT > 1 ? qa[ks][2 * NT - 2] : 0u, qa[ks][1],
                      NT > 1 ? qa[ks][2 * NT - 1] : 0u, e4m3x2_f16x2(ws[i]),
                      e4m3x2_f16x2(ws[i] >> 16));
            } else {
              const int ks = 8 * k + 2 * i;
              mma_f16(s[j], qa[ks][0], NT > 1 ? qa[ks][2 * NT - 2] : 0u, qa[ks][1],
                      NT > 1 ? qa[ks][2 * NT - 1] : 0u, nib_f16x2<0>(ws[i]), nib_f16x2<1>(ws[i]));
              mma_f16(s[j], qa[ks + 1][0], NT > 1 ? qa[ks + 1][2 * NT - 2] : 0u, qa[ks + 1][1],
                      NT > 1 ? qa[ks + 1][2 * NT - 1] : 0u, nib_f16x2<0>(ws[i] >> 8),
                      nib_f16x2<1>(ws[i] >> 8));
            }
          }
        }
      }
      uint2 kpar_now[QUANT ? NJ : 1];
      if constexpr (QUANT) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) kpar_now[j] = kpar[j];
      }
      // ---- request the next batch's K (its pages first); this batch's V is on its way
      if (rn < r_end) {
        find(rn);
        load_k(rn);
      }
      // ---- scaled logits (log2 domain), masked
      float alpha_o[NT];
      uint32_t phi[NT][NJ], plo[NT][QUANT ? 1 : NJ];
      bool moved = false;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[NJ][2];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = s[j][2 * t + e];
            if constexpr (FMT == kFmtFp8) {
              v *= __uint_as_float(e ? kpar_now[j].y : kpar_now[j].x);
            } else if constexpr (FMT == kFmtInt4) {
              const uint32_t par = e ? kpar_now[j].y : kpar_now[j].x;
              v = fmaf(v, bf16_lo(par), bf16_hi(par) * qsum[t]);
            }
            x[j][e] = r + 8 * j + 2 * qp + e < lim[t] ? v * cq[t] : -INFINITY;
            mx = fmaxf(mx, x[j][e]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(st.m[t], mx);
        const float m_sub = m_new == -INFINITY ? 0.f : m_new;   // nothing seen yet
        const float alpha = exp2f(st.m[t] - m_sub);
        moved |= m_new != st.m[t];
        st.m[t] = m_new;
        float sum = 0.f;
        if constexpr (!QUANT) {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const float e0 = exp2f(x[j][0] - m_sub), e1 = exp2f(x[j][1] - m_sub);
            sum += e0 + e1;
            phi[t][j] = pack_bf16x2(e0, e1);
            plo[t][j] = pack_bf16x2(e0 - bf16_lo(phi[t][j]), e1 - bf16_hi(phi[t][j]));
          }
          alpha_o[t] = alpha;
        } else {
          // weights p s relative to their own maximum: y = x + log2 s
          float y[NJ][2], my = -INFINITY, z = 0.f;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t par = e ? vpar[j].y : vpar[j].x;
              const float pe = exp2f(x[j][e] - m_sub);
              sum += pe;
              float ls;
              if constexpr (FMT == kFmtFp8) {
                // the exponent of 2^e; a NaN scale (a row with a non-finite element) stays NaN
                ls = par < 0x7f800000u ? static_cast<float>(static_cast<int>(par >> 23) - 127)
                                       : __uint_as_float(0x7fc00000u);
              } else {
                ls = __log2f(bf16_lo(par));
                // a masked row's zero may be anything: only seen rows count
                z += r + 8 * j + 2 * qp + e < lim[t] ? pe * bf16_hi(par) : 0.f;
              }
              y[j][e] = r + 8 * j + 2 * qp + e < lim[t] ? x[j][e] + ls : -INFINITY;
              my = fmaxf(my, y[j][e]);
            }
          my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 1));
          my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 2));
          const float mo_new = fmaxf(st.mo[t], my);
          const float mo_sub = mo_new == -INFINITY ? 0.f : mo_new;
          alpha_o[t] = exp2f(st.mo[t] - mo_sub);
          moved |= mo_new != st.mo[t];
          st.mo[t] = mo_new;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            phi[t][j] = pack_f16x2(exp2f(y[j][0] - mo_sub), exp2f(y[j][1] - mo_sub));
          st.oz[t] = st.oz[t] * alpha + z;
        }
        st.l[t] = st.l[t] * alpha + sum;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float a_lo = __shfl_sync(0xffffffffu, alpha_o[t], 8 * qp);
          const float a_hi = __shfl_sync(0xffffffffu, alpha_o[t], 8 * qp + 4);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            st.o[t][k][0] *= a_lo;
            st.o[t][k][1] *= a_hi;
            st.o[t][k][2] *= a_lo;
            st.o[t][k][3] *= a_hi;
          }
        }
      }
      // ---- O^T += V^T P^T, 16 cache rows at a time
#pragma unroll
      for (int g = 0; g < BR / 16; ++g) {
        auto pv = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_fmt<FMT>(st.o[t][mt], a0, a1, a2, a3, phi[t][2 * g], phi[t][2 * g + 1]);
            if constexpr (!QUANT)
              mma_bf16(st.o[t][mt], a0, a1, a2, a3, plo[t][2 * g], plo[t][2 * g + 1]);
          }
        };
        constexpr int WORDS = RB / 32;      // 32-bit words of a V row per lane
#pragma unroll
        for (int wd = 0; wd < WORDS; ++wd) {
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4& q4 = vreg[4 * g + i][wd / 4];
            v[i] = wd % 4 == 0 ? q4.x : (wd % 4 == 1 ? q4.y : (wd % 4 == 2 ? q4.z : q4.w));
          }
          if constexpr (FMT == kFmtBf16) {
            pv(wd, __byte_perm(v[0], v[1], 0x5410), __byte_perm(v[0], v[1], 0x7632),
               __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[2], v[3], 0x7632));
          } else if constexpr (FMT == kFmtFp8) {
            const uint32_t x0 = __byte_perm(v[0], v[1], 0x5140), x1 = __byte_perm(v[0], v[1], 0x7362);
            const uint32_t y0 = __byte_perm(v[2], v[3], 0x5140), y1 = __byte_perm(v[2], v[3], 0x7362);
            pv(2 * wd, e4m3x2_f16x2(x0), e4m3x2_f16x2(x0 >> 16), e4m3x2_f16x2(y0),
               e4m3x2_f16x2(y0 >> 16));
            pv(2 * wd + 1, e4m3x2_f16x2(x1), e4m3x2_f16x2(x1 >> 16), e4m3x2_f16x2(y1),
               e4m3x2_f16x2(y1 >> 16));
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t x = __byte_perm(v[0], v[1], h ? 0x7632 : 0x5410);
              const uint32_t y = __byte_perm(v[2], v[3], h ? 0x7632 : 0x5410);
              pv(4 * wd + 2 * h, nib_f16x2<0>(x), nib_f16x2<1>(x), nib_f16x2<0>(y), nib_f16x2<1>(y));
              pv(4 * wd + 2 * h + 1, nib_f16x2<0>(x >> 8), nib_f16x2<1>(x >> 8),
                 nib_f16x2<0>(y >> 8), nib_f16x2<1>(y >> 8));
            }
          }
        }
      }
      if (rn < r_end) load_v(rn);
    }

    // ---- this warp's result, relative to 2^m: o = sum p v
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      st.l[t] += __shfl_xor_sync(0xffffffffu, st.l[t], 1);
      st.l[t] += __shfl_xor_sync(0xffffffffu, st.l[t], 2);
      if constexpr (QUANT) {
        st.oz[t] += __shfl_xor_sync(0xffffffffu, st.oz[t], 1);
        st.oz[t] += __shfl_xor_sync(0xffffffffu, st.oz[t], 2);
        const float f = st.mo[t] == -INFINITY ? 0.f : exp2f(st.mo[t] - st.m[t]);
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * qp);
        const float f1 = __shfl_sync(0xffffffffu, f, 8 * qp + 4);
        const float z0 = __shfl_sync(0xffffffffu, st.oz[t], 8 * qp);
        const float z1 = __shfl_sync(0xffffffffu, st.oz[t], 8 * qp + 4);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          st.o[t][k][0] = fmaf(st.o[t][k][0], f0, z0);
          st.o[t][k][1] = fmaf(st.o[t][k][1], f1, z1);
          st.o[t][k][2] = fmaf(st.o[t][k][2], f0, z0);
          st.o[t][k][3] = fmaf(st.o[t][k][3], f1, z1);
        }
      }
    }
    // element of o[.][mt][e] (query row 2 qp + (e & 1)): a run of the lane's own piece
    auto elem = [&](int mt, int e) {
      if constexpr (FMT == kFmtBf16)
        return 64 * (mt / 4) + 8 * quad + 2 * (mt % 4) + (e >> 1);
      else if constexpr (FMT == kFmtFp8)
        return 128 * (mt / 8) + 16 * quad + 2 * (mt % 8) + (e >> 1);
      else
        return (D / 8) * quad + 2 * mt + (e >> 1);
    };
    // ---- merge the warps pairwise: the upper half hands over, the lower half adds
    for (int half = WARPS / 2; half >= 1; half >>= 1) {
      if (warp >= half && warp < 2 * half) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (qp == 0) {
            xm[warp][quad + 8 * t] = st.m[t];
            xl[warp][quad + 8 * t] = st.l[t];
          }
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              xo[warp - half][2 * qp + (e & 1) + 8 * t][elem(k, e)] = st.o[t][k][e];
        }
      }
      __syncthreads();
      if (warp < half) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float m2 = xm[warp + half][quad + 8 * t], l2 = xl[warp + half][quad + 8 * t];
          const float M = fmaxf(st.m[t], m2);
          const float sub = M == -INFINITY ? 0.f : M;
          const float fa = exp2f(st.m[t] - sub), fb = exp2f(m2 - sub);
          st.m[t] = M;
          st.l[t] = st.l[t] * fa + l2 * fb;
          const float a0 = __shfl_sync(0xffffffffu, fa, 8 * qp), a1 = __shfl_sync(0xffffffffu, fa, 8 * qp + 4);
          const float b0 = __shfl_sync(0xffffffffu, fb, 8 * qp), b1 = __shfl_sync(0xffffffffu, fb, 8 * qp + 4);
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              st.o[t][k][e] = st.o[t][k][e] * ((e & 1) ? a1 : a0) +
                              xo[warp][2 * qp + (e & 1) + 8 * t][elem(k, e)] * ((e & 1) ? b1 : b0);
        }
      }
      __syncthreads();
    }
    // ---- warp 0 holds the CTA's result; it goes out through shared memory in row order
    if (warp == 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (qp == 0) {
          xm[0][quad + 8 * t] = st.m[t];
          xl[0][quad + 8 * t] = st.l[t];
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            xo[0][2 * qp + (e & 1) + 8 * t][elem(k, e)] = st.o[t][k][e];
      }
    }
    __syncthreads();
    if (t0 == 0 && t1 == n_tiles) {
      for (int i = threadIdx.x; i < it.rows * (D / 8); i += THREADS) {
        const int row = i / (D / 8), e = (i % (D / 8)) * 8;
        const float inv = xl[0][row] > 0.f ? 1.f / xl[0][row] : (xl[0][row] == 0.f ? 0.f : NAN);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = xo[0][row][e + k] * inv;
        attn_store8(a, shape, it, row, e, v);
      }
    } else {
      const int64_t slot = line_slot(all, cta, n_cta, at);
      for (int i = threadIdx.x; i < RQ * D / 4; i += THREADS)
        reinterpret_cast<float4*>(o_out + slot * RQ * D)[i] =
            reinterpret_cast<const float4*>(&xo[0][0][0])[i];
      if (threadIdx.x < RQ) ml_out[slot * RQ + threadIdx.x] = make_float2(xm[0][threadIdx.x], xl[0][threadIdx.x]);
    }
    __syncthreads();
  }
}

template <int FMT, int D, int NT>
cudaError_t launch_rows(const CacheAttnArgs& a, cudaStream_t st, int* launches) {
  using Cfg = RowsCfg<FMT, D>;
  const AttnShape shape = attn_shape(a.q_lens, a.n_q, a.G, 8 * NT, kRowsTile);
  const int64_t items = a.c.units * shape.blocks;
  const int ctas = rows_ctas(a.c.format, D);
  float2* ml = static_cast<float2*>(a.ws);
  float* o = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) +
                                      attn_ml_bytes(ctas, shape.block));
  cache_attn_rows<FMT, D, NT><<<ctas, Cfg::THREADS, 0, st>>>(
      a, shape, items, a.scale * 1.4426950408889634f, ml, o);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  *launches += 2;
  return launch_attn_merge(a, shape, items, ctas, ml, o, st);
}

}  // namespace

// CTAs of the work line: as many as fit on the 148 SMs together (their registers
// allow three per SM, two for bf16 rows of 256).
int rows_ctas(int format, int d) { return 148 * (format == kFmtBf16 && d == 256 ? 2 : 3); }

int rows_block(int64_t rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_cache_attn_rows(const CacheAttnArgs& a, cudaStream_t s, int* launches) {
  const bool one = rows_block(static_cast<int64_t>(a.n_q) * a.G) == 8;
#define KVZIP_ROWS(F, DD)                                            \
  case F * 1000 + DD:                                                \
    return one ? launch_rows<F, DD, 1>(a, s, launches) : launch_rows<F, DD, 2>(a, s, launches);
  switch (a.c.format * 1000 + a.c.d) {
    KVZIP_ROWS(kFmtBf16, 128)
    KVZIP_ROWS(kFmtBf16, 256)
    KVZIP_ROWS(kFmtFp8, 128)
    KVZIP_ROWS(kFmtFp8, 256)
    KVZIP_ROWS(kFmtInt4, 128)
    KVZIP_ROWS(kFmtInt4, 256)
    default: return cudaErrorInvalidValue;
  }
#undef KVZIP_ROWS
}

}  // namespace kvzip
