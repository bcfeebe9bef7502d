// Attention of new tokens over the paged cache, for few query rows a unit.
//
// For unit u with len rows, m new tokens (already written: they are its last m
// rows) and G query heads, query row (i, g) sees rows j < len - m + i + 1:
//   out = sum_j softmax_j(scale q.k_j) v_j,  zeros where nothing is seen.
// With a handful of query rows (decoding: G of them) every cache byte is used
// once, so the kernel is bound by HBM.  Each warp walks batches of rows of its
// CTA's piece of the work line, with mma.sync fragments:
//   logits  S = Q K^T       M = 16 query rows, N = 8 cache rows, K = 16 elements
//   output  O^T += V^T P^T  M = 16 elements, N = 8 query rows, K = 16 cache rows
// The order of the elements inside a product is free as long as both operands
// agree, so a lane's share of a K row is 16 consecutive bytes (B fragment: lane
// group `quad` = cache row, lane in quad = 16-byte piece), and its share of V is
// 16 consecutive bytes of four rows (A fragment: `quad` = piece, lane in quad =
// rows): every load is a whole sector of a row, and pairs of V rows are
// interleaved with byte permutes.  The accumulator fragment of S is the B
// fragment of P^T as it stands.  Each warp keeps a ring of two or three batches in
// shared memory that asynchronous copies fill, so that over 100 KB per SM are in
// flight; batches held in registers (one ahead) reached half of that.  Two or three
// CTAs an SM: more start and end more items' parts, fewer leave issue slots idle
// (16 sequences, 4-bit, 2 / 3 / 4 CTAs an SM: 64 / 58 / 60 us; bf16, 2 with three
// batches 39 us, 3 with two 41 us).
//
// Measured, a call in a stream: one token over a bf16 layer of 284K rows in 8 heads
// (145 MB) 34 us, of which 27 go to the loads (5.4 TB/s; CTAs end between 23 and 31 us,
// as some SMs get more of HBM than others) and the rest to start, join and merge; one
// token for each of 16 sequences over 4-bit pages (149 MB) 48 us: 46% issue active with
// three warps a scheduler, whose logits, softmax and output of a batch wait for one another.
//
// Quantised formats multiply the codes themselves, as fp16, and fold the rows'
// parameters into logits and weights:
//   x_j = c (s_j S_j + z_j sum(q)),     out = sum_j (p_j s_j) code_j + sum_j p_j z_j.
// e4m3 codes are exact in fp16.  4-bit codes are not converted at all: masked out of
// their word, four bits are the fp16 subnormal c 2^-24 (or 16 c 2^-24), which the
// tensor core multiplies exactly; the powers of two go into Q and the result.
// Unpacking to fp16 integers instead takes two more instructions a pair.  The two sums over
// 4-bit rows are taken apart and may nearly cancel: their float32 rounding, up to n 2^-26 of
// either over the n rows that a warp walks, is of sum p s c and sum p z, not of the output.
// Q goes to fp16 scaled by a power of two per row (a bf16 value is exact in fp16
// down to 2^-28 of the row's largest).  The weights p_j s_j are formed relative
// to a power of two that keeps their largest between 2^8 and 2^15, as fp16: rounded by at
// most 2^-11 of themselves (an eighth of the rounding of a bf16 output) down to 2^-22 of
// the largest, and by 2^-33 of it below.  bf16 caches take the weights as two bf16 parts
// (about 16 bits).
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cache.cuh"
#include "cache_attention.cuh"
#include "cache_sched.cuh"
#include "kvzip_internal.h"
#include "sm100_ptx.cuh"

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

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Whether the e4m3 codes of a stored row are zeros, of either sign.
template <int BYTES>
__device__ __forceinline__ bool all_zero_codes(uint32_t row) {
#pragma unroll 1
  for (int i = 0; i < BYTES; i += 16) {
    const uint4 v = lds16(row + i);
    if (((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) != 0) return false;
  }
  return true;
}

constexpr float kCodeUnit = 16777216.f;   // 2^24
// How far (log2) a row's running maximum may be above the reference of its weights.  Sums of
// weights times values stay finite for values up to 2^96 of 2^23 rows.
constexpr float kLag = 8.f;
// The largest of the weights that are formed as fp16: held between these, set to 2^11 .. 2^12.
constexpr float kWeightMax = 32768.f, kWeightMin = 256.f;
constexpr int kWeightSet = 11;
constexpr int kRowsTile = 64;     // cache rows of a tile: two or four batches, one per warp

template <int FMT, int D>
struct RowsCfg {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int RB = CacheRow<FMT, D>::BYTES;
  static constexpr int BR = RB >= 256 ? 16 : 32;         // cache rows of one batch
  static constexpr int NJ = BR / 8;                       // 8-row tiles of the logits
  static constexpr int KC = RB / 64;                      // 16-byte pieces of a K row per lane
  static constexpr int KS = D / 16;                       // k-steps of the logits; m-tiles of the output
  static constexpr bool QUANT = FMT != kFmtBf16;
  // a warp's ring of batches: K codes, V codes, K parameters, V parameters
  static constexpr int SLOTS = FMT == kFmtFp8 && D == 128 ? 2 : 3;
  static constexpr int CODES = BR * RB;
  static constexpr int SLOT = 2 * CODES + (QUANT ? 8 * BR : 0);
  static constexpr int RING = WARPS * SLOTS * SLOT;
  static constexpr int PAD = 4;                           // an item's start and end in tiles of work
};

// 16-byte chunk of row r as it lies in shared memory: chunks of a row are exchanged so
// that neither the K reads (rows quad, chunks of the lane in quad) nor the V reads (rows
// 2 lane-in-quad, chunks by quad) meet in a bank.
template <int RB>
__device__ __forceinline__ int swizzled(int r, int chunk) {
  if constexpr (RB == 64) return chunk ^ ((r >> 1) & 3);
  else return chunk ^ ((((r >> 1) & 3) << 1) ^ ((r & 1) << 2));
}

// Asynchronous copies global -> shared; `bytes` 0 fills with zeros instead.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// CTAs that fit on an SM together, by registers and shared memory.
constexpr int rows_per_sm(int format, int d, int block) {
  if (d == 128) return block == 8 && format != kFmtBf16 ? 3 : 2;
  return format == kFmtBf16 ? 1 : 2;
}

// NT: 8-row groups of query rows in an item (1 or 2).
template <int FMT, int D, int NT>
__global__ void __launch_bounds__(RowsCfg<FMT, D>::THREADS, rows_per_sm(FMT, D, 8 * NT))
    cache_attn_rows(const CacheAttnArgs a, const AttnShape shape, int64_t items, float c,
                    float2* __restrict__ ml_out, float* __restrict__ o_out) {
  using Cfg = RowsCfg<FMT, D>;
  constexpr int WARPS = Cfg::WARPS, THREADS = Cfg::THREADS, RB = Cfg::RB, BR = Cfg::BR;
  constexpr int NJ = Cfg::NJ, KC = Cfg::KC, KS = Cfg::KS, RQ = 8 * NT;
  constexpr bool QUANT = FMT != kFmtBf16;
  __shared__ int64_t scratch[WARPS];
  __shared__ LineSpot spot_s;
  __shared__ float xm[WARPS][RQ], xl[WARPS][RQ];
  extern __shared__ __align__(16) uint8_t ring_raw[];
  // the warps' results, once their rings are read
  float(*xo)[RQ][D] = reinterpret_cast<float(*)[RQ][D]>(ring_raw);
  static_assert(WARPS * RQ * D * 4 <= Cfg::RING, "results do not fit where the rings were");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, qp = lane & 3;
  const int64_t cta = blockIdx.x;

  begin_after_previous();
  Line<THREADS> line(a.c, shape, items, scratch, &spot_s);
  const int64_t all = line.all;
  const int64_t n_cta = line_ctas(all, gridDim.x);
  if (cta >= n_cta) return;
  const int64_t p0 = line_cut(all, cta, n_cta), p1 = line_cut(all, cta + 1, n_cta);
  const LineSpot spot = line.find(p0);
  int64_t w = spot.item, w_at = spot.at;
  AttnItem it = spot.info;

  for (int64_t p = p0; p < p1; ++w) {
    if (w != spot.item) it = attn_item(a.c, shape, w);
    const int64_t at = w_at;
    if (it.span == 0) continue;
    int t0, t1;
    const bool any = line_tiles(it, shape, at, p, p1, t0, t1);
    p = w_at += it.span;
    if (!any) continue;
    const int r_end = min(t1 * kRowsTile, it.vis);

    // ---- batches of this warp: rows r0 + (warp + WARPS n) * BR
    const int r_first = t0 * kRowsTile + warp * BR;
    const int lim_all = min(seen_rows(it, it.row0 / shape.G), r_end);   // rows that all queries see
    const uint32_t ring = smem_u32(ring_raw) + warp * (Cfg::SLOTS * Cfg::SLOT);
    constexpr int GROUPS = BR / 16;
    // pool row of each 16-row group of a batch, or -1
    auto find = [&](int r, int64_t (&base)[GROUPS]) {
      base[0] = r < r_end ? cache_slot(a.c, it.u, r) : -1;
      if constexpr (GROUPS > 1) {
        if (a.c.page_shift >= 5) base[1] = base[0] >= 0 ? base[0] + 16 : -1;   // the same page
        else base[1] = r + 16 < r_end ? cache_slot(a.c, it.u, r + 16) : -1;
      }
    };
    // batch of rows r .. into a slot; rows past the end and of a bad page become zeros
    auto request = [&](int r, uint32_t slot, const int64_t (&base)[GROUPS]) {
      // parameters, four rows a copy: a lane of the first BR / 4 takes K's, of the next V's
      const int par_row = 4 * (lane % (BR / 4));
      const uint32_t par_dst = slot + 2 * Cfg::CODES + 16 * lane;
      const uint32_t* par_pool = lane < BR / 4 ? a.c.k_params : a.c.v_params;
      auto base_of_lane = [&](const int64_t (&b)[GROUPS]) { return par_row < 16 ? b[0] : b[GROUPS - 1]; };
      constexpr int CPR = RB / 16, PER = 32 / CPR > 0 ? 32 / CPR : 1;   // chunks a row, rows a copy
      if (r + BR <= r_end && base[0] >= 0 && base[GROUPS - 1] >= 0) {
        // nothing to leave out: a copy takes 512 consecutive bytes of a group
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const uint8_t* k = static_cast<const uint8_t*>(a.c.k_pages) + base[g] * RB + 16 * lane;
          const uint8_t* v = static_cast<const uint8_t*>(a.c.v_pages) + base[g] * RB + 16 * lane;
#pragma unroll
          for (int i = 0; i < RB / 32; ++i) {
            const int idx = 32 * (i + g * (RB / 32)) + lane, row = idx / CPR, chunk = idx % CPR;
            const uint32_t dst = slot + row * RB + 16 * swizzled<RB>(row, chunk);
            copy16(dst, k + 512 * i);
            copy16(dst + Cfg::CODES, v + 512 * i);
          }
        }
        if constexpr (QUANT) {
          if (lane < 2 * (BR / 4)) copy16(par_dst, par_pool + base_of_lane(base) + par_row % 16);
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < Cfg::CODES / 512; ++i) {
        const int idx = 32 * i + lane, row = idx / CPR, chunk = idx % CPR;
        const int g = CPR >= 32 ? (i * 32 / CPR) / 16 : (i * PER) / 16;
        const int bytes = base[g] >= 0 && r + row < r_end ? 16 : 0;
        const int64_t at = bytes ? (base[g] + (row & 15)) * RB + 16 * chunk : 0;
        const uint32_t dst = slot + row * RB + 16 * swizzled<RB>(row, chunk);
        copy16(dst, static_cast<const uint8_t*>(a.c.k_pages) + at, bytes);
        copy16(dst + Cfg::CODES, static_cast<const uint8_t*>(a.c.v_pages) + at, bytes);
      }
      if constexpr (QUANT) {
        if (lane < 2 * (BR / 4)) {
          const int64_t b = base_of_lane(base);
          const int bytes = b >= 0 ? 4 * max(0, min(4, r_end - r - par_row)) : 0;
          copy16(par_dst, par_pool + (bytes ? b + par_row % 16 : 0), bytes);
        }
      }
    };
    // ---- query fragments and per-row limits (rows quad and quad + 8 of the item)
    uint32_t qa[KS][2 * NT];
    float cq[NT];        // log2-domain logit = cq S (+ cz z_j for int4)
    float cz[NT];
    int lim[NT];
    // the pairs of fragment columns 2 qp and 2 qp + 8 of every k-step, as bf16: requested
    // before the copies, which would keep them waiting
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = it.row0 + quad + 8 * t;
      const bool live = quad + 8 * t < it.rows;
      const int tok = row / shape.G;
      lim[t] = live ? seen_rows(it, tok) : 0;
      const uint16_t* qr = static_cast<const uint16_t*>(a.q) + it.u * a.q_unit +
                           (row - tok * shape.G) * a.q_head + tok * a.q_row;
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
        uint4 v = make_uint4(0, 0, 0, 0);
        // int4, a word of codes: elements e0..e7
        const int el = FMT == kFmtInt4 ? 128 * (ks / 8) + 32 * qp + 4 * (ks % 8)
                       : FMT == kFmtBf16 ? 32 * (ks / 2) + 8 * qp
                                         : 64 * (ks / 4) + 16 * qp + 4 * (ks & 3);
        if (live) v = __ldcg(reinterpret_cast<const uint4*>(qr + el));
        qa[ks][2 * t] = v.x;
        qa[ks][2 * t + 1] = v.y;
        qa[ks + 1][2 * t] = v.z;
        qa[ks + 1][2 * t + 1] = v.w;
      }
    }
    // the first batches: all their pages, then all their copies, on their way while Q is
    // prepared
    {
      int64_t base[Cfg::SLOTS][GROUPS];
#pragma unroll
      for (int n = 0; n < Cfg::SLOTS; ++n) find(r_first + n * WARPS * BR, base[n]);
#pragma unroll
      for (int n = 0; n < Cfg::SLOTS; ++n) {
        if (r_first + n * WARPS * BR < r_end)
          request(r_first + n * WARPS * BR, ring + n * Cfg::SLOT, base[n]);
        copies_commit();
      }
    }

#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t top_q = 0;
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
        uint32_t(&w0)[2 * NT] = qa[ks];
        uint32_t(&w1)[2 * NT] = qa[ks + 1];
        if constexpr (FMT == kFmtInt4) {     // (e0, e4), (e1, e5) then (e2, e6), (e3, e7)
          const uint4 v = make_uint4(w0[2 * t], w0[2 * t + 1], w1[2 * t], w1[2 * t + 1]);
          w0[2 * t] = __byte_perm(v.x, v.z, 0x5410);
          w0[2 * t + 1] = __byte_perm(v.x, v.z, 0x7632);
          w1[2 * t] = __byte_perm(v.y, v.w, 0x5410);
          w1[2 * t + 1] = __byte_perm(v.y, v.w, 0x7632);
        }
        if constexpr (QUANT) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            top_q = max(top_q, max(max((w0[2 * t + k] << 16) & 0x7fff0000u, w0[2 * t + k] & 0x7fff0000u),
                                   max((w1[2 * t + k] << 16) & 0x7fff0000u, w1[2 * t + k] & 0x7fff0000u)));
        }
      }
      cq[t] = c;
      cz[t] = 0.f;
      if constexpr (QUANT) {
        // fp16, the row's largest element lifted to [2^14, 2^15)
        top_q = max(top_q, __shfl_xor_sync(0xffffffffu, top_q, 1));
        top_q = max(top_q, __shfl_xor_sync(0xffffffffu, top_q, 2));
        const int e = static_cast<int>(top_q >> 23) - 127;       // -127 for zeros and subnormals
        const float f = __uint_as_float(static_cast<uint32_t>(min(max(127 + 14 - e, 1), 254)) << 23);
        // int4: codes meet Q as fp16 subnormals c 2^-24, those of the odd pairs as 16 c 2^-24
        const float f1 = FMT == kFmtInt4 ? f * 0.0625f : f;
        float sum = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t w0 = qa[ks][2 * t], w1 = qa[ks][2 * t + 1];
          sum += (bf16_lo(w0) + bf16_hi(w0)) + (bf16_lo(w1) + bf16_hi(w1));
          qa[ks][2 * t] = pack_f16x2(bf16_lo(w0) * f, bf16_hi(w0) * f);
          qa[ks][2 * t + 1] = pack_f16x2(bf16_lo(w1) * f1, bf16_hi(w1) * f1);
        }
        cq[t] = c / f;
        if constexpr (FMT == kFmtInt4) {
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          cq[t] *= kCodeUnit;
          cz[t] = c * sum;
        }
      }
    }

    // State of the query rows this lane has in the logits.  Weights are p = 2^(x - m) with
    // a reference m that follows a row's running maximum only once that is 2^8 above it
    // (32-bit sums bear it): no exchange between lanes and no rescaling in most batches.
    // l: this lane's sums of p, by column parity.  Quantised: weights p s are formed as
    // fp16 times a power of two F; F moves when one exceeds top, or (none so far, top = 0)
    // at the first; lead: the largest p s at the last move.  int4: oz = sum p z.
    float m[NT], F[NT], lead[NT], top[NT];
    float2 l2[NT], oz2[NT];
    float o[NT][KS][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -INFINITY;
      l2[t] = oz2[t] = make_float2(0.f, 0.f);
      lead[t] = top[t] = 0.f;
      F[t] = 1.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][k][e] = 0.f;
    }
    // multiplies row t's output by f (of the lanes that have the row in the logits)
    auto rescale = [&](int t, float f) {
      const float f_lo = __shfl_sync(0xffffffffu, f, 8 * qp);
      const float f_hi = __shfl_sync(0xffffffffu, f, 8 * qp + 4);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        o[t][k][0] *= f_lo;
        o[t][k][1] *= f_hi;
        o[t][k][2] *= f_lo;
        o[t][k][3] *= f_hi;
      }
    };

    int n_slot = 0;
    for (int r = r_first; r < r_end; r += WARPS * BR) {
      const int rn = r + Cfg::SLOTS * WARPS * BR;          // the batch that takes this one's slot
      int64_t base[GROUPS];
      find(rn, base);
      const uint32_t slot = ring + n_slot * Cfg::SLOT;
      n_slot = n_slot + 1 == Cfg::SLOTS ? 0 : n_slot + 1;
      copies_wait<Cfg::SLOTS - 1>();
      __syncwarp();
      if constexpr (FMT != kFmtInt4) {
        // the chunk's own tokens, which not every query row sees, must not reach those as
        // 0 * NaN: what is not finite becomes zero, and rows that see it NaN.  (fp8 rows
        // written here have finite codes; those of another writer may not)
        if (lim_all < min(r + BR, r_end)) {
          int bad = INT_MAX;
          for (int i = lane; i < Cfg::CODES / 16; i += 32) {
            const int row = r + i / (RB / 16);
            const uint32_t at = slot + Cfg::CODES + 16 * i;
            if (row < lim_all || row >= r_end) continue;
            if (FMT == kFmtFp8 ? e4m3x16_finite(lds16(at)) : bf16x8_finite(lds16(at))) continue;
            bad = min(bad, row);
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
          }
          __syncwarp();                  // other lanes read what this one has cleared
          bad = __reduce_min_sync(0xffffffffu, bad);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (bad < lim[t]) l2[t].x = NAN;
        }
      }
      // ---- products of the logits
      float s[NJ][4];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
        auto qk = [&](int ks, uint32_t b0, uint32_t b1) {
          mma_fmt<FMT>(s[j], qa[ks][0], NT > 1 ? qa[ks][2 * NT - 2] : 0u, qa[ks][1],
                       NT > 1 ? qa[ks][2 * NT - 1] : 0u, b0, b1);
        };
#pragma unroll
        for (int k = 0; k < KC; ++k) {
          const int row = 8 * j + quad;
          const uint4 kw = lds16(slot + row * RB + 16 * swizzled<RB>(row, 4 * k + qp));
          const uint32_t ws[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (FMT == kFmtBf16) {
              if (i & 1) continue;
              qk(2 * k + i / 2, ws[i], ws[i + 1]);
            } else if constexpr (FMT == kFmtFp8) {
              uint32_t lo, hi;
              e4m3x4_f16x2(ws[i], lo, hi);
              qk(4 * k + i, lo, hi);
            } else {
              qk(8 * k + 2 * i, ws[i] & 0x000f000fu, ws[i] & 0x00f000f0u);
              qk(8 * k + 2 * i + 1, (ws[i] >> 8) & 0x000f000fu, (ws[i] >> 8) & 0x00f000f0u);
            }
          }
        }
      }
      uint2 kpar[QUANT ? NJ : 1], vpar[QUANT ? NJ : 1];     // rows 8 j + 2 qp, + 1
      if constexpr (QUANT) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          kpar[j] = lds8(slot + 2 * Cfg::CODES + 4 * (8 * j + 2 * qp));
          vpar[j] = lds8(slot + 2 * Cfg::CODES + 4 * (BR + 8 * j + 2 * qp));
        }
      }
      if constexpr (FMT == kFmtFp8) {
        // a row of zeros is stored with the scale 1, hundreds of times its neighbours': it
        // must not set the range of the weights
        constexpr uint32_t kOne = 0x3f800000u;
        bool one = false;
#pragma unroll
        for (int j = 0; j < NJ; ++j) one = one || vpar[j].x == kOne || vpar[j].y == kOne;
        if (__any_sync(0xffffffffu, one)) {
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const uint32_t row = slot + Cfg::CODES + (8 * j + 2 * qp) * RB;
            if (vpar[j].x == kOne && all_zero_codes<RB>(row)) vpar[j].x = 0u;
            if (vpar[j].y == kOne && all_zero_codes<RB>(row + RB)) vpar[j].y = 0u;
          }
          __syncwarp();
        }
      }
      // ---- logits (log2 domain) in place, weights
      uint32_t phi[NT][NJ], plo[NT][QUANT ? 1 : NJ];
      auto softmax = [&](auto mask_tag) {
        constexpr bool MASK = decltype(mask_tag)::value;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float2 x[NJ];
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            x[j] = make_float2(s[j][2 * t], s[j][2 * t + 1]);
            const float2 c2 = make_float2(cq[t], cq[t]);
            if constexpr (FMT == kFmtFp8) {
              x[j] = fmul2(x[j], fmul2(make_float2(__uint_as_float(kpar[j].x),
                                                   __uint_as_float(kpar[j].y)), c2));
            } else if constexpr (FMT == kFmtInt4) {
              const float2 sc = fmul2(make_float2(bf16_lo(kpar[j].x), bf16_lo(kpar[j].y)), c2);
              const float2 zc = fmul2(make_float2(bf16_hi(kpar[j].x), bf16_hi(kpar[j].y)),
                                      make_float2(cz[t], cz[t]));
              x[j] = ffma2(x[j], sc, zc);
            } else {
              x[j] = fmul2(x[j], c2);
            }
            if (MASK) {
              x[j].x = r + 8 * j + 2 * qp < lim[t] ? x[j].x : -INFINITY;
              x[j].y = r + 8 * j + 2 * qp + 1 < lim[t] ? x[j].y : -INFINITY;
            }
            mx = fmaxf(mx, fmaxf(x[j].x, x[j].y));
          }
          bool moved = false;
          float f = 1.f;
          if (__any_sync(0xffffffffu, mx > m[t] + kLag)) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m[t], mx);
            f = m_new == -INFINITY ? 1.f : ex2_approx(m[t] - m_new);   // -infinity: nothing seen yet
            m[t] = m_new;
            l2[t] = make_float2(l2[t].x * f, l2[t].y * f);
            oz2[t] = make_float2(oz2[t].x * f, oz2[t].y * f);
            moved = true;
          }
          const float nm = m[t] == -INFINITY ? 0.f : -m[t];
          [[maybe_unused]] float ta = 0.f;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            x[j] = fadd2(x[j], make_float2(nm, nm));
            x[j].x = ex2_approx(x[j].x);
            x[j].y = ex2_approx(x[j].y);
            l2[t] = fadd2(l2[t], x[j]);
            if constexpr (!QUANT) {
              phi[t][j] = pack_bf16x2(x[j].x, x[j].y);
              plo[t][j] = pack_bf16x2(x[j].x - bf16_lo(phi[t][j]), x[j].y - bf16_hi(phi[t][j]));
            } else {
              uint32_t p0 = vpar[j].x, p1 = vpar[j].y;
              if (MASK) {            // a row that this query does not see may hold anything
                p0 = r + 8 * j + 2 * qp < lim[t] ? p0 : 0u;
                p1 = r + 8 * j + 2 * qp + 1 < lim[t] ? p1 : 0u;
              }
              if constexpr (FMT == kFmtFp8) {
                x[j] = fmul2(x[j], make_float2(__uint_as_float(p0), __uint_as_float(p1)));
              } else {
                oz2[t] = ffma2(x[j], make_float2(bf16_hi(p0), bf16_hi(p1)), oz2[t]);
                x[j] = fmul2(x[j], make_float2(bf16_lo(p0), bf16_lo(p1)));
              }
              ta = fmaxf(ta, fmaxf(x[j].x, x[j].y));
            }
          }
          if constexpr (QUANT) {
            if (moved || __any_sync(0xffffffffu, ta > top[t])) {
              ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, 1));
              ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, 2));
              lead[t] = fmaxf(lead[t] * f, ta);
              const float now = lead[t] * F[t];
              if (lead[t] > 0.f && !(now <= kWeightMax && now >= kWeightMin)) {
                const int e = static_cast<int>(__float_as_uint(lead[t]) >> 23);
                const float fn = __uint_as_float(static_cast<uint32_t>(min(max(254 + kWeightSet - e, 1), 253)) << 23);
                f = f * fn / F[t];         // in this order: fn / F may be infinite where f is 0
                F[t] = fn;
              }
              top[t] = lead[t] > 0.f ? kWeightMax / F[t] : 0.f;
              moved = true;
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              x[j] = fmul2(x[j], make_float2(F[t], F[t]));
              phi[t][j] = pack_f16x2(x[j].x, x[j].y);
            }
          }
          if (moved) rescale(t, f);
        }
      };
      if (r + BR > lim_all) softmax(std::true_type{});
      else softmax(std::false_type{});
      // ---- O^T += V^T P^T, 16 cache rows at a time
#pragma unroll
      for (int g = 0; g < BR / 16; ++g) {
        auto pv = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma_fmt<FMT>(o[t][mt], a0, a1, a2, a3, phi[t][2 * g], phi[t][2 * g + 1]);
            if constexpr (!QUANT) mma_bf16(o[t][mt], a0, a1, a2, a3, plo[t][2 * g], plo[t][2 * g + 1]);
          }
        };
        uint32_t vw[4][4];
        // this lane's 16 (RB = 64: 8) bytes of rows 16 g + {0, 1, 8, 9} + 2 qp
        constexpr int VW = RB >= 128 ? 4 : 2;         // 32-bit words of one piece
#pragma unroll
        for (int wd = 0; wd < RB / 32; ++wd) {
          if (wd % VW == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 16 * g + 2 * qp + (i & 1) + 8 * (i >> 1);
              const uint32_t at = slot + Cfg::CODES + row * RB;
              if constexpr (RB >= 128) {
                const uint4 q4 = lds16(at + 16 * swizzled<RB>(row, 8 * (wd / 4) + quad));
                vw[i][0] = q4.x;
                vw[i][1] = q4.y;
                vw[i][2] = q4.z;
                vw[i][3] = q4.w;
              } else {
                const uint2 q2 = lds8(at + 16 * swizzled<RB>(row, quad >> 1) + 8 * (quad & 1));
                vw[i][0] = q2.x;
                vw[i][1] = q2.y;
              }
            }
          }
          const uint32_t v[4] = {vw[0][wd % VW], vw[1][wd % VW], vw[2][wd % VW], vw[3][wd % VW]};
          if constexpr (FMT == kFmtBf16) {
            pv(wd, __byte_perm(v[0], v[1], 0x5410), __byte_perm(v[0], v[1], 0x7632),
               __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[2], v[3], 0x7632));
          } else if constexpr (FMT == kFmtFp8) {
            uint32_t x0, x1, x2, x3, y0, y1, y2, y3;
            e4m3x4_f16x2(__byte_perm(v[0], v[1], 0x5140), x0, x1);
            e4m3x4_f16x2(__byte_perm(v[0], v[1], 0x7362), x2, x3);
            e4m3x4_f16x2(__byte_perm(v[2], v[3], 0x5140), y0, y1);
            e4m3x4_f16x2(__byte_perm(v[2], v[3], 0x7362), y2, y3);
            pv(2 * wd, x0, x1, y0, y1);
            pv(2 * wd + 1, x2, x3, y2, y3);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t x = __byte_perm(v[0], v[1], h ? 0x7632 : 0x5410);
              const uint32_t y = __byte_perm(v[2], v[3], h ? 0x7632 : 0x5410);
              pv(4 * wd + 2 * h, x & 0x000f000fu, x & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u);
              pv(4 * wd + 2 * h + 1, (x >> 8) & 0x000f000fu, (x >> 8) & 0x00f000f0u,
                 (y >> 8) & 0x000f000fu, (y >> 8) & 0x00f000f0u);
            }
          }
        }
      }
      __syncwarp();                      // the slot is read
      if (rn < r_end) request(rn, slot, base);
      copies_commit();
    }
    copies_wait<0>();
    __syncthreads();                     // every warp's ring is read: results go there

    // ---- this warp's result, relative to 2^m: o = sum p v
    float l[NT], oz[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      l[t] = l2[t].x + l2[t].y;
      oz[t] = oz2[t].x + oz2[t].y;
      l[t] += __shfl_xor_sync(0xffffffffu, l[t], 1);
      l[t] += __shfl_xor_sync(0xffffffffu, l[t], 2);
      if constexpr (QUANT) {
        oz[t] += __shfl_xor_sync(0xffffffffu, oz[t], 1);
        oz[t] += __shfl_xor_sync(0xffffffffu, oz[t], 2);
        const float f = 1.f / F[t];
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * qp);
        const float f1 = __shfl_sync(0xffffffffu, f, 8 * qp + 4);
        const float z0 = __shfl_sync(0xffffffffu, oz[t], 8 * qp);
        const float z1 = __shfl_sync(0xffffffffu, oz[t], 8 * qp + 4);
        // int4: codes were c 2^-24, and 16 c 2^-24 in the fragment's second row
        constexpr float u0 = FMT == kFmtInt4 ? kCodeUnit : 1.f;
        constexpr float u1 = FMT == kFmtInt4 ? kCodeUnit / 16.f : 1.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          o[t][k][0] = fmaf(o[t][k][0] * u0, f0, z0);
          o[t][k][1] = fmaf(o[t][k][1] * u0, f1, z1);
          o[t][k][2] = fmaf(o[t][k][2] * u1, f0, z0);
          o[t][k][3] = fmaf(o[t][k][3] * u1, f1, z1);
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
    // ---- join the warps: everything through shared memory, eight elements a thread
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (qp == 0) {
        xm[warp][quad + 8 * t] = m[t];
        xl[warp][quad + 8 * t] = l[t];
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            xo[warp][2 * qp + b + 8 * t][elem(k, e)] = o[t][k][e + b];
    }
    __syncthreads();
    const bool whole = t1 - t0 == it.n_tiles;
    const int64_t slot = line_slot(all, cta, n_cta, at + shape.pad);
    for (int i = threadIdx.x; i < it.rows * (D / 8); i += THREADS) {
      const int row = i / (D / 8), e = (i % (D / 8)) * 8;
      float M = xm[0][row];
#pragma unroll
      for (int k = 1; k < WARPS; ++k) M = fmaxf(M, xm[k][row]);
      const float sub = M == -INFINITY ? 0.f : M;
      float L = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        const float f = ex2_approx(xm[k][row] - sub);
        L = fmaf(xl[k][row], f, L);
        const float4 x = *reinterpret_cast<const float4*>(&xo[k][row][e]);
        const float4 y = *reinterpret_cast<const float4*>(&xo[k][row][e + 4]);
        v[0] = fmaf(x.x, f, v[0]);
        v[1] = fmaf(x.y, f, v[1]);
        v[2] = fmaf(x.z, f, v[2]);
        v[3] = fmaf(x.w, f, v[3]);
        v[4] = fmaf(y.x, f, v[4]);
        v[5] = fmaf(y.y, f, v[5]);
        v[6] = fmaf(y.z, f, v[6]);
        v[7] = fmaf(y.w, f, v[7]);
      }
      if (whole) {
        const float inv = attn_inverse(L, seen_rows(it, (it.row0 + row) / shape.G) <= 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= inv;
        attn_store8(a, shape, it, row, e, v);
      } else if (slot_in_bounds(shape, slot, gridDim.x, row)) {
        float4* dst = reinterpret_cast<float4*>(o_out + (slot * RQ + row) * D + e);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        if (e == 0) ml_out[slot * RQ + row] = make_float2(M, L);
      }
    }
    __syncthreads();
  }
}

template <int FMT, int D, int NT>
cudaError_t launch_rows(const CacheAttnArgs& a, cudaStream_t st, int* launches) {
  using Cfg = RowsCfg<FMT, D>;
  const AttnShape shape = attn_shape(a.q_lens, a.n_q, a.G, 8 * NT, kRowsTile, Cfg::PAD);
  const int64_t items = a.c.units * shape.blocks;
  const int ctas = rows_ctas(FMT, D, shape.block);
  float2* ml = static_cast<float2*>(a.ws);
  float* o = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) +
                                      attn_ml_bytes(ctas, shape.block));
  cudaError_t e = cudaFuncSetAttribute(cache_attn_rows<FMT, D, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::RING);
  if (e != cudaSuccess) return e;
  e = launch_after(cache_attn_rows<FMT, D, NT>, dim3(ctas), Cfg::THREADS, Cfg::RING, st, a, shape,
                   items, a.scale * 1.4426950408889634f, ml, o);
  if (e != cudaSuccess) return e;
  *launches += 2;
  return launch_attn_merge(a, shape, items, ctas, false, ml, o, st);
}

}  // namespace

cudaError_t bounds_flag_cache_attention(unsigned int* out) { return take_bounds_flag(out); }

// CTAs of the work line: all resident on the 148 SMs at once.
int rows_ctas(int format, int d, int block) { return 148 * rows_per_sm(format, d, block); }

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
