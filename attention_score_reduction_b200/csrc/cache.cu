// Writing rows into the paged cache, quantised on the way, and reading them back.
//
// Both directions touch every byte once, so they are bound by HBM (large calls)
// or by the launch (a decoding step's few rows).  A row of d elements is the
// work of d / 8 lanes, 16 bytes of bf16 each, so that a half warp (d = 128) or a
// warp (d = 256) moves whole 128-byte lines and a row's extremes cost four or
// five shuffles.  A warp takes `chunk` consecutive rows: lane i finds where row i
// goes (unit, page, pool row) for all of them at once, which keeps the dependent
// loads (offsets, start, page table) off the rows' own path, and the lanes of a
// row get its address by a shuffle.
//
// Quantisation (one row x of one unit):
//   fp8   e = smallest integer >= -126 with max|x| <= 448 * 2^e (0 for a zero
//         row); code = e4m3(x * 2^-e).  The scale is a power of two, so x * 2^-e
//         is exact, the one rounding is the e4m3 conversion's, and the value
//         code * 2^e is exact in bf16.  A non-finite element makes the scale NaN:
//         the whole row reads back as NaN.
//   int4  z = min x (exact in bf16), s = bf16((max - min) / 15), code = the
//         integer nearest (x - z) / s (ties to even, 0 where s = 0), held to 15.
//         A non-finite element, or one of magnitude 2^126 or more (its range
//         would overflow), makes s and z NaN.
// The scale s = bf16((max - min) / 15) is the same from 32 bits as from exact
// arithmetic: a quotient within 2^-23 of a midpoint between two bf16 numbers m
// needs max - min = 15 m (1 + tiny), but 15 m has 12 or 13 significant bits and
// max and min have 8 each, so they are equal or at least 2^-20 apart.
#include <cuda_runtime.h>

#include <cstdint>

#include "cache.cuh"
#include "kvzip_internal.h"
#include "sm100_ptx.cuh"

namespace kvzip {

namespace {

constexpr int kRowThreads = 256;
constexpr float kInt4Limit = 8.507059173023462e37f;   // 2^126

// Unit and row of flat row r: dense r = u * n_rows + t; packed offsets[u] <= r <
// offsets[u + 1].  Returns false where no unit owns the row.
__device__ __forceinline__ bool row_owner(const int64_t* offsets, int64_t units, int64_t n_rows,
                                          int64_t r, int64_t* u, int64_t* t) {
  if (offsets == nullptr) {
    *u = r / n_rows;
    *t = r - *u * n_rows;
    return *u < units;
  }
  int64_t lo = 0, hi = units;            // offsets[lo] <= r (or lo = 0), r < offsets[hi] (or hi = units)
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (offsets[mid] <= r) lo = mid; else hi = mid;
  }
  *u = lo;
  *t = r - offsets[lo];
  return *t >= 0 && r < offsets[lo + 1];
}

// Rows the call brings for unit u.
__device__ __forceinline__ int64_t rows_of(const CacheWriteArgs& a, int64_t u) {
  if (a.offsets != nullptr) {
    const int64_t lo = a.offsets[u], hi = a.offsets[u + 1];
    if (lo < 0 || hi < lo || hi > a.n_rows) atomicOr(a.c.status, kStatusBadCache);
    const int64_t n = (hi > a.n_rows ? a.n_rows : hi) - (lo < 0 ? 0 : lo);
    return n < 0 ? 0 : n;
  }
  return a.counts == nullptr ? a.n_rows
                             : held_to(a.counts[u], static_cast<int>(a.n_rows), a.c.status);
}

__device__ __forceinline__ void advance_len(const CacheWriteArgs& a, int64_t u, int first) {
  const int cap = cache_cap(a.c);
  a.c.lens[u] = held_to(first + rows_of(a, u), cap, a.c.status);
}

// One row's eight elements of a lane, as floats.
__device__ __forceinline__ void unpack8(const uint4& raw, float (&x)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

// What the 4-bit codes of a row are computed with.
struct Int4Row {
  uint32_t par;
  float lift, zl, s, inv;
  bool exact;             // the row needs int4_codes<true>
};

__device__ __forceinline__ Int4Row int4_row(float lo, float hi) {
  Int4Row q;
  const bool bad = !(hi < kInt4Limit && lo > -kInt4Limit);      // infinity, NaN, too large
  q.par = bad ? 0x7fc07fc0u : pack_bf16x2((hi - lo) / 15.f, lo);
  q.s = bf16_lo(q.par);
  // tiny scales are lifted by 2^100 (exactly), so that 1 / s stays finite
  q.lift = q.s < 8.6736174e-19f ? 1.2676506e30f : 1.f;
  q.zl = -lo * q.lift;
  q.s *= q.lift;
  q.inv = q.s > 0.f ? 1.f / q.s : 0.f;
  // x - z is exact in 32 bits unless one of the two is below 2^-16 of the other.  Then
  // it is the other, rounded, and that matters only where the other is half way between
  // two codes: -z by itself, or any x beside a tiny z.
  const float zq = q.zl * q.inv, frac = zq - floorf(zq);
  q.exact = q.lift > 1.f || fabsf(frac - 0.5f) < 1e-4f + fabsf(zq) * 4.7683716e-7f || (lo != 0.f && fabsf(lo) < hi * 3.0517578e-5f);
  return q;
}

// Eight codes as a word.  The quotient is corrected by its exact remainder, so that a
// tie is a tie (of bf16 rows a few elements in a thousand are: x, z and s have eight
// significant bits each; by the same count any other quotient is at least 2^-13 from
// a border).  Rounded to even by adding 1.5 * 2^23: the code is in the sum's low bits.
// A quotient is between 0 and 15.06, as s is within 2^-8 of range / 15.
// EXACT: a tiny s, a subnormal bf16, can be further off (codes are held to 15), and
// where x - z was rounded its error decides a tie.
template <bool EXACT>
__device__ __forceinline__ uint32_t int4_codes(const uint4& raw, const Int4Row& q) {
  constexpr float kRound = 12582912.f;
  constexpr uint32_t kRoundBits = 0x4b400000u;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const float2 lift = make_float2(q.lift, q.lift), zl = make_float2(q.zl, q.zl);
  const float2 inv = make_float2(q.inv, q.inv), ns = make_float2(-q.s, -q.s);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
    const float2 d = ffma2(x, lift, zl);                    // x - z
    float2 t = fmul2(d, inv);
    t = ffma2(ffma2(t, ns, d), inv, t);
    float2 u = fadd2(t, make_float2(kRound, kRound));
    if constexpr (EXACT) {
      auto settle = [&](float xi, float di, float& ui) {
        const float r = fmaf(kRound - ui, q.s, di), half = 0.5f * q.s;
        const bool odd = __float_as_uint(ui) & 1u;
        const float a = xi * q.lift, bb = di - a;
        const float err = (a - (di - bb)) + (q.zl - bb);
        if (r > half || (r == half && (err > 0.f || (err == 0.f && odd)))) ui += 1.f;
        if (r < -half || (r == -half && (err < 0.f || (err == 0.f && odd)))) ui -= 1.f;
        ui = fminf(ui, kRound + 15.f);
      };
      settle(x.x, d.x, u.x);
      settle(x.y, d.y, u.y);
    }
    word += (__float_as_uint(u.x) - kRoundBits) << (8 * i);
    word += (__float_as_uint(u.y) - kRoundBits) << (8 * i + 4);
  }
  return q.s > 0.f ? word : 0u;
}

// Groups of eight elements that a lane has of a row, d / 8 / kGroups apart.  Quantised:
// two, as half the shuffles and half the lanes that work out the row's scale.
template <int FMT>
constexpr int kGroups = FMT == kFmtBf16 ? 1 : 2;

// Stores N rows of which this lane has C groups each; slot < 0: none.  Every step
// goes over all rows before the next, so that their latencies overlap.
template <int FMT, int D, int N, int C>
__device__ __forceinline__ void store_rows(uint8_t* pages, uint32_t* params, const int64_t (&slot)[N],
                                           int lr, const uint4 (&raw)[N][C]) {
  constexpr int LPR = D / 8 / C;
  if constexpr (FMT == kFmtBf16) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (slot[n] >= 0)
        *reinterpret_cast<uint4*>(pages + slot[n] * CacheRow<FMT, D>::BYTES + lr * 16) = raw[n][0];
  } else if constexpr (FMT == kFmtFp8) {
    // the largest magnitude by the order of the bits, where a NaN ranks above
    // infinity and so is seen
    uint32_t top[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t t = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t w[4] = {raw[n][c].x, raw[n][c].y, raw[n][c].z, raw[n][c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) t = max(t, max((w[i] << 16) & 0x7fff0000u, w[i] & 0x7fff0000u));
      }
      top[n] = t;
    }
#pragma unroll
    for (int k = LPR / 2; k >= 1; k >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) top[n] = max(top[n], __shfl_xor_sync(0xffffffffu, top[n], k));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      // 448 * 2^e = 1.75 * 2^(e + 8): e from the exponent, one more above 1.75
      int e = static_cast<int>(top[n] >> 23) - 127 - 8 + ((top[n] & 0x7fffffu) > 0x600000u ? 1 : 0);
      e = top[n] == 0 ? 0 : max(e, -126);
      const bool bad = top[n] >= 0x7f800000u;
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);   // 2^-e
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float x[8];
        unpack8(raw[n][c], x);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = pack_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
        // a bad row's codes are zeros: NaN lives in parameters only, which the
        // attention applies after its mask
        if (slot[n] >= 0)
          *reinterpret_cast<uint2*>(pages + slot[n] * CacheRow<FMT, D>::BYTES + (lr + c * LPR) * 8) =
              bad ? make_uint2(0, 0) : make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      }
      if (slot[n] >= 0 && lr == 0)
        params[slot[n]] = bad ? 0x7fc00000u : static_cast<uint32_t>(127 + e) << 23;
    }
  } else {
    // (smallest, minus the largest) as two bf16, so that one exchange serves both
    uint32_t ends[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t lo = raw[n][0].x, hi = raw[n][0].x;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t w[4] = {raw[n][c].x, raw[n][c].y, raw[n][c].z, raw[n][c].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo = bf16x2_min_nan(lo, w[i]);
          hi = bf16x2_max_nan(hi, w[i]);
        }
      }
      hi ^= 0x80008000u;
      ends[n] = bf16x2_min_nan(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
    }
#pragma unroll
    for (int k = LPR / 2; k >= 1; k >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n)
        ends[n] = bf16x2_min_nan(ends[n], __shfl_xor_sync(0xffffffffu, ends[n], k));
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const Int4Row q = int4_row(bf16_lo(ends[n]), -bf16_hi(ends[n]));
      uint32_t word[C];
#pragma unroll
      for (int c = 0; c < C; ++c) word[c] = int4_codes<false>(raw[n][c], q);
      if (q.exact) {
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
          const uint32_t exact = int4_codes<true>(c == 0 ? raw[n][0] : raw[n][C - 1], q);
          if (c == 0) word[0] = exact; else word[C - 1] = exact;
        }
      }
      if (slot[n] >= 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          *reinterpret_cast<uint32_t*>(pages + slot[n] * CacheRow<FMT, D>::BYTES + (lr + c * LPR) * 4) =
              word[c];
        if (lr == 0) params[slot[n]] = q.par;
      }
    }
  }
}

// Codes of eight elements of a stored row as loaded, and as four bf16 pairs.
template <int FMT>
struct RowBits {
  uint4 c;         // bf16: 16 bytes; fp8: 8 in x, y; int4: 4 in x
  uint32_t par;
};
template <int FMT, int D>
__device__ __forceinline__ RowBits<FMT> load_row(const uint8_t* pages, const uint32_t* params,
                                                 int64_t slot, int lr) {
  RowBits<FMT> b{};
  const uint8_t* p = pages + slot * CacheRow<FMT, D>::BYTES;
  if constexpr (FMT == kFmtBf16) {
    b.c = ld_stream16(p + lr * 16);
  } else {
    if constexpr (FMT == kFmtFp8) {
      const uint2 v = ld_stream8(p + lr * 8);
      b.c.x = v.x;
      b.c.y = v.y;
    } else {
      b.c.x = ld_stream4(p + lr * 4);
    }
    b.par = ld_stream4(params + slot);
  }
  return b;
}
template <int FMT>
__device__ __forceinline__ uint4 row_values(const RowBits<FMT>& b) {
  if constexpr (FMT == kFmtBf16) {
    return b.c;
  } else if constexpr (FMT == kFmtFp8) {
    const float s = __uint_as_float(b.par);
    uint32_t h[4], o[4];
    e4m3x4_f16x2(b.c.x, h[0], h[1]);
    e4m3x4_f16x2(b.c.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f0, f1;
      asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\t"
          "cvt.f32.f16 %1, b;\n\t}"
          : "=f"(f0), "=f"(f1)
          : "r"(h[i]));
      o[i] = pack_bf16x2(f0 * s, f1 * s);   // exact: 4 significant bits and a power of two
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    const uint32_t s2 = __byte_perm(b.par, 0, 0x1010), z2 = __byte_perm(b.par, 0, 0x3232);
    // 0x4300 | c is the bf16 128 + c; minus 128 it is exact, and s c + z is rounded once
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = bfma2(bfma2(and_or(b.c.x >> (4 * i), 0x000f000fu, 0x43004300u), 0x3f803f80u, 0xc300c300u),
                   s2, z2);                       // elements i and i + 4
    return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410),
                      __byte_perm(o[0], o[1], 0x7632), __byte_perm(o[2], o[3], 0x7632));
  }
}

// mode 0: lens left to another launch; 1: starts and lens are different buffers,
// any thread may write lens; 2: append, a warp's chunk is one whole unit.
// Rows that are not there load from the first row instead (no branch between loads).
// Two rows of K and of V per step (fp8: one).  At the 64 registers that four blocks an SM
// leave, the 4-bit kernel spills (140 bytes stored, 52 loaded a thread); four rows a step
// spill more or halve the warps.  255K packed rows to 4-bit pages and back as bf16 (two
// launches, 296 MB): 71 us, 4.2 TB/s; one row a step 77, one group a lane 87.  The write
// alone is 43 us at 67% issue active and 39% of DRAM: arithmetic and its latency, not HBM.
template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads, 4)
    cache_write_rows(const CacheWriteArgs a, int64_t total, int chunk, int mode) {
  constexpr int C = kGroups<FMT>, LPR = D / 8 / C, RPW = 32 / LPR, UNR = FMT == kFmtFp8 ? 1 : 2;
  const int lane = threadIdx.x & 31;
  begin_after_previous();
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  if (mode == 1) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRowThreads;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; u < a.c.units;
         u += step)
      advance_len(a, u, held_to(a.starts[u], cache_cap(a.c), a.c.status));
  }
  const int64_t r0 = warp * chunk;
  // lane i: where row r0 + i comes from and goes to
  int64_t slot = -1, ksrc = 0, vsrc = 0;
  if (lane < chunk && r0 + lane < total) {
    int64_t u, t;
    if (row_owner(a.offsets, a.c.units, a.n_rows, r0 + lane, &u, &t) && t < rows_of(a, u)) {
      const int cap = cache_cap(a.c);
      const int64_t pos =
          held_to(a.starts ? a.starts[u] : __ldcg(a.c.lens + u), cap, a.c.status) + t;
      if (pos < cap)
        slot = cache_slot(a.c, u, static_cast<int>(pos));
      else
        atomicOr(a.c.status, kStatusBadCache);
      if (!in_bounds(t >= 0 && t < a.n_rows)) slot = -1;
      ksrc = a.offsets ? (r0 + lane) * a.k_row : u * a.k_unit + t * a.k_row;
      vsrc = a.offsets ? (r0 + lane) * a.v_row : u * a.v_unit + t * a.v_row;
    }
  }
  __syncwarp();
  if (mode == 2 && lane == 0 && warp < a.c.units)
    advance_len(a, warp, held_to(__ldcg(a.c.lens + warp), cache_cap(a.c), a.c.status));
  if (__all_sync(0xffffffffu, slot < 0)) return;
  const int sub = lane / LPR, lr = lane % LPR;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + lr * 8;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + lr * 8;
  for (int i0 = 0; i0 < chunk; i0 += UNR * RPW) {
    int64_t sl[UNR];
    uint4 kr[UNR][C], vr[UNR][C];
#pragma unroll
    for (int j = 0; j < UNR; ++j) {
      const int i = i0 + j * RPW + sub;          // i >= chunk: its lane holds slot = -1, or i >= 32
      sl[j] = __shfl_sync(0xffffffffu, slot, i & 31);
      const uint16_t* k1 = kp + __shfl_sync(0xffffffffu, ksrc, i & 31);
      const uint16_t* v1 = vp + __shfl_sync(0xffffffffu, vsrc, i & 31);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        kr[j][c] = ld_stream16(k1 + c * LPR * 8);
        vr[j][c] = ld_stream16(v1 + c * LPR * 8);
      }
      if (i >= chunk) sl[j] = -1;
    }
    store_rows<FMT, D, UNR, C>(static_cast<uint8_t*>(a.c.k_pages), a.c.k_params, sl, lr, kr);
    store_rows<FMT, D, UNR, C>(static_cast<uint8_t*>(a.c.v_pages), a.c.v_params, sl, lr, vr);
  }
}

// Appends of many rows: lens moves on once every row has read the old one.
__global__ void cache_advance(const CacheWriteArgs a) {
  begin_after_previous();
  const int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (u < a.c.units) advance_len(a, u, held_to(__ldcg(a.c.lens + u), cache_cap(a.c), a.c.status));
}

template <int FMT, int D>
__global__ void __launch_bounds__(kRowThreads)
    cache_read_rows(const CacheReadArgs a, int64_t total, int chunk) {
  // rows in flight: more where a row is few bytes
  constexpr int LPR = D / 8, RPW = 32 / LPR, UNR = FMT == kFmtInt4 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  begin_after_previous();
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x) >> 5;
  const int64_t r0 = warp * chunk;
  int64_t slot = -1;
  if (lane < chunk && r0 + lane < total) {
    int64_t u, t;
    if (row_owner(a.offsets, a.c.units, a.n_rows, r0 + lane, &u, &t)) {
      const int cap = cache_cap(a.c);
      const int64_t pos = (a.starts ? held_to(a.starts[u], cap, a.c.status) : 0) + t;
      if (pos < held_to(__ldcg(a.c.lens + u), cap, a.c.status))
        slot = cache_slot(a.c, u, static_cast<int>(pos));
    }
  }
  if (__all_sync(0xffffffffu, slot < 0)) return;
  const int sub = lane / LPR, lr = lane % LPR;
  for (int i0 = 0; i0 < chunk; i0 += UNR * RPW) {
    int64_t sl[UNR];
    RowBits<FMT> kb[UNR], vb[UNR];
#pragma unroll
    for (int j = 0; j < UNR; ++j) {
      const int i = i0 + j * RPW + sub;
      sl[j] = __shfl_sync(0xffffffffu, slot, i & 31);
      if (i >= chunk) sl[j] = -1;
      const int64_t at = sl[j] < 0 ? 0 : sl[j];       // rows that are not there: no branch
      kb[j] = load_row<FMT, D>(static_cast<const uint8_t*>(a.c.k_pages), a.c.k_params, at, lr);
      vb[j] = load_row<FMT, D>(static_cast<const uint8_t*>(a.c.v_pages), a.c.v_params, at, lr);
    }
#pragma unroll
    for (int j = 0; j < UNR; ++j) {
      const uint4 kv = row_values<FMT>(kb[j]), vv = row_values<FMT>(vb[j]);
      if (sl[j] >= 0 && in_bounds(r0 + i0 + j * RPW + sub < total)) {
        const int64_t o = (r0 + i0 + j * RPW + sub) * D + lr * 8;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_out) + o) = kv;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_out) + o) = vv;
      }
    }
  }
}

// Rows a warp takes: 32 (one address per lane) when that still gives every SM a
// few warps, else fewer, so that a short call spreads over the machine.
int rows_per_warp(int64_t total) {
  int chunk = 32;
  while (chunk > 2 && total / chunk < 148 * 16) chunk >>= 1;
  return chunk;
}

template <int FMT, int D>
cudaError_t write_fd(const CacheWriteArgs& a, cudaStream_t s, int* launches) {
  const int64_t total = a.offsets ? a.n_rows : a.c.units * a.n_rows;
  int mode = a.starts ? 1 : 0;
  int chunk = rows_per_warp(total);
  int64_t warps = (total + chunk - 1) / chunk;
  if (!a.starts && !a.offsets && a.n_rows > 0 && a.n_rows <= 32) {
    mode = 2;
    chunk = static_cast<int>(a.n_rows);
    warps = a.c.units;
  }
  const int per_block = kRowThreads / 32;
  int64_t blocks = (warps + per_block - 1) / per_block;
  if (blocks < 1) blocks = 1;     // no rows: lens may still change (starts given)
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  *launches += 1;
  const cudaError_t e = launch_after(cache_write_rows<FMT, D>, dim3(static_cast<unsigned>(blocks)),
                                     kRowThreads, 0, s, a, total, chunk, mode);
  if (e != cudaSuccess || mode != 0) return e;
  *launches += 1;
  return launch_after(cache_advance, dim3(static_cast<unsigned>((a.c.units + 127) / 128)), 128, 0, s, a);
}

template <int FMT, int D>
cudaError_t read_fd(const CacheReadArgs& a, cudaStream_t s, int* launches) {
  const int64_t total = a.offsets ? a.n_rows : a.c.units * a.n_rows;
  const int chunk = rows_per_warp(total);
  const int64_t warps = (total + chunk - 1) / chunk;
  const int per_block = kRowThreads / 32;
  const int64_t blocks = (warps + per_block - 1) / per_block;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  *launches += 1;
  return launch_after(cache_read_rows<FMT, D>, dim3(static_cast<unsigned>(blocks)), kRowThreads, 0,
                      s, a, total, chunk);
}

}  // namespace

cudaError_t bounds_flag_cache(unsigned int* out) { return take_bounds_flag(out); }

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t s, int* launches) {
  switch (a.c.format * 1000 + a.c.d) {
    case kFmtBf16 * 1000 + 128: return write_fd<kFmtBf16, 128>(a, s, launches);
    case kFmtBf16 * 1000 + 256: return write_fd<kFmtBf16, 256>(a, s, launches);
    case kFmtFp8 * 1000 + 128: return write_fd<kFmtFp8, 128>(a, s, launches);
    case kFmtFp8 * 1000 + 256: return write_fd<kFmtFp8, 256>(a, s, launches);
    case kFmtInt4 * 1000 + 128: return write_fd<kFmtInt4, 128>(a, s, launches);
    case kFmtInt4 * 1000 + 256: return write_fd<kFmtInt4, 256>(a, s, launches);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t s, int* launches) {
  switch (a.c.format * 1000 + a.c.d) {
    case kFmtBf16 * 1000 + 128: return read_fd<kFmtBf16, 128>(a, s, launches);
    case kFmtBf16 * 1000 + 256: return read_fd<kFmtBf16, 256>(a, s, launches);
    case kFmtFp8 * 1000 + 128: return read_fd<kFmtFp8, 128>(a, s, launches);
    case kFmtFp8 * 1000 + 256: return read_fd<kFmtFp8, 256>(a, s, launches);
    case kFmtInt4 * 1000 + 128: return read_fd<kFmtInt4, 128>(a, s, launches);
    case kFmtInt4 * 1000 + 256: return read_fd<kFmtInt4, 256>(a, s, launches);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvzip
