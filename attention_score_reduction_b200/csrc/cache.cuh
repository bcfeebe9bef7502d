// The paged key/value cache as the device code sees it, shared by the kernels
// that write it, read it back and attend over it.
//
// A unit is one KV head of one sequence.  Row `pos` of unit u lies in page
// page_table[u][pos / page_rows], at row pos % page_rows of that page.  Formats:
//   bf16  the row itself (2 d bytes)
//   fp8   d e4m3 codes; parameter word = float32 scale 2^e; value = code * 2^e
//   int4  d/2 bytes, element 2b in the low nibble of byte b; parameter word =
//         bf16 scale s (low half) and bf16 zero z (high half); value = s c + z
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "kvzip_internal.h"

namespace kvzip {

enum : int { kFmtBf16 = 0, kFmtFp8 = 1, kFmtInt4 = 2 };

template <int FMT, int D>
struct CacheRow {
  static constexpr int BYTES = FMT == kFmtBf16 ? 2 * D : (FMT == kFmtFp8 ? D : D / 2);
};

// Rows a unit can hold (the host keeps it below 2^31 - 2^12).
__device__ __forceinline__ int cache_cap(const CacheArgs& c) { return c.max_pages << c.page_shift; }

// n held to [0, hi]; anything outside sets the status bit.
__device__ __forceinline__ int held_to(int64_t n, int hi, uint32_t* status) {
  if (n >= 0 && n <= hi) return static_cast<int>(n);
  atomicOr(status, kStatusBadCache);
  return n < 0 ? 0 : hi;
}

// Pool row of position pos of unit u (0 <= pos < max_pages * page_rows), or -1
// (and the status bit) where the page table names no page of the pool.
__device__ __forceinline__ int64_t cache_slot(const CacheArgs& c, int64_t u, int pos) {
  if (!in_bounds(u >= 0 && u < c.units && pos >= 0 && pos < cache_cap(c))) return -1;
  const int page = c.page_table[u * c.max_pages + (pos >> c.page_shift)];
  if (page < 0 || page >= c.n_pages) {
    atomicOr(c.status, kStatusBadCache);
    return -1;
  }
  return (static_cast<int64_t>(page) << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// First thing in a kernel launched by launch_after: waits for the kernel before it, whose
// writes (and, as that one waited, those of all before it) are visible then, and only then
// lets the next one be launched.  Not the other way round: three kernels of a stream would
// be on an SM together, and the wait of the third says nothing of the first's.  Beside that
// order, what these kernels write (pages, parameters, lengths, partial results, outputs) is
// read past L1 (ld_stream*, __ldcg, cp.async.cg, bulk and TMA copies), never by read-only
// loads; what only the caller writes (page tables, offsets, starts, counts) goes through L1.
__device__ __forceinline__ void begin_after_previous() {
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
}

// Launch of a kernel that begins with begin_after_previous(): its start overlaps
// the end of the kernel before it on the stream.
template <typename... Params, typename... Args>
inline cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int block, size_t smem,
                                cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// min and max of two bf16 each; NaN if one of them is
__device__ __forceinline__ uint32_t bf16x2_min_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// none of eight bf16 is infinite or NaN
__device__ __forceinline__ bool bf16x8_finite(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool ok = true;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    ok = ok && (w[k] & 0x7f80u) != 0x7f80u && (w[k] & 0x7f800000u) != 0x7f800000u;
  return ok;
}

// none of sixteen e4m3 codes is NaN (all ones but the sign)
__device__ __forceinline__ bool e4m3x16_finite(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) any |= (w[k] & 0x7f7f7f7fu) + 0x01010101u;
  return (any & 0x80808080u) == 0;
}

// two floats as bf16x2 (x in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_bf16x2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
// two floats as f16x2 (x in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_f16x2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
// four e4m3 codes (low byte first) as two f16x2: exact
__device__ __forceinline__ void e4m3x4_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// two floats as e4m3 codes (x in the low byte), round to nearest even
__device__ __forceinline__ uint32_t pack_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

// (x & mask) | magic in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(magic));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Nibbles 0 and 4 (NIB = 0) or 1 and 5 (NIB = 1) of w as exact f16x2 codes:
// 0x6400 | c is 1024 + c, 0x6400 | 16 c is 1024 + 16 c.
template <int NIB>
__device__ __forceinline__ uint32_t nib_f16x2(uint32_t w) {
  if constexpr (NIB == 0)
    return hadd2(and_or(w, 0x000f000fu, 0x64006400u), 0xe400e400u);              // - 1024
  else
    return hfma2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd400d400u);   // / 16 - 64
}

// loads that are not kept in L1 (each byte is used once)
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_stream4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

}  // namespace kvzip
