// Attention of many new tokens over the paged cache on the tensor cores
// (tcgen05 + TMEM + TMA).
//
// A chunk of n tokens with G query heads gives every unit n G query rows; 128 of
// them fill an MMA, so that a cache tile fetched once serves them all and the
// kernel is bound by the tensor pipe (2 * 128 * rows * d multiply-adds a tile)
// once there are a few hundred, by HBM below.
//
// An item is 256 query rows of a unit at d = 128 (128 at d = 256); its tiles are
// shared out as cache_sched.cuh describes.  Per cache tile and block of 128 rows:
//   S = Q K^T       A = Q (shared memory, or TMEM at d = 256), B = K tile, K-major
//   P = 2^(c S - m) two warpgroups a block, half a query row per thread (one, with whole
//                   rows, is a warp per scheduler and bound by latency); P goes back to
//                   TMEM as bf16 over the columns S had
//   O += P V        A = P from TMEM, B = V tile as it lies (MN-major), O in TMEM
// TMEM (512 columns): d = 128: S0 S1 O0 O1 of 128 each; d = 256: O 256, S0 S1 64
// each (cache tiles of 64 rows), Q 128 (with Q in shared memory an MMA of N = 64
// would read more operand bytes than shared memory delivers).
//
// The two S buffers keep the tensor pipe fed while the softmax works on the other.
// With more than 128 rows (d = 128) each buffer belongs to one block of 128 rows;
// with fewer, buffer b takes the tiles of parity b, each with an O of its own at
// d = 128 (joined at the end).  There one thread issues all MMAs of a buffer, which
// complete in order: S of its next tile being ready means the O of its last is, too.
//
// The running maximum is only moved when it grows by more than 2^8 (P then stays
// below 2^8, its rounding relative): O is rescaled in TMEM for a few tiles of an
// item instead of all.  P is rounded to bf16 (at most 2^-8 of a weight, errors of
// both signs); the sum of the weights is taken before the rounding, in fp32.  For
// quantised caches P is fp16 and lifted by 2^7, to below 2^15: the largest weight times
// its row's power of two (below) is at least 2^7, others are rounded by at most 2^-11 of
// themselves down to 2^-21 of it and by 2^-32 of it below.  Without the lift a row that
// takes nearly all the weight and adds little (the first of a context) left the others
// 2^-25 of it: 131072 of them were lost.
//
// bf16 pages come by TMA, one box per page and 64 elements, 128-byte swizzle.
// Quantised pages come as they are, by bulk copies into a ring of 64-row pieces,
// and a warpgroup of its own unpacks them into the same layout as fp16, where a
// pair of codes costs one or two instructions (a bf16 pair of e4m3 codes costs
// five; unpacking was what bound the kernel then).  fp16 lacks bf16's range, so
// powers of two stay outside of it:
//   K   a 64-row piece is scaled by one power of two, the largest row's: smaller
//       rows lose at most 2^-38 of the largest row's logits.  The softmax thread
//       multiplies it back in.  Q is scaled per row (exact down to 2^-32 of its
//       largest element).
//   V   every row has its own power of two 2^e (e4m3: the row's scale, exact; int4:
//       that of the row's largest value, s c + z rounded to 2^-11).  It goes into
//       the weight: with x' = x + e the products are 2^(x' - m) * row, the running
//       maximum is x''s, and the sum of weights is sum 2^(x' - m) 2^-e.  At d = 128
//       64 rows share one e, the largest, where none is more than 2^4 below it: then it
//       is a constant of the tile and the softmax has nothing to load per column.  A row
//       of zeros has e = -88, so that it counts in the sum of weights and hardly in m.
// Rows of the last tile that are not part of the item (other data of the page, or
// what an earlier tile left) are zeroed in V, since 0 * NaN is NaN; in K they give
// logits that the mask replaces.
//
// Measured: 2048 tokens, G = 4, over 8 bf16 heads of 573000 rows together (d = 128):
// 2.2 ms cold, 2.6 to 2.7 ms under the power cap, 1070 .. 890 TFLOP/s.  A round of two blocks
// is a chain of softmax (1900 cycles), issue and execution of 16 MMAs (1000) and the
// ways between them (1100), of which the two blocks overlap all but the MMAs.
// 1024 tokens, G = 2, over 8 heads of 324000 rows together, calls one after another: d = 256
// bf16 0.76 to 0.85 ms (0.59 cold), fp8 1.20, int4 1.06; d = 128 bf16 0.33, fp8 0.54, int4
// 0.42.  Each item unpacks its unit's rows again, beside a softmax that wants the same issue
// slots (without the conversions fp8 at d = 256 takes a tenth less, without the per-column
// powers of two too, without both a quarter less).  A caller who reads such a cache back to
// bf16 pages once and attends those is faster: d = 256 fp8 0.97, int4 0.90; d = 128 0.44, 0.38.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cache.cuh"
#include "cache_attention.cuh"
#include "cache_rings.h"
#include "cache_sched.cuh"
#include "kvzip_internal.h"
#include "sm100_ptx.cuh"
#include "tc_common.cuh"

namespace kvzip {

namespace {

// log2 of how far apart rows of V may be that share a power of two: the smaller lose that
// much of P's range
constexpr int kOneESpan = 4;

template <int FMT, int D>
struct TcaCfg {
  static constexpr bool QUANT = FMT != kFmtBf16;
  using Rings = TcaRings<QUANT, FMT == kFmtInt4, D>;
  static constexpr int BN = Rings::BN;                 // cache rows of a tile
  static constexpr int NB = D == 128 ? 2 : 1;          // blocks of 128 query rows
  static constexpr int BLOCK = 128 * NB;               // query rows of an item
  static constexpr int HC = BN / 2;                    // columns of S per softmax thread
  static constexpr int SW = 2 * NB;                    // softmax warpgroups: block, half of the columns
  static constexpr int PAD = 3;                        // an item's start and end in tiles of work
  static constexpr int KB = D / 64;                    // 128-byte column blocks of a row
  static constexpr int STAGE = BN * D * 2;             // one K or V tile: 32 KB
  static constexpr int Q_BYTES = D == 128 ? NB * 128 * D * 2 : 0;
  static constexpr int STAGES = Rings::STAGES;
  static constexpr int UW = Rings::GROUPS;             // unpacking warpgroups
  // warps: loader, two MMA issuers, ends of items (bf16) or row parameters; softmax; unpacking
  static constexpr int SOFT_WARP0 = 4;
  static constexpr int UNPACK_WARP0 = SOFT_WARP0 + 4 * SW;
  static constexpr int THREADS = 32 * UNPACK_WARP0 + 128 * UW;
  // quantised pages: pieces of 64 rows as they are stored, codes then parameters
  static constexpr int RB = CacheRow<FMT, D>::BYTES;
  static constexpr int RAW_BYTES = 64 * (RB + 4);
  static constexpr int RAW_SLOTS = Rings::RAW_SLOTS;
  // a group of the two has the same stages and slots in every round (a barrier's
  // parity tells two successive phases apart, not three)
  static_assert(UW < 2 || (STAGES % UW == 0 && RAW_SLOTS % UW == 0), "groups share a slot");
  // TMEM columns
  static constexpr int S0 = D == 128 ? 0 : 256, O0 = D == 128 ? 256 : 0;
  static constexpr int Q0 = 384;                        // d = 256 only
  // shared memory
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = Q_BYTES;
  static constexpr int OFF_RAW = OFF_KV + STAGES * STAGE;
  // what the unpacking tells the softmax: per V tile e of its pieces (64 rows) or, where
  // a piece's rows differ too much, e of each row, then 2^-e; per K tile the powers of
  // two of its pieces.  Rings, as long as the parameters can be ahead of the softmax.
  static constexpr int V_RING = Rings::V_RING, K_RING = Rings::K_RING;
  static constexpr int OFF_ROWEXP = OFF_RAW + RAW_SLOTS * RAW_BYTES;
  static constexpr int OFF_KSCALE = OFF_ROWEXP + (QUANT ? V_RING * BN * 8 : 0);
  static constexpr int OFF_VSCALE = OFF_KSCALE + (QUANT ? K_RING * 8 : 0);
  static constexpr int OFF_LIFT = OFF_VSCALE + (QUANT ? V_RING * 8 : 0);   // scale of each Q row
  static constexpr int OFF_XCH = OFF_LIFT + (QUANT ? 256 * 4 : 0);       // a float per row
  // (m, l) per row and warpgroup at an item's end: d = 128 where Q was, else its own
  static constexpr int OFF_ML = D == 128 ? OFF_Q : OFF_XCH + BLOCK * 4;
  static constexpr int OFF_BAR = OFF_XCH + BLOCK * 4 + (D == 128 ? 0 : SW * 128 * 8);
  // kv_full[STAGES], kv_empty[STAGES], s_full[2], p_full[2], o_full[2], pv_done[2], q_full[2],
  // mma_done, turn[2], tail_full[STAGES], raw_full[RAW_SLOTS], raw_ready[RAW_SLOTS],
  // raw_empty[RAW_SLOTS]
  static constexpr int N_BARS = 3 * STAGES + 13 + 3 * RAW_SLOTS;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;
  static constexpr int BYTES = OFF_MISC + 48;          // TMEM address, abort flag, bad rows of four items
  static constexpr int SMEM = BYTES + 1024;
  static_assert(SMEM <= 232448 - 256, "exceeds 227 KB of shared memory with the static part");
  // registers a thread of each warpgroup after the split (0: no split); the sums
  // stay within what the block is launched with
  static constexpr int R_LAUNCH = D == 128 && QUANT ? 80 : 0;          // 0: every thread the same
  static constexpr int R_CTL = R_LAUNCH == 0 ? 0 : 40;
  static constexpr int R_SOFT = R_LAUNCH == 0 ? 0 : 88;
  static constexpr int R_UNPACK = R_LAUNCH == 0 ? 0 : 88;
  static_assert(R_CTL + SW * R_SOFT + UW * R_UNPACK <= R_LAUNCH * THREADS / 128 || R_LAUNCH == 0, "register split");
  static constexpr int CH = 32;                        // columns a thread takes at a time
  // and keeps from the maximum to the exponentials (quantised: kept, others spill)
  static constexpr bool HOLD = HC == CH && !QUANT;
  // quantised: one power of two for 64 rows of V where it will do, instead of one a row.
  // d = 128: a seventh faster; d = 256: as fast with either, the plainer one
  static constexpr bool ONE_E = QUANT && D == 128;
  static constexpr float LIFT = QUANT ? 7.f : 0.f;      // log2 of what P is multiplied by
  // of 8 pairs of exponentials, those on the FMA pipe (beside the unpacking, issue slots
  // are scarcer: none there is up to a tenth faster than two)
  static constexpr int POLY = QUANT ? 0 : 2;
};

// Shared-memory matrix descriptors under the 128-byte swizzle, low words (the high
// word is the same for all): start address and leading offset.  K-major operands
// have one 64-element block in reach of an MMA and no use for the offset; of an
// MN-major operand (64 elements of N per 128-byte row, rows of K in groups of eight,
// 1024 bytes) it leads to the next 64 elements of N, `block` bytes on.
// An MMA takes its operands from uniform registers: with the descriptors built from
// warp-uniform words in a few adds it is issued every 67 cycles (128x128x16, 64 at
// best), with 64-bit arithmetic per descriptor every 97.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t smem_addr) {
  return ((smem_addr & 0x3FFFFu) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint32_t desc_mn(uint32_t smem_addr, uint32_t block) {
  return ((smem_addr & 0x3FFFFu) >> 4) | ((block >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
  return (static_cast<uint64_t>(kDescHi) << 32) | lo;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// The parameter of a stored fp8 row of V whose codes have to be looked at.  A row of zeros is
// stored with the scale 1, hundreds of times its neighbours': 0 instead.  A row that not every
// token sees (`clear`) may hold NaN codes of another writer: they become zeros, and NaN instead.
template <int BYTES>
__device__ __forceinline__ uint32_t looked_at(uint8_t* codes, uint32_t par, bool clear) {
  uint32_t any = 0;
  bool bad = false;
#pragma unroll 1
  for (int i = 0; i < BYTES; i += 16) {
    uint4* at = reinterpret_cast<uint4*>(codes + i);
    const uint4 v = *at;
    any |= v.x | v.y | v.z | v.w;
    if (clear && !e4m3x16_finite(v)) {
      *at = make_uint4(0, 0, 0, 0);
      bad = true;
    }
  }
  if (bad) return 0x7fc00000u;
  return par == 0x3f800000u && (any & 0x7f7f7f7fu) == 0 ? 0u : par;
}

// Byte offset of 16-byte chunk ch (of 64-element column blocks) of tile row r.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
  return static_cast<uint32_t>((ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// The tiles a CTA works through for one item.
struct Piece {
  int r0;        // first cache row
  int end;       // rows before this one take part
  int n;         // tiles
};

template <int FMT, int D>
__global__ void __launch_bounds__(TcaCfg<FMT, D>::THREADS, 1)
    cache_attn_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const CacheAttnArgs a, const AttnShape shape, int64_t items, float c,
                  float2* __restrict__ ml_out, float* __restrict__ o_out) {
  using Cfg = TcaCfg<FMT, D>;
  constexpr int BN = Cfg::BN, KB = Cfg::KB, STAGES = Cfg::STAGES, STAGE = Cfg::STAGE;
  constexpr int THREADS = Cfg::THREADS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ int64_t scratch[THREADS / 32];
  __shared__ LineSpot spot_s;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = kv_full + STAGES;
  uint64_t* s_full = kv_empty + STAGES;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* pv_done = o_full + 2;
  uint64_t* q_full = pv_done + 2;
  uint64_t* mma_done = q_full + 2;
  uint64_t* turn = mma_done + 1;
  uint64_t* tail_full = turn + 2;
  uint64_t* raw_full = tail_full + STAGES;
  uint64_t* raw_ready = raw_full + Cfg::RAW_SLOTS;
  uint64_t* raw_empty = raw_ready + Cfg::RAW_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
  int* bad_row = reinterpret_cast<int*>(smem + Cfg::OFF_MISC + 16);   // see the end of a bf16 item
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int64_t cta = blockIdx.x;

  begin_after_previous();
  Line<THREADS> line(a.c, shape, items, scratch, &spot_s);
  const int64_t all = line.all;
  const int64_t n_cta = line_ctas(all, gridDim.x);
  if (cta >= n_cta) return;
  const int64_t p0 = line_cut(all, cta, n_cta), p1 = line_cut(all, cta + 1, n_cta);
  const LineSpot spot = line.find(p0);
  const int64_t w_first = spot.item, w_first_at = spot.at;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&kv_full[s], Cfg::QUANT ? 128 : 1);
      mbar_init(&kv_empty[s], Cfg::NB);      // a commit of each issuer that reads the stage
      mbar_init(&tail_full[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 256);
      mbar_init(&o_full[i], 1);
      mbar_init(&q_full[i], 256);
      mbar_init(&turn[i], 1);
    }
    mbar_init(&pv_done[0], 1);
    mbar_init(&pv_done[1], 1);
    mbar_init(mma_done, 2);
    for (int i = 0; i < Cfg::RAW_SLOTS; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_ready[i], 1);
      mbar_init(&raw_empty[i], 4);      // one thread of each unpacking warp
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Ctl ctl{abort_flag, a.c.status, a.timeout_ns};

  // Walks the CTA's pieces of items; f returns false to stop.
  auto each_item = [&](auto&& f) {
    int64_t p = p0, at = w_first_at;
    for (int64_t w = w_first; p < p1; ++w) {
      const AttnItem it = attn_item(a.c, shape, w);
      if (it.span == 0) continue;
      const int64_t begin = at;
      int t0, t1;
      const bool any = line_tiles(it, shape, begin, p, p1, t0, t1);
      p = at += it.span;
      if (!any) continue;
      Piece pc;
      pc.r0 = t0 * BN;
      pc.end = min(t1 * BN, it.vis);
      pc.n = t1 - t0;
      if (!f(it, pc, pc.n == it.n_tiles, line_slot(all, cta, n_cta, begin + shape.pad))) return;
    }
  };
  auto two_blocks = [&](const AttnItem& it) { return Cfg::NB == 2 && it.rows > 128; };
  // Rows of the piece that all query rows of the item see; tiles that go further are ragged.
  auto seen_by_all = [&](const AttnItem& it, const Piece& pc) {
    return min(seen_rows(it, it.row0 / shape.G), pc.end);
  };
  // K and V tiles in the order the MMAs use them: f(is_v, tile).
  auto each_stage = [&](const AttnItem& it, const Piece& pc, auto&& f) -> bool {
    return for_each_stage(pc.n, two_blocks(it) ? 1 : Cfg::Rings::AHEAD, f);
  };

  if (warp < Cfg::SOFT_WARP0) {
   regs_to<Cfg::R_LAUNCH, Cfg::R_CTL>();
   if (warp == 0) {
    // ============================================================ TMA producer
    if constexpr (!Cfg::QUANT) {
      const int box_shift = min(a.c.page_shift, BN == 128 ? 7 : 6);
      const int box = 1 << box_shift;
      const int rows_total = static_cast<int>(a.c.n_pages << a.c.page_shift);
      uint32_t g = 0;
      if (a.test_stall == 0)
        each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
          const int all_see = seen_by_all(it, pc);
          return each_stage(it, pc, [&](bool is_v, int j) {
            const int s = g % STAGES;
            const int r = pc.r0 + j * BN + lane * box;       // lane i brings page box i
            const bool mine = lane < BN / box && r < pc.end;
            int row = rows_total;                            // a bad page reads as zeros
            if (mine) {
              const int64_t slot = cache_slot(a.c, it.u, r);
              if (slot >= 0) row = static_cast<int>(slot);
            }
            const int n_box = __popc(__ballot_sync(0xffffffffu, mine));
            if (!wait_warp(&kv_empty[s], ((g / STAGES) & 1) ^ 1, ctl)) return false;
            // the last V tiles go by way of warp 3
            uint64_t* full = is_v && pc.r0 + (j + 1) * BN > all_see ? &tail_full[s] : &kv_full[s];
            if (lane == 0) mbar_arrive_expect_tx(full, n_box * box * D * 2);
            __syncwarp();
            if (mine) {
              uint8_t* dst = smem + Cfg::OFF_KV + s * STAGE + lane * box * 128;
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
                tma_load_3d(dst + kb * (BN * 128), is_v ? &vmap : &kmap, full, kb * 64, row, 0);
            }
            ++g;
            return true;
          });
        });
      // every copy lands before shared memory is released
      if (lane == 0)
        for (uint32_t s = 0; s < STAGES && s < g; ++s) {
          const uint32_t last = s + ((g - 1 - s) / STAGES) * STAGES;
          wait_drain(&kv_full[s], (last / STAGES) & 1, a.c.status);
        }
      __syncwarp();
    } else {
      const int box = min(1 << a.c.page_shift, 64);
      const uint8_t* kp = static_cast<const uint8_t*>(a.c.k_pages);
      const uint8_t* vp = static_cast<const uint8_t*>(a.c.v_pages);
      uint32_t g = 0;
      if (a.test_stall == 0)
        each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
          return each_stage(it, pc, [&](bool is_v, int j) {
            for (int h = 0; h < BN; h += 64) {
              const int s = g % Cfg::RAW_SLOTS;
              const int r = pc.r0 + j * BN + h + lane * box;      // lane i brings page box i
              const bool mine = lane < 64 / box && r < pc.end;
              const int64_t slot = mine ? cache_slot(a.c, it.u, r) : -1;
              const int n_box = __popc(__ballot_sync(0xffffffffu, slot >= 0));
              if (!wait_warp(&raw_empty[s], ((g / Cfg::RAW_SLOTS) & 1) ^ 1, ctl)) return false;
              uint8_t* codes = smem + Cfg::OFF_RAW + s * Cfg::RAW_BYTES + lane * box * Cfg::RB;
              uint8_t* par = smem + Cfg::OFF_RAW + s * Cfg::RAW_BYTES + 64 * Cfg::RB + lane * box * 4;
              if (mine && slot < 0) {                              // a bad page: rows of zeros
                for (int i = 0; i < box * Cfg::RB; i += 16)
                  *reinterpret_cast<uint4*>(codes + i) = make_uint4(0, 0, 0, 0);
                for (int i = 0; i < box * 4; i += 16)
                  *reinterpret_cast<uint4*>(par + i) = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
              }
              __syncwarp();
              if (lane == 0) mbar_arrive_expect_tx(&raw_full[s], n_box * box * (Cfg::RB + 4));
              __syncwarp();
              if (slot >= 0) {
                bulk_load(codes, (is_v ? vp : kp) + slot * Cfg::RB, box * Cfg::RB, &raw_full[s]);
                bulk_load(par, (is_v ? a.c.v_params : a.c.k_params) + slot, box * 4, &raw_full[s]);
              }
              ++g;
            }
            return true;
          });
        });
      if (lane == 0)
        for (uint32_t s = 0; s < Cfg::RAW_SLOTS && s < g; ++s) {
          const uint32_t last = s + ((g - 1 - s) / Cfg::RAW_SLOTS) * Cfg::RAW_SLOTS;
          wait_drain(&raw_full[s], (last / Cfg::RAW_SLOTS) & 1, a.c.status);
        }
      __syncwarp();
    }
   } else if (warp <= 2) {
    // ============================================================ MMA issuers
    // tcgen05.mma issue stalls until the previous one is nearly done, so that one
    // thread's waits, fences and commits idle the tensor pipe (128x128x16: 113
    // instead of 64 cycles); two issuers cover for each other.  d = 128: one per S
    // buffer (and its O); d = 256, where both buffers add to one O: one for the
    // logits, one for the output.
    // both operands bf16 or, for quantised caches, fp16 (format 0)
    constexpr uint32_t fmt_bits = Cfg::QUANT ? (1u << 7) | (1u << 10) : 0u;
    constexpr uint32_t id_qk = idesc_bf16_f32(128, BN) ^ fmt_bits;
    constexpr uint32_t id_pv = (idesc_bf16_f32(128, D) ^ fmt_bits) | (1u << 16);     // B is MN-major
    const uint32_t kv_base = smem_u32(smem + Cfg::OFF_KV);
    const uint32_t q_base = smem_u32(smem + Cfg::OFF_Q);
    auto qk = [&](int buf, int qt, uint32_t stage) {
      const uint32_t kd = uniform(desc_k(kv_base + stage * STAGE));
      const uint32_t qd = uniform(desc_k(q_base + qt * (128 * D * 2)));
      const uint32_t sd = uniform(tmem + Cfg::S0 + buf * BN), qt_mem = uniform(tmem + Cfg::Q0);
      if (elect_one()) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {      // 16 elements: 32 bytes of each row
            const uint64_t b = desc(kd + kb * (BN * 128 >> 4) + 2 * kk);
            if constexpr (D == 128)
              umma_bf16_ss(sd, desc(qd + kb * (128 * 128 >> 4) + 2 * kk), b, id_qk, (kb | kk) != 0);
            else
              umma_bf16_ts(sd, qt_mem + (kb * 4 + kk) * 8, b, id_qk, (kb | kk) != 0);
          }
        umma_commit(&s_full[buf]);
      }
      __syncwarp();
    };
    auto pv = [&](int buf, int ob, uint32_t stage, bool first) {
      const uint32_t vd = uniform(desc_mn(kv_base + stage * STAGE, BN * 128));
      const uint32_t od = uniform(tmem + Cfg::O0 + ob * D), pd = uniform(tmem + Cfg::S0 + buf * BN);
      const uint32_t keep = uniform(first ? 0u : 1u);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)     // 16 rows: 8 columns of P, 2048 bytes of each V block
          umma_bf16_ts(od, pd + (16 * k / Cfg::HC) * Cfg::HC + (16 * k % Cfg::HC) / 2,
                       desc(vd + k * (2048 >> 4)), id_pv, k == 0 ? keep : 1u);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    // Places in the order of each_stage.
    auto k_at = [](int j, int ahead) { return j < ahead ? j : 2 * j - ahead + 1; };
    auto v_at = [](int j, int ahead, int n) { return min(j + ahead, n) + j; };
    const int t = warp - 1;
    uint32_t base = 0, n_item = 0;                 // stages and items so far
    uint32_t n_even = 0, n_odd = 0;                // earlier items' tiles of each parity
    uint32_t n_p = 0, n_p1 = 0;                    // P tiles of this issuer's buffer (d = 256: of each)
    uint32_t n_turn = 0;
    auto stage_ready = [&](uint32_t g) {
      if (!wait_warp(&kv_full[g % STAGES], (g / STAGES) & 1, ctl)) return false;
      tc_fence_after();
      return true;
    };
    auto release = [&](uint32_t g) { commit(&kv_empty[g % STAGES]); };
    each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
      const bool two = two_blocks(it);
      const int ahead = two ? 1 : 2, n = pc.n;
      const uint32_t qph = n_item++ & 1;
      if (!wait_warp(&q_full[0], qph, ctl)) return false;
      if (Cfg::NB == 2 && !wait_warp(&q_full[1], qph, ctl)) return false;
      tc_fence_after();
      if constexpr (Cfg::NB == 2) {
        // issuer t: its block of rows over every tile, or the tiles of parity t.  The
        // issuers take turns of one output and the next logits: while the pipe works
        // on one buffer's, the softmax works on the other's.  Left alone they drift
        // into step, and the pipe waits for both.
        const int j0 = two ? 0 : t, dj = two ? 1 : 2, qt = two ? t : 0;
        const int rounds = two ? n : (n + 1) / 2;
        for (int r = -1; r < rounds; ++r) {
          const int j = j0 + r * dj, jn = j + dj;       // output of j, logits of jn
          const uint32_t gv = base + v_at(j, ahead, n), gk = base + k_at(jn, ahead);
          const bool out = r >= 0 && j < n, log = jn < n;
          if (out) {
            if (!stage_ready(gv)) return false;
            if (!wait_warp(&p_full[t], n_p++ & 1, ctl)) return false;
          }
          if (log && !stage_ready(gk)) return false;
          // issuer 1's turn follows issuer 0's; the very first of issuer 0 follows none
          if ((t == 1 || n_turn > 0) && !wait_warp(&turn[t], (n_turn - (t == 0)) & 1, ctl)) return false;
          ++n_turn;
          tc_fence_after();
          if (out) pv(t, t, gv % STAGES, r == 0);
          if (log) qk(t, qt, gk % STAGES);
          if (elect_one()) umma_commit(&turn[t ^ 1]);
          __syncwarp();
          if (out) release(gv);
          if (log) release(gk);
          if (!two) {                     // kv_empty counts both issuers
            if (out) release(gv);
            if (log) release(gk);
          }
        }
        commit(&o_full[t]);
      } else if (t == 0) {
        // logits: S of tile j takes the buffer that P of tile j - 2 leaves
        for (int j = 0; j < n; ++j) {
          const uint32_t g = base + k_at(j, ahead);
          // this first: with the output of tile j - 2 done, the stage's previous use is
          // complete, and its barrier's parity names this use
          if (j >= 2 && !wait_warp(&pv_done[j & 1], ((j & 1 ? n_odd : n_even) + (j >> 1) - 1) & 1, ctl))
            return false;
          if (!stage_ready(g)) return false;
          qk(j & 1, 0, g % STAGES);
          release(g);
        }
      } else {
        for (int j = 0; j < n; ++j) {
          const uint32_t g = base + v_at(j, ahead, n);
          if (!stage_ready(g)) return false;
          if (!wait_warp(&p_full[j & 1], (j & 1 ? n_p1++ : n_p++) & 1, ctl)) return false;
          tc_fence_after();
          pv(j & 1, 0, g % STAGES, j == 0);
          release(g);
          commit(&pv_done[j & 1]);
        }
        commit(&o_full[0]);
      }
      base += 2 * n;
      n_even += (n + 1) / 2;
      n_odd += n / 2;
      return true;
    });
    // all MMAs are done before TMEM is freed
    commit(mma_done);
    if (lane == 0) wait_drain(mma_done, 0, a.c.status);
    __syncwarp();
   } else {
    // ============================================================ end of a bf16 item, or row parameters
    if constexpr (!Cfg::QUANT) {
      // V rows that some query row of the item does not see must not reach it as 0 * NaN.
      // Those past the piece's end become zeros before the MMAs see them.  Of the others
      // (the chunk's own tokens) what is not finite becomes zero, and the first such row
      // is noted, by the parity of its tile: query rows that see it end as NaN.
      uint32_t g = 0, phase = 0, n_item = 0;
      each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
        const int all_see = seen_by_all(it, pc);
        int bad = INT_MAX;
        int* noted = &bad_row[2 * (n_item++ & 3)];     // no more than three items are in flight
        return each_stage(it, pc, [&](bool is_v, int j) {
          const int s = g++ % STAGES;
          const int r = pc.r0 + j * BN, live = pc.end - r;
          if (!is_v || r + BN <= all_see) return true;
          if (!wait_warp(&tail_full[s], (phase >> s) & 1, ctl)) return false;
          phase ^= 1u << s;
          for (int i = max(0, all_see - r) * (D / 8) + lane; i < BN * (D / 8); i += 32) {
            const int row = i / (D / 8);
            uint4* at = reinterpret_cast<uint4*>(smem + Cfg::OFF_KV + s * STAGE +
                                                 tile_off<BN>(row, i % (D / 8)));
            if (row < live) {
              if (bf16x8_finite(*at)) continue;
              bad = min(bad, r + row);
            }
            *at = make_uint4(0, 0, 0, 0);
          }
          bad = __reduce_min_sync(0xffffffffu, bad);
          if (lane == 0) noted[j & 1] = bad;
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_full[s]);
          return true;
        });
      });
    } else {
      // The 64 rows' parameter words of a piece, two per lane, become what the unpacking
      // multiplies by (in place), and the powers of two that the softmax needs.
      uint32_t g = 0, k_tile = 0, v_tile = 0;
      if (a.test_stall == 0)
        each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
          const int all_see = seen_by_all(it, pc);
          return each_stage(it, pc, [&](bool is_v, int j) {
            for (int h = 0; h < BN; h += 64, ++g) {
              const int rs = g % Cfg::RAW_SLOTS;
              if (!wait_warp(&raw_full[rs], (g / Cfg::RAW_SLOTS) & 1, ctl)) return false;
              uint32_t* params =
                  reinterpret_cast<uint32_t*>(smem + Cfg::OFF_RAW + rs * Cfg::RAW_BYTES + 64 * Cfg::RB);
              const int live = pc.end - (pc.r0 + j * BN + h);       // rows of the piece that count
              uint32_t par[2];
              // a row of zeros (its part of the sum of weights, 2^88 times at most 2^15 of them
              // each, stays finite for 2^22 rows)
              constexpr int kMinE = -50, kMaxE = 50, kZeroE = -88;
              int e[2], ev[2];           // the row's power of two; the one used for V
              bool nan[2], zero[2];
              int hi = -1000, lo = 1000;
              // fp8: the codes of V rows that not every token sees are looked at, and once the
              // parameters are read those of rows with the scale 1
              const int rows = min(live, 64), open = all_see - (pc.r0 + j * BN + h);
              bool look = FMT == kFmtFp8 && is_v && open < rows;
              while (true) {
                if (FMT == kFmtFp8 && look) {
#pragma unroll 1
                  for (int row = lane; row < rows; row += 32)
                    params[row] = looked_at<Cfg::RB>(smem + Cfg::OFF_RAW + rs * Cfg::RAW_BYTES + row * Cfg::RB,
                                                     params[row], row >= open);
                  __syncwarp();
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  par[k] = lane + 32 * k < live ? params[lane + 32 * k] : 0u;
                  if constexpr (FMT == kFmtFp8) {
                    nan[k] = par[k] >= 0x7f800000u;
                    zero[k] = par[k] == 0;          // no row, or a page that is not there
                    e[k] = nan[k] || zero[k] ? -126 : static_cast<int>(par[k] >> 23) - 127;
                  } else {
                    const float sc = bf16_lo(par[k]), z = bf16_hi(par[k]);
                    const float top = fmax_nan(fabsf(z), fabsf(fmaf(15.f, sc, z)));
                    nan[k] = !(top < INFINITY);
                    zero[k] = top == 0.f;
                    e[k] = nan[k] ? -110 : max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -110);
                  }
                  // V: within 2^+-50, so that 2^(x' - m) of no row underflows beside another's
                  // that matters no more; fp16 holds some of what is beyond.  A row that it
                  // does not hold is NaN for who sees it, as its infinities would reach others
                  if (is_v && e[k] > kMaxE + (FMT == kFmtFp8 ? 7 : 14)) nan[k] = true;
                  ev[k] = nan[k] ? 0 : (zero[k] ? kZeroE : min(max(e[k], kMinE), kMaxE));
                }
                if (Cfg::ONE_E && is_v) {
                  hi = -1000;
                  lo = 1000;
#pragma unroll
                  for (int k = 0; k < 2; ++k)
                    if (lane + 32 * k < live) {
                      hi = max(hi, ev[k]);
                      lo = min(lo, nan[k] ? -1000 : ev[k]);
                    }
                  hi = __reduce_max_sync(0xffffffffu, hi);
                  lo = __reduce_min_sync(0xffffffffu, lo);
                }
                if (FMT != kFmtFp8 || !is_v || look) break;
                look = Cfg::ONE_E ? hi >= 0 : __any_sync(0xffffffffu, par[0] == 0x3f800000u || par[1] == 0x3f800000u);
                if (!look) break;
              }
              // V: one power of two for the 64 rows, too, if none is far below the largest
              // (their products with it are exact, or as good as their own)
              bool own_e = is_v && !Cfg::ONE_E;
              if (Cfg::ONE_E && is_v) {
                own_e = hi - lo > kOneESpan;
                if (hi == -1000) hi = 0;
                if (!own_e) ev[0] = ev[1] = hi;
                if (lane == 0)
                  reinterpret_cast<float*>(smem + Cfg::OFF_VSCALE)[2 * (v_tile % Cfg::V_RING) + h / 64] =
                      own_e ? INFINITY : static_cast<float>(hi);
              }
              // a row of NaN: K's logits are; V's weights are (its e), for who sees it, and the
              // row is zeros, as 0 * NaN would reach the others
              const uint32_t not_a_row = is_v ? 0u : 0x7e007e00u;
              // K: one power of two for the 64 rows, the largest
              const int top_e = __reduce_max_sync(0xffffffffu, max(e[0], e[1]));
              const int ring = v_tile % Cfg::V_RING;
              float* row_e = reinterpret_cast<float*>(smem + Cfg::OFF_ROWEXP) + ring * (2 * BN) + h;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t mul;            // fp8: the row's factor twice; int4: (s, z) scaled
                if constexpr (FMT == kFmtFp8) {
                  // K: 2^(e - top + 6), at most 2^6: 448 * 2^6 is within fp16; V: 1
                  const int x = is_v ? (zero[k] ? 0 : e[k] - ev[k]) : e[k] - top_e + 6;
                  const uint32_t f = x >= -14 ? static_cast<uint32_t>(x + 15) << 10
                                              : (x >= -24 ? 1u << (x + 24) : 0u);
                  mul = nan[k] ? not_a_row : f | (f << 16);
                } else {
                  // values below 2^(e + 1): to below 2^14 (K), below 2 (V)
                  const int x = is_v ? -ev[k] : 13 - top_e;
                  const float f = __uint_as_float(static_cast<uint32_t>(127 + x) << 23);
                  mul = nan[k] ? not_a_row : pack_f16x2(bf16_lo(par[k]) * f, bf16_hi(par[k]) * f);
                }
                params[lane + 32 * k] = mul;
                if (own_e) {
                  row_e[lane + 32 * k] = nan[k] ? NAN : static_cast<float>(ev[k]);
                  row_e[BN + lane + 32 * k] = __uint_as_float(static_cast<uint32_t>(127 - ev[k]) << 23);
                }
              }
              if (!is_v && lane == 0) {
                const int x = top_e - (FMT == kFmtFp8 ? 6 : 13);
                reinterpret_cast<float*>(smem + Cfg::OFF_KSCALE)[2 * (k_tile % Cfg::K_RING) + h / 64] =
                    x >= -126 ? __uint_as_float(static_cast<uint32_t>(127 + x) << 23) : 0.f;
              }
              fence_proxy_async();           // the next copy into the slot comes by the async proxy
              __syncwarp();
              if (lane == 0) mbar_arrive(&raw_ready[rs]);
            }
            if (is_v) ++v_tile; else ++k_tile;
            return true;
          });
        });
    }
   }
  } else if (warp < Cfg::UNPACK_WARP0) {
    // ============================================================ softmax warpgroups
    regs_to<Cfg::R_LAUNCH, Cfg::R_SOFT>();
    constexpr int HC = Cfg::HC, CH = Cfg::CH;
    constexpr int kAll = 128 * Cfg::SW;
    const int sw = (warp - Cfg::SOFT_WARP0) >> 2;
    const int t = sw >> 1, half = sw & 1;
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;                 // TMEM lane = row of the 128-row block
    const int pair_bar = 2 + t * 4 + quarter;              // the two warps with the same rows
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* xch = reinterpret_cast<float*>(smem + Cfg::OFF_XCH) + t * 128 + lrow;
    float* lifts = reinterpret_cast<float*>(smem + Cfg::OFF_LIFT);
    // growth of the maximum that is let pass; m is in units of S (bf16) or of log2
    const float lazy = Cfg::QUANT ? 8.f : 8.f / c;
    uint32_t n_s[2] = {0, 0}, n_item = 0, n_tile = 0;     // n_tile: tiles of earlier items
    uint32_t n_even = 0, n_odd = 0;                        // by parity
    each_item([&](const AttnItem& it, const Piece& pc, bool whole, int64_t slot) {
      const bool two = two_blocks(it);
      const bool join = Cfg::NB == 2 && !two;              // both blocks' groups share the rows
      const int row = (two ? t * 128 : 0) + lrow;          // query row within the item
      const bool live = row < it.rows;
      int lim = 0;
      if (live) lim = min(seen_rows(it, (it.row0 + row) / shape.G), pc.end);
      // rows every query of this block sees: tiles before need no mask
      const int lim_all = min(seen_rows(it, (it.row0 + (two ? t * 128 : 0)) / shape.G), pc.end);
      // ---- Q into the MMA's operand.  Quantised: as fp16, a row's largest element
      // lifted to [2^14, 2^15); int4 tiles hold each 8 elements as 0 4 1 5 2 6 3 7,
      // so Q does, too.
      const uint16_t* qu = static_cast<const uint16_t*>(a.q) + it.u * a.q_unit;
      auto magnitude = [](const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          top = max(top, max((w[k] << 16) & 0x7fff0000u, w[k] & 0x7fff0000u));
        return top;
      };
      auto lift_of = [](uint32_t top) {
        const int e = static_cast<int>(top >> 23) - 127;
        return __uint_as_float(static_cast<uint32_t>(min(max(127 + 14 - e, 1), 254)) << 23);
      };
      auto operand = [](uint4 v, float f) {
        if constexpr (Cfg::QUANT) {
          v.x = pack_f16x2(bf16_lo(v.x) * f, bf16_hi(v.x) * f);
          v.y = pack_f16x2(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
          v.z = pack_f16x2(bf16_lo(v.z) * f, bf16_hi(v.z) * f);
          v.w = pack_f16x2(bf16_lo(v.w) * f, bf16_hi(v.w) * f);
        }
        if constexpr (FMT == kFmtInt4)
          v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                         __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
        return v;
      };
      float cq = c;
      if constexpr (D == 128) {
        // a warp brings rows two at a time, 16 lanes a row; the groups share the
        // item's blocks evenly
        const int per_warp = (two ? 256 : 128) / (4 * Cfg::SW);      // 8 or more
        const int lane_half = lane >> 4, ch = lane & 15;
        int b_row = sw * (4 * per_warp) + quarter * per_warp + lane_half;
        int b_tok = (it.row0 + b_row) / shape.G;
        int b_head = it.row0 + b_row - b_tok * shape.G;
        for (int i0 = 0; i0 < per_warp; i0 += 8) {
          uint4 v[4];
          int rows[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            rows[i] = b_row;
            v[i] = b_row < it.rows
                       ? __ldcg(reinterpret_cast<const uint4*>(qu + b_head * a.q_head + b_tok * a.q_row + ch * 8))
                       : make_uint4(0, 0, 0, 0);
            b_row += 2;
            b_head += 2;
            while (b_head >= shape.G) {
              b_head -= shape.G;
              ++b_tok;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f = 1.f;
            if constexpr (Cfg::QUANT) {
              uint32_t top = magnitude(v[i]);
#pragma unroll
              for (int k = 8; k >= 1; k >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
              f = lift_of(top);
              if (ch == 0) lifts[rows[i]] = f;
            }
            *reinterpret_cast<uint4*>(smem + Cfg::OFF_Q + (rows[i] >> 7) * (128 * D * 2) +
                                      tile_off<128>(rows[i] & 127, ch)) = operand(v[i], f);
          }
        }
        fence_proxy_async();
        if constexpr (Cfg::QUANT) {
          named_barrier_sync(1, kAll);
          cq = c / lifts[row];
        }
      } else {
        // each half of the columns of the row's TMEM lane
        const int r = it.row0 + row, tok = r / shape.G, head = r - tok * shape.G;
        const uint4* src = reinterpret_cast<const uint4*>(qu + head * a.q_head + tok * a.q_row) +
                           half * (D / 16);
        float f = 1.f;
        if constexpr (Cfg::QUANT) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            top = max(top, magnitude(live ? __ldcg(src + i) : make_uint4(0, 0, 0, 0)));
          lifts[half * 128 + lrow] = __uint_as_float(top);
          named_barrier_sync(1, kAll);
          top = max(top, __float_as_uint(lifts[(half ^ 1) * 128 + lrow]));
          f = lift_of(top);
          cq = c / f;
        }
#pragma unroll
        for (int h = 0; h < D / 128; ++h) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = operand(live ? __ldcg(src + 8 * h + i) : make_uint4(0, 0, 0, 0), f);
            v[4 * i] = x.x;
            v[4 * i + 1] = x.y;
            v[4 * i + 2] = x.z;
            v[4 * i + 3] = x.w;
          }
          tmem_st32_async(lane_base + Cfg::Q0 + half * (D / 4) + 32 * h, v);
        }
        tmem_wait_st();
        tc_fence_before();
      }
      mbar_arrive(&q_full[t]);

      float m = -INFINITY, l = 0.f;
      const uint32_t o_addr = lane_base + Cfg::O0 + t * D;
      const int j0 = join ? t : 0, dj = join ? 2 : 1;
      bool ok = true;
      for (int j = j0; j < pc.n; j += dj) {
        const int b = Cfg::NB == 2 ? t : (j & 1);
        const uint32_t s_addr = lane_base + Cfg::S0 + b * BN + half * HC;
        ok = ok && wait_warp(&s_full[b], n_s[b]++ & 1, ctl);
        const int col0 = pc.r0 + j * BN + half * HC;
        const bool masked = pc.r0 + j * BN + BN > lim_all;
        const float* row_e = nullptr;        // e of these V rows; 2^-e are BN floats on
        float ce = c, e_all = 0.f;           // x (x') = ce S + e; e_all: e of all of them, or infinity
        if constexpr (Cfg::QUANT) {
          const uint32_t gv = 2 * n_tile + min(j + (two ? 1 : 2), pc.n) + j;
          const int sv = gv % STAGES;
          ok = ok && wait_warp(&kv_full[sv], (gv / STAGES) & 1, ctl);
          row_e = reinterpret_cast<const float*>(smem + Cfg::OFF_ROWEXP) +
                  ((n_tile + j) % Cfg::V_RING) * (2 * BN) + half * HC;
          // this half's columns are of one piece; never 0, which would turn -infinity to NaN
          ce = fmaxf(cq * reinterpret_cast<const float*>(smem + Cfg::OFF_KSCALE)[
                         2 * ((n_tile + j) % Cfg::K_RING) + (half * HC) / 64], 1.17549435e-38f);
          if constexpr (Cfg::ONE_E)
            e_all = reinterpret_cast<const float*>(smem + Cfg::OFF_VSCALE)[
                2 * ((n_tile + j) % Cfg::V_RING) + (half * HC) / 64];
        }
        const bool own_e = Cfg::QUANT && (!Cfg::ONE_E || e_all == INFINITY);
        tc_fence_after();
        // CH columns: S or, if each row has its own e, x' = x + e; -infinity where this row
        // does not see
        auto load = [&](int h, float (&v)[CH]) {
          tmem_ld_tile(s_addr + h, v);
          if (Cfg::QUANT && own_e) {
            const float2 ce2 = make_float2(ce, ce);
#pragma unroll
            for (int i = 0; i < CH; i += 4) {
              const float4 e = *reinterpret_cast<const float4*>(row_e + h + i);
              const float2 x0 = ffma2(make_float2(v[i], v[i + 1]), ce2, make_float2(e.x, e.y));
              const float2 x1 = ffma2(make_float2(v[i + 2], v[i + 3]), ce2, make_float2(e.z, e.w));
              v[i] = x0.x;
              v[i + 1] = x0.y;
              v[i + 2] = x1.x;
              v[i + 3] = x1.y;
            }
          }
          if (masked) {
            const int n = lim - (col0 + h);
#pragma unroll
            for (int i = 0; i < CH; ++i) v[i] = i < n ? v[i] : -INFINITY;
          }
        };
        // columns that are not held are read again for the exponentials
        float s_row[Cfg::HOLD ? HC / CH : 1][CH];
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (ok) {
#pragma unroll
          for (int h = 0; h < HC / CH; ++h) {
            float(&v)[CH] = s_row[Cfg::HOLD ? h : 0];
            load(h * CH, v);
#pragma unroll
            for (int i = 0; i < CH; i += 8)
#pragma unroll
              for (int q = 0; q < 4; ++q) mx[q] = fmax3_nan(mx[q], v[i + 2 * q], v[i + 2 * q + 1]);
          }
        }
        float cand = fmax_nan(fmax_nan(mx[0], mx[1]), fmax_nan(mx[2], mx[3]));
        if (Cfg::QUANT && !own_e) cand = fmaf(cand, ce, e_all);
        cand = fmax_nan(m, cand);
        bool need = !(cand - m <= lazy) && cand != -INFINITY;
        // both warps of these rows have to move together (or to give up together)
        need = named_barrier_or(pair_bar, 64, need || !ok);
        if (need) {
          if (half == 0) *xch = cand;
          if (named_barrier_or(pair_bar, 64, !ok)) { ok = false; break; }
          if (half == 1) {
            cand = fmax_nan(cand, *xch);
            *xch = cand;
          }
          named_barrier_sync(pair_bar, 64);
          if (half == 0) cand = *xch;
          const float f = cand == -INFINITY ? 1.f : ex2_approx(Cfg::QUANT ? m - cand : (m - cand) * c);
          if (j != j0) {
            // d = 256: S was ready before the last O; wait for that product
            if constexpr (Cfg::NB == 1)
              ok = wait_warp(&pv_done[(j - 1) & 1],
                             ((j & 1 ? n_even : n_odd) + ((j - 1) >> 1)) & 1, ctl);
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < D / 2; h += 32) {
              float o[32];
              tmem_ld32(o_addr + half * (D / 2) + h, o);
              uint32_t u[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
              tmem_st32_async(o_addr + half * (D / 2) + h, u);
            }
            tmem_wait_st();
          }
          l *= f;
          m = cand;
        }
        float nb = m == -INFINITY ? 0.f : (Cfg::QUANT ? Cfg::LIFT - m : -m * c);
        if (Cfg::QUANT && !own_e) nb += e_all;
        const float2 ce2 = make_float2(ce, ce), nb2 = make_float2(nb, nb);
        float2 acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = make_float2(0.f, 0.f);
        // POLY of eight pairs go to the FMA pipe, where nothing is masked (the polynomial
        // has no 2^-infinity)
        auto weights = [&](auto poly, auto own) {
          constexpr bool OWN = decltype(own)::value;
          constexpr int POLY = decltype(poly)::value;
#pragma unroll
          for (int hh = 0; hh < HC / CH; ++hh) {
            const int h = hh * CH;
            float(&v)[CH] = s_row[Cfg::HOLD ? hh : 0];
            if (!Cfg::HOLD) load(h, v);
            uint32_t pk[CH / 2];
#pragma unroll
            for (int i = 0; i < CH; i += 16)
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const int e0 = i + 2 * q;
                const float2 x = OWN ? fadd2(make_float2(v[e0], v[e0 + 1]), nb2)
                                                      : ffma2(make_float2(v[e0], v[e0 + 1]), ce2, nb2);
                float2 e;
                if (q < POLY) {
                  e = exp2_poly2(x);
                } else {
                  e.x = ex2_approx(x.x);
                  e.y = ex2_approx(x.y);
                }
                if constexpr (OWN)
                  acc[q & 3] = ffma2(e, *reinterpret_cast<const float2*>(row_e + BN + h + e0), acc[q & 3]);
                else
                  acc[q & 3] = fadd2(acc[q & 3], e);
                pk[e0 / 2] = Cfg::QUANT ? pack_f16x2(e.x, e.y) : pack_bf16x2(e.x, e.y);
              }
            // over columns of this half's S that are read
            tmem_st_tile(s_addr + h / 2, pk);
          }
        };
        using none = std::integral_constant<int, 0>;
        using poly = std::integral_constant<int, Cfg::POLY>;
        constexpr auto own = std::integral_constant<bool, Cfg::QUANT>{};      // e of each row, if any
        if (Cfg::ONE_E && !own_e) {
          if (masked) weights(none{}, std::false_type{});
          else weights(poly{}, std::false_type{});
        } else if (masked || Cfg::ONE_E) {
          weights(none{}, own);
        } else {
          weights(poly{}, own);
        }
        const float2 sum = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
        if (Cfg::QUANT && !own_e)      // of 2^x, not 2^x'
          l = fmaf(sum.x + sum.y, __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(e_all)) << 23), l);
        else
          l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[b]);
      }
      n_tile += pc.n;
      n_even += (pc.n + 1) / 2;
      n_odd += pc.n / 2;

      // ---- the item's result
      ok = ok && wait_warp(&o_full[t], n_item & 1, ctl);
      tc_fence_after();
      if constexpr (!Cfg::QUANT) {
        // notes of tiles whose output this group has waited for: all, or of one parity
        const int first = max(seen_by_all(it, pc) - pc.r0, 0) / BN;       // ragged tile
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if ((!join || p == t) && first + ((first ^ p) & 1) < pc.n &&
              bad_row[2 * (n_item & 3) + p] < lim)
            l = NAN;
      }
      ++n_item;
      // the polynomial has 2^-125 for 2^-infinity
      if (Cfg::POLY > 0 && m == -INFINITY && l > 0.f) l = 0.f;
      const float m2 = Cfg::QUANT || m == -INFINITY ? m : m * c;
      // Q's own block is no longer read; of rows that all groups share, block 1 never was
      float2* mls = reinterpret_cast<float2*>(smem + Cfg::OFF_ML +
                                              (D == 128 && (join || t == 1) ? 128 * D * 2 : 0));
      mls[(join ? sw : half) * 128 + lrow] = make_float2(m2, l);
      // one view of the abort flag, and (m, l) are visible
      if (named_barrier_or(1, kAll, !ok || *abort_flag != 0)) return false;
      float f0 = 1.f, f1 = 0.f, M = m2;
      auto block_l = [&](int blk) {             // a row's sum over both halves of the columns
        return mls[blk * 256 + lrow].y + mls[blk * 256 + 128 + lrow].y;
      };
      float L = block_l(0);
      if (join) {
        const float2 x = mls[lrow], y = mls[256 + lrow];
        M = fmax_nan(x.x, y.x);
        const float sub = M == -INFINITY ? 0.f : M;
        f0 = ex2_approx(x.x - sub);
        f1 = ex2_approx(y.x - sub);
        L = L * f0 + block_l(1) * f1;
      }
      // every group writes its share of the elements
      const int share = D / (join ? Cfg::SW : 2);
      const int h0 = (join ? sw : half) * share, h1 = h0 + share;
      const uint32_t oa = lane_base + Cfg::O0 + (join ? 0 : t * D);
      const float inv = whole ? attn_inverse(L, lim <= 0) : 1.f;
      f0 *= inv;
      f1 *= inv;
      const bool second = join && pc.n > 1;       // block 1's groups had a tile
#pragma unroll 1
      for (int h = h0; h < h1; h += 32) {
        float o[32];
        tmem_ld32(oa + h, o);
        if (second) {
          float y[32];
          tmem_ld32(oa + D + h, y);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = fmaf(y[i], f1, o[i] * f0);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f0;
        }
        if (live) {
          // element i of 8 is in column i, or (int4) in 0 4 1 5 2 6 3 7's place of it
          auto at = [&](int i) { return FMT == kFmtInt4 ? o[(i & ~7) | ((i & 3) << 1) | ((i >> 2) & 1)] : o[i]; };
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              const float x[8] = {at(i), at(i + 1), at(i + 2), at(i + 3),
                                  at(i + 4), at(i + 5), at(i + 6), at(i + 7)};
              attn_store8(a, shape, it, row, h + i, x);
            }
          } else if (slot_in_bounds(shape, slot, gridDim.x, row)) {
            // by fours of elements, then rows: a warp's stores are whole lines
            float4* dst = reinterpret_cast<float4*>(o_out) + (slot * (D / 4) + h / 4) * Cfg::BLOCK + row;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              dst[i / 4 * Cfg::BLOCK] = make_float4(at(i), at(i + 1), at(i + 2), at(i + 3));
          }
        }
      }
      if (!whole && live && half == 0 && (t == 0 || two) && slot_in_bounds(shape, slot, gridDim.x, row))
        ml_out[slot * Cfg::BLOCK + row] = make_float2(M, L);
      named_barrier_sync(1, kAll);      // (m, l) and both O are read
      tc_fence_before();
      return true;
    });
  } else {
    // ============================================================ unpacking warpgroups
    // Codes of a 64-row piece -> fp16 tile.  Group u of UW takes every UW-th tile.
    if constexpr (Cfg::QUANT) {
      regs_to<Cfg::R_LAUNCH, Cfg::R_UNPACK>();
      constexpr int RB = Cfg::RB;
      constexpr int CPR = RB / 16;                     // 16-byte pieces of a stored row
      constexpr int NL = CPR / 2;                      // pieces per thread of 64 rows
      constexpr int RSTEP = 128 / CPR;                 // rows between a thread's pieces
      static_assert(RSTEP % 8 == 0, "a thread's rows keep their place in the swizzle");
      const int tid = (threadIdx.x - 32 * Cfg::UNPACK_WARP0) & 127;
      const uint32_t group = (threadIdx.x - 32 * Cfg::UNPACK_WARP0) >> 7;
      const int piece = tid % CPR, row0 = tid / CPR;
      // fp8: the two 16-byte chunks of a piece, int4: the four, in an order by column
      // block so that no bank is hit twice
      constexpr int NC = FMT == kFmtFp8 ? 2 : 4;
      const int x = FMT == kFmtFp8 ? (piece >> 2) & 1 : (CPR == 4 ? 2 * (piece >> 1) : piece >> 1);
      uint32_t off[NC];
#pragma unroll
      for (int k = 0; k < NC; ++k) off[k] = tile_off<BN>(row0, NC * piece + (k ^ x));
      uint32_t g = 0, g_raw = 0;
      if (a.test_stall == 0)
        each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
          return each_stage(it, pc, [&](bool is_v, int j) {
            const int s = g % STAGES;
            if (Cfg::UW > 1 && g % Cfg::UW != group) {
              ++g;
              g_raw += BN / 64;
              return true;
            }
            uint8_t* dst = smem + Cfg::OFF_KV + s * STAGE;
#pragma unroll 1
            for (int h = 0; h < BN; h += 64, ++g_raw) {
              const int rs = g_raw % Cfg::RAW_SLOTS;
              if (!wait_warp(&raw_ready[rs], (g_raw / Cfg::RAW_SLOTS) & 1, ctl)) return false;
              const uint8_t* raw = smem + Cfg::OFF_RAW + rs * Cfg::RAW_BYTES;
              const uint32_t* muls = reinterpret_cast<const uint32_t*>(raw + 64 * RB);
              const int live = pc.end - (pc.r0 + j * BN + h);       // rows of the piece that count
              uint4 code[NL];
              uint32_t mul[NL];
#pragma unroll
              for (int i = 0; i < NL; ++i) {
                code[i] = *reinterpret_cast<const uint4*>(raw + (tid + 128 * i) * 16);
                mul[i] = muls[row0 + i * RSTEP];
              }
              if (live < 64) {
#pragma unroll
                for (int i = 0; i < NL; ++i)
                  if (row0 + i * RSTEP >= live) code[i] = make_uint4(0, 0, 0, 0);
              }
              // the piece is in registers; the next copy into the slot is the async proxy's,
              // which nothing else keeps behind these reads (without the fence tiles of fp8,
              // and of 4 bits at d = 128, now and then hold codes of a later piece)
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) mbar_arrive(&raw_empty[rs]);
              if (h == 0 && !wait_warp(&kv_empty[s], ((g / STAGES) & 1) ^ 1, ctl)) return false;
              uint8_t* d = dst + h * 128;
#pragma unroll
              for (int i = 0; i < NL; ++i) {
                const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
                if constexpr (FMT == kFmtFp8) {
                  const uint32_t u[4] = {x ? w[2] : w[0], x ? w[3] : w[1], x ? w[0] : w[2], x ? w[1] : w[3]};
                  uint32_t o[8];
#pragma unroll
                  for (int k = 0; k < 4; ++k) e4m3x4_f16x2(u[k], o[2 * k], o[2 * k + 1]);
                  if (!is_v || mul[i] != 0x3c003c00u) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = hmul2(o[k], mul[i]);
                  }
                  *reinterpret_cast<uint4*>(d + off[0] + i * RSTEP * 128) = make_uint4(o[0], o[1], o[2], o[3]);
                  *reinterpret_cast<uint4*>(d + off[1] + i * RSTEP * 128) = make_uint4(o[4], o[5], o[6], o[7]);
                } else {
                  const uint32_t s2 = __byte_perm(mul[i], 0, 0x1010), z2 = __byte_perm(mul[i], 0, 0x3232);
                  const uint32_t y[4] = {x & 1 ? w[1] : w[0], x & 1 ? w[0] : w[1],
                                         x & 1 ? w[3] : w[2], x & 1 ? w[2] : w[3]};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t u = x & 2 ? y[k ^ 2] : y[k];      // word k ^ x
                    const uint32_t u8 = u >> 8;
                    *reinterpret_cast<uint4*>(d + off[k] + i * RSTEP * 128) =
                        make_uint4(hfma2(nib_f16x2<0>(u), s2, z2), hfma2(nib_f16x2<1>(u), s2, z2),
                                   hfma2(nib_f16x2<0>(u8), s2, z2), hfma2(nib_f16x2<1>(u8), s2, z2));
                  }
                }
              }
            }
            fence_proxy_async();
            mbar_arrive(&kv_full[s]);
            ++g;
            return true;
          });
        });
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int FMT, int D>
cudaError_t launch_tc_fd(const CacheAttnArgs& a, cudaStream_t st, int* launches) {
  using Cfg = TcaCfg<FMT, D>;
  const AttnShape shape = attn_shape(a.q_lens, a.n_q, a.G, Cfg::BLOCK, Cfg::BN, Cfg::PAD);
  const int64_t items = a.c.units * shape.blocks;
  float2* ml = static_cast<float2*>(a.ws);
  float* o = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + attn_ml_bytes(kTcCtas, Cfg::BLOCK));
  CUtensorMap kmap{}, vmap{};
  if constexpr (!Cfg::QUANT) {
    const int rows = static_cast<int>(a.c.n_pages << a.c.page_shift);
    const int box = min(1 << a.c.page_shift, Cfg::BN);
    if (!make_map(&kmap, a.c.k_pages, 1, rows, D, box) ||
        !make_map(&vmap, a.c.v_pages, 1, rows, D, box))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(cache_attn_tc<FMT, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  if constexpr (Cfg::R_LAUNCH > 0) {
    // a warpgroup that grows waits for registers the others gave up: the split must
    // fit what the block is launched with
    static const int regs = [] {
      cudaFuncAttributes at;
      return cudaFuncGetAttributes(&at, cache_attn_tc<FMT, D>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs < Cfg::R_LAUNCH) return cudaErrorLaunchOutOfResources;
  }
  e = launch_after(cache_attn_tc<FMT, D>, dim3(kTcCtas), Cfg::THREADS, Cfg::SMEM, st, kmap, vmap, a,
                   shape, items, a.scale * 1.4426950408889634f, ml, o);
  if (e != cudaSuccess) return e;
  *launches += 2;
  return launch_attn_merge(a, shape, items, kTcCtas, true, ml, o, st);
}

}  // namespace

cudaError_t bounds_flag_cache_attention_tc(unsigned int* out) { return take_bounds_flag(out); }

int tc_block(int d) { return d == 128 ? 256 : 128; }

cudaError_t launch_cache_attn_tc(const CacheAttnArgs& a, cudaStream_t s, int* launches) {
  switch (a.c.format * 1000 + a.c.d) {
    case kFmtBf16 * 1000 + 128: return launch_tc_fd<kFmtBf16, 128>(a, s, launches);
    case kFmtBf16 * 1000 + 256: return launch_tc_fd<kFmtBf16, 256>(a, s, launches);
    case kFmtFp8 * 1000 + 128: return launch_tc_fd<kFmtFp8, 128>(a, s, launches);
    case kFmtFp8 * 1000 + 256: return launch_tc_fd<kFmtFp8, 256>(a, s, launches);
    case kFmtInt4 * 1000 + 128: return launch_tc_fd<kFmtInt4, 128>(a, s, launches);
    case kFmtInt4 * 1000 + 256: return launch_tc_fd<kFmtInt4, 256>(a, s, launches);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvzip
