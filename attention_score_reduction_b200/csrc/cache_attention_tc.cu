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
//   P = 2^(c S - m) a warpgroup, one query row per thread; P goes back to TMEM as
//                   bf16 over the columns S had
//   O += P V        A = P from TMEM, B = V tile as it lies (MN-major), O in TMEM
// TMEM (512 columns): d = 128: S0 S1 O0 O1 of 128 each; d = 256: O 256, S0 S1 64
// each (cache tiles of 64 rows), Q 128 (with Q in shared memory an MMA of N = 64
// would read more operand bytes than shared memory delivers).
//
// The two S buffers keep the tensor pipe fed while a warpgroup works on the other.
// With more than 128 rows (d = 128) each buffer belongs to one block of 128 rows;
// with fewer, buffer b takes the tiles of parity b, each with an O of its own at
// d = 128 (joined at the end).  One thread issues every MMA, so MMAs complete in
// order: S of a buffer's next tile being ready means the O of its last is, too.
//
// The running maximum is only moved when it grows by more than 2^8 (P then stays
// below 2^8, its bf16 rounding relative): O is rescaled in TMEM for a few tiles of
// an item instead of all.  P is rounded to bf16 (at most 2^-8 of a weight, errors
// of both signs); the sum of the weights is taken before the rounding, in fp32.
//
// bf16 pages come by TMA, one box per page and 64 elements, 128-byte swizzle.
// Quantised pages are unpacked by a warpgroup of their own into the same layout:
// e4m3 codes times 2^e are exact in bf16 (down to its smallest numbers); s c + z is
// rounded once to bf16.
// Rows of the last tile that are not part of the item (other data of the page, or
// what an earlier tile left) are zeroed in V, since 0 * NaN is NaN; in K they give
// logits that the mask replaces.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "cache_attention.cuh"
#include "cache_sched.cuh"
#include "kvzip_internal.h"
#include "sm100_ptx.cuh"
#include "tc_common.cuh"

namespace kvzip {

namespace {

template <int FMT, int D>
struct TcaCfg {
  static constexpr bool QUANT = FMT != kFmtBf16;
  static constexpr int BN = D == 128 ? 128 : 64;       // cache rows of a tile
  static constexpr int WG = D == 128 ? 2 : 1;          // softmax warpgroups
  static constexpr int BLOCK = 128 * WG;               // query rows of an item
  static constexpr int KB = D / 64;                    // 128-byte column blocks of a row
  static constexpr int STAGE = BN * D * 2;             // one K or V tile: 32 KB
  static constexpr int Q_BYTES = D == 128 ? WG * 128 * D * 2 : 0;
  static constexpr int STAGES = D == 128 ? 5 : 7;
  static constexpr int THREADS = 128 + 128 * WG + (QUANT ? 128 : 0);
  static constexpr int UNPACK_WARP0 = 4 + 4 * WG;      // first warp that unpacks codes
  // TMEM columns
  static constexpr int S0 = D == 128 ? 0 : 256, O0 = D == 128 ? 256 : 0;
  static constexpr int Q0 = 384;                        // d = 256 only
  // shared memory
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = Q_BYTES;
  static constexpr int OFF_ML = OFF_Q + 128 * D * 2;   // float2 per row, where the second Q block is unused
  static constexpr int OFF_BAR = OFF_KV + STAGES * STAGE;
  // kv_full[STAGES], kv_empty[STAGES], s_full[2], p_full[2], o_full[2], pv_done, q_full[2], mma_done
  static constexpr int N_BARS = 2 * STAGES + 10;
  static constexpr int OFF_MISC = OFF_BAR + 8 * N_BARS;
  static constexpr int BYTES = OFF_MISC + 16;
  static constexpr int SMEM = BYTES + 1024;
  static_assert(SMEM <= 232448, "exceeds 227 KB of shared memory");
  // registers a thread of each warpgroup after the split (0: no split); the sums
  // stay within the 168 (384 threads) or 128 (512 threads) a thread of the launch
  static constexpr int R_CTL = D == 256 ? 0 : (QUANT ? 48 : 104);
  static constexpr int R_SOFT = D == 256 ? 0 : (QUANT ? 176 : 200);
  static constexpr int R_UNPACK = D == 256 ? 0 : 112;
  static_assert(D == 256 || !QUANT || R_CTL + 2 * R_SOFT + R_UNPACK <= 4 * 128, "register split");
  static_assert(D == 256 || QUANT || R_CTL + 2 * R_SOFT <= 3 * 168, "register split");
  static constexpr int POLY = 2;     // of 8 pairs of exponentials, those on the FMA pipe
};

// Descriptor of an MN-major operand under the 128-byte swizzle: 64 elements (128
// bytes) of N per row, rows of K 128 bytes apart in groups of eight (1024 bytes),
// the next 64 elements of N `block` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr, uint32_t block) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Byte offset of 16-byte chunk ch (of 64-element column blocks) of tile row r.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
  return static_cast<uint32_t>((ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Two e4m3 codes in the high bytes of x's halves -> bf16x2 of value * 2^-120
// (exponent bias 7 read with bias 127; subnormal codes are subnormal bf16).
__device__ __forceinline__ uint32_t e4m3_bits(uint32_t x) {
  const uint32_t t = (x & 0x7f007f00u) >> 4;
  return t | (x & 0x80008000u);
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
  __shared__ int64_t found[2];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* kv_full = bars;
  uint64_t* kv_empty = kv_full + STAGES;
  uint64_t* s_full = kv_empty + STAGES;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* pv_done = o_full + 2;
  uint64_t* q_full = pv_done + 1;
  uint64_t* mma_done = q_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cta = blockIdx.x;

  cudaTriggerProgrammaticLaunchCompletion();   // the merge may be launched; it waits for this grid
  Line<THREADS> line(a.c, shape, items, scratch, found);
  const int64_t all = line.all;
  const int64_t n_cta = line_ctas(all, gridDim.x);
  if (cta >= n_cta) return;
  const int64_t p0 = line_cut(all, cta, n_cta), p1 = line_cut(all, cta + 1, n_cta);
  int64_t w_first, w_first_at;
  line.find(p0, &w_first, &w_first_at);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&kv_full[s], Cfg::QUANT ? 128 : 1);
      mbar_init(&kv_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
      mbar_init(&q_full[i], 128);
    }
    mbar_init(pv_done, 1);
    mbar_init(mma_done, 1);
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
      if (it.n_tiles == 0) continue;
      const int t0 = static_cast<int>(p - at);
      const int t1 = static_cast<int>(min(static_cast<int64_t>(it.n_tiles), p1 - at));
      Piece pc;
      pc.r0 = t0 * BN;
      pc.end = min(t1 * BN, it.vis);
      pc.n = t1 - t0;
      const bool whole = pc.n == it.n_tiles;
      if (!f(it, pc, whole, line_slot(all, cta, n_cta, at))) return;
      p = at + t1;
      at += it.n_tiles;
    }
  };
  auto two_blocks = [&](const AttnItem& it) { return Cfg::WG == 2 && it.rows > 128; };
  // K and V tiles in the order the MMAs use them: f(is_v, tile)
  auto each_stage = [&](const AttnItem& it, const Piece& pc, auto&& f) -> bool {
    const int ahead = two_blocks(it) ? 1 : 2;
    for (int j = 0; j < ahead && j < pc.n; ++j)
      if (!f(false, j)) return false;
    for (int j = 0; j < pc.n; ++j) {
      if (!f(true, j)) return false;
      if (j + ahead < pc.n && !f(false, j + ahead)) return false;
    }
    return true;
  };

  if (warp < 4) {
   if constexpr (Cfg::R_CTL > 0) regs_shrink<Cfg::R_CTL>();
   if (warp == 0) {
    // ============================================================ TMA producer
    if constexpr (!Cfg::QUANT) {
      const int box_shift = min(a.c.page_shift, BN == 128 ? 7 : 6);
      const int box = 1 << box_shift;
      const int rows_total = static_cast<int>(a.c.n_pages << a.c.page_shift);
      uint32_t g = 0;
      if (a.test_stall == 0)
        each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
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
            if (lane == 0) mbar_arrive_expect_tx(&kv_full[s], n_box * box * D * 2);
            __syncwarp();
            if (mine) {
              uint8_t* dst = smem + Cfg::OFF_KV + s * STAGE + lane * box * 128;
#pragma unroll
              for (int kb = 0; kb < KB; ++kb)
                tma_load_3d(dst + kb * (BN * 128), is_v ? &vmap : &kmap, &kv_full[s], kb * 64, row, 0);
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
    }
   } else if (warp == 1) {
    // ============================================================ MMA issuer
    constexpr uint32_t id_qk = idesc_bf16_f32(128, BN);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, D) | (1u << 16);     // B is MN-major
    const uint32_t kv_base = smem_u32(smem + Cfg::OFF_KV);
    const uint32_t q_base = smem_u32(smem + Cfg::OFF_Q);
    uint32_t g = 0, n_item = 0, n_p[2] = {0, 0};
    auto stage_ready = [&]() { return wait_warp(&kv_full[g % STAGES], (g / STAGES) & 1, ctl); };
    auto qk = [&](int buf, int qt, uint32_t stage) {
      if (lane == 0) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const uint64_t bd = sdesc_sw128(kv_base + stage * STAGE + kb * (BN * 128));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (D == 128) {
              const uint64_t ad = sdesc_sw128(q_base + qt * (128 * D * 2) + kb * (128 * 128));
              umma_bf16_ss(tmem + Cfg::S0 + buf * BN, ad + 2 * kk, bd + 2 * kk, id_qk, (kb | kk) != 0);
            } else {
              umma_bf16_ts(tmem + Cfg::S0 + buf * BN, tmem + Cfg::Q0 + (kb * 4 + kk) * 8, bd + 2 * kk,
                           id_qk, (kb | kk) != 0);
            }
          }
        }
        umma_commit(&s_full[buf]);
      }
      __syncwarp();
    };
    auto pv = [&](int buf, int ob, uint32_t stage, bool first) {
      if (lane == 0) {
        const uint64_t bd = sdesc_mn_sw128(kv_base + stage * STAGE, BN * 128);
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)     // 16 rows: 8 columns of P, 2048 bytes of each V block
          umma_bf16_ts(tmem + Cfg::O0 + ob * D, tmem + Cfg::S0 + buf * BN + k * 8,
                       bd + k * (2048 >> 4), id_pv, !(first && k == 0));
      }
      __syncwarp();
    };
    auto release = [&](uint64_t* bar) {
      if (lane == 0) umma_commit(bar);
      __syncwarp();
    };
    // rows of the last V tile past the piece's end: zeros
    auto clear_tail = [&](const Piece& pc, int j, uint32_t stage) {
      if constexpr (!Cfg::QUANT) {
        const int live = pc.end - (pc.r0 + j * BN);
        if (live < BN) {
          for (int i = lane; i < (BN - live) * (D / 8); i += 32)
            *reinterpret_cast<uint4*>(smem + Cfg::OFF_KV + stage * STAGE +
                                      tile_off<BN>(live + i / (D / 8), i % (D / 8))) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async();
          __syncwarp();
        }
      }
    };
    each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
      const bool two = two_blocks(it);
      const uint32_t qph = n_item++ & 1;
      if (!wait_warp(&q_full[0], qph, ctl)) return false;
      if (Cfg::WG == 2 && !wait_warp(&q_full[1], qph, ctl)) return false;
      tc_fence_after();
      if (two) {
        if (!stage_ready()) return false;
        tc_fence_after();
        qk(0, 0, g % STAGES);
        qk(1, 1, g % STAGES);
        release(&kv_empty[g % STAGES]);
        ++g;
        for (int j = 0; j < pc.n; ++j) {
          if (!stage_ready()) return false;
          const uint32_t sv = g % STAGES;
          clear_tail(pc, j, sv);
          ++g;
          const bool more = j + 1 < pc.n;
          for (int t = 0; t < 2; ++t) {
            if (!wait_warp(&p_full[t], n_p[t]++ & 1, ctl)) return false;
            tc_fence_after();
            pv(t, t, sv, j == 0);
            if (more) {
              if (t == 0 && !stage_ready()) return false;
              tc_fence_after();
              qk(t, t, g % STAGES);
            }
          }
          release(&kv_empty[sv]);
          if (more) {
            release(&kv_empty[g % STAGES]);
            ++g;
          }
        }
      } else {
        for (int j = 0; j < 2 && j < pc.n; ++j) {
          if (!stage_ready()) return false;
          tc_fence_after();
          qk(j, 0, g % STAGES);
          release(&kv_empty[g % STAGES]);
          ++g;
        }
        for (int j = 0; j < pc.n; ++j) {
          const int b = j & 1;
          if (!stage_ready()) return false;
          const uint32_t sv = g % STAGES;
          clear_tail(pc, j, sv);
          ++g;
          if (!wait_warp(&p_full[b], n_p[b]++ & 1, ctl)) return false;
          tc_fence_after();
          pv(b, Cfg::WG == 2 ? b : 0, sv, Cfg::WG == 2 ? j < 2 : j == 0);
          release(&kv_empty[sv]);
          if (Cfg::WG == 1) release(pv_done);
          if (j + 2 < pc.n) {
            if (!stage_ready()) return false;
            tc_fence_after();
            qk(b, 0, g % STAGES);
            release(&kv_empty[g % STAGES]);
            ++g;
          }
        }
      }
      release(&o_full[0]);
      if (Cfg::WG == 2) release(&o_full[1]);
      return true;
    });
    // all MMAs are done before TMEM is freed
    release(mma_done);
    if (lane == 0) wait_drain(mma_done, 0, a.c.status);
    __syncwarp();
   }
  } else if (warp < Cfg::UNPACK_WARP0) {
    // ============================================================ softmax warpgroups
    if constexpr (Cfg::R_SOFT > 0) regs_grow<Cfg::R_SOFT>();
    const int wg = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;                 // TMEM lane = row of the 128-row block
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float2* mls = reinterpret_cast<float2*>(smem + Cfg::OFF_ML);
    const float lazy = 8.f / c;                            // growth of the maximum that is let pass
    uint32_t n_s[2] = {0, 0}, n_item = 0, n_pv = 0;
    each_item([&](const AttnItem& it, const Piece& pc, bool whole, int64_t slot) {
      const bool two = two_blocks(it);
      const int row = (two ? wg * 128 : 0) + lrow;         // query row within the item
      const bool live = row < it.rows;
      const int r = it.row0 + row, tok = r / shape.G, head = r - tok * shape.G;
      const int lim = live ? min(seen_rows(it, tok), pc.end) : 0;
      // rows every query of this block sees: tiles before need no mask
      const int lim_all = min(seen_rows(it, (it.row0 + (two ? wg * 128 : 0)) / shape.G), pc.end);
      // ---- this row of Q into the MMA's operand
      if (two || wg == 0) {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) + it.u * a.q_unit + head * a.q_head + tok * a.q_row);
        // int4 tiles hold each 8 elements as 0 4 1 5 2 6 3 7, so Q does, too
        auto chunk = [&](int i) {
          uint4 v = live ? src[i] : make_uint4(0, 0, 0, 0);
          if constexpr (FMT == kFmtInt4)
            v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                           __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
          return v;
        };
        if constexpr (D == 128) {
          uint8_t* dst = smem + Cfg::OFF_Q + wg * (128 * D * 2);
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint4*>(dst + tile_off<128>(lrow, i)) = chunk(i);
          fence_proxy_async();
        } else {
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 x = chunk(8 * h + i);
              v[4 * i] = x.x;
              v[4 * i + 1] = x.y;
              v[4 * i + 2] = x.z;
              v[4 * i + 3] = x.w;
            }
            tmem_st32_async(lane_base + Cfg::Q0 + 32 * h, v);
          }
          tmem_wait_st();
          tc_fence_before();
        }
      }
      mbar_arrive(&q_full[wg]);

      float m = -INFINITY, l = 0.f;                        // m in units of S
      const uint32_t o_addr = lane_base + Cfg::O0 + wg * D;
      const int j0 = two || Cfg::WG == 1 ? 0 : wg, dj = two || Cfg::WG == 1 ? 1 : 2;
      bool ok = true;
      for (int j = j0; j < pc.n; j += dj) {
        const int b = Cfg::WG == 2 ? wg : (j & 1);
        const uint32_t s_addr = lane_base + Cfg::S0 + b * BN;
        if (!wait_warp(&s_full[b], n_s[b]++ & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        float s[BN];
#pragma unroll
        for (int h = 0; h < BN; h += 64) {
          float v[64];
          tmem_ld64(s_addr + h, v);
#pragma unroll
          for (int i = 0; i < 64; ++i) s[h + i] = v[i];
        }
        const int col0 = pc.r0 + j * BN;
        const bool masked = col0 + BN > lim_all;
        if (masked) {
          const int n = lim - col0;
#pragma unroll
          for (int i = 0; i < BN; ++i) s[i] = i < n ? s[i] : -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = fmax_nan(s[2 * q], s[2 * q + 1]);
#pragma unroll
        for (int i = 8; i < BN; i += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmax3_nan(mx[q], s[i + 2 * q], s[i + 2 * q + 1]);
        const float cand = fmax3_nan(fmax_nan(mx[0], mx[1]), fmax_nan(mx[2], mx[3]), m);
        const bool need = !(cand - m <= lazy) && cand != -INFINITY;
        if (__any_sync(0xffffffffu, need)) {
          const float f = cand == -INFINITY ? 1.f : ex2_approx((m - cand) * c);
          if (j != j0) {
            // d = 256: S was ready before the last O; wait for that product
            if (Cfg::WG == 1 && !wait_warp(pv_done, (n_pv + j - 1) & 1, ctl)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < D; h += 32) {
              float v[32];
              tmem_ld32(o_addr + h, v);
              uint32_t u[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(v[i] * f);
              tmem_st32_async(o_addr + h, u);
            }
            tmem_wait_st();
          }
          l *= f;
          m = cand;
        }
        const float nb = m == -INFINITY ? 0.f : -m * c;
        const float2 c2 = make_float2(c, c), nb2 = make_float2(nb, nb);
        float2 acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = make_float2(0.f, 0.f);
#pragma unroll
        for (int h = 0; h < BN; h += 64) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 64; i += 16)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const int e0 = h + i + 2 * q;
              const float2 x = ffma2(make_float2(s[e0], s[e0 + 1]), c2, nb2);
              float2 e;
              if (q < Cfg::POLY && !masked) {     // the polynomial has no -infinity
                e = exp2_poly2(x);
              } else {
                e.x = ex2_approx(x.x);
                e.y = ex2_approx(x.y);
              }
              acc[q & 3] = fadd2(acc[q & 3], e);
              pk[(i + 2 * q) / 2] = pack_bf16x2(e.x, e.y);
            }
          tmem_st32_async(s_addr + h / 2, pk);
        }
        const float2 sum = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[b]);
      }
      if (Cfg::WG == 1) n_pv += pc.n;

      // ---- the item's result
      if (ok) ok = wait_warp(&o_full[wg], n_item & 1, ctl);
      ++n_item;
      tc_fence_after();
      const bool join = Cfg::WG == 2 && !two;     // both groups hold part of the same rows
      const float m2 = m == -INFINITY ? m : m * c;
      if (join) mls[wg * 128 + lrow] = make_float2(m2, l);
      // one view of the abort flag; also: Q is not overwritten while the other
      // group's MMAs may read it, and the exchanged (m, l) are visible
      if (named_barrier_or(1, 128 * Cfg::WG, !ok || *abort_flag != 0)) return false;
      float f0 = 1.f, f1 = 0.f, L = l, M = m2;
      int h0 = 0, h1 = D;
      if (join) {
        const float2 x = mls[lrow], y = mls[128 + lrow];
        M = fmax_nan(x.x, y.x);
        const float sub = M == -INFINITY ? 0.f : M;
        f0 = ex2_approx(x.x - sub);
        f1 = ex2_approx(y.x - sub);
        L = x.y * f0 + y.y * f1;
        h0 = wg * (D / 2);                          // each group writes half of the elements
        h1 = h0 + D / 2;
      }
      const uint32_t oa = lane_base + Cfg::O0 + (join ? 0 : wg * D);
      const float inv = !whole ? 1.f : (L > 0.f ? 1.f / L : (L == 0.f ? 0.f : NAN));
      f0 *= inv;
      f1 *= inv;
      const bool second = join && pc.n > 1;       // group 1 had a tile
#pragma unroll 1
      for (int h = h0; h < h1; h += 32) {
        float v[32];
        tmem_ld32(oa + h, v);
        if (second) {
          float y[32];
          tmem_ld32(oa + D + h, y);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = fmaf(y[i], f1, v[i] * f0);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= f0;
        }
        if constexpr (FMT == kFmtInt4) {            // back from the order 0 4 1 5 2 6 3 7
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = v[(i & ~7) | ((i & 3) << 1) | ((i >> 2) & 1)];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = y[i];
        }
        if (live) {
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              const float x[8] = {v[i], v[i + 1], v[i + 2], v[i + 3],
                                  v[i + 4], v[i + 5], v[i + 6], v[i + 7]};
              attn_store8(a, shape, it, row, h + i, x);
            }
          } else {
            float4* o = reinterpret_cast<float4*>(o_out + (slot * Cfg::BLOCK + row) * D + h);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
      }
      if (!whole && live && (wg == 0 || two))
        ml_out[slot * Cfg::BLOCK + row] = make_float2(M, L);
      if (join) named_barrier_sync(1, 128 * Cfg::WG);      // (m, l) and both O are read
      tc_fence_before();
      return true;
    });
  } else {
    // ============================================================ unpacking warpgroup
    if constexpr (Cfg::QUANT) {
      if constexpr (Cfg::R_UNPACK > 0) regs_shrink<Cfg::R_UNPACK>();
      constexpr int RB = CacheRow<FMT, D>::BYTES;
      constexpr int CPR = RB / 16;                     // 16-byte pieces of a stored row
      constexpr int NL = BN * CPR / 128;               // pieces per thread
      constexpr int RSTEP = 128 / CPR;                 // rows between a thread's pieces
      const int tid = threadIdx.x - 32 * Cfg::UNPACK_WARP0;
      const int piece = tid % CPR, row0 = tid / CPR;
      uint4 raw[NL];
      uint32_t par[NL];
      uint32_t g = 0;
      auto fetch = [&](const AttnItem& it, const Piece& pc, bool is_v, int j) {
        const uint8_t* pages = static_cast<const uint8_t*>(is_v ? a.c.v_pages : a.c.k_pages);
        const uint32_t* params = is_v ? a.c.v_params : a.c.k_params;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int r = pc.r0 + j * BN + row0 + i * RSTEP;
          const int64_t slot = r < pc.end ? cache_slot(a.c, it.u, r) : -1;
          raw[i] = slot >= 0 ? ldg_stream16(pages + slot * RB + piece * 16) : make_uint4(0, 0, 0, 0);
          par[i] = slot >= 0 ? __ldg(params + slot) : 0u;
        }
      };
      auto put = [&](uint8_t* dst) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int r = row0 + i * RSTEP;
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          if constexpr (FMT == kFmtFp8) {
            // code * 2^e = bits * 2^120 * 2^e, in one exact product where 2^(120 + e) is a bf16
            const int e = static_cast<int>(par[i] >> 23) - 127;      // 128 for a NaN scale, -127 for none
            const uint32_t up = par[i] >= 0x7f800000u
                                    ? 0x7fc0u
                                    : static_cast<uint32_t>(max(0, min(254, 247 + e))) << 7;
            const uint32_t f = up | (up << 16);
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * k] = bmul2(e4m3_bits(__byte_perm(w[k], 0, 0x1404)), f);
              o[2 * k + 1] = bmul2(e4m3_bits(__byte_perm(w[k], 0, 0x3424)), f);
            }
            if (e > 7) {      // rows beyond 57344: the rest of the scale
              const uint32_t x2 = static_cast<uint32_t>(min(127 + e - 7, 254)) << 7;
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = bmul2(o[k], x2 | (x2 << 16));
            }
            *reinterpret_cast<uint4*>(dst + tile_off<BN>(r, 2 * piece)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + tile_off<BN>(r, 2 * piece + 1)) =
                make_uint4(o[4], o[5], o[6], o[7]);
          } else {
            const uint32_t s2 = __byte_perm(par[i], 0, 0x1010), z2 = __byte_perm(par[i], 0, 0x3232);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t o[4];
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                // 0x4300 | c is 128 + c; minus 128 is c, exactly
                const uint32_t x = ((w[k] >> (4 * n)) & 0x000f000fu) | 0x43004300u;
                o[n] = bfma2(bfma2(x, 0x3f803f80u, 0xc300c300u), s2, z2);
              }
              *reinterpret_cast<uint4*>(dst + tile_off<BN>(r, 4 * piece + k)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
      };
      if (a.test_stall == 0)
        each_item([&](const AttnItem& it, const Piece& pc, bool, int64_t) {
          return each_stage(it, pc, [&](bool is_v, int j) {
            const int s = g % STAGES;
            fetch(it, pc, is_v, j);
            if (!wait_warp(&kv_empty[s], ((g / STAGES) & 1) ^ 1, ctl)) return false;
            put(smem + Cfg::OFF_KV + s * STAGE);
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
  const AttnShape shape = attn_shape(a.q_lens, a.n_q, a.G, Cfg::BLOCK, Cfg::BN);
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
  if constexpr (Cfg::R_SOFT > 0) {
    // a warpgroup that grows waits for registers the others gave up: the split must
    // fit what the block is launched with
    static const int regs = [] {
      cudaFuncAttributes at;
      return cudaFuncGetAttributes(&at, cache_attn_tc<FMT, D>) == cudaSuccess ? at.numRegs : 0;
    }();
    if (Cfg::R_CTL + 2 * Cfg::R_SOFT + (Cfg::QUANT ? Cfg::R_UNPACK : 0) > regs * Cfg::THREADS / 128)
      return cudaErrorLaunchOutOfResources;
  }
  cache_attn_tc<FMT, D><<<kTcCtas, Cfg::THREADS, Cfg::SMEM, st>>>(
      kmap, vmap, a, shape, items, a.scale * 1.4426950408889634f, ml, o);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  *launches += 2;
  return launch_attn_merge(a, shape, items, kTcCtas, ml, o, st);
}

}  // namespace

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
