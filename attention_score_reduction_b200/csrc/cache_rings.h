// Rings of the tensor-memory attention over the paged cache (cache_attention_tc.cu):
// how many tiles and pieces are in flight, and how long the rings of powers of two
// that the row-parameter warp fills for the softmax have to be for that.
// No CUDA here: a host test walks the same order of tiles against these numbers.
#pragma once

namespace kvzip {

// A cache tile (K or V) of BN rows goes through these stations, each in the order of
// for_each_stage:
//   raw slot    pieces of 64 rows as they are stored; the parameter warp works on them there
//   registers   a piece of each unpacking group, which has given its raw slot back and waits
//               for a stage
//   stage       the unpacked tile, until its MMAs are done
template <bool QUANT, bool INT4, int D>
struct TcaRings {
  static constexpr int BN = D == 128 ? 128 : 64;                  // cache rows of a tile
  static constexpr int AHEAD = 2;                                 // K tiles before the first V tile, at most
  static constexpr int STAGES = QUANT ? 4 : (D == 128 ? 5 : 6);
  static constexpr int GROUPS = QUANT ? (D == 128 ? 1 : 2) : 0;   // unpacking warpgroups
  static constexpr int RAW_SLOTS = !QUANT ? 0 : (INT4 ? (D == 128 ? 5 : 6) : (D == 128 ? 3 : 4));

  // The softmax of tile j reads what the parameter warp noted for K tile j and V tile j,
  // and V tile j keeps its stage until that softmax is done.  So while it reads, the
  // parameter warp is at most LEAD tiles past V tile j: those in the other stages, in
  // registers and in raw slots.
  static constexpr int PIECES = BN / 64;
  static constexpr int LEAD = STAGES - 1 + (GROUPS + RAW_SLOTS + PIECES - 1) / PIECES;
  // K and V do not simply alternate: K tiles run up to AHEAD before V tiles, never behind
  // them, and an item ends with its last V tiles in a row.  After V tile j the K tiles are
  // at most AHEAD - 1 ahead, so of the LEAD tiles that follow no more than this are V ...
  static constexpr int V_AFTER = (LEAD + AHEAD - 1) / 2;
  // ... and K tiles past K tile j: those ahead already (AHEAD - 1 at most), and half of
  // the rest, as they cannot be more than AHEAD ahead at its end.
  static constexpr int K_AFTER = AHEAD - 1 + (LEAD + 1) / 2;
  // Entries; tile i's is overwritten by tile i + RING.
  static constexpr int V_RING = V_AFTER + 1;
  static constexpr int K_RING = K_AFTER + 1;
};

// K and V tiles of an item of n tiles in the order the MMAs use them: f(is_v, tile), false
// to stop.  V tile j comes after min(j + ahead, n) K tiles and j V tiles; ahead <= AHEAD.
#ifdef __CUDACC__
#define KVZIP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KVZIP_HOST_DEVICE inline
#endif
template <typename F>
KVZIP_HOST_DEVICE bool for_each_stage(int n, int ahead, F&& f) {
  for (int j = 0; j < ahead && j < n; ++j)
    if (!f(false, j)) return false;
  for (int j = 0; j < n; ++j) {
    if (!f(true, j)) return false;
    if (j + ahead < n && !f(false, j + ahead)) return false;
  }
  return true;
}

}  // namespace kvzip
