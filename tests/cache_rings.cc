// Walks the tiles of many successions of items through the stations of the tensor-memory
// cache attention (raw slots, registers of the unpacking groups, stages) with the softmax
// stopped at each tile in turn, and compares how far the row-parameter warp gets with the
// rings it writes to.  Prints, per format and head size, the farthest distances and the rings.
#include <algorithm>
#include <cstdio>
#include <vector>

#include "cache_rings.h"

struct Tile {
  bool v;
  int index;      // of its kind, over all items
};

// Tiles whose parameters can be written while the softmax is at tile `stop` (a V tile, which
// keeps its stage): every other tile is taken from its stage as soon as it is there.
template <typename R>
static int reach(int total, int stop) {
  constexpr int pieces = R::PIECES, groups = R::GROUPS;
  std::vector<int> unpacked(groups, 0);         // pieces of the group's current tile written to its stage
  std::vector<int> at(groups);                  // that tile
  std::vector<char> in_regs(groups, 0);
  for (int u = 0; u < groups; ++u) at[u] = u;
  std::vector<int> freed(R::RAW_SLOTS, 0);      // times each raw slot was given back
  std::vector<int> stage_done(total, 0);        // unpacked and taken
  int loaded = 0;                               // pieces with parameters written, in order
  for (bool moved = true; moved;) {
    moved = false;
    while (loaded < total * pieces && loaded / R::RAW_SLOTS <= freed[loaded % R::RAW_SLOTS]) {
      ++loaded;
      moved = true;
    }
    for (int u = 0; u < groups; ++u) {
      if (at[u] >= total) continue;
      const int piece = at[u] * pieces + unpacked[u];
      if (!in_regs[u] && piece < loaded) {      // raw slot -> registers
        in_regs[u] = 1;
        ++freed[piece % R::RAW_SLOTS];
        moved = true;
      }
      const int before = at[u] - R::STAGES;     // the stage's tile before
      if (in_regs[u] && (before < 0 || stage_done[before])) {
        in_regs[u] = 0;
        moved = true;
        if (++unpacked[u] == pieces) {
          stage_done[at[u]] = at[u] != stop;
          at[u] += groups;
          unpacked[u] = 0;
        }
      }
    }
  }
  return (loaded + pieces - 1) / pieces;        // a tile counts from its first piece on
}

template <typename R>
struct Walk {
  int v_far = 0, k_far = 0, lead = 0;
  std::vector<Tile> tiles;

  void check(int first) {                       // every stop in the tiles from `first` on
    const int total = static_cast<int>(tiles.size());
    for (int g = first; g < total; ++g) {
      if (!tiles[g].v) continue;
      const int end = reach<R>(total, g);
      if (end == total) continue;               // too short to show how far it gets
      lead = std::max(lead, end - 1 - g);
      for (int x = 0; x < end; ++x) {
        const int far = tiles[x].index - tiles[g].index;
        if (tiles[x].v) v_far = std::max(v_far, far); else k_far = std::max(k_far, far);
      }
    }
  }
  void items(const std::vector<int>& sizes, const std::vector<int>& aheads) {
    tiles.clear();
    int k = 0, v = 0;
    for (size_t i = 0; i < sizes.size(); ++i)
      kvzip::for_each_stage(sizes[i], aheads[i], [&](bool is_v, int) {
        tiles.push_back({is_v, is_v ? v++ : k++});
        return true;
      });
    check(0);
  }
  // all successions of items whose tiles just pass the window
  void extend(std::vector<int>& sizes, std::vector<int>& aheads, int sum, int window, bool one_block) {
    if (sum > window) {
      items(sizes, aheads);
      return;
    }
    for (int n = 1; n <= 9; ++n)
      for (int ahead = one_block ? 2 : 1; ahead <= R::AHEAD; ++ahead) {
        sizes.push_back(n);
        aheads.push_back(ahead);
        extend(sizes, aheads, sum + 2 * n, window, one_block);
        sizes.pop_back();
        aheads.pop_back();
      }
  }
};

template <bool INT4, int D>
static bool show(const char* name) {
  using R = kvzip::TcaRings<true, INT4, D>;
  Walk<R> w;
  std::vector<int> sizes, aheads;
  w.extend(sizes, aheads, 0, D == 256 ? 18 : 14, D == 256);
  std::printf("%s lead %d of %d, V %d of ring %d, K %d of ring %d\n", name, w.lead, R::LEAD, w.v_far,
              R::V_RING, w.k_far, R::K_RING);
  return w.lead <= R::LEAD && w.v_far < R::V_RING && w.k_far < R::K_RING;
}

// The places the kernel's issuers and softmax compute: V tile j comes after
// min(j + ahead, n) K tiles and j V tiles, K tile j after max(0, j - ahead + 1) V tiles.
static bool places() {
  bool ok = true;
  for (int n = 1; n <= 40; ++n)
    for (int ahead = 1; ahead <= 2; ++ahead) {
      int at = 0;
      kvzip::for_each_stage(n, ahead, [&](bool v, int j) {
        ok = ok && at == (v ? std::min(j + ahead, n) + j : (j < ahead ? j : 2 * j - ahead + 1));
        ++at;
        return true;
      });
      ok = ok && at == 2 * n;
    }
  return ok;
}

int main() {
  bool ok = places();
  ok = show<false, 128>("fp8 128") && ok;
  ok = show<true, 128>("int4 128") && ok;
  ok = show<false, 256>("fp8 256") && ok;
  ok = show<true, 256>("int4 256") && ok;
  return ok ? 0 : 1;
}
