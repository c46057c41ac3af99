// Prints the stages of the ring (csrc/hs_ring.hpp) that each loader fills, in the order of its jobs: for step t the two jobs of
// K(t), then those of V(t - 1). A line for each loader of each split: "lv n last_segs loader: first stage of each job ..", with
// the arrivals of a job's stages behind it, and its first row and column of K or V ("18x2@32/128"; a K job is two stages), and
// first a line of the ring's constants.
#include <cstdio>

#include "hs_ring.hpp"

template <int lv>
void walk(int n, int last) {
  const hs::Tiles<lv> tiles{0, n, last};
  for (int wl = 0; wl < hs::LOADERS; ++wl) {
    const hs::Loader<lv> loader{wl};
    std::printf("%d %d %d %d:", lv, n, last, wl);
    for (int t = 0; t <= n; ++t) {
      for (int h = 0; h < 2 && t < n; ++h) {
        const int at = tiles.k_stage(t) + loader.k_stage(h);
        for (int i = 0; i < 2; ++i)
          std::printf(" %dx%d@%d/%d", at + i, hs::K_ARRIVE, loader.k_row(), loader.group() * 128 + 256 * h + 64 * i);
      }
      for (int h = 0; h < loader.v_jobs && t > 0; ++h)
        if (loader.segment(h) < tiles.segs(t - 1))
          std::printf(" %dx%d@%d/%d", tiles.v_stage(t - 1) + loader.v_stage(h), hs::V_ARRIVE,
                      loader.segment(h) * hs::SEG + loader.v_row(), loader.v_col());
    }
    std::printf("\n");
  }
  std::printf("%d %d %d keys:", lv, n, last);
  for (int t = 0; t < n; ++t) std::printf(" %dx%d", tiles.k_stage(t) + hs::ROPE_AT, hs::KEY_ARRIVE * hs::KEY_WARPS);
  std::printf("\n%d %d %d issuer:", lv, n, last);  // how many stages of each tile the MMAs read
  for (int t = 0; t < n; ++t) std::printf(" %d+%d", hs::KBLK, tiles.v_stages(t));
  std::printf("\n");
}

int main() {
  std::printf("%d %d\n", hs::NSTAGE, hs::FULL);
  for (int n = 1; n <= 6; ++n)
    for (int last = 1; last <= hs::NSEG; ++last) walk<0>(n, last), walk<1>(n, last);
}
