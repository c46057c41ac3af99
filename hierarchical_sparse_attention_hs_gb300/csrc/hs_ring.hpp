// The ring of hs_decode4.cu: which stage holds what, and who fills it (plain C++, so that the order is checked without a device).
#ifndef HS_RING_HPP_
#define HS_RING_HPP_

#ifdef __CUDACC__
#define HS_RING_FN __host__ __device__ __forceinline__
#else
#define HS_RING_FN inline
#endif

namespace hs {

constexpr int SEG = 64, NSEG = 4;  // rows of a segment, segments of a tile
constexpr int KBLK = 9;            // 64-column blocks of a row: K stages of a tile
constexpr int ROPE_AT = 4;         // the K stage of the rotary keys
constexpr int NSTAGE = 5;          // stages that the ring has places for
constexpr int LOADERS = 8;         // loader warps of a CTA
constexpr int KEY_WARPS = 2;       // warps of a CTA that bring rotary keys
// A stage is full with FULL arrivals, half of them for each CTA: a loader's for its part of a K stage and of a V stage, a key
// warp's for its part of the keys.
constexpr int FULL = 8, K_ARRIVE = 1, V_ARRIVE = 2, KEY_ARRIVE = 2;

// A split's tiles, and where their stages lie in the order K(0) K(1) V(0) K(2) V(1) ... V(n - 1): K's rotary keys in the
// middle of its latents (stage ROPE_AT). Of the list's last tile only the first `last_segs` segments hold entries: the others
// are not multiplied with V. (lv, here and below: 1 with the value columns in halves.)
template <int lv>
struct Tiles {
  static constexpr int vstages = (2 * NSEG) >> lv;  // V stages of a whole tile
  int first, n;   // the split's first tile, and how many it has
  int last_segs;  // segments of its last tile
  HS_RING_FN int segs(int t) const { return t == n - 1 ? last_segs : NSEG; }
  HS_RING_FN int v_stages(int t) const { return (2 * segs(t)) >> lv; }
  HS_RING_FN int k_stage(int t) const { return t == 0 ? 0 : t * (KBLK + vstages) - vstages; }
  HS_RING_FN int v_stage(int t) const { return (t + 1) * (KBLK + vstages) - vstages + (t == n - 1 ? 0 : KBLK); }
};

// What loader `wl` has to do with a tile: two jobs of K, 32 of the CTA's rows by 128 columns each, which are two stages; two of
// V, 32 rows by 128 columns each, which are a part of one stage, or one with the value columns in halves.
template <int lv>
struct Loader {
  static constexpr int v_jobs = 2 - lv;
  int wl;
  HS_RING_FN int group() const { return wl >> 2; }
  HS_RING_FN int k_row() const { return (wl & 3) * 32; }  // the first of its rows of the CTA's half of the tile
  HS_RING_FN int v_row() const { return (wl & 1) * 32; }  // of a segment
  HS_RING_FN int v_col() const { return lv ? 0 : (wl >> 1 & 1) * 128; }  // the first of the pair's value columns of its CTA
  HS_RING_FN int k_stage(int job) const { return (ROPE_AT + 1) * job + 2 * group(); }  // and the one after
  HS_RING_FN int segment(int job) const { return (lv ? wl >> 1 : group()) + 2 * job; }
  HS_RING_FN int v_stage(int job) const { return lv ? segment(job) : 2 * segment(job) + v_col() / 128; }
};

}  // namespace hs

#endif  // HS_RING_HPP_
