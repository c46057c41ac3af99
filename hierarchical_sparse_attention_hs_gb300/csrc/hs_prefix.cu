// Attention of a batch over a prefix that all of its requests share, sm_103a (tcgen05 tensor cores, TMA, TMEM).
//
// For request b and head h, over the tokens t < length whose page the pool holds:
//     s[t] = sm_scale * q[b][h] . row_t,   out = sum softmax(s)[t] row_t[0:512],   lse = ln sum e^s[t],
// joined with what the request's own rows gave. The tokens are cut into splits where there are fewer requests than the
// device takes at once; a split leaves its unnormalised output O, its running maximum m (in log2 units) and its
// normaliser l, and a second kernel joins them:
//     M = max m_s,   total = sum 2^(m_s - M) l_s,   out = sum 2^(m_s - M) O_s / total,   lse = ln 2 (M + log2 total),
// where the own rows count as one more split with m = own_lse / ln 2, l = 1, O = own_out.
//
// What bounds it. A row is 1152 bytes and serves 2 * 128 * (576 + 512) operations for each request, 242 per byte: with
// one request the tensor cores and HBM are in balance, with more the tensor cores decide, as long as the rows come from
// L2. Requests of one split run side by side and walk the same rows, so HBM is read about once for all.
//
// A pair of CTAs (a cluster of two) takes one request's 128 heads, 64 for each CTA, over one split, 256 keys a tile. The
// 512 output columns of 128 heads in fp32 would fill a CTA's tensor memory; with 64 heads a CTA they take half (the pair's
// MMAs, cta_group::2 with M = 128, put the two halves of a head's columns on lanes r and r + 64), which leaves room for two
// buffers of scores. For S = Q K^T each CTA holds its 64 heads of Q and 128 of the tile's keys; for O += P V its 64 heads of
// P and all 256 keys of 256 value columns. The MMA reads each CTA's operand half and shares it; the value half of a CTA's
// own keys is loaded twice (K and V are addressed by one descriptor for both CTAs, and their halves cut the rows
// differently). Every MMA has N = 256: one of M = 128 takes 64 cycles there, the full rate, and 47.6 with N = 128 or 64
// (measured), so a tile of 128 keys would run its scores at two thirds of the rate.
//
// Units. A pair walks whole requests, or one of the `nsplit` parts of a request, one after the other; requests are cut only
// as far as the pairs would otherwise run out of even work (cut_of). A pair's tiles form one sequence over all its units:
// the next unit's rows, queries and first scores are under way while the last one's output is stored.
//
// Warp roles per CTA: 0-7 softmax (warp w: TMEM lanes 32 (w % 4) .. +31, that is head lane % 64 and key half lane / 64,
// and keys 64 (w / 4) .. +63 of that half), 8 the issuer (the pair's first CTA issues for both), 9-15 the loaders. K and
// V pass through one ring of 16 KB stages in the order in which the MMAs read them, with a loader for each slot (one
// thread's wait, expectation and copies of a stage take about 310 cycles one after the other, more than the stage's
// MMAs): a K stage is 64 columns of the CTA's 128 keys, a V stage 128 of its value columns of 64 keys; each feeds four
// MMAs, 256 cycles. The issuer runs the scores of tile g + 1 before the value product of tile g, so the softmax of a tile
// overlaps the value product of the one before and the scores of the one after. P is rounded to bf16: one MMA takes
// operands of one type, and V is bf16. Keeping more of P, as a second bf16 operand with what the rounding cuts off, would
// double the value product, 512 of the 1,088 multiplications of a head and key. The rounding leaves an output 0.0010 to
// 0.0013 off in the mean (fp32 outputs, N(0, 1) rows; 0.00007 against the same sum with its weights rounded), against
// 0.0017 of the rounding to a bf16 output. Its normaliser sums the unrounded weights. O is rescaled only when a head's
// maximum has risen by more than 8 (log2), which keeps P below 2^8.
//
// Loads are TMA boxes of 64 columns x min(page_rows, 64) rows, 128-byte swizzle; pages of one or two rows are gathered four
// rows a copy. A box whose page the pool does not hold starts behind the last row of the tensor map: it reads nothing and
// fills with zeros. In the page that the prefix ends inside, boxes of four rows and of one do the same. So rows outside the
// prefix are never read, and a masked key's value row is zero, whatever memory holds; its score is masked to -inf by the
// softmax. Segments of 64 tokens behind the prefix's end are left out altogether.
//
// Measured on one GB300, medians of replayed graphs: 76 requests over 8,192 tokens 100 to 101 us, 1,717 to 1,734
// TFLOP/s, 0.90 of the measured bf16 product; 32 over 65,537 360 to 363 us, 1,610; 100 over 2,047 51 us; 1 over
// 131,072 49 us. Of the first the tensor pipe is active for 71 % of the cycles (under the profiler). L2 gives an SM 71
// bytes a cycle when both SMs of a TPC read different data (116 when they read the same), against the 64 that the full
// rate takes. Nine ring stages instead of seven, with four blocks of Q in tensor memory and one score buffer: 105 us against
// 99 for the first, not kept.
//
// Waits are bounded: on running out a role sets the abort flag, which ends every role, and the HS_DEVERR_TIMEOUT bit.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/hs.h"
#include "hs_internal.hpp"
#include "hs_tcgen05.cuh"

namespace {

using namespace hs;

constexpr int HEADS = 128, DQK = 576, DV = 512, ROW_BYTES = DQK * 2;
constexpr int NK = 256;            // keys of a tile
constexpr int QH = HEADS / 2;      // heads of a CTA
constexpr int KH = NK / 2;         // keys of a CTA's K half
constexpr int DVH = DV / 2;        // value columns of a CTA
constexpr int SEG = 64;            // keys of a segment: the rows of the largest box, and a softmax thread's keys
constexpr int NSEG = NK / SEG;
constexpr int KBLK = DQK / 64;     // 64-column blocks of a row: K stages of a tile
constexpr int BLK_BYTES = 64 * 128;      // 64 rows x 64 columns
constexpr int STAGE_BYTES = 2 * BLK_BYTES;
constexpr int NSTAGE = 7;          // stages of the ring
constexpr int OFF_Q = 0;
constexpr int OFF_RING = OFF_Q + KBLK * BLK_BYTES;
constexpr int OFF_P = OFF_RING + NSTAGE * STAGE_BYTES;
constexpr int OFF_BAR = OFF_P + NSEG * BLK_BYTES;
// mbarriers: qfull full[7] empty[7] sfull[2] sfree[2] pfull pdone drain stall mx[2]
constexpr int B_QFULL = 0, B_FULL = 1, B_EMPTY = B_FULL + NSTAGE, B_SFULL = B_EMPTY + NSTAGE,
              B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2, B_PDONE = B_PFULL + 1, B_DRAIN = B_PDONE + 1,
              B_STALL = B_DRAIN + 1, B_MX = B_STALL + 1, NBAR = B_MX + 2;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;            // tensor-memory address, abort flag
constexpr int OFF_RED = (OFF_MISC + 8 + 15) & ~15;      // [2 parities][NSEG][QH] floats
constexpr int SMEM_BYTES = OFF_RED + 2 * NSEG * QH * 4;
static_assert(NSTAGE <= KBLK, "the ring starts within the first K");
static_assert(SMEM_BYTES <= 232448, "shared memory per block");
constexpr int SOFTMAX_WARPS = 8, MMA_WARP = 8, LOAD_WARP0 = 9, THREADS = (LOAD_WARP0 + NSTAGE) * 32;
static_assert(THREADS <= 512, "128 registers a thread");
constexpr uint32_t TMEM_COLS = 512, TMEM_O = 0, TMEM_S = 256;  // O: 2 x 128 columns; S: two buffers of 128

constexpr int MAX_SPLIT = 128;     // splits of a request

struct PrefixArgs {
  const int32_t* pages;
  int32_t page_shift, max_length;
  int32_t page_limit;     // pages 0 .. page_limit - 1 lie within the rows
  int32_t box_shift;      // log2 of the rows of a box (4 to 64)
  int32_t none;           // a row coordinate behind the last row
  const int32_t* length;  // or nullptr: max_length
  float scale_log2;
  int32_t batch;
  int32_t whole;          // requests 0 .. whole - 1 are one unit each; the others are cut into nsplit units
  int32_t nsplit;
  int32_t units;
  float* part_o;          // [nsplit][batch - whole][HEADS][DV]
  float2* part_ml;        // [nsplit][batch - whole][HEADS]: (m, l)
  const float* own_out;
  const float* own_lse;
  void* out;
  int32_t out_f32;
  float* lse;
  int32_t* err;
  uint32_t wait_limit;
  int32_t stall;
};

__device__ __forceinline__ int length_of(const PrefixArgs& a) {
  return a.length ? min(max(ld_fresh(a.length), 0), a.max_length) : a.max_length;
}
// The prefix's tiles: all of them, and how they are dealt out over the splits: `per` each, one more for the first `more`. Of
// the last tile only the first `last_segs` segments begin within the prefix: the others are neither loaded (their scores
// are masked, whatever the buffer holds) nor multiplied with V.
struct Tiles {
  int n, per, more, last_segs;
  __device__ __forceinline__ int segs(int tile) const { return tile == n - 1 ? last_segs : NSEG; }
};
// A pair's walk over its units (every pairs-th) and their tiles: the same sequence in every role. (Nothing is divided here:
// with divisions in its walks the kernel took a quarter longer, though they would run once a unit.)
struct Walk {
  int u, b, split;  // unit, its request, its split (-1: the request is whole)
  int j0, nt, j;    // the unit's first tile, its tiles, and the tile within it
  __device__ __forceinline__ void set(const PrefixArgs& a, int unit, const Tiles& t) {
    u = b = unit;
    split = -1;
    j = j0 = 0;
    nt = t.n;
    if (u >= a.whole && u < a.units) {
      for (split = 0; b >= a.batch; ++split) b -= a.batch - a.whole;
      nt = t.per + (split < t.more ? 1 : 0);
      j0 = split * t.per + min(split, t.more);
    }
  }
  // the first unit from u on that has tiles; false behind the last
  __device__ __forceinline__ bool settle(const PrefixArgs& a, const Tiles& t) {
    while (u < a.units && nt == 0) set(a, u + (int)(gridDim.x >> 1), t);
    return u < a.units;
  }
  __device__ __forceinline__ bool start(const PrefixArgs& a, const Tiles& t) {
    set(a, (int)(blockIdx.x >> 1), t);
    return settle(a, t);
  }
  __device__ __forceinline__ bool next(const PrefixArgs& a, const Tiles& t) {
    if (++j < nt) return true;
    set(a, u + (int)(gridDim.x >> 1), t);
    return settle(a, t);
  }
};
// Row of token `tok`, or -1.
__device__ __forceinline__ int row_of(const PrefixArgs& a, int tok, int len) {
  if (tok >= len) return -1;
  const int page = a.pages[tok >> a.page_shift];
  return page >= 0 && page < a.page_limit ? (page << a.page_shift) + (tok & ((1 << a.page_shift) - 1)) : -1;
}

// Shared-memory matrix descriptor, 128-byte swizzle. K-major: 8-row groups 1024 bytes apart (lbo unused). MN-major: `lbo`
// between 64-element runs along M or N, 1024 bytes between 8-deep groups along K.
__device__ __forceinline__ uint64_t sdesc128(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// arrive on the barrier at this offset in both CTAs once every MMA issued so far has finished
__device__ __forceinline__ void commit2(uint64_t* b) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(b)),
      "h"((uint16_t)3)
      : "memory");
}
// Arrive on a barrier of the pair's first CTA. What it orders are this thread's tensor-memory reads and shared-memory
// writes before the MMAs that the issuer starts after its wait, which the tcgen05 and proxy fences before it cover; a
// release of cluster scope on top would cost about 870 cycles an arrival (measured).
__device__ __forceinline__ void arrive_lead(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}
// A box at column block `blk` and row `row` into this CTA's shared memory; its bytes count on a barrier of the pair's
// first CTA.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int blk, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(blk)
      : "memory");
}

// Four rows of one column block, from column `col` on, to four consecutive 128-byte rows. (All four exist: see find_rows.)
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int col, const int (&row)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(col), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3])
      : "memory");
}
// The lane's box of a segment of 64 tokens: box u for lane u, of min(page_rows, 64) rows, but of four where pages have
// fewer. Pages are fetched well before they are used, rows worked out from them before the wait for a stage.
struct Box {
  int page[4], row[4];  // [0] alone where the box's rows lie together
  int have;             // rows of the box within the prefix, all of them where it loads as one
};
__device__ __forceinline__ void fetch_pages(const PrefixArgs& a, Box& s, int tok0, int len, int lane) {
  const int tok = tok0 + (lane << a.box_shift);
  s.page[0] = a.pages[min(tok, len - 1) >> a.page_shift];
  if (a.page_shift < 2) {
#pragma unroll
    for (int i = 1; i < 4; ++i) s.page[i] = a.pages[min(tok + i, len - 1) >> a.page_shift];
  }
}
__device__ __forceinline__ void find_rows(const PrefixArgs& a, Box& s, int tok0, int len, int lane) {
  const int tok = tok0 + (lane << a.box_shift), rows = 1 << a.box_shift;
  auto row = [&](int i) {
    const bool on = tok + i < len && s.page[i] >= 0 && s.page[i] < a.page_limit;
    return on ? (s.page[i] << a.page_shift) + ((tok + i) & ((1 << a.page_shift) - 1)) : a.none;
  };
  s.row[0] = row(0);
  s.have = s.row[0] != a.none ? min(rows, len - tok) : rows;
  if (a.page_shift < 2) {
#pragma unroll
    for (int i = 1; i < 4; ++i) s.row[i] = row(i);
    // Four rows are gathered by one copy if the pool holds any of them. A missing one takes the place of one that is there:
    // its weight is 0, and where the row's values are not finite the outputs are not a number either way (such a value
    // makes the row's own score infinite or not a number). Without any the box is one of zeros.
    const int some = min(min(s.row[0], s.row[1]), min(s.row[2], s.row[3]));
    s.have = some != a.none ? 4 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.row[i] = s.row[i] != a.none ? s.row[i] : some;
  }
}
// Loads it: NBLK column blocks from `blk` on to `dst`, where a column block's 64 rows lie together. `map` has boxes of one
// column block, `wide` of NBLK, map1 of one row, `small` of four rows (or, for pages of fewer, gathers four). A box that the
// prefix ends inside is loaded in fours, and row by row where it ends.
template <int NBLK>
__device__ __forceinline__ void load_box(const PrefixArgs& a, const CUtensorMap* map, const CUtensorMap* wide,
                                         const CUtensorMap* map1, const CUtensorMap* small, const Box& s, uint32_t dst,
                                         int blk, uint32_t bar, int lane) {
  if (s.have == SEG) {  // the segment is one box, with its blocks' rows together
    tma_box(dst, wide, blk, s.row[0], bar);
    return;
  }
  const int rows = 1 << a.box_shift;
#pragma unroll 1
  for (int n = 0; n < NBLK; ++n) {
    const uint32_t d = dst + (uint32_t)(n * BLK_BYTES + ((lane << a.box_shift) * 128));
    if (a.page_shift < 2) {
      if (s.have)
        tma_gather4(d, small, (blk + n) * 64, s.row, bar);
      else
        tma_box(d, map, blk + n, a.none, bar);
    } else if (s.have == rows) {
      tma_box(d, map, blk + n, s.row[0], bar);
    } else {
#pragma unroll 1
      for (int r = 0; r < rows; r += 4) {
        if (r + 4 <= s.have || r >= s.have) {
          tma_box(d + r * 128u, small, blk + n, r < s.have ? s.row[0] + r : a.none, bar);
        } else {
          for (int i = r; i < r + 4; ++i) tma_box(d + i * 128u, map1, blk + n, i < s.have ? s.row[0] + i : a.none, bar);
        }
      }
    }
  }
}

// One softmax warp's part of an output without own rows: its 32 heads' columns c_lo .. c_lo + 127 from tensor memory times
// w0 (zeros without O), 128 bytes of every row at a time, staged in `tile` (32 rows of 128 bytes, 16-byte chunk k of row r at
// k ^ (r % 8): no conflicts, and the 128-byte swizzle of `map`) and stored by TMA from (column, row) on. The last copy is
// left in flight: wait_tile_read before the tile is written again and before the kernel ends. (Through registers instead,
// tile to coalesced stores, a unit's 64 KB took 2.7 us a CTA.)
__device__ __forceinline__ void wait_tile_read(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void store_tma(uint32_t tcol, bool have_o, float w0, uint8_t* tile, const CUtensorMap* map,
                                          bool f32, int col, int row, int lane, int c_lo) {
  const int step = f32 ? 32 : 64;
#pragma unroll 1
  for (int c = c_lo; c < c_lo + DVH / 2; c += step) {
    uint32_t w[32];  // the row's 128 bytes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (f32 && h == 1) break;
      uint32_t o[32];
      if (have_o) {
        tmem_ld32(tcol + c + 32 * h, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0;
      }
      if (f32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(o[i]) * w0);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[2 * i]) * w0, __uint_as_float(o[2 * i + 1]) * w0);
          w[16 * h + i] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
    }
    wait_tile_read(lane);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint4*>(tile + lane * 128 + ((i ^ (lane & 7)) << 4)) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    fence_proxy_async();
    __syncwarp();
    if (lane == 0)
      asm volatile(
          "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\t"
          "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
          "r"(su32(tile)), "r"(col + c), "r"(row)
          : "memory");
  }
}

// The same joined with the own rows: plus w1 times their output where w1 != 0. 32-column slices go through the tile so that
// global accesses are whole row segments. `base`: element offset of the warp's first head, first column in out and own.
__device__ __forceinline__ void store_join(uint32_t tcol, bool have_o, float w0, float w1, float* tile, const float* own,
                                           void* out, bool f32, size_t base, int lane, int c_lo) {
  const int c4 = lane & 7;
  uint32_t joined = 0;  // which of the lane's eight rows of a slice have own rows
#pragma unroll
  for (int r = 0; r < 8; ++r) joined |= (__shfl_sync(0xffffffffu, w1, 4 * r + (lane >> 3)) != 0.f ? 1u : 0u) << r;
  float4 p[8];  // the own rows' slice, loaded a slice ahead
  auto load_own = [&](int c) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (joined >> r & 1) p[r] = *reinterpret_cast<const float4*>(own + base + (size_t)(4 * r + (lane >> 3)) * DV + c + 4 * c4);
  };
  load_own(c_lo);
  wait_tile_read(lane);
#pragma unroll 1
  for (int c = c_lo; c < c_lo + DVH / 2; c += 32) {
    uint32_t o[32];
    if (have_o) {
      tmem_ld32(tcol + c, o);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(tile + lane * 32 + ((i ^ (lane & 7)) << 2)) =
          make_float4(__uint_as_float(o[4 * i]) * w0, __uint_as_float(o[4 * i + 1]) * w0,
                      __uint_as_float(o[4 * i + 2]) * w0, __uint_as_float(o[4 * i + 3]) * w0);
    __syncwarp();
    float4 v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int h = 4 * r + (lane >> 3);
      v[r] = *reinterpret_cast<const float4*>(tile + h * 32 + ((c4 ^ (h & 7)) << 2));
      const float w = __shfl_sync(0xffffffffu, w1, h);
      if (joined >> r & 1)
        v[r] = make_float4(fmaf(w, p[r].x, v[r].x), fmaf(w, p[r].y, v[r].y), fmaf(w, p[r].z, v[r].z), fmaf(w, p[r].w, v[r].w));
    }
    __syncwarp();
    if (c + 32 < c_lo + DVH / 2) load_own(c + 32);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const size_t at = base + (size_t)(4 * r + (lane >> 3)) * DV + c + 4 * c4;
      if (f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v[r];
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[r].x, v[r].y), hi = __floats2bfloat162_rn(v[r].z, v[r].w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
}

__global__ void __launch_bounds__(THREADS, 1)
    hs_prefix_kernel(const PrefixArgs a, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap map,
                     const __grid_constant__ CUtensorMap map2, const __grid_constant__ CUtensorMap map1,
                     const __grid_constant__ CUtensorMap small, const __grid_constant__ CUtensorMap omap,
                     const __grid_constant__ CUtensorMap pmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  float* const red = reinterpret_cast<float*>(smem + OFF_RED);
  const int t = threadIdx.x, lane = t & 31;
  const int warp = __shfl_sync(0xffffffffu, t >> 5, 0);  // the same in all lanes, and known to be
  const uint32_t rank = cluster_rank();
  const unsigned lim = a.wait_limit;

  if (t == 32) {  // the copies' descriptors on their way while the barriers are set up
    for (const CUtensorMap* m : {&qmap, &map, &map2, &small, &omap})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (t == 0) {
    for (int i = 0; i < NBAR; ++i) bar_init(bar + i, 1);
    // one arrival for each softmax warp of the pair
    for (int i = 0; i < 2; ++i) bar_init(bar + B_SFREE + i, 2 * SOFTMAX_WARPS);
    bar_init(bar + B_PFULL, 2 * SOFTMAX_WARPS);
    for (int i = 0; i < 2; ++i) bar_init(bar + B_MX + i, NSEG);  // the warps that hold the same heads
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == MMA_WARP)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(smem + OFF_MISC)),
                 "r"(TMEM_COLS)
                 : "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_MISC), 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel's blocks may settle in; they wait for the end

  const int len = length_of(a);
  Tiles tiles;
  tiles.n = (len + NK - 1) / NK;
  tiles.per = tiles.n / a.nsplit;
  tiles.more = tiles.n - tiles.per * a.nsplit;
  tiles.last_segs = (len - (tiles.n - 1) * NK + SEG - 1) / SEG;
  const uint32_t lead = peer_addr(bar, 0);  // the first CTA's barriers
  // test hook: the roles that would start a copy or an MMA first wait on a barrier that nothing completes
  bool ok = true;
  Walk w;

  if (warp == MMA_WARP) {
    // ---- the issuer, of the pair's first CTA. The whole warp walks the loop, so that the descriptors stay in uniform
    //      registers; one lane issues. Tile g of the pair's walk: scores of tile g, then the value product of tile g - 1.
    if (rank == 0) {
      constexpr uint32_t ID_S = idesc_bf16(HEADS, NK, 0, 0), ID_O = idesc_bf16(HEADS, 256, 0, 1);
      const bool leader = elect_one();
      const uint64_t dq = sdesc128(su32(smem + OFF_Q), 0), dp = sdesc128(su32(smem + OFF_P), 0),
                     dk = sdesc128(su32(smem + OFF_RING), 0), dv = sdesc128(su32(smem + OFF_RING), BLK_BYTES);
      int st = 0;
      unsigned ph = 0;
      auto wait = [&](int i, unsigned parity) { return __all_sync(0xffffffffu, bar_wait(bar + i, parity, abort_flag, lim)); };
      // four MMAs on the next stage: A's step of 32 bytes, B's of `step` (in units of 16), then the stage is free
      auto four = [&](uint32_t d, uint64_t oa, uint64_t ob, int step, uint32_t id, uint32_t acc) {
        if (leader) {
          mma2(d, oa, ob, id, acc);
          mma2(d, oa + 2, ob + step, id, 1u);
          mma2(d, oa + 4, ob + 2 * step, id, 1u);
          mma2(d, oa + 6, ob + 3 * step, id, 1u);
          commit2(bar + B_EMPTY + st);
        }
        __syncwarp();
        if (++st == NSTAGE) st = 0, ph ^= 1u;
      };
      ok = !a.stall || wait(B_STALL, 0);
      bool more = w.start(a, tiles), pending = false, pending_first = false;
      int g = 0, nq = 0, pending_v = 0;  // tiles whose scores have been issued, units, V stages of the pending product
      while ((more || pending) && ok) {
        const bool first = w.j == 0;
        if (more) {
          if (first) ok = wait(B_QFULL, (unsigned)nq++ & 1u);
          if (g >= 2) ok = ok && wait(B_SFREE + (g & 1), (unsigned)((g >> 1) - 1) & 1u);
          tc_fence_after();
          for (int c = 0; c < KBLK && ok; ++c) {
            ok = wait(B_FULL + st, ph);
            if (ok) four(tmem + TMEM_S + (uint32_t)(g & 1) * KH, dq + (uint64_t)(c * (BLK_BYTES >> 4)),
                         dk + (uint64_t)(st * (STAGE_BYTES >> 4)), 2, ID_S, c != 0 ? 1u : 0u);
          }
          if (!ok) break;
          if (leader) commit2(bar + B_SFULL + (g & 1));
        }
        if (pending) {
          // P of a unit's first tile comes after the softmax warps have stored the unit before, so O is free too
          ok = wait(B_PFULL, (unsigned)(g - 1) & 1u);
          tc_fence_after();
          for (int c = 0; c < pending_v && ok; ++c) {
            // 64 keys: block c / 2 of P; 128 of the CTA's value columns, 16 rows a step
            ok = wait(B_FULL + st, ph);
            if (ok) four(tmem + TMEM_O + (uint32_t)(c & 1) * 128, dp + (uint64_t)((c >> 1) * (BLK_BYTES >> 4)),
                         dv + (uint64_t)(st * (STAGE_BYTES >> 4)), 128, ID_O, !pending_first || c > 1 ? 1u : 0u);
          }
          if (!ok) break;
          if (leader) commit2(bar + B_PDONE);
        }
        pending = more;
        if (more) {
          pending_first = first;
          pending_v = 2 * tiles.segs(w.j0 + w.j);
          ++g;
          more = w.next(a, tiles);
        }
      }
      __syncwarp();
      if (leader) commit2(bar + B_DRAIN);
    }
    __syncwarp();
  } else if (warp >= LOAD_WARP0) {
    // ---- the loader of ring slot s: every NSTAGE-th stage of K(0) K(1) V(0) K(2) V(1) ... over the tiles of the pair's
    //      walk, the order in which the issuer takes them. Each lane that has boxes walks them by itself; lane 0 of the
    //      first CTA expects both CTAs' bytes. (A stage is full only with every lane's boxes, so no lane falls a round
    //      behind.)
    ok = !a.stall || bar_wait(bar + B_STALL, 0, abort_flag, lim);
    const int s = warp - LOAD_WARP0;
    if ((lane << a.box_shift) < SEG && ok) {
      const uint32_t dst = su32(smem + OFF_RING + s * STAGE_BYTES), fb = lead + (B_FULL + s) * 8;
      Walk v;  // w: the tile whose K is next, v: whose V is
      bool kmore = w.start(a, tiles), vmore = v.start(a, tiles), is_k = true, head = true;
      int c = s;  // the stage's place in its tile's K or V
      // Q of the unit of `x`, and its own rows' output on its way into L2
      auto load_q = [&](const Walk& x) {
        if (lane != 0) return;
        const int row = x.b * HEADS + (int)rank * QH;
        if (rank == 0) bar_arrive_expect(bar + B_QFULL, 2 * KBLK * BLK_BYTES);
        for (int i = 0; i < KBLK; i += 3) tma_box(su32(smem + OFF_Q + i * BLK_BYTES), &qmap, i, row, lead + B_QFULL * 8);
        if (x.split < 0 && a.own_out)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.own_out + (size_t)row * DV), "r"(QH * DV * 4)
                       : "memory");
      };
      bool q_next = false;  // the next unit's Q is this loader's to load, once its slot is free
      // a stage's first token: the CTA's half of the keys, or the segment that the V stage belongs to
      auto first = [&]() { return is_k ? (w.j0 + w.j) * NK + (int)rank * KH : (v.j0 + v.j) * NK + (c >> 1) * SEG; };
      Box p0 = {}, p1 = {};
      if (kmore && s == 0) load_q(w);
      if (kmore) fetch_pages(a, p0, first(), len, lane), fetch_pages(a, p1, first() + SEG, len, lane);
      unsigned ph = 1;  // a barrier that has not completed a phase passes for the parity before its first
      while (vmore) {
        find_rows(a, p0, first(), len, lane);
        if (is_k) find_rows(a, p1, first() + SEG, len, lane);
        const int blk = is_k ? c : (int)rank * (DVH / 64) + (c & 1) * 2;
        // K: 64 columns of every segment within the prefix, each in one of the CTAs
        const uint32_t bytes = is_k ? (uint32_t)tiles.segs(w.j0 + w.j) * BLK_BYTES : 2 * STAGE_BYTES;
        const int here = is_k ? (len - first() + SEG - 1) >> 6 : 0;  // of them in this one (at most two are loaded)
        ok = bar_wait(bar + B_EMPTY + s, ph, abort_flag, lim);  // the MMAs that read the slot have finished
        if (!ok) break;
        ph ^= 1u;
        if (rank == 0 && lane == 0) bar_arrive_expect(bar + B_FULL + s, bytes);
        if (is_k) {
          if (here > 0) load_box<1>(a, &map, &map, &map1, &small, p0, dst, blk, fb, lane);
          if (here > 1) load_box<1>(a, &map, &map, &map1, &small, p1, dst + BLK_BYTES, blk, fb, lane);
        } else {
          load_box<2>(a, &map, &map2, &map1, &small, p0, dst, blk, fb, lane);
        }
        if (q_next) load_q(w);
        // the slot of a unit's last K stage is free when the unit's last scores have been taken, and so is Q
        q_next = is_k && c == KBLK - 1 && w.j + 1 == w.nt;
        c += NSTAGE;
        for (int end; vmore && c >= (end = is_k ? KBLK : 2 * tiles.segs(v.j0 + v.j));) {
          if (is_k) {
            c -= KBLK;
            kmore = w.next(a, tiles);
            q_next = q_next && kmore;
            is_k = head && kmore;
            head = false;
          } else {
            c -= end;
            vmore = v.next(a, tiles);
            is_k = kmore;
          }
        }
        if (vmore) {
          fetch_pages(a, p0, first(), len, lane);
          if (is_k) fetch_pages(a, p1, first() + SEG, len, lane);
        }
      }
    }
    __syncwarp();
  } else {
    // ---- softmax: a thread holds head r of this CTA and 64 keys of every tile, segment sg
    const int q = warp & 3, sub = warp >> 2, r = (q & 1) * 32 + lane, hf = q >> 1, sg = hf * 2 + sub;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
    uint8_t* const prows = smem + OFF_P + sg * BLK_BYTES + (q & 1) * 32 * 128;  // the warp's 32 rows of P
    float m_run = -INFINITY, l_run = 0.f;
    int nx = 0;  // exchanges
    // hands `v` to the other three threads of the head
    auto exchange = [&](float v) {
      float* const share = red + (nx & 1) * NSEG * QH;
      share[sg * QH + r] = v;
      __syncwarp();
      if (lane == 0) bar_arrive(bar + B_MX + (q & 1));
      ok = __all_sync(0xffffffffu, bar_wait(bar + B_MX + (q & 1), (unsigned)nx & 1u, abort_flag, lim)) && ok;
      ++nx;
      return share + r;
    };
    auto key_mask = [&](int tile) {
      const int tok = tile * NK + sg * SEG + lane;
      const unsigned lo = __ballot_sync(0xffffffffu, row_of(a, tok, len) >= 0);
      const unsigned hi = __ballot_sync(0xffffffffu, row_of(a, tok + 32, len) >= 0);
      return (uint64_t)hi << 32 | lo;
    };
    // a unit's output: its part, or the final one, joined with the own rows. The warp's rows of P stage the stores.
    auto finish = [&](int b, int split, bool have_o) {
      const int h0 = (int)rank * QH + (q & 1) * 32;  // the warp's first head
      const bool part = split >= 0;
      const int64_t row = part ? ((int64_t)split * (a.batch - a.whole) + b - a.whole) * HEADS + h0 : (int64_t)b * HEADS + h0;
      float f = 1.f, fo = 0.f;
      if (part) {
        if (sg == 0) a.part_ml[row + lane] = make_float2(m_run, l_run);
        if (!have_o) return;
      } else {
        const float own = a.own_lse ? a.own_lse[row + lane] * 1.4426950408889634f : -INFINITY;
        const float mx = fmaxf(l_run != 0.f ? m_run : -INFINITY, own);
        const float ref = mx == -INFINITY ? 0.f : mx;
        f = l_run != 0.f ? exp2f(m_run == -INFINITY ? 0.f : m_run - ref) : 0.f;
        fo = own != -INFINITY ? exp2f(own - ref) : 0.f;
        const float total = fmaf(f, l_run, fo);
        const float inv = total != 0.f ? 1.f / total : 0.f;
        f *= inv;
        fo = fo != 0.f ? fo * inv : 0.f;  // (0 itself without own rows, not 0 times a reciprocal that may be NaN)
        if (a.own_lse) exchange(0.f);     // all threads of a head have read own_lse, which may be lse itself
        if (sg == 0) a.lse[row + lane] = total != 0.f ? (ref + log2f(total)) * 0.6931471805599453f : -INFINITY;
      }
      if (__any_sync(0xffffffffu, fo != 0.f))
        store_join(trow + TMEM_O, have_o, f, fo, reinterpret_cast<float*>(prows), a.own_out, a.out, a.out_f32 != 0,
                   (size_t)row * DV + hf * DVH, lane, sub * (DVH / 2));
      else
        store_tma(trow + TMEM_O, have_o, f, prows, part ? &pmap : &omap, part || a.out_f32 != 0, hf * DVH, (int)row, lane,
                  sub * (DVH / 2));
    };
    const float scale = a.scale_log2 > 0.f ? a.scale_log2 : 1.f;  // the maximum is taken before the scale: see below
    int g = 0;  // tiles of the pair's walk
    w.set(a, (int)(blockIdx.x >> 1), tiles);
    while (w.u < a.units && ok) {
      m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < w.nt; ++j, ++g) {
        const uint64_t mask = key_mask(w.j0 + j);
        ok = __all_sync(0xffffffffu, bar_wait(bar + B_SFULL + (g & 1), (unsigned)(g >> 1) & 1u, abort_flag, lim));
        if (!ok) break;
        tc_fence_after();
        // The scores are read twice, 32 at a time: for the maximum, and once the four threads of a head agree on it. (Holding
        // all 64 across the exchange takes more registers than 16 warps leave.)
        const uint32_t scol = trow + TMEM_S + (uint32_t)((g & 1) * KH + sub * SEG);
        uint32_t sv[32];
        float mb = -INFINITY;
        // 32 of the thread's scores before the scale, -inf without a row. (A scale that is not positive is applied here,
        // and is 1 later.) Both conditions are the same in all lanes.
        auto load32 = [&](int h) {
          tmem_ld32(scol + 32 * h, sv);
          tmem_wait_ld();
          if (!(a.scale_log2 > 0.f)) {
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[i] = __float_as_uint(__uint_as_float(sv[i]) * a.scale_log2);
          }
          const uint32_t m32 = (uint32_t)(mask >> (32 * h));
          if (~m32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) sv[i] = m32 >> i & 1 ? sv[i] : 0xff800000u;
          }
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load32(h);
#pragma unroll
          for (int i = 0; i < 32; ++i) mb = fmaxf(mb, __uint_as_float(sv[i]));
        }
        const float* share = exchange(mb);
        if (!ok) break;
        mb = scale * fmaxf(fmaxf(share[0], share[QH]), fmaxf(share[2 * QH], share[3 * QH]));
        float m_new = m_run;
        if (mb > -INFINITY && (m_run == -INFINITY || mb > m_run + 8.f)) m_new = mb;
        const bool resc = m_new != m_run && m_run != -INFINITY;
        const float ref = m_new == -INFINITY ? 0.f : m_new;  // no finite score yet: nothing to subtract, a NaN still shows
        float sum[2] = {0.f, 0.f};
        uint32_t p[SEG / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          load32(h);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float p0 = ex2_approx(fmaf(__uint_as_float(sv[2 * i]), scale, -ref)),
                        p1 = ex2_approx(fmaf(__uint_as_float(sv[2 * i + 1]), scale, -ref));
            sum[i & 1] += p0 + p1;
            const __nv_bfloat162 v = __floats2bfloat162_rn(p0, p1);
            p[16 * h + i] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead(lead + (B_SFREE + (g & 1)) * 8);
        // P's buffer is free, and O holds the tiles before, once the value product of the tile before has finished
        if (g >= 1) {
          ok = __all_sync(0xffffffffu, bar_wait(bar + B_PDONE, (unsigned)(g - 1) & 1u, abort_flag, lim));
          if (!ok) break;
        }
        if (__any_sync(0xffffffffu, resc)) {
          // each of the two threads with the same lane takes half of its columns
          tc_fence_after();
          const float f = resc ? ex2_approx(m_run - m_new) : 1.f;
#pragma unroll 1
          for (int c = sub * (DVH / 2); c < (sub + 1) * (DVH / 2); c += 16) {
            float o[16];
            tmem_ld16(trow + TMEM_O + c, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st16(trow + TMEM_O + c, o);
          }
          tmem_wait_st();
          l_run *= f;
        }
        m_run = m_new;
        l_run += sum[0] + sum[1];
        if (j == 0) wait_tile_read(lane);  // the stores of the unit before are staged in the warp's rows of P
#pragma unroll
        for (int c = 0; c < SEG / 8; ++c)
          *reinterpret_cast<uint4*>(prows + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead(lead + B_PFULL * 8);
      }
      if (!ok) break;
      const int b = w.b, split = w.split;
      const bool have_o = w.nt > 0;
      w.set(a, w.u + (int)(gridDim.x >> 1), tiles);
      if (have_o) {
        ok = __all_sync(0xffffffffu, bar_wait(bar + B_PDONE, (unsigned)(g - 1) & 1u, abort_flag, lim));
        if (!ok) break;
        const float* const share = exchange(l_run);
        if (!ok) break;
        l_run = (share[0] + share[QH]) + (share[2 * QH] + share[3 * QH]);
        tc_fence_after();
      }
      finish(b, split, have_o);
      tc_fence_before();
    }
    wait_tile_read(lane);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {  // every MMA has finished before the tensor memory is freed, after an abort too
    bool drained = bar_test(bar + B_DRAIN, 0);
    for (const uint64_t t0 = now_ns(); !drained && now_ns() - t0 < WAIT_NS;) drained = bar_test(bar + B_DRAIN, 0);
    if (!drained) *abort_flag = 1;
    __syncwarp();
    if (*abort_flag) {
      // a wait ran out: let the copies in flight land before the shared memory goes, and report
      for (int i = 0; i < 50; ++i) __nanosleep(1000);
      if (lane == 0) atomicOr(a.err, HS_DEVERR_TIMEOUT);
    }
    __syncwarp();
  }
  cluster_sync();
  tc_fence_after();
  if (warp == MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
}

// One CTA joins one head of one request: thread t of a group of 128 holds outputs 4t .. 4t + 3 of every G-th split, four
// loads in flight; the groups' sums meet in shared memory. Every warp works the splits' weights out for itself (lane u:
// splits u, u + 32, ...), so that nothing else waits for the block. Up to 16 splits one group does; more of them are
// divided over four (a single group walking 74 splits took 40 us for one request: a chain of latencies).
template <int G>
__global__ void __launch_bounds__(G * DV / 4) hs_prefix_join_kernel(const PrefixArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ float4 part[G > 1 ? G - 1 : 1][DV / 4];
  constexpr int PER = G > 1 ? MAX_SPLIT / 32 : 1;  // splits of a lane
  const int t = threadIdx.x & (DV / 4 - 1), g = threadIdx.x / (DV / 4), lane = threadIdx.x & 31, n = a.nsplit;
  const size_t part_row = blockIdx.x, heads = (size_t)(a.batch - a.whole) * HEADS, bh = (size_t)a.whole * HEADS + part_row;
  const float own = a.own_lse ? a.own_lse[bh] * 1.4426950408889634f : -INFINITY;
  float2 ml[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i)
    ml[i] = lane + 32 * i < n ? a.part_ml[(size_t)(lane + 32 * i) * heads + part_row] : make_float2(0.f, 0.f);
  float mx = own;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (ml[i].y != 0.f) mx = fmaxf(mx, ml[i].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  float weight[PER], total = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {  // a split with no row: no weight, and no output to read
    weight[i] = ml[i].y != 0.f ? exp2f(ml[i].x == -INFINITY ? 0.f : ml[i].x - ref) : 0.f;
    total += ml[i].y != 0.f ? weight[i] * ml[i].y : 0.f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const float wo = own != -INFINITY ? exp2f(own - ref) : 0.f;
  total += wo;
  const float inv = total != 0.f ? 1.f / total : 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, float4 v) {
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  };
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    for (int s0 = 32 * i + g; s0 < min(n, 32 * i + 32); s0 += 4 * G) {
      float w[4];
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int s = s0 + u * G;
        w[u] = __shfl_sync(0xffffffffu, weight[i], s & 31);
        if (s >= 32 * i + 32) w[u] = 0.f;
        if (w[u] != 0.f) v[u] = __ldcs(reinterpret_cast<const float4*>(a.part_o + ((size_t)s * heads + part_row) * DV) + t);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (w[u] != 0.f) add(w[u], v[u]);
    }
  }
  if (g == 0 && wo != 0.f) add(wo, *(reinterpret_cast<const float4*>(a.own_out + bh * DV) + t));
  if (G > 1 && g > 0) part[g - 1][t] = o;
  __syncthreads();  // (and every thread has read own_lse, which may be lse itself)
  if (g > 0) return;
#pragma unroll
  for (int i = 0; i < G - 1; ++i) add(1.f, part[i][t]);
  o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (a.out_f32) {
    reinterpret_cast<float4*>(static_cast<float*>(a.out) + bh * DV)[t] = o;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + bh * DV)[t] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
  if (t == 0) a.lse[bh] = total != 0.f ? (ref + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

// How many pairs the current device holds at once, cached per device.
int pairs_resident() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n) return n;
  if (cudaFuncSetAttribute(hs_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, hs_prefix_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

// How a batch is cut into units: requests 0 .. whole - 1 are one unit each, the others `nsplit` units.
struct Cut {
  static constexpr size_t SPLIT_BYTES = HEADS * (DV * sizeof(float) + sizeof(float2));  // of one split of one request
  int whole, nsplit;
  size_t workspace(int batch) const { return nsplit > 1 ? (size_t)nsplit * (size_t)(batch - whole) * SPLIT_BYTES : 0; }
  // The most that any cut_of takes for up to this batch and length: a request has at most as many splits as tiles and
  // MAX_SPLIT, and all splits together are at most 4 * pairs.
  static size_t most(int pairs, int32_t batch, int32_t max_length) {
    const int tiles = (max_length + NK - 1) / NK;
    return tiles < 2 ? 0 : (size_t)std::min<int64_t>(4 * pairs, (int64_t)batch * std::min(tiles, MAX_SPLIT)) * SPLIT_BYTES;
  }
};
// The cut with the shortest expected time, in tiles (1.2 to 2.6 us): a pair's units one after the other, each its tiles and
// about one more (the softmax of its last tile and its store), and with splits their join, 1.5 and 0.025 for each. (What every
// launch pays counts for all cuts alike and is left out.) Either all requests are cut, or as many as fill the pairs whole
// times over stay whole and the rest is cut.
Cut cut_of(int pairs, int32_t batch, int32_t max_length) {
  const int tiles = (max_length + NK - 1) / NK, full = batch / pairs * pairs;
  Cut best = {batch, 1};
  double least = (double)((batch + pairs - 1) / pairs) * (tiles + 1);
  for (int whole = 0;; whole = full) {
    const int rest = batch - whole;
    for (int n = 2; rest > 0 && n <= std::min({tiles, MAX_SPLIT, 4 * pairs / rest}); ++n) {
      const int64_t units = (int64_t)rest * n;
      const double cost = (double)(whole / pairs) * (tiles + 1) +
                          (double)((units + pairs - 1) / pairs) * ((tiles + n - 1) / n + 1) + 1.5 + 0.025 * units;
      if (cost < least) least = cost, best = {whole, n};
    }
    if (whole == full) break;
  }
  return best;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeFn>(p);
  fn.store(f, std::memory_order_release);
  return f;
}
// Rows of 576 bf16 values as (column, row, 64-column block): boxes of 64 columns x `box` rows x `blocks` blocks, which lie
// block by block in shared memory, 128-byte swizzle, zeros outside.
bool make_map(EncodeFn f, CUtensorMap* m, const void* rows, uint64_t count, uint32_t box, uint32_t blocks) {
  const cuuint64_t dims[3] = {64, count, KBLK}, strides[2] = {ROW_BYTES, 128};
  const cuuint32_t boxes[3] = {64, box, blocks}, steps[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(rows), dims, strides, boxes, steps,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same rows as (column, row), for gathering: a box is 64 columns of one row.
bool make_gather_map(EncodeFn f, CUtensorMap* m, const void* rows, uint64_t count) {
  const cuuint64_t dims[2] = {DQK, count}, strides[1] = {ROW_BYTES};
  const cuuint32_t boxes[2] = {64, 1}, steps[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(rows), dims, strides, boxes, steps,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Outputs as (column, row): boxes of 128 bytes x 32 rows, 128-byte swizzle.
bool make_out_map(EncodeFn f, CUtensorMap* m, void* out, uint64_t rows, bool f32) {
  const cuuint64_t dims[2] = {DV, rows}, strides[1] = {(cuuint64_t)DV * (f32 ? 4 : 2)};
  const cuuint32_t boxes[2] = {f32 ? 32u : 64u, 32}, steps[2] = {1, 1};
  return f(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, boxes, steps,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" size_t hs_mla_prefix_workspace(hs_pool* pool, int32_t batch, int32_t max_length) {
  if (!pool || batch <= 0 || max_length < 0 || max_length > 1 << 30 || batch > (1 << 24) / HEADS || !hs_on_device(pool)) return 0;
  const int pairs = pairs_resident();
  return pairs > 0 ? cut_of(pairs, batch, max_length).workspace(batch) : 0;
}

extern "C" int hs_mla_prefix_workspace_bound(hs_pool* pool, int32_t batch, int32_t max_length, size_t* bytes) {
  if (!bytes) return HS_ERR_INVALID_ARG;
  *bytes = 0;
  if (!pool || batch < 0 || batch > (1 << 24) / HEADS || max_length < 0 || max_length > 1 << 30 || !hs_on_device(pool))
    return HS_ERR_INVALID_ARG;
  const int pairs = pairs_resident();
  if (pairs < 1) return HS_ERR_UNSUPPORTED;
  *bytes = Cut::most(pairs, batch, max_length);
  return HS_OK;
}

extern "C" int hs_mla_prefix(hs_pool* pool, int32_t batch, const void* q, const hs_paged_rows* prefix,
                             int32_t max_length, const int32_t* prefix_length, float sm_scale, const float* own_out,
                             const float* own_lse, void* out, int32_t out_type, float* lse, void* workspace,
                             size_t workspace_bytes, hs_stream_t stream) {
  const auto aligned = [](const void* p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!pool || !prefix || batch < 0 || batch > (1 << 24) / HEADS || max_length < 0 || max_length > 1 << 30 || !hs_paged_ok(prefix) ||
      ((int64_t)max_length + prefix->page_rows - 1) / prefix->page_rows > prefix->page_stride ||
      (out_type != HS_TYPE_BF16 && out_type != HS_TYPE_F32) ||
      (own_out != nullptr) != (own_lse != nullptr))
    return HS_ERR_INVALID_ARG;
  if (pool->d.row_bytes != ROW_BYTES) return HS_ERR_UNSUPPORTED;
  if (batch == 0) return HS_OK;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || (own_out && (!aligned(own_out, 16) || !aligned(own_lse, 4))) ||
      (prefix_length && !aligned(prefix_length, 4)) || !hs_on_device(pool))
    return HS_ERR_INVALID_ARG;
  const int pairs = pairs_resident();
  const EncodeFn encode = encoder();
  if (pairs < 1 || !encode) return HS_ERR_UNSUPPORTED;
  const Cut cut = cut_of(pairs, batch, max_length);
  const size_t need = cut.workspace(batch);
  if (need && (!aligned(workspace, 256) || workspace_bytes < need)) return HS_ERR_INVALID_ARG;

  PrefixArgs a;
  std::memset(&a, 0, sizeof(a));
  a.pages = prefix->pages;
  while ((1 << a.page_shift) < prefix->page_rows) ++a.page_shift;
  a.box_shift = std::max(2, std::min(a.page_shift, 6));
  a.max_length = max_length;
  a.page_limit = (int32_t)(prefix->count / prefix->page_rows);
  a.none = (int32_t)prefix->count;
  a.length = prefix_length;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.batch = batch;
  const int rest = batch - cut.whole;
  a.whole = cut.whole;
  a.nsplit = cut.nsplit;
  a.units = cut.whole + rest * cut.nsplit;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = rest ? reinterpret_cast<float2*>(a.part_o + (size_t)cut.nsplit * rest * HEADS * DV) : nullptr;
  a.own_out = own_out;
  a.own_lse = own_lse;
  a.out = out;
  a.out_f32 = out_type == HS_TYPE_F32;
  a.lse = lse;
  a.err = pool->err;
  hs_attention_waits(&a.wait_limit, &a.stall);
  CUtensorMap qmap, map, map2, map1, small, omap, pmap;
  // an empty pool of rows still needs a map: one row, which page_limit = 0 keeps from being read
  const uint64_t count = std::max<int64_t>(prefix->count, 1);
  a.none = (int32_t)count;
  if (!make_map(encode, &qmap, q, (uint64_t)batch * HEADS, QH, 3) ||
      !make_map(encode, &map, prefix->rows, count, 1u << a.box_shift, 1) ||
      !make_map(encode, &map2, prefix->rows, count, 1u << a.box_shift, 2) || !make_map(encode, &map1, prefix->rows, count, 1, 1) ||
      !(a.page_shift < 2 ? make_gather_map(encode, &small, prefix->rows, count)
                         : make_map(encode, &small, prefix->rows, count, 4, 1)) ||
      !make_out_map(encode, &omap, out, (uint64_t)batch * HEADS, a.out_f32 != 0) ||
      !make_out_map(encode, &pmap, rest ? workspace : out, (uint64_t)(rest ? rest * cut.nsplit : batch) * HEADS, rest || a.out_f32))
    return HS_ERR_INVALID_ARG;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min(a.units, pairs)), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const int rc = hs_launched(cudaLaunchKernelEx(&cfg, hs_prefix_kernel, a, qmap, map, map2, map1, small, omap, pmap));
  if (rc != HS_OK || !rest) return rc;
  cfg.gridDim = dim3((unsigned)rest * HEADS, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  const int groups = cut.nsplit <= 16 ? 1 : 4;
  cfg.blockDim = dim3((unsigned)groups * DV / 4, 1, 1);
  return hs_launched(groups == 1 ? cudaLaunchKernelEx(&cfg, hs_prefix_join_kernel<1>, a)
                                 : cudaLaunchKernelEx(&cfg, hs_prefix_join_kernel<4>, a));
}
