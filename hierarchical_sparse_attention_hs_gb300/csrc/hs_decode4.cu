// Sparse MLA decode attention over 4-bit rows, sm_103a (tcgen05 tensor cores, TMEM).
//
// For request b and head h, over the rows that the request's list names:
//     s[i] = sm_scale * q[b][h] . row_i,   out = sum softmax(s)[i] row_i[0:512],   lse = ln sum e^s[i],
// the rows' latents being number times scale (hs_rows.cuh).
//
// What bounds it. A row is 416 bytes and serves 2 * 128 * (576 + 512) operations, 670 a byte: the tensor cores and the shared
// memory that feeds them. A decode step's lists are short, though, and much of its time is the chain of one launch: the
// list, the rows it names, the first scores, and at the end the last product, its store and the join of splits.
//
// Operands, all of them exact. For the scores the rows' latents become bf16, beside the queries and rotary keys that are; for
// the value product they become halves, at 2^-6 of their value, beside weights in halves. Rounding the weights, 2^-11 of
// each (2^-31 of the largest, for those far below it), leaves an output 0.00014 off in the mean, a tenth of its own rounding
// to bf16; weights in bf16 would leave 0.0011.
//
// A pair of CTAs takes one request's 128 heads, 64 for each CTA, over one split of its list, 256 entries a tile, with MMAs
// of M = 128, N = 256 that both run together (cta_group::2): for S = Q K^T each CTA holds its 64 heads of Q and 128 of the
// tile's rows, for O += P V its 64 heads of P and all 256 rows of 256 value columns. So the latents are unpacked 1.9 times:
// once as K, and those of the half of the columns that a CTA has as V again.
//
// A request is cut where pairs would otherwise be left over (cut_of): its list into 1, 2, 4 or 8 splits, and a split's value
// columns into halves, whose two pairs take 128 columns a CTA and both work out all scores. Halves do not have to be joined,
// and make what splits join half as large. A cluster of up to eight pairs leaves the splits' outputs in shared memory,
// unnormalised, with each head's maximum and normaliser, and joins them:
//     M = max m_s,   total = sum 2^(m_s - M) l_s,   out = sum 2^(m_s - M) O_s / total,   lse = ln 2 (M + log2 total).
//
// Warp roles per CTA: 0-7 softmax (warp w: TMEM lanes 32 (w % 4) .. +31, that is head lane % 64 and half lane / 64 of the
// tile's rows, and rows 64 (w / 4) .. +63 of that half), 8 the issuer (the pair's first CTA issues for both), 9-16 the
// loaders, which unpack latents, 17 and 18 the rotary keys. K and V pass through one ring of 16 KB stages in the order in which
// the MMAs read them (hs_ring.hpp): a K stage is 64 columns of the CTA's 128 rows, a V stage 128 of its value columns of 64
// rows, both 128 rows of 128 bytes, 128-byte swizzle; each feeds four MMAs, 256 cycles. The rows' words come into shared memory
// as they are, by asynchronous copies a job ahead (through registers they were waited for as soon as they were asked for), and
// are unpacked from there.
//
// Measured on one GB300 (replayed graphs): a tile takes 4.1 us, 7,700 cycles, of which its MMAs are 4,352 at their full rate.
// Shared memory is what it waits for: 2,200 cycles of stores of unpacked rows, 1,100 of the words' way through it, and 96 of
// its 128 bytes a cycle that MMAs of this shape read while they run, 3,300 or more. 32 requests of 2,048 entries 27.8 us (657
// TFLOP/s; four tiles a pair, the start, the join), one 14.4, seven 16.3, five of 16,384 45.5, one of 65 8.3. Outputs in fp32 0.1 to
// 0.6 us more; the list in mapped host memory, which each role of a CTA reads for itself, 0.9 us more for one request of 2,048, 6.6
// for 32; rows in host memory 26 and 313 us (87 GB/s of rows for 32 requests).
//
// Where it leaves SMs idle: a list is cut into at most eight splits, since they join within one cluster, so a request has at most
// 16 of 152 SMs (five of 16,384: 80), and splits are powers of two (40 requests of 2,048: one split each, 80 SMs, 39.9 us).
//
// Steps that brought it there, for 32 requests of 2,048: lanes that load a row each 62 us; eight rows by four lanes 40; copies
// into shared memory, scores in bf16, queries by TMA 34; jobs of 32 rows in a fixed order, the keys by warps of their own
// 29.1; the code of a loader's two jobs and of the join once each, 78 KB for 94 (what a launch runs once waits for its
// instructions) 28.0. Halves of the value columns: one request of 2,048 14.7 from 15.3, of 1,000 12.0 from 14.4, of 65 8.2
// from 9.1; as an argument in place of a template's the others took 28.4 to 28.7.
//
// Not kept: eleven loaders with 96 registers or fewer that take jobs in turn, 30.2 (and a wait that could be lapped); all
// loaders on one stage pair, 16 rows each, 36; rows brought into L2 by bulk prefetches, whose issue took a warp 2,000 cycles
// for 32; first copies ahead of the cluster's start, 29.2 against 28.9 (programmatic launch hides that start already); a job's
// copies started after the job before is unpacked, 29.5 against 28.2; waits as calls of a function 28.7; the join by bulk copies
// into the CTA that sums a head, 31.
//
// Waits are bounded: on running out a role sets the abort flag, which ends every role, and the HS_DEVERR_TIMEOUT bit.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/hs.h"
#include "hs_internal.hpp"
#include "hs_load.cuh"
#include "hs_pair.cuh"
#include "hs_ring.hpp"
#include "hs_rows.cuh"
#include "hs_source.hpp"

namespace {

using namespace hs;

constexpr int HEADS = 128;
constexpr int NK = 256;            // rows of a tile
constexpr int QH = HEADS / 2;      // heads of a CTA
constexpr int KH = NK / 2;         // rows of a CTA's K half
constexpr int DVH = LATENT / 2;    // value columns of a CTA
static_assert(SEG * NSEG == NK, "a softmax thread's rows of a tile are a segment");
static_assert(KBLK * 64 == WIDTH, "a stage's columns");
constexpr int BLK_BYTES = 64 * 128;      // 64 rows x 64 columns
constexpr int STAGE_BYTES = 2 * BLK_BYTES;
constexpr int OFF_Q = 0;
constexpr int OFF_RING = OFF_Q + KBLK * BLK_BYTES;
constexpr int OFF_P = OFF_RING + NSTAGE * STAGE_BYTES;
constexpr int SOFTMAX_WARPS = 8, MMA_WARP = 8, LOAD_WARP0 = 9, KEY_WARP = LOAD_WARP0 + LOADERS,
              THREADS = (KEY_WARP + KEY_WARPS) * 32;
static_assert(THREADS <= 640, "96 registers a thread: five warps a scheduler");
// A loader's two jobs as their rows are in memory, 64 bytes of codes (row r: 16-byte chunk j at j ^ (r / 2 % 4)) and eight scales
// each.
constexpr int RAW_CODES = 32 * 64, RAW_JOB = RAW_CODES + 32 * 8;
constexpr int OFF_RAW = OFF_P + NSEG * BLK_BYTES;
constexpr int OFF_BAR = OFF_RAW + LOADERS * 2 * RAW_JOB;
// mbarriers: qfull full[] empty[] sfull[2] sfree[2] pfull pdone drain stall mx[2]
constexpr int B_QFULL = 0, B_FULL = 1, B_EMPTY = B_FULL + NSTAGE, B_SFULL = B_EMPTY + NSTAGE,
              B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2, B_PDONE = B_PFULL + 1, B_DRAIN = B_PDONE + 1,
              B_STALL = B_DRAIN + 1, B_MX = B_STALL + 1, NBAR = B_MX + 2;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;            // tensor-memory address, abort flag, the softmax warps' own
constexpr int OFF_RED = (OFF_MISC + 12 + 15) & ~15;     // [2 parities][NSEG][QH] floats
constexpr int OFF_ML = OFF_RED + 2 * NSEG * QH * 4;     // [QH] (m, l) of a split
constexpr int SMEM_BYTES = OFF_ML + QH * 8;
static_assert(SMEM_BYTES <= 232448, "shared memory per block");
constexpr uint32_t TMEM_COLS = 512, TMEM_O = 0, TMEM_S = 256;  // O: 2 x 128 columns; S: two buffers of 128
// A CTA's outputs take the place of Q and the ring: rows of a head, 16 bytes apart beyond their own size (no bank conflicts).
constexpr int OUT_F32 = LATENT * 4 + 16, OUT_BF16 = LATENT * 2 + 16;
static_assert(QH * OUT_F32 <= OFF_P, "a CTA's outputs fit in front of P");
constexpr int MAX_PAIRS_LOG = 3;  // of a cluster: 16 CTAs
constexpr float P_SHIFT = 6.f;  // weights are kept at 2^6: their smallest half is then 2^-30 of a weight of the maximum's
constexpr float UNSCALE = 64.f;  // latents are kept at 2^-6

struct Decode4Args {
  const int32_t* idx;  // [batch][k]
  int32_t k;
  RowSource src;
  float scale_log2;    // sm_scale * log2(e)
  int32_t nsplit;      // splits of the list
  void* out;
  int32_t out_f32;
  float* lse;
  int32_t* err;
  uint32_t wait_limit;
  int32_t stall;
};

__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, int a_mn, int b_mn) {
  return idesc_bf16(m, n, a_mn, b_mn) & ~(1u << 7 | 1u << 10);
}
// Copies into shared memory (volatile: they stay behind the launch wait).
__device__ __forceinline__ void copy16(uint32_t dst, unsigned long long src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, unsigned long long src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float4 ld_peer(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// 32 latents of a row, unpacked into four of the eight 16-byte chunks of a stage's row, from chunk ch on: as bf16 for the
// scores, as halves at 2^-6 for the values.
template <bool K>
__device__ __forceinline__ void unpack(uint8_t* row, int swizzle, int ch, uint4 codes, uint32_t scales) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t code = g ? scales >> 8 : scales & 255u;
    std::conditional_t<K, Int4Bf16, Int4Half> k;
    k.set(code);
#pragma unroll
    for (int i = 2 * g; i < 2 * g + 2; ++i) {
      uint4 v;
      if constexpr (K) {
        const __nv_bfloat162 h[4] = {int4_pair(w[i], k), int4_pair(w[i] >> 4, k), int4_pair(w[i] >> 8, k),
                                     int4_pair(w[i] >> 12, k)};
        v = *reinterpret_cast<const uint4*>(h);
      } else {
        const __half2 h[4] = {int4_pair<0>(w[i], k), int4_pair<1>(w[i], k), int4_pair<0>(w[i] >> 8, k),
                              int4_pair<1>(w[i] >> 8, k)};
        v = *reinterpret_cast<const uint4*>(h);
      }
      *reinterpret_cast<uint4*>(row + (((ch + i) ^ swizzle) << 4)) = v;
    }
  }
}

template <int lv>
__global__ void __launch_bounds__(THREADS, 1) hs_decode4_kernel(const Decode4Args a, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* const bar = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  volatile int* const out_stop = abort_flag + 1;
  float* const red = reinterpret_cast<float*>(smem + OFF_RED);
  const int t = threadIdx.x, lane = t & 31;
  const int warp = __shfl_sync(0xffffffffu, t >> 5, 0);  // the same in all lanes, and known to be
  const uint32_t crank = cluster_rank(), rank = crank & 1u, first = crank & ~1u;
  const unsigned lim = a.wait_limit;

  if (t == 0) {
    for (int i = 0; i < NBAR; ++i) bar_init(bar + i, 1);
    // one arrival for each softmax warp of the pair
    for (int i = 0; i < NSTAGE; ++i) bar_init(bar + B_FULL + i, FULL);
    for (int i = 0; i < 2; ++i) bar_init(bar + B_SFREE + i, 2 * SOFTMAX_WARPS);
    bar_init(bar + B_PFULL, 2 * SOFTMAX_WARPS);
    for (int i = 0; i < 2; ++i) bar_init(bar + B_MX + i, NSEG);  // the warps that hold the same heads
    *abort_flag = *out_stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == MMA_WARP)
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(smem + OFF_MISC)),
                 "r"(TMEM_COLS)
                 : "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_MISC), 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  const int half = (int)(crank >> 1) & lv;  // the pair's half of the value columns
  const uint32_t b = blockIdx.x / (uint32_t)((2 * a.nsplit) << lv);
  const int split = (int)(crank >> 1) >> lv, all = (a.k + NK - 1) / NK, per = all / a.nsplit, more = all - per * a.nsplit;
  Tiles<lv> tiles;
  tiles.n = per + (split < more ? 1 : 0);
  tiles.first = split * per + min(split, more);
  tiles.last_segs = min(NSEG, (a.k - (tiles.first + tiles.n - 1) * NK + SEG - 1) / SEG);
  const int32_t* const list = a.idx + (size_t)b * a.k;
  const uint32_t lead = peer_addr(bar, first);  // the first CTA's barriers
  // test hook: the roles that would start a copy or an MMA first wait on a barrier that nothing completes
  bool ok = true;
  if (warp == MMA_WARP) {
    // ---- the issuer, of the pair's first CTA. The whole warp walks the loop, so that the descriptors stay in uniform
    //      registers; one lane issues: scores of tile g, then the value product of tile g - 1.
    if (rank == 0) {
      constexpr uint32_t ID_S = idesc_bf16(HEADS, NK, 0, 0), ID_O = idesc_f16(HEADS, 256, 0, 1);
      const bool leader = elect_one();
      const uint32_t both = 3u << first;
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
          commit2(bar + B_EMPTY + st, both);
        }
        __syncwarp();
        if (++st == NSTAGE) st = 0, ph ^= 1u;
      };
      ok = (!a.stall || wait(B_STALL, 0)) && wait(B_QFULL, 0);
      for (int g = 0; g <= tiles.n && ok; ++g) {
        if (g < tiles.n) {
          if (g >= 2) ok = wait(B_SFREE + (g & 1), (unsigned)((g >> 1) - 1) & 1u);
          tc_fence_after();
          for (int c = 0; c < KBLK && ok; ++c) {
            ok = wait(B_FULL + st, ph);
            tc_fence_after();
            const int blk = c < ROPE_AT ? c : c == ROPE_AT ? KBLK - 1 : c - 1;
            if (ok) four(tmem + TMEM_S + (uint32_t)(g & 1) * KH, dq + (uint64_t)(blk * (BLK_BYTES >> 4)),
                         dk + (uint64_t)(st * (STAGE_BYTES >> 4)), 2, ID_S, c != 0 ? 1u : 0u);
          }
          if (!ok) break;
          if (leader) commit2(bar + B_SFULL + (g & 1), both);
        }
        if (g >= 1) {
          ok = wait(B_PFULL, (unsigned)(g - 1) & 1u);
          tc_fence_after();
          const int nv = tiles.v_stages(g - 1), two = 1 - lv;
          for (int c = 0; c < nv && ok; ++c) {
            // 64 rows: a block of P; 128 of the CTA's value columns, 16 rows a step
            ok = wait(B_FULL + st, ph);
            tc_fence_after();
            if (ok) four(tmem + TMEM_O + (uint32_t)(c & two) * 128, dp + (uint64_t)((c >> two) * (BLK_BYTES >> 4)),
                         dv + (uint64_t)(st * (STAGE_BYTES >> 4)), 128, ID_O, g > 1 || c > two ? 1u : 0u);
          }
          if (!ok) break;
          if (leader) commit2(bar + B_PDONE, both);
        }
      }
      __syncwarp();
      if (leader) commit2(bar + B_DRAIN, both);
    }
    __syncwarp();
  } else if (warp >= KEY_WARP) {
    // ---- the rotary keys of the CTA's half of every tile, 64 rows a warp, as they are: 16 bytes a copy, eight lanes a row.
    //      Their place in the ring is free when the V before this K has been multiplied (of the second K: when the first one
    //      has; either wait is for a phase that the next one of its barrier cannot follow before these keys are there). (Rows
    //      as a whole brought into L2 a tile or two ahead: 46.2 us for five requests of 16,384 against 45.6, cold and warm.)
    ok = !a.stall || __all_sync(0xffffffffu, bar_wait(bar + B_STALL, 0, abort_flag, lim));
    const int r8 = lane & 7, qd = lane >> 3, part = warp - KEY_WARP;
    int32_t e[2];  // the entries of the lane's rows, a tile ahead
    auto entries = [&](int tile) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = (tiles.first + tile) * NK + (int)rank * KH + part * 64 + lane + 32 * i;
        e[i] = tile < tiles.n && x < a.k ? ld_fresh(list + x) : -1;
      }
    };
    entries(0);
    for (int t = 0; t < tiles.n && ok; ++t) {
      unsigned long long row[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) row[i] = reinterpret_cast<unsigned long long>(row_at(a.src, b, e[i], ROW_INT4));
      entries(t + 1);
      if (t == 1) ok = __all_sync(0xffffffffu, bar_wait(bar + B_SFULL, 0, abort_flag, lim));
      if (t >= 2) ok = __all_sync(0xffffffffu, bar_wait(bar + B_PDONE, (unsigned)(t - 2) & 1u, abort_flag, lim));
      if (!ok) break;
      const int slot = (tiles.k_stage(t) + ROPE_AT) % NSTAGE;
      uint8_t* const dst = smem + OFF_RING + slot * STAGE_BYTES + (part * 64 + qd) * 128;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 4 * i + qd;
        const unsigned long long p = __shfl_sync(0xffffffffu, row[i >> 3], r & 31);
        uint8_t* const d = dst + i * 512 + ((r8 ^ (r & 7)) << 4);
        if (p)
          copy16(su32(d), p + INT4_ROPE + 16 * r8);
        else
          *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
      }
      copies_commit();
      copies_wait<0>();
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_lead(lead + (B_FULL + slot) * 8, KEY_ARRIVE);
    }
    copies_wait<0>();
    __syncwarp();
  } else if (warp >= LOAD_WARP0) {
    // ---- a loader. All of them work side by side, 32 rows by 128 columns each: of K's latents first on 128 columns a group of
    //      four, then on the other two 128s; of V on two segments, then on the other two (of half of the columns on all four).
    //      Two jobs' words are on their way.
    ok = !a.stall || __all_sync(0xffffffffu, bar_wait(bar + B_STALL, 0, abort_flag, lim));
    const Loader<lv> loader{warp - LOAD_WARP0};
    const int r8 = lane & 7, qd = lane >> 3, wl = loader.wl, grp = loader.group();
    if (wl == 0 && lane == 0 && ok) {
      if (rank == 0) bar_arrive_expect(bar + B_QFULL, 2 * KBLK * BLK_BYTES);
      for (int i = 0; i < KBLK; i += 3)
        tma_box(su32(smem + OFF_Q + i * BLK_BYTES), &qmap, i, (int)b * HEADS + (int)rank * QH, lead + B_QFULL * 8);
    }
    __syncwarp();
    using Address = unsigned long long;
    // the list's entry of the lane's row, `row` of a tile, and where that row is
    auto entry = [&](int tile, int row) {
      const int i = (tiles.first + tile) * NK + row + lane;
      return tile < tiles.n && i < a.k ? ld_fresh(list + i) : -1;
    };
    auto at = [&](int32_t e) { return reinterpret_cast<Address>(row_at(a.src, b, e, ROW_INT4)); };
    // a loader's rows of K and of its first segment of V
    const int krow = (int)rank * KH + loader.k_row(), vrow = loader.segment(0) * SEG + loader.v_row();
    // The words of 128 columns from `col` on, on their way into buffer `par`: four lanes a row; where there is no row its scales
    // are zeros (and the numbers may be anything).
    uint8_t* const raw = smem + OFF_RAW + wl * 2 * RAW_JOB;
    auto load = [&](int par, Address mine, int col) {
      uint8_t* const scales = raw + par * RAW_JOB + RAW_CODES + lane * 8;
      if (mine)
        copy8(su32(scales), mine + INT4_SCALES + col / INT4_BLOCK);
      else
        *reinterpret_cast<uint2*>(scales) = make_uint2(0, 0);
      const uint32_t to = su32(raw + par * RAW_JOB + (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 3 & 3)) << 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (the swizzle of rows 8 apart is the same)
        const Address p = __shfl_sync(0xffffffffu, mine, 8 * i + (lane >> 2));
        if (p) copy16(to + i * 512, p + col / 2 + 16 * (lane & 3));
      }
      copies_commit();
    };
    // a lane's part of a buffer: 32 latents of rows lane % 8, + 8, + 16 and + 24
    auto read = [&](int par, uint4 (&codes)[4], uint32_t (&scales)[4]) {
      __syncwarp();
      const uint8_t* const from = raw + par * RAW_JOB;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        codes[i] = *reinterpret_cast<const uint4*>(from + i * 512 + r8 * 64 + ((qd ^ (r8 >> 1 & 3)) << 4));
        scales[i] = *reinterpret_cast<const uint16_t*>(from + RAW_CODES + i * 64 + r8 * 8 + 2 * qd);
      }
      __syncwarp();
    };
    // Waits until the MMAs that read the stage NSTAGE before stage n have finished: n takes its place. A barrier's parity only
    // tells a phase from its neighbours. The phase after cannot be over: it takes this loader's part of stage n. The phase
    // before is: stages that a loader has a part in are at most four apart, and it has waited for the last one's place.
    auto need = [&](int n) {
      if (n >= NSTAGE && ok)
        ok = __all_sync(0xffffffffu, bar_wait(bar + B_EMPTY + n % NSTAGE, (unsigned)(n / NSTAGE - 1) & 1u, abort_flag, lim));
    };
    auto full = [&](int stage, uint32_t count) { arrive_lead(lead + (B_FULL + stage % NSTAGE) * 8, count); };
    // 32 rows by 128 columns of K into stages n and n + 1, or of V into stage n, the upper 64 columns behind the lower
    auto put = [&](auto k, const uint4 (&codes)[4], const uint32_t (&scales)[4], int n) {
      constexpr bool K = decltype(k)::value;
      need(n);
      if (K) need(n + 1);
      if (!ok) return;
      uint8_t* const dst = smem + OFF_RING + (K ? n + (qd >> 1) : n) % NSTAGE * STAGE_BYTES +
                           ((K ? loader.k_row() : (qd >> 1) * SEG + loader.v_row()) + r8) * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack<K>(dst + i * 1024, r8, (qd & 1) * 4, codes[i], scales[i]);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        full(n, K ? K_ARRIVE : V_ARRIVE);
        if (K) full(n + 1, K_ARRIVE);
      }
    };
    const std::true_type K;
    const std::false_type V;
    const int kcol = grp * 128, vcol = (int)rank * DVH + half * 128 + loader.v_col();
    uint4 w[4];
    uint32_t sc[4];
    Address krows = at(entry(0, krow));
    int32_t ek = entry(1, krow), ev0 = entry(0, vrow), ev1 = entry(0, vrow + 2 * SEG);
#pragma unroll 1
    for (int h = 0; h < 2; ++h) load(h, krows, kcol + 256 * h);
    // Step t: the two halves of K(t), then V(t - 1), of all columns in two jobs, of half of them in one. A job's words are
    // awaited and read, the copies of the job after the next started into their place, and the words unpacked.
    for (int t = 0; t <= tiles.n && ok; ++t) {
      const int odd = t > 0 ? lv & (t + 1) : 0;  // with single jobs of V: 3 t - 1 jobs come before step t
      const bool k_next = t + 1 < tiles.n;       // what comes after V(t - 1): K(t + 1), or the last V
      if (t < tiles.n) {
        const int n = tiles.k_stage(t);
        krows = at(ek);
        ek = entry(t + 2, krow);
        // after K(t) comes V(t - 1), or K(1) or V(0)
        const bool v_next = t > 0 || !k_next;
#pragma unroll 1
        for (int h = 0; h < 2 && ok; ++h) {
          const int par = h ^ odd;  // the job's buffer
          const bool past = lv && h;  // the job after the next is the one behind a V that is a single job
          const bool v = past ? t > 0 && !k_next : v_next;
          copies_wait<1>();
          read(par, w, sc);
          load(par, v ? at(h > lv ? ev1 : ev0) : past && !k_next ? 0 : krows, v ? vcol : past && t > 0 ? kcol : kcol + 256 * h);
          if (lv && h == 0 && t > 0) ev0 = entry(t, vrow);
          put(K, w, sc, n + loader.k_stage(h));
        }
        if (!ok) break;
        if (t > 0 && !lv) {
          ev0 = entry(t, vrow);
          ev1 = entry(t, vrow + 2 * SEG);
        }
      }
      if (t > 0) {
        const int n = tiles.v_stage(t - 1), segs = tiles.segs(t - 1);
#pragma unroll 1
        for (int h = 0; h < loader.v_jobs && ok; ++h) {
          const int par = h ^ odd;  // the job's buffer
          copies_wait<1>();
          read(par, w, sc);
          load(par, k_next ? krows : lv || t == tiles.n ? 0 : at(h ? ev1 : ev0), k_next ? kcol + 256 * (h | lv) : vcol);
          if (loader.segment(h) < segs) put(V, w, sc, n + loader.v_stage(h));
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  } else {
    // ---- softmax: a thread holds head r of this CTA and 64 rows of every tile, segment sg
    const int q = warp & 3, sub = warp >> 2, r = (q & 1) * 32 + lane, hf = q >> 1, sg = hf * 2 + sub;
    const uint32_t trow = tmem + ((uint32_t)(q * 32) << 16);
    uint8_t* const prows = smem + OFF_P + sg * BLK_BYTES + (q & 1) * 32 * 128;  // the warp's 32 rows of P
    const size_t head0 = (size_t)b * HEADS + rank * QH;                         // the CTA's first
    float m_run = -INFINITY, l_run = 0.f;
    const int o_cols = (DVH / 2) >> lv;  // columns of O of a thread
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
    const bool up = a.scale_log2 > 0.f;
    // the maximum is taken before a positive scale; another is applied first
    const float factor = a.scale_log2, scale = up ? factor : 1.f;
    int32_t e0, e1;  // the thread's entries of the tile's mask: rows lane and lane + 32 of its segment
    auto entries = [&](int tile) {
      const int key = (tiles.first + tile) * NK + sg * SEG + lane;
      e0 = key < a.k ? ld_fresh(list + key) : -1;
      e1 = key + 32 < a.k ? ld_fresh(list + key + 32) : -1;
    };
    entries(0);
    for (int g = 0; g < tiles.n; ++g) {
      const unsigned mlo = __ballot_sync(0xffffffffu, row_at(a.src, b, e0, ROW_INT4) != nullptr);
      const unsigned mhi = __ballot_sync(0xffffffffu, row_at(a.src, b, e1, ROW_INT4) != nullptr);
      if (g + 1 < tiles.n) entries(g + 1);
      ok = __all_sync(0xffffffffu, bar_wait(bar + B_SFULL + (g & 1), (unsigned)(g >> 1) & 1u, abort_flag, lim));
      if (!ok) break;
      tc_fence_after();
      // The scores are read twice, 32 at a time: for the maximum, and once the four threads of a head agree on it. (Holding
      // all 64 across the exchange takes more registers than 19 warps leave.)
      const uint32_t scol = trow + TMEM_S + (uint32_t)((g & 1) * KH + sub * SEG);
      uint32_t sv[32];
      float mb = -INFINITY;
      auto load32 = [&](int h) {
        tmem_ld32(scol + 32 * h, sv);
        tmem_wait_ld();
        if (!up) {
#pragma unroll
          for (int i = 0; i < 32; ++i) sv[i] = __float_as_uint(__uint_as_float(sv[i]) * factor);
        }
        const uint32_t m32 = h ? mhi : mlo;
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
      // the maximum follows only when it has risen by more than 8 (log2), so that O is rarely rescaled: weights stay below
      // 2^(8 + P_SHIFT), within a half
      float m_new = m_run;
      if (mb > -INFINITY && (m_run == -INFINITY || mb > m_run + 8.f)) m_new = mb;
      const bool resc = m_new != m_run && m_run != -INFINITY;
      // (no finite score yet: nothing to subtract, and a NaN still shows)
      const float ref = m_new == -INFINITY ? 0.f : m_new - P_SHIFT;
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
          const __half2 v = __floats2half2_rn(p0, p1);
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
        for (int c = sub * o_cols; c < (sub + 1) * o_cols; c += 16) {
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
#pragma unroll
      for (int c = 0; c < SEG / 8; ++c)
        *reinterpret_cast<uint4*>(prows + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
      fence_proxy_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_lead(lead + B_PFULL * 8);
    }
    if (ok) ok = __all_sync(0xffffffffu, bar_wait(bar + B_PDONE, (unsigned)(tiles.n - 1) & 1u, abort_flag, lim));
    if (ok) {
      const float* const share = exchange(l_run);
      if (ok) l_run = (share[0] + share[QH]) + (share[2 * QH] + share[3 * QH]);
    }
    if (!ok) *out_stop = 1;  // for all softmax warps alike: they meet at barriers below
    // O, out of tensor memory into the head's row; every MMA of the pair has read Q and the ring by now, and every loader is
    // done. Whole lists leave normalised, in the output's type; splits as they are.
    named_sync(1, SOFTMAX_WARPS * 32);
    if (*out_stop == 0) {
      tc_fence_after();
      const bool part = a.nsplit > 1, f32 = part || a.out_f32;
      const float ref = m_run == -INFINITY ? 0.f : m_run - P_SHIFT;
      const float f = part ? 1.f : l_run != 0.f ? UNSCALE / l_run : 0.f;
      if (sg == 0) {
        if (part)
          reinterpret_cast<float2*>(smem + OFF_ML)[r] = make_float2(m_run == -INFINITY ? -INFINITY : ref, l_run);
        else if (half == 0)
          a.lse[head0 + r] = l_run != 0.f ? (ref + log2f(l_run)) * 0.6931471805599453f : -INFINITY;
      }
      uint8_t* const orow = smem + r * (f32 ? OUT_F32 : OUT_BF16);
#pragma unroll 1
      for (int c = sub * o_cols; c < (sub + 1) * o_cols; c += 32) {
        uint32_t v[32];
        tmem_ld32(trow + TMEM_O + c, v);
        tmem_wait_ld();
        const int col = hf * 2 * o_cols + c;
        if (f32) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(orow + 4 * col + 16 * i) =
                make_float4(__uint_as_float(v[4 * i]) * f, __uint_as_float(v[4 * i + 1]) * f, __uint_as_float(v[4 * i + 2]) * f,
                            __uint_as_float(v[4 * i + 3]) * f);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 x =
                  __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * j]) * f, __uint_as_float(v[8 * i + 2 * j + 1]) * f);
              y[j] = *reinterpret_cast<const uint32_t*>(&x);
            }
            *reinterpret_cast<uint4*>(orow + 2 * col + 16 * i) = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
      }
      tc_fence_before();
      if (!part) {
        fence_proxy_async();
        named_sync(1 + 1 + (q & 1), SOFTMAX_WARPS * 16);  // the four warps of the same 32 heads
        // eight rows a warp, one copy a lane; half of the columns are two pieces of a row
        if (lane < 8 << lv) {
          const int h = (q & 1) * 32 + sg * 8 + (lane & 7), piece = lane >> 3, size = f32 ? 4 : 2;
          const uint32_t bytes = (uint32_t)(size * (lv ? LATENT / 4 : LATENT));
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(
                           static_cast<uint8_t*>(a.out) + ((head0 + h) * LATENT + piece * DVH + half * (DVH / 2)) * size),
                       "r"(su32(smem + h * (f32 ? OUT_F32 : OUT_BF16) + piece * bytes)), "r"(bytes)
                       : "memory");
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
      }
    }
    __syncwarp();
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
  if (a.nsplit > 1) {
    // Join: this CTA's share of its 64 heads, from the splits' CTAs of the same heads and columns. A group of threads, 128 for
    // all columns or 64 for half of them, holds every fourth or eighth head of them, a thread four outputs, eight loads from
    // the other CTAs in flight; the weights of all 64 pairs of head and split are worked out by 64 threads meanwhile. Each CTA
    // and group begins with another split, `turn` (all of them with the first: one request of 2,048 0.5 us more).
    const int n = a.nsplit, lg = n == 2 ? 1 : n == 4 ? 2 : 3, share = QH >> lg, groups = 4 << lv,
              grp = t >> (7 - lv), c = 4 * (t & (127 >> lv));
    const int turn = split + grp;
    auto pair_of = [&](int of) { return 2u * (uint32_t)((of << lv) + half) + rank; };  // this CTA's like in another split
    float* const weight = red;
    const uint8_t* const mine = smem + split * share * OUT_F32 + 4 * c;
    const int col = lv ? (c >> 7) * DVH + half * (DVH / 2) + (c & 127) : c;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t head0 = (size_t)b * HEADS + rank * QH + split * share;  // the CTA's first
    bool write = false;
#pragma unroll 1
    for (int x0 = 0; x0 < 16 >> lv; x0 += 8) {  // of the group's pairs: its heads grp, grp + groups, ..
      float4 v[8];
      if (grp < groups) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = ld_peer(peer_addr(mine + (((x0 + u) >> lg) * groups + grp) * OUT_F32, pair_of((u + turn) & (n - 1))));
      }
      if (x0 == 0) {
        if (t < QH) {
          const int h = split * share + (t >> lg);
          const float2 ml = ld_peer2(peer_addr(smem + OFF_ML + h * 8, pair_of(t & (n - 1))));
          const bool some = ml.y != 0.f;  // (a split with no row has no weight, and zeros)
          float mx = some ? ml.x : -INFINITY;
          for (int d = 1; d < n; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          const float ref = mx == -INFINITY ? 0.f : mx;
          const float f = some ? exp2f(ml.x == -INFINITY ? 0.f : ml.x - ref) : 0.f;
          float total = some ? f * ml.y : 0.f;
          for (int d = 1; d < n; d <<= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
          weight[t] = total != 0.f ? f * (UNSCALE / total) : 0.f;
          if ((t & (n - 1)) == 0 && half == 0)
            a.lse[(size_t)b * HEADS + rank * QH + h] = total != 0.f ? (ref + log2f(total)) * 0.6931471805599453f : -INFINITY;
        }
        __syncthreads();
        write = grp < groups && *abort_flag == 0;
      }
      if (!write) continue;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = ((x0 + u) >> lg) * groups + grp;
        const float w = weight[(i << lg) + ((u + turn) & (n - 1))];
        o.x = fmaf(w, v[u].x, o.x);
        o.y = fmaf(w, v[u].y, o.y);
        o.z = fmaf(w, v[u].z, o.z);
        o.w = fmaf(w, v[u].w, o.w);
        if ((u & (n - 1)) == n - 1) {
          uint8_t* const to = static_cast<uint8_t*>(a.out) + ((((head0 + i) * LATENT + col) * 4) >> (a.out_f32 ? 0 : 1));
          if (a.out_f32) {
            *reinterpret_cast<float4*>(to) = o;
          } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
            *reinterpret_cast<uint2*>(to) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          }
          o = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
    __syncwarp();
    cluster_sync();  // the splits' shared memory stays until all have read it
  }
}

using Kernel = void (*)(Decode4Args, CUtensorMap);
const Kernel KERNELS[2] = {hs_decode4_kernel<0>, hs_decode4_kernel<1>};

// How many clusters of 2^lg splits the current device, `dev`, holds at once, cached per device; 0 where it holds none, or takes
// none that large. -1 where it could not be asked: not cached, so that equal calls are cut alike before and after.
int resident(int dev, int lg, int halves) {
  static std::atomic<int> cache[64][2][MAX_PAIRS_LOG + 1];  // 0: not yet asked, else the count + 1
  const unsigned ctas = 2u << (lg + halves);
  const int c = cache[dev][halves][lg].load(std::memory_order_relaxed);
  if (c) return c - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int got = 0;
  const Kernel kernel = KERNELS[halves];
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) {
    e = cudaOccupancyMaxActiveClusters(&got, kernel, &cfg);
    if (e == cudaErrorInvalidClusterSize) {
      cudaGetLastError();
      got = 0, e = cudaSuccess;
    }
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  cache[dev][halves][lg].store(got + 1, std::memory_order_relaxed);
  return got;
}

// How the requests of a grid are cut: the splits of a list, and whether two pairs of CTAs share the value columns of each.
struct Cut {
  int splits, halves;
};
// Calls f(lg, halves, clusters held at once, us of one wave of them) for every way to cut lists of `tiles` tiles into 2^lg
// splits; false where the device could not be asked. A wave takes its start, its last softmax and its output (5 us), its tiles
// (4.2 us, 3.4 with half of the value columns) and the join of splits. Measured, in us, as splits / splits with halves: one
// request of 65 entries 9.4 / 8.3; of 400, one 13.6 / 11.6, two 13.3 / 10.9; of 2,048, one 39 / 32, two 25.7 / 20.7, four 18.3 /
// 14.9, eight 15.8; 9 of 2,048 (more clusters of 16 CTAs than the device holds), two 26.1 / 21.6, four 19.3 / 30.6; 32 of 2,048,
// one 41 / 34, two 27.9 / 65; 76 of 2,048, one 45 / 100.
template <class F>
bool each_cut(int dev, int tiles, F f) {
  for (int halves = 0; halves < 2; ++halves)
    for (int lg = 0; lg + halves <= MAX_PAIRS_LOG && 1 << lg <= tiles; ++lg) {
      const int held = resident(dev, lg, halves);
      if (held < 0) return false;
      const double join = lg == 0 ? 0. : halves ? 1.5 + 1.1 * lg : 2.6 + 1.3 * lg;
      if (held > 0) f(lg, halves, held, 5. + (((tiles - 1) >> lg) + 1) * (halves ? 3.4 : 4.2) + join);
    }
  return true;
}
// The cut of one grid with the shortest expected time, which goes to *us; no splits where the device holds no pair, and false
// where it could not be asked.
bool cut_of(int dev, int32_t batch, int tiles, Cut* best, double* us) {
  *best = {0, 0};
  return each_cut(dev, tiles, [&](int lg, int halves, int held, double wave) {
    const double cost = (batch + held - 1) / held * wave;
    if (best->splits == 0 || cost < *us) *us = cost, *best = {1 << lg, halves};
  });
}
// A call is one grid, or two where the requests of a last, partly filled wave do better with a cut of their own (a second grid
// costs GRID_US: with 1.5 77 requests of 300 took 27.1 us in place of 26.4). 80 of 2,048 62.5 us from 81.3, 160 106 from 124,
// 100 of 1,111 53.1 from 56.0.
struct Plan {
  int32_t first;  // requests of the first grid
  Cut cut[2];
};
constexpr double GRID_US = 3;
int plan_of(int dev, int32_t batch, int32_t k, Plan* plan) {
  if (dev < 0 || dev >= 64) return HS_ERR_UNSUPPORTED;
  const int tiles = (k + NK - 1) / NK;
  *plan = {batch, {{0, 0}, {0, 0}}};
  double least = 0;
  if (!cut_of(dev, batch, tiles, &plan->cut[0], &least)) return HS_ERR_CUDA;
  each_cut(dev, tiles, [&](int lg, int halves, int held, double wave) {  // (every answer is cached by now)
    const int32_t waves = batch / held, rest = batch - waves * held;
    if (waves == 0 || rest == 0 || waves * wave + GRID_US >= least) return;
    double us = 0;
    Cut last;
    cut_of(dev, rest, tiles, &last, &us);
    us += waves * wave + GRID_US;
    if (us < least) least = us, *plan = {waves * held, {{1 << lg, halves}, last}};
  });
  return plan->cut[0].splits < 1 ? HS_ERR_UNSUPPORTED : HS_OK;
}

int launch_part(Decode4Args a, int32_t batch, const Cut& cut, const void* q, hs_stream_t stream) {
  a.nsplit = cut.splits;
  const unsigned ctas = (2u * (unsigned)cut.splits) << cut.halves;  // of a request: a cluster
  CUtensorMap qmap;
  const EncodeFn encode = encoder();
  if (!encode) return HS_ERR_UNSUPPORTED;
  if (!make_map(encode, &qmap, q, (uint64_t)batch * HEADS, QH, 3)) return HS_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * (unsigned)batch, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return hs_launched(cudaLaunchKernelEx(&cfg, KERNELS[cut.halves], a, qmap));
}

int launch(hs_pool* p, int32_t batch, const void* q, const int32_t* idx, int32_t k, const RowSource& src, float sm_scale,
           void* out, int32_t out_type, float* lse, hs_stream_t stream) {
  Plan plan;
  int rc = plan_of(p->device, batch, k, &plan);  // (the pool's device is the current one: see check)
  if (rc != HS_OK) return rc;
  Decode4Args a;
  std::memset(&a, 0, sizeof(a));
  a.idx = idx;
  a.k = k;
  a.src = src;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_type == HS_TYPE_F32;
  a.lse = lse;
  a.err = p->err;
  hs_attention_waits(&a.wait_limit, &a.stall);
  rc = launch_part(a, plan.first, plan.cut[0], q, stream);
  if (rc != HS_OK || plan.first == batch) return rc;
  const size_t heads = (size_t)plan.first * HEADS;
  a.idx += (size_t)plan.first * (size_t)k;
  a.src.rows += (size_t)plan.first * (size_t)src.req_stride;
  a.out = static_cast<uint8_t*>(out) + heads * LATENT * (a.out_f32 ? 4 : 2);
  a.lse += heads;
  return launch_part(a, batch - plan.first, plan.cut[1], static_cast<const uint8_t*>(q) + heads * (WIDTH * 2), stream);
}

// HS_OK, or what the call is refused with; *empty for one that has nothing to do.
int check(hs_pool* p, int32_t layer, int32_t batch, const void* q, const int32_t* idx, int32_t k, const void* out,
          int32_t out_type, const float* lse, bool* empty) {
  if (!p || layer < 0 || layer >= p->d.layers || batch < 0 || batch > p->d.max_batch || batch > 65536 || k < 0 || k > 1 << 30 ||
      (out_type != HS_TYPE_BF16 && out_type != HS_TYPE_F32))
    return HS_ERR_INVALID_ARG;
  if (p->d.row_bytes != ROW_INT4) return HS_ERR_UNSUPPORTED;
  *empty = batch == 0 || k == 0;
  if (*empty) return HS_OK;
  const auto bad = [](const void* x, uintptr_t n) { return !x || (reinterpret_cast<uintptr_t>(x) & (n - 1)) != 0; };
  return bad(q, 16) || bad(idx, 4) || bad(out, 16) || bad(lse, 4) || !hs_on_device(p) ? HS_ERR_INVALID_ARG : HS_OK;
}

}  // namespace

extern "C" int hs_mla_decode_int4(hs_pool* pool, int32_t layer, int32_t batch, const void* q, const int32_t* out_slots,
                                  int32_t k, const void* resident_rows, int64_t resident_count, float sm_scale, void* out,
                                  int32_t out_type, float* lse, hs_stream_t stream) {
  if (resident_count < 0 || (reinterpret_cast<uintptr_t>(resident_rows) & 15)) return HS_ERR_INVALID_ARG;
  bool empty = true;
  const int rc = check(pool, layer, batch, q, out_slots, k, out, out_type, lse, &empty);
  if (rc != HS_OK || empty) return rc;
  return launch(pool, batch, q, out_slots, k, hs_slot_rows(pool, layer, resident_rows, resident_count), sm_scale, out, out_type,
                lse, stream);
}

extern "C" int hs_mla_decode_int4_history(hs_pool* pool, int32_t layer, int32_t batch, const void* q, const int32_t* topk_idx,
                                          int32_t k, float sm_scale, void* out, int32_t out_type, float* lse,
                                          hs_stream_t stream) {
  bool empty = true;
  const int rc = check(pool, layer, batch, q, topk_idx, k, out, out_type, lse, &empty);
  if (rc != HS_OK || empty) return rc;
  return launch(pool, batch, q, topk_idx, k, hs_history_rows(pool, layer), sm_scale, out, out_type, lse, stream);
}
