// Appending KV rows, sm_103a: the writer of the tiers that a resolve, a prefetch and the attention read.
//
// Token i at position p of request r: z = kv[i][0:512] (times weight / sqrt(mean(z^2) + eps) with a norm), and the 32
// pairs of kv[i][512:576] turned by the angles p * inv_freq[j]. The row goes to every tier that holds the token, as 576
// bf16 values or as 512 e4m3 values, a scale for each 128 and 64 bf16 (the pool's row_bytes says which). The queries'
// rotary values of the same token turn by the same angles.
//
// Angles. p * inv_freq is wanted modulo a full turn, and p reaches millions: a 32-bit product would be off by p * 2^-24
// turns and more. inv_freq / 2 pi is taken once per warp, in 64 bits, as a fraction of a turn in fixed point (G / 2^64);
// p * G modulo 2^64 is then the position's fraction of a turn by integer multiplication that wraps where the angle does.
// The fraction's signed upper 32 bits go to sincospif. They are off by 2^-32 turns, cut off, and by p * inv_freq * 2^-54, as
// the rate passes through 53 bits: 2^-30 turns at p = 2^24 for inv_freq = 1. (Double arithmetic per token would cost more than
// the memory traffic: this device has few FP64 units.)
//
// Work. One warp per row and one warp per 16 heads of a token's queries, each with several once there are many. A lane
// holds 16 latents (two 16-byte chunks for 16-bit inputs) and one pair of the key, so a row is loaded and stored in
// whole 128-byte segments and the norm's sum and the scales' maxima are warp shuffles. Only the norm's weights
// pass through shared memory.
//
// Measured on one GB300 (reads and writes over the time): 1 to 32 tokens with 128 heads 2.1-2.2 us, a launch's own cost;
// 256 2.8 us; 2,047 with 128 heads 18.5 us from fp32 (5.8 TB/s) and 13.5 from bf16; 131,071 without queries 50 us into bf16
// rows (6.1 TB/s) and 50 into fp8 rows (4.8: 339 instructions a row, which take 38 us where every scheduler issues one a
// cycle; 0.73 are measured); 4,096 into host memory 17.5 us for fp8 rows and 26 for bf16, 153 and 180 GB/s of writes over the
// link.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/hs.h"
#include "hs_internal.hpp"
#include "hs_load.cuh"

namespace {

using hs::ld_fresh;

constexpr int LATENT = 512, ROPE = 64, PAIRS = ROPE / 2, WIDTH = LATENT + ROPE;
constexpr int ROW_BF16 = WIDTH * 2;              // 1152
constexpr int ROW_FP8 = LATENT + 4 * 4 + ROPE * 2;  // 656
constexpr int FP8_ROPE = LATENT + 4 * 4;         // byte offset of the rotary key in an fp8 row
constexpr int Q_HEADS = 16;                      // heads of one warp's work item: four 16-byte loads a lane in flight
constexpr int MAX_TOKENS = 1 << 30;              // and items of 16 heads of a token's queries
constexpr int THREADS = 128, WARPS = THREADS / 32;
// Blocks of a kernel that an SM holds at least. A launch of many tokens has as many blocks of rows as the device holds:
// all warps get the same number of tokens, so time goes in whole waves, and in one wave a warp works its turn rates out
// once. For 656-byte rows a bound of 7 (72 registers a thread) measured best; 131,071 / 16,384 / 8,191 rows in us: from
// 16 bits 50.5 / 9.3 / 6.0 (a bound of 8 50.5 / 10.2 / 6.4, of 6 51.8 / 9.7 / 6.8, twelve blocks where seven fit 50.2 /
// 10.6 / 6.0), from fp32 61.0 / 10.6 / 6.4 (of 6 63.2 / 11.1 / 7.3, of 5 64.5 / 11.3 / 6.7, twelve blocks 65.7 / 13.1 /
// 6.5). For 1152-byte rows the compiler's own choice is kept, 8 blocks from 16 bits, 50.2 / 8.9 / 5.3 (a bound of 7 50.3
// / 8.8 / 5.0, of 6 52.9 / 9.2 / 5.6; one of 8 took the queries of 256 and 2,047 tokens from 2.8 and 13.4 to 3.05 and
// 14.0), 6 from fp32, 70.3 / 11.4 / 6.4 (a bound of 7 73.4 / 10.9 / 5.6, of 5 70.9 / 11.7 / 5.8).
template <bool FP8>
constexpr int MIN_BLOCKS = FP8 ? 7 : 0;  // 0: none
constexpr int Q_BLOCKS = 16;  // blocks of queries an SM, at most

struct AppendArgs {
  const void* kv;
  int64_t kv_stride;
  const float* norm_weight;
  const float* inv_freq;
  const int32_t* req_ids;
  const int32_t* positions;
  const void* q_rope;
  int64_t qr_token, qr_head;
  __nv_bfloat16* q;
  int64_t q_token, q_head;
  int32_t heads;
  int32_t head_items;     // work items per token's queries: ceil(heads / Q_HEADS)
  float eps;
  int32_t ntok, max_batch, ctx, slots;
  uint8_t* history;       // request 0's rows of this layer, or nullptr
  int64_t req_stride;
  uint8_t* hot;           // request 0's slots of this layer
  const int32_t* tok2slot;
  uint8_t* paged;         // or nullptr
  const int32_t* pages;
  int64_t page_stride, page_limit;  // pages 0 .. page_limit - 1 lie within the rows
  int32_t page_shift;
  int32_t lists;          // lists of pages, one a request; 0 without paged rows
  int32_t per_warp;       // tokens of a warp's rows
  int32_t row_blocks;     // blocks 0 .. row_blocks - 1 write rows, the others turn queries
  int32_t* err;
};

// Eight consecutive values as they lie in memory, then in 32 bits. (Plain loads: queries may be turned in place.)
template <class T>
struct Raw8 {
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const;
};
template <>
__device__ __forceinline__ void Raw8<__nv_bfloat16>::get(float (&x)[8]) const {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void Raw8<__half>::get(float (&x)[8]) const {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// Pair `lane`'s turns per position as a fraction of a turn in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turn_rate(const float* inv_freq, int lane) {
  const double g = (double)__ldg(inv_freq + lane) * 0.15915494309189533577;  // 1 / 2 pi
  return __double2ull_rn((g - floor(g)) * 18446744073709551616.0);
}
__device__ __forceinline__ void angle_of(unsigned long long rate, int pos, float* cosv, float* sinv) {
  const int32_t frac = (int32_t)((rate * (unsigned long long)(unsigned)pos) >> 32);  // of a turn, in [-1/2, 1/2) * 2^32
  sincospif((float)frac * 4.656612873077393e-10f, sinv, cosv);                       // half turns: frac * 2^-31
}

// The token's request and position; false for padding and, with the error word set, for what is out of range.
__device__ __forceinline__ bool token_of(const AppendArgs& a, int i, int* req, int* pos) {
  *pos = ld_fresh(a.positions + i);
  *req = a.req_ids ? ld_fresh(a.req_ids + i) : i;
  if (*pos < 0) return false;
  return *pos < a.ctx && *req >= 0 && *req < a.max_batch;
}

// A warp's `per` consecutive tokens. Where they go is looked up 32 tokens at a time, one lane each (position, request, then
// slot and page: a chain of loads that every row would otherwise wait for), and a row's values are loaded while the one
// before is worked on.
template <class T, bool FP8, bool INTER>
__device__ __forceinline__ void append_rows(const AppendArgs& a, float* weight, int lane, int warp) {
  constexpr int RB = FP8 ? ROW_FP8 : ROW_BF16;
  constexpr uint32_t ALL = 0xffffffffu;
  const unsigned long long rate = turn_rate(a.inv_freq, lane);
  const int64_t begin = (int64_t)warp * a.per_warp;
  const int end = (int)min((int64_t)a.ntok, begin + a.per_warp);
  const T* const kv = static_cast<const T*>(a.kv);
  Raw8<T> ahead[2];
  T pair[2];
  auto load = [&](int i) {
    const T* x = kv + (int64_t)i * a.kv_stride;
    ahead[0].load(x + 8 * lane);
    ahead[1].load(x + LATENT / 2 + 8 * lane);
    pair[0] = x[LATENT + (INTER ? 2 * lane : lane)];
    pair[1] = x[LATENT + (INTER ? 2 * lane + 1 : lane + PAIRS)];
  };
  if (begin < end) load((int)begin);
  if (a.norm_weight) {  // shared by the block's warps: 16 registers a lane less, or 2 KB less to load for each row
    reinterpret_cast<float4*>(weight)[threadIdx.x] = reinterpret_cast<const float4*>(a.norm_weight)[threadIdx.x];
    __syncthreads();
  }
  for (int i0 = (int)min(begin, (int64_t)a.ntok); i0 < end; i0 += 32) {
    int my_req = -1, my_pos = -1, my_slot = -1, my_row = -1;
    if (i0 + lane < end) {
      if (token_of(a, i0 + lane, &my_req, &my_pos)) {
        my_slot = __ldcg(a.tok2slot + (int64_t)my_req * a.ctx + my_pos);
        if (my_req < a.lists) {
          const int64_t pi = my_pos >> a.page_shift;
          const int page = pi < a.page_stride ? a.pages[my_req * a.page_stride + pi] : -1;
          if (page >= 0 && page < a.page_limit) my_row = (page << a.page_shift) + (my_pos & ((1 << a.page_shift) - 1));
        }
      } else {
        if (my_pos >= 0) atomicOr(a.err, HS_DEVERR_RANGE);
        my_pos = -1;
      }
    }
    const int m = min(32, end - i0);
    for (int k = 0; k < m; ++k) {
      const Raw8<T> raw[2] = {ahead[0], ahead[1]};
      const float k0 = to_f32(pair[0]), k1 = to_f32(pair[1]);
      if (i0 + k + 1 < end) load(i0 + k + 1);
      const int pos = __shfl_sync(ALL, my_pos, k);
      const int64_t req = __shfl_sync(ALL, my_req, k);
      const int slot = __shfl_sync(ALL, my_slot, k), row = __shfl_sync(ALL, my_row, k);
      if (pos < 0) continue;
      // where the row goes: the hot slot that maps the token, the paged rows, the history
      uint8_t* dst[3] = {slot >= 0 && slot < a.slots ? a.hot + (req * a.slots + slot) * RB : nullptr,
                         row >= 0 ? a.paged + (int64_t)row * RB : nullptr,
                         a.history ? a.history + req * a.req_stride + (int64_t)pos * RB : nullptr};
      float z[2][8];
      raw[0].get(z[0]);
      raw[1].get(z[1]);
      if (a.norm_weight) {
        float ss = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(z[h][e], z[h][e], ss);
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.f / LATENT) + a.eps);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const float4 w = *reinterpret_cast<const float4*>(weight + h * (LATENT / 2) + 8 * lane + e);
            z[h][e] *= r * w.x;
            z[h][e + 1] *= r * w.y;
            z[h][e + 2] *= r * w.z;
            z[h][e + 3] *= r * w.w;
          }
      }
      // the rotary key: lane j turns pair j; lane l then writes the values 2l and 2l + 1
      float c, s;
      angle_of(rate, pos, &c, &s);
      const float t0 = k0 * c - k1 * s, t1 = k0 * s + k1 * c;
      uint32_t kw;
      if (INTER) {
        kw = pack_bf16(t0, t1);
      } else {
        const int src = (2 * lane) & 31;
        const float lo0 = __shfl_sync(0xffffffffu, t0, src), lo1 = __shfl_sync(0xffffffffu, t0, src + 1);
        const float hi0 = __shfl_sync(0xffffffffu, t1, src), hi1 = __shfl_sync(0xffffffffu, t1, src + 1);
        kw = lane < 16 ? pack_bf16(lo0, lo1) : pack_bf16(hi0, hi1);
      }
      if (FP8) {
        // lanes 0-15 hold groups 0 and 2 of 128 latents, lanes 16-31 groups 1 and 3
        uint2 w[2];
        float scale[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(z[h][e]));
#pragma unroll
          for (int o = 8; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          scale[h] = m > 0.f ? fmaxf(m / 448.f, 1.17549435e-38f) : 1.f;  // at least 2^-126: its reciprocal is finite
          const float inv = 1.f / scale[h];
          w[h] = make_uint2(pack_e4m3(z[h][0] * inv, z[h][1] * inv, z[h][2] * inv, z[h][3] * inv),
                            pack_e4m3(z[h][4] * inv, z[h][5] * inv, z[h][6] * inv, z[h][7] * inv));
        }
#pragma unroll
        for (int d = 0; d < 3; ++d) {
          uint8_t* o = dst[d];
          if (!o) continue;
          *reinterpret_cast<uint2*>(o + 8 * lane) = w[0];
          *reinterpret_cast<uint2*>(o + LATENT / 2 + 8 * lane) = w[1];
          if ((lane & 15) == 0) {
            float* sc = reinterpret_cast<float*>(o + LATENT) + (lane >> 4);
            sc[0] = scale[0];
            sc[2] = scale[1];
          }
          *reinterpret_cast<uint32_t*>(o + FP8_ROPE + 4 * lane) = kw;
        }
      } else {
        uint4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = make_uint4(pack_bf16(z[h][0], z[h][1]), pack_bf16(z[h][2], z[h][3]), pack_bf16(z[h][4], z[h][5]),
                            pack_bf16(z[h][6], z[h][7]));
#pragma unroll
        for (int d = 0; d < 3; ++d) {
          uint8_t* o = dst[d];
          if (!o) continue;
          *reinterpret_cast<uint4*>(o + 16 * lane) = w[0];
          *reinterpret_cast<uint4*>(o + LATENT + 16 * lane) = w[1];
          *reinterpret_cast<uint32_t*>(o + 2 * LATENT + 4 * lane) = kw;
        }
      }
    }
  }
}

// 16 heads of one token's queries: eight lanes hold a head's 64 values, four heads a pass, four passes in flight.
template <class T, bool INTER>
__device__ __forceinline__ void turn_queries(const AppendArgs& a, int lane, int warp, int warps) {
  const unsigned long long rate = turn_rate(a.inv_freq, lane);
  const int c8 = lane & 7, sub = lane >> 3;
  const unsigned items = (unsigned)a.ntok * (unsigned)a.head_items;  // the host has seen to it that this is below 2^31
  for (unsigned it = (unsigned)warp; it < items; it += (unsigned)warps) {
    const int i = (int)(it / (unsigned)a.head_items), h0 = (int)(it - (unsigned)i * (unsigned)a.head_items) * Q_HEADS + sub;
    const T* src = static_cast<const T*>(a.q_rope) + (int64_t)i * a.qr_token + 8 * c8;
    Raw8<T> raw[Q_HEADS / 4];
#pragma unroll
    for (int u = 0; u < Q_HEADS / 4; ++u)
      if (h0 + 4 * u < a.heads) raw[u].load(src + (int64_t)(h0 + 4 * u) * a.qr_head);
    int req, pos;
    if (!token_of(a, i, &req, &pos)) continue;  // the row's warp reports it
    float cl, sl;
    angle_of(rate, pos, &cl, &sl);
    // interleaved: this lane's four pairs are 4 c8 ..; half-split: its eight values belong to pairs 8 (c8 % 4) ..
    constexpr int NP = INTER ? 4 : 8;
    float c[NP], s[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const int j = INTER ? 4 * c8 + e : 8 * (c8 & 3) + e;
      c[e] = __shfl_sync(0xffffffffu, cl, j);
      s[e] = __shfl_sync(0xffffffffu, sl, j);
    }
    __nv_bfloat16* dst = a.q + (int64_t)i * a.q_token + LATENT + 8 * c8;
#pragma unroll
    for (int u = 0; u < Q_HEADS / 4; ++u) {
      const bool on = h0 + 4 * u < a.heads;
      float x[8], y[8];
      if (on) {
        raw[u].get(x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
      }
      if (INTER) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = x[2 * e] * c[e] - x[2 * e + 1] * s[e];
          y[2 * e + 1] = x[2 * e] * s[e] + x[2 * e + 1] * c[e];
        }
      } else {
        // lanes 0-3 of the eight hold the first members of the pairs, lanes 4-7 the second
        const float sign = c8 < 4 ? -1.f : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float other = __shfl_xor_sync(0xffffffffu, x[e], 4);
          y[e] = x[e] * c[e] + sign * (other * s[e]);
        }
      }
      if (on)
        *reinterpret_cast<uint4*>(dst + (int64_t)(h0 + 4 * u) * a.q_head) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    }
  }
}

template <class T, bool FP8, bool INTER>
__global__ void __launch_bounds__(THREADS, MIN_BLOCKS<FP8>) hs_append_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  __shared__ __align__(16) float weight[LATENT];
  static_assert(THREADS * 4 == LATENT, "one 16-byte load a thread");
  if ((int)blockIdx.x < a.row_blocks)
    append_rows<T, FP8, INTER>(a, weight, lane, (int)blockIdx.x * WARPS + w);
  else
    turn_queries<T, INTER>(a, lane, ((int)blockIdx.x - a.row_blocks) * WARPS + w,
                           ((int)gridDim.x - a.row_blocks) * WARPS);
}

using Kernel = void (*)(AppendArgs);
template <class T>
Kernel kernel_of(bool fp8, bool inter) {
  if (fp8) return inter ? hs_append_kernel<T, true, true> : hs_append_kernel<T, true, false>;
  return inter ? hs_append_kernel<T, false, true> : hs_append_kernel<T, false, false>;
}
// How many blocks of a kernel an SM of the device holds, cached per device and `form` (0 .. 11); 0 on an error.
int blocks_held(Kernel kernel, int form, int device) {
  static std::atomic<int> cache[64][12];
  if (device < 0 || device >= 64) return 0;
  int n = cache[device][form].load(std::memory_order_relaxed);
  if (n) return n;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(kernel), THREADS, 0) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cache[device][form].store(n, std::memory_order_relaxed);
  return n;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
// `n` strides of at least `least` elements of `size` bytes, multiples of 16 bytes, used by `count` items
bool stride_ok(int64_t stride, int64_t least, int size, int64_t count) {
  return count <= 1 || (stride >= least && stride <= INT64_MAX / size / (count > 0 ? count : 1) && (stride * size) % 16 == 0);
}

}  // namespace

bool hs_paged_ok(const hs_paged_rows* p) {
  return p->rows && p->pages && aligned16(p->rows) && aligned4(p->pages) && p->count >= 0 &&
         p->count <= INT32_MAX - 63 && p->page_stride >= 1 && p->lists >= 0 && p->page_rows >= 1 && p->page_rows <= 65536 &&
         (p->page_rows & (p->page_rows - 1)) == 0;
}

bool hs_on_device(const hs_pool* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return dev == p->device;
}

int hs_launched(cudaError_t e) {
  if (e == cudaSuccess) return HS_OK;
  cudaGetLastError();
  return HS_ERR_CUDA;
}

extern "C" int hs_append(hs_pool* pool, int32_t layer, int32_t ntok, const hs_append_desc* desc,
                         const hs_paged_rows* paged, int32_t to_history, hs_stream_t stream) {
  if (!pool || !desc || layer < 0 || layer >= pool->d.layers || ntok < 0) return HS_ERR_INVALID_ARG;
  if (pool->d.row_bytes != ROW_BF16 && pool->d.row_bytes != ROW_FP8) return HS_ERR_UNSUPPORTED;
  const hs_append_desc& d = *desc;
  if (d.type < HS_TYPE_BF16 || d.type > HS_TYPE_F32 || (!paged && !to_history && !d.q_rope)) return HS_ERR_INVALID_ARG;
  if (paged && !hs_paged_ok(paged)) return HS_ERR_INVALID_ARG;
  if (ntok == 0) return HS_OK;
  const int size = d.type == HS_TYPE_F32 ? 4 : 2;
  if (!d.kv || !aligned16(d.kv) || !stride_ok(d.kv_stride, WIDTH, size, ntok) || !d.inv_freq || !d.positions ||
      !aligned4(d.inv_freq) || !aligned4(d.positions) || !aligned4(d.req_ids) ||
      (d.norm_weight && (!aligned16(d.norm_weight) || !(d.norm_eps >= 0.f))) || (!d.req_ids && ntok > pool->d.max_batch))
    return HS_ERR_INVALID_ARG;
  if ((d.q_rope != nullptr) != (d.q != nullptr) || (d.q_rope != nullptr) != (d.q_heads > 0) || d.q_heads < 0)
    return HS_ERR_INVALID_ARG;
  if (d.q_rope && (!aligned16(d.q_rope) || !aligned16(d.q) || !stride_ok(d.q_rope_token_stride, ROPE, size, ntok) ||
                   !stride_ok(d.q_rope_head_stride, ROPE, size, d.q_heads) ||
                   !stride_ok(d.q_token_stride, WIDTH, 2, ntok) || !stride_ok(d.q_head_stride, WIDTH, 2, d.q_heads)))
    return HS_ERR_INVALID_ARG;
  const int64_t head_items = ((int64_t)d.q_heads + Q_HEADS - 1) / Q_HEADS;
  if (ntok > MAX_TOKENS || ntok * head_items > MAX_TOKENS) return HS_ERR_INVALID_ARG;
  if (!hs_on_device(pool)) return HS_ERR_INVALID_ARG;

  AppendArgs a;
  std::memset(&a, 0, sizeof(a));
  a.kv = d.kv;
  a.kv_stride = d.kv_stride;
  a.norm_weight = d.norm_weight;
  a.inv_freq = d.inv_freq;
  a.req_ids = d.req_ids;
  a.positions = d.positions;
  a.q_rope = d.q_rope;
  a.qr_token = d.q_rope_token_stride;
  a.qr_head = d.q_rope_head_stride;
  a.q = static_cast<__nv_bfloat16*>(d.q);
  a.q_token = d.q_token_stride;
  a.q_head = d.q_head_stride;
  a.heads = d.q_heads;
  a.head_items = (int32_t)head_items;
  a.eps = d.norm_eps;
  a.ntok = ntok;
  a.max_batch = pool->d.max_batch;
  a.ctx = pool->d.ctx;
  a.slots = pool->d.slots;
  const size_t rl0 = (size_t)layer * (size_t)pool->d.max_batch;
  if (to_history) a.history = const_cast<uint8_t*>(pool->src) + (size_t)layer * (size_t)pool->d.host_layer_stride;
  a.req_stride = pool->d.host_req_stride ? pool->d.host_req_stride : (int64_t)pool->d.ctx * pool->d.row_bytes;
  a.hot = static_cast<uint8_t*>(pool->d.hot_buf) + rl0 * (size_t)pool->d.slots * (size_t)pool->d.row_bytes;
  a.tok2slot = pool->tok2slot + rl0 * (size_t)pool->d.ctx;
  if (paged) {
    a.paged = static_cast<uint8_t*>(paged->rows);
    a.pages = paged->pages;
    a.page_stride = paged->page_stride;
    a.page_limit = paged->count / paged->page_rows;
    a.lists = paged->lists ? paged->lists : pool->d.max_batch;
    while ((1 << a.page_shift) < paged->page_rows) ++a.page_shift;
  }
  a.err = pool->err;

  // As many warps of rows as the device holds at once, each with its share of the tokens (and of the queries' items, whose
  // warps come on top): the turn rates (64-bit arithmetic) are worked out once per warp, not per row.
  const bool fp8 = pool->d.row_bytes == ROW_FP8, inter = d.interleaved != 0;
  const Kernel kernel = d.type == HS_TYPE_BF16  ? kernel_of<__nv_bfloat16>(fp8, inter)
                        : d.type == HS_TYPE_F16 ? kernel_of<__half>(fp8, inter)
                                                : kernel_of<float>(fp8, inter);
  const int held = blocks_held(kernel, d.type * 4 + fp8 * 2 + inter, pool->device);
  if (held < 1) return HS_ERR_CUDA;
  const int64_t most = (int64_t)pool->num_sms * held;
  const int64_t items = (int64_t)ntok * a.head_items;
  a.per_warp = (int32_t)((ntok + most * WARPS - 1) / (most * WARPS));
  const int64_t row_warps = ((int64_t)ntok + a.per_warp - 1) / a.per_warp;
  a.row_blocks = (int32_t)((row_warps + WARPS - 1) / WARPS);
  const int64_t q_blocks = std::min<int64_t>((items + WARPS - 1) / WARPS, (int64_t)pool->num_sms * Q_BLOCKS);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.row_blocks + q_blocks), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return hs_launched(cudaLaunchKernelEx(&cfg, kernel, a));
}
