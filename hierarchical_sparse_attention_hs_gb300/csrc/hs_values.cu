// Rows read back as numbers, sm_103a: the values that the selected rows stand for, whatever their format, in bf16, f16 or
// fp32, for a consumer that takes no quantised rows (the attention of a prefill chunk, a check, another library's kernel).
//
// Entry i of a request's list names a row (a hot slot, a row of the paged pool, a token of the history) or none, whose
// values are zeros. 416-byte rows: number times scale, exact in bf16 and f16; 656-byte rows: e4m3 value times scale in 32
// bits, rounded once; 1152-byte rows: their bf16 values. Nothing is computed to speak of: the floor is the bytes, 416 read
// and 1152 written for a 4-bit row into bf16.
//
// Work. A warp takes ROWS consecutive entries at a time: their list entries in one load, then all their rows' loads in
// flight together, then the stores. A lane's values lie 32 lanes' worth apart (chunk t of a lane: values (32 t + lane) V on),
// so that every store instruction of a warp fills 512 consecutive bytes, and every load of codes 128 (4-bit) to 512.
//
// Measured on one GB300 (reads and writes over the time): 131,072 4-bit rows into bf16 32.9 us, 6.25 TB/s, 0.92 of the
// measured copy, into fp32 58.4 (6.1 TB/s); 65,536 fp8 rows into fp32 33.6 us, 5.8 TB/s, into bf16 20.5; 65,536 bf16 rows into
// bf16 26.7, into fp32 36.3 (6.25 TB/s); 771 rows 2.2 us, a launch's own cost. Out of host memory, whose link gives 211 GB/s:
// 32,768 4-bit rows into bf16 84 us (163 GB/s; into fp32 101, where a warp's loads of codes are half as wide), 16,384 fp8 rows
// 66 (162 GB/s; into fp32 78), 16,384 bf16 rows 93 into any type (204 GB/s).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/hs.h"
#include "hs_internal.hpp"
#include "hs_load.cuh"
#include "hs_rows.cuh"
#include "hs_source.hpp"

namespace {

using namespace hs;

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int ROWS = 4;          // rows of a warp in flight
// Blocks an SM, at most: 131,072 4-bit rows into bf16 took 32.9 us with 16 (37.0 with 8, 32.6 with 32), 65,536 fp8 rows into
// fp32 33.6 with 8 (34.4 with 16, 35.2 with 4). Four rows in flight: 37.0 and 33.6 us with eight blocks, against 36.3 and 34.3
// with two rows, 34.6 and 38.3 with eight.
constexpr int BLOCKS_16 = 16, BLOCKS_32 = 8;
constexpr int64_t MAX_ENTRIES = 1 << 30;

struct ValuesArgs {
  const int32_t* idx;       // [entries]
  uint32_t entries, k;      // of all requests, of one
  RowSource src;
  uint8_t* dst;
};

// Loads of a row's bytes: of host memory afresh, so that a line that L2 kept is never used.
template <bool HOST, class W>
__device__ __forceinline__ W load(const uint8_t* p) {
  if constexpr (HOST) return __ldcv(reinterpret_cast<const W*>(p));
  return __ldcg(reinterpret_cast<const W*>(p));
}

// A lane's part of a row: NT chunks of V latents (16 bytes of the output each), then its share of the key, 2 values.
template <int RB, class T>
struct Part {
  static constexpr int V = 16 / sizeof(T), NT = LATENT / (32 * V);
  using Codes = std::conditional_t<RB == ROW_INT4, uint32_t,
                                   std::conditional_t<RB == ROW_FP8, std::conditional_t<V == 8, uint2, uint32_t>,
                                                      std::conditional_t<V == 8, uint4, uint2>>>;
  Codes codes[NT];
  uint32_t scale[NT], key;

  template <bool HOST>
  __device__ __forceinline__ void fetch(const uint8_t* row, int lane) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int v = (32 * t + lane) * V;  // the chunk's first latent
      if constexpr (RB == ROW_INT4) {
        codes[t] = load<HOST, uint32_t>(row + v / 8 * 4);
        scale[t] = load<HOST, uint8_t>(row + INT4_SCALES + v / INT4_BLOCK);
      } else if constexpr (RB == ROW_FP8) {
        codes[t] = load<HOST, Codes>(row + v);
        scale[t] = load<HOST, uint32_t>(row + FP8_SCALES + v / 128 * 4);
      } else {
        codes[t] = load<HOST, Codes>(row + 2 * v);
        scale[t] = 0;
      }
    }
    key = load<HOST, uint32_t>(row + RB - 2 * ROPE + 4 * lane);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) codes[t] = Codes{}, scale[t] = 0;
    key = 0;
  }
  // chunk t in 32 bits
  __device__ __forceinline__ void get(int t, int lane, float (&x)[V]) const {
    if constexpr (RB == ROW_INT4) {
      Int4Half k;
      k.set(scale[t]);
      const uint32_t w = V == 8 ? codes[t] : codes[t] >> (8 * (lane & 1));  // four of a word's eight where a chunk is four
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const float2 f = __half22float2(e & 1 ? int4_pair<1>(w >> (4 * (e & 2)), k) : int4_pair<0>(w >> (4 * (e & 2)), k));
        x[2 * e] = 64.f * f.x;
        x[2 * e + 1] = 64.f * f.y;
      }
    } else if constexpr (RB == ROW_FP8) {
      const float s = __uint_as_float(scale[t]);
      uint32_t w[V / 4];
      memcpy(w, &codes[t], sizeof(w));
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[e / 2] >> (16 * (e & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * e] = f.x * s;
        x[2 * e + 1] = f.y * s;
      }
    } else {
      uint32_t w[V / 2];
      memcpy(w, &codes[t], sizeof(w));
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    }
  }
};

template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <int RB, class T, bool HOST>
__global__ void __launch_bounds__(THREADS) hs_values_kernel(const ValuesArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  using P = Part<RB, T>;
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * WARPS;
  for (uint32_t r0 = (blockIdx.x * WARPS + (threadIdx.x >> 5)) * ROWS; r0 < a.entries; r0 += warps * ROWS) {
    // lanes 0 .. ROWS - 1 look the rows up
    const uint8_t* mine = nullptr;
    if (lane < ROWS && r0 + lane < a.entries) mine = row_at(a.src, (r0 + lane) / a.k, ld_fresh(a.idx + r0 + lane), RB);
    P part[ROWS];
    const uint8_t* row[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      row[u] = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), u));
      if (row[u]) part[u].template fetch<HOST>(row[u], lane);
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      if (r0 + u >= a.entries) break;
      if (!row[u]) part[u].clear();
      uint8_t* const dst = a.dst + (size_t)(r0 + u) * (WIDTH * sizeof(T));
#pragma unroll
      for (int t = 0; t < P::NT; ++t) {
        float x[P::V];
        part[u].get(t, lane, x);
        uint4 w;
        if constexpr (sizeof(T) == 4)
          w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        else
          w = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
        *reinterpret_cast<uint4*>(dst + (32 * t + lane) * 16) = w;
      }
      const float k0 = __uint_as_float(part[u].key << 16), k1 = __uint_as_float(part[u].key & 0xffff0000u);
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float2*>(dst + LATENT * 4 + 8 * lane) = make_float2(k0, k1);
      else
        *reinterpret_cast<uint32_t*>(dst + LATENT * 2 + 4 * lane) =
            std::is_same_v<T, __half> ? pack2<T>(k0, k1) : part[u].key;
    }
  }
}

using Kernel = void (*)(ValuesArgs);
template <int RB, bool HOST>
Kernel of_type(int32_t type) {
  return type == HS_TYPE_BF16  ? hs_values_kernel<RB, __nv_bfloat16, HOST>
         : type == HS_TYPE_F16 ? hs_values_kernel<RB, __half, HOST>
                               : hs_values_kernel<RB, float, HOST>;
}
template <bool HOST>
Kernel kernel_of(int rb, int32_t type) {
  return rb == ROW_BF16  ? of_type<ROW_BF16, HOST>(type)
         : rb == ROW_FP8 ? of_type<ROW_FP8, HOST>(type)
                         : of_type<ROW_INT4, HOST>(type);
}

int launch_values(hs_pool* p, int32_t batch, const int32_t* idx, int32_t k, const RowSource& src, bool host, void* dst,
                  int32_t type, hs_stream_t stream) {
  ValuesArgs a;
  std::memset(&a, 0, sizeof(a));
  a.idx = idx;
  a.entries = (uint32_t)batch * (uint32_t)k;
  a.k = (uint32_t)k;
  a.src = src;
  a.dst = static_cast<uint8_t*>(dst);
  cudaLaunchConfig_t cfg = {};
  const uint32_t per = WARPS * ROWS, most = (uint32_t)p->num_sms * (type == HS_TYPE_F32 ? BLOCKS_32 : BLOCKS_16);
  cfg.gridDim = dim3(std::min<uint32_t>((a.entries + per - 1) / per, most), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const Kernel kernel = host ? kernel_of<true>(p->d.row_bytes, type) : kernel_of<false>(p->d.row_bytes, type);
  return hs_launched(cudaLaunchKernelEx(&cfg, kernel, a));
}

// HS_OK, or what the call is refused with; *empty for one that has nothing to do.
int check(hs_pool* p, int32_t layer, int32_t batch, const int32_t* idx, int32_t k, const void* dst, int32_t type, bool* empty) {
  if (!p || layer < 0 || layer >= p->d.layers || batch < 0 || batch > p->d.max_batch || k < 0 ||
      (int64_t)batch * k > MAX_ENTRIES || type < HS_TYPE_BF16 || type > HS_TYPE_F32)
    return HS_ERR_INVALID_ARG;
  if (p->d.row_bytes != ROW_BF16 && p->d.row_bytes != ROW_FP8 && p->d.row_bytes != ROW_INT4) return HS_ERR_UNSUPPORTED;
  *empty = batch == 0 || k == 0;
  if (*empty) return HS_OK;
  const uintptr_t d = reinterpret_cast<uintptr_t>(dst), i = reinterpret_cast<uintptr_t>(idx);
  return d && !(d & 15) && i && !(i & 3) && hs_on_device(p) ? HS_OK : HS_ERR_INVALID_ARG;
}

}  // namespace

RowSource hs_slot_rows(const hs_pool* p, int32_t layer, const void* resident_rows, int64_t resident_count) {
  const size_t request = (size_t)p->d.slots * (size_t)p->d.row_bytes;
  return {static_cast<const uint8_t*>(p->d.hot_buf) + (size_t)layer * (size_t)p->d.max_batch * request, (int64_t)request,
          p->d.slots, static_cast<const uint8_t*>(resident_rows), resident_rows ? resident_count : 0};
}
RowSource hs_history_rows(const hs_pool* p, int32_t layer) {
  return {p->src + (size_t)layer * (size_t)p->d.host_layer_stride,
          p->d.host_req_stride ? p->d.host_req_stride : (int64_t)p->d.ctx * p->d.row_bytes, p->d.ctx, nullptr, 0};
}

extern "C" int hs_gather_values(hs_pool* pool, int32_t layer, int32_t batch, const int32_t* out_slots, int32_t k,
                                const void* resident_rows, int64_t resident_count, void* dst, int32_t dst_type,
                                hs_stream_t stream) {
  if (resident_count < 0 || (reinterpret_cast<uintptr_t>(resident_rows) & 15)) return HS_ERR_INVALID_ARG;
  bool empty = true;
  const int rc = check(pool, layer, batch, out_slots, k, dst, dst_type, &empty);
  if (rc != HS_OK || empty) return rc;
  return launch_values(pool, batch, out_slots, k, hs_slot_rows(pool, layer, resident_rows, resident_count), false, dst, dst_type,
                       stream);
}

extern "C" int hs_gather_values_history(hs_pool* pool, int32_t layer, int32_t batch, const int32_t* topk_idx, int32_t k,
                                        void* dst, int32_t dst_type, hs_stream_t stream) {
  bool empty = true;
  const int rc = check(pool, layer, batch, topk_idx, k, dst, dst_type, &empty);
  if (rc != HS_OK || empty) return rc;
  return launch_values(pool, batch, topk_idx, k, hs_history_rows(pool, layer), !pool->noio, dst, dst_type, stream);
}
