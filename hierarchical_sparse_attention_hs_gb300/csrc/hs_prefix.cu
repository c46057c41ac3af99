// Attention of a batch over a prefix that all of its requests share, sm_103a.
//
// For request b and head h, over the tokens t < length whose page the pool holds:
//     s[t] = sm_scale * q[b][h] . row_t,   out = sum softmax(s)[t] row_t[0:512],   lse = ln sum e^s[t],
// joined with what the request's own rows gave. The tokens are cut into splits; a split leaves its unnormalised output O,
// its running maximum m (in log2 units) and its normaliser l, and a second kernel joins them:
//     M = max m_s,   total = sum 2^(m_s - M) l_s,   out = sum 2^(m_s - M) O_s / total,   lse = ln 2 (M + log2 total),
// where the own rows count as one more split with m = own_lse / ln 2, l = 1, O = own_out.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/hs.h"
#include "hs_pool.hpp"

namespace {

constexpr int HEADS = 128, DQK = 576, DV = 512, ROW_BYTES = DQK * 2;
constexpr int NK = 32;        // keys of a block
constexpr int HG = 16;        // heads of a CTA
constexpr int THREADS = 256;
constexpr int SMEM = HG * DQK * 4 + NK * ROW_BYTES + HG * NK * 4;

struct PrefixArgs {
  const __nv_bfloat16* q;
  const uint8_t* rows;
  const int32_t* pages;
  int32_t page_shift, max_length;
  int64_t page_limit;
  const int32_t* length;  // or nullptr: max_length
  float scale_log2;
  int32_t batch, nsplit;
  float* part_o;          // [nsplit][batch][HEADS][DV]
  float2* part_ml;        // [nsplit][batch][HEADS]: (m, l)
  const float* own_out;
  const float* own_lse;
  void* out;
  int32_t out_f32;
  float* lse;
};

__device__ __forceinline__ int32_t ld_fresh(const int32_t* p) {
  int32_t v;
  asm("ld.global.cv.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ int length_of(const PrefixArgs& a) {
  return a.length ? min(max(ld_fresh(a.length), 0), a.max_length) : a.max_length;
}

// One CTA: 16 heads of one request over one split, 32 keys at a time.
__global__ void __launch_bounds__(THREADS) hs_prefix_kernel(const PrefixArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ __align__(16) uint8_t smem[];
  float* qs = reinterpret_cast<float*>(smem);
  __nv_bfloat16* ks = reinterpret_cast<__nv_bfloat16*>(smem + HG * DQK * 4);
  float* ps = reinterpret_cast<float*>(smem + HG * DQK * 4 + NK * ROW_BYTES);
  const int t = threadIdx.x, b = blockIdx.x, h0 = blockIdx.y * HG, split = blockIdx.z;
  const int len = length_of(a);
  const int nblk = (len + NK - 1) / NK, per = (nblk + a.nsplit - 1) / a.nsplit;
  const int j0 = split * per, j1 = min(nblk, j0 + per);
  const __nv_bfloat16* q = a.q + ((size_t)b * HEADS + h0) * DQK;
  for (int i = t; i < HG * DQK; i += THREADS) qs[i] = __bfloat162float(q[i]);
  float acc[HG][2], m[HG], l[HG];
#pragma unroll
  for (int h = 0; h < HG; ++h) acc[h][0] = acc[h][1] = l[h] = 0.f, m[h] = -INFINITY;
  for (int j = j0; j < j1; ++j) {
    __syncthreads();
    for (int c = t; c < NK * (ROW_BYTES / 16); c += THREADS) {
      const int r = c / (ROW_BYTES / 16), tok = j * NK + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (tok < len) {
        const int64_t page = ld_fresh(a.pages + (tok >> a.page_shift));
        if (page >= 0 && page < a.page_limit)
          v = *reinterpret_cast<const uint4*>(
              a.rows + ((page << a.page_shift) + (tok & ((1 << a.page_shift) - 1))) * (int64_t)ROW_BYTES +
              (c % (ROW_BYTES / 16)) * 16);
      }
      reinterpret_cast<uint4*>(ks)[c] = v;
    }
    __syncthreads();
    for (int c = t; c < HG * NK; c += THREADS) {
      const int h = c / NK, r = c % NK, tok = j * NK + r;
      float s = 0.f;
      for (int d = 0; d < DQK; ++d) s = fmaf(qs[h * DQK + d], __bfloat162float(ks[r * DQK + d]), s);
      bool on = tok < len;
      if (on) {
        const int64_t page = ld_fresh(a.pages + (tok >> a.page_shift));
        on = page >= 0 && page < a.page_limit;
      }
      ps[c] = on ? s * a.scale_log2 : -INFINITY;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      float mb = m[h];
      for (int r = 0; r < NK; ++r) mb = fmaxf(mb, ps[h * NK + r]);
      const float ref = mb == -INFINITY ? 0.f : mb;  // no finite score yet: nothing is subtracted, a NaN still shows
      const float f = exp2f(m[h] - ref);
      m[h] = mb;
      l[h] *= f;
      acc[h][0] *= f;
      acc[h][1] *= f;
      for (int r = 0; r < NK; ++r) {
        const float p = exp2f(ps[h * NK + r] - ref);
        const float pr = __bfloat162float(__float2bfloat16_rn(p));
        l[h] += p;
        acc[h][0] = fmaf(pr, __bfloat162float(ks[r * DQK + t]), acc[h][0]);
        acc[h][1] = fmaf(pr, __bfloat162float(ks[r * DQK + t + THREADS]), acc[h][1]);
      }
    }
  }
  const size_t rh = ((size_t)split * a.batch + b) * HEADS + h0;
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    a.part_o[(rh + h) * DV + t] = acc[h][0];
    a.part_o[(rh + h) * DV + t + THREADS] = acc[h][1];
    if (t == 0) a.part_ml[rh + h] = make_float2(m[h], l[h]);
  }
}

// One CTA joins one head of one request: thread t holds outputs 4t .. 4t + 3.
__global__ void __launch_bounds__(DV / 4) hs_prefix_join_kernel(const PrefixArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int t = threadIdx.x;
  const size_t bh = blockIdx.x, heads = (size_t)a.batch * HEADS;
  const float own = a.own_lse ? a.own_lse[bh] * 1.4426950408889634f : -INFINITY;
  float mx = own;
  for (int s = 0; s < a.nsplit; ++s) {
    const float2 ml = a.part_ml[(size_t)s * heads + bh];
    if (ml.y != 0.f) mx = fmaxf(mx, ml.x);
  }
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
  auto add = [&](float w, const float* p) {
    const float4 v = *reinterpret_cast<const float4*>(p + 4 * t);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  };
  if (own != -INFINITY) {
    total = exp2f(own - mx);
    add(total, a.own_out + bh * DV);
  }
  for (int s = 0; s < a.nsplit; ++s) {
    const float2 ml = a.part_ml[(size_t)s * heads + bh];
    if (ml.y == 0.f) continue;  // a split with no row
    const float w = exp2f(ml.x - mx);
    total = fmaf(w, ml.y, total);
    add(w, a.part_o + ((size_t)s * heads + bh) * DV);
  }
  const float inv = total != 0.f ? 1.f / total : 0.f;
  o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (a.out_f32) {
    reinterpret_cast<float4*>(static_cast<float*>(a.out) + bh * DV)[t] = o;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + bh * DV)[t] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
  __syncthreads();  // own_lse may be lse itself
  if (t == 0) a.lse[bh] = total != 0.f ? (mx + log2f(total)) * 0.6931471805599453f : -INFINITY;
}

int splits_of(const hs_pool* p, int32_t batch, int32_t max_length) {
  const int blocks = (max_length + NK - 1) / NK;
  return std::max(1, std::min({blocks, 2 * p->num_sms / std::max(1, batch * (HEADS / HG)), 64}));
}

}  // namespace

extern "C" size_t hs_mla_prefix_workspace(hs_pool* pool, int32_t batch, int32_t max_length) {
  if (!pool || batch <= 0 || max_length < 0) return 0;
  return (size_t)splits_of(pool, batch, max_length) * (size_t)batch * HEADS * (DV * sizeof(float) + sizeof(float2));
}

extern "C" int hs_mla_prefix(hs_pool* pool, int32_t batch, const void* q, const hs_paged_rows* prefix,
                             int32_t max_length, const int32_t* prefix_length, float sm_scale, const float* own_out,
                             const float* own_lse, void* out, int32_t out_type, float* lse, void* workspace,
                             size_t workspace_bytes, hs_stream_t stream) {
  const auto aligned = [](const void* p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!pool || !prefix || batch < 0 || batch > (1 << 24) / HEADS || max_length < 0 || !hs_paged_ok(prefix) ||
      max_length > prefix->page_stride * prefix->page_rows || (out_type != HS_TYPE_BF16 && out_type != HS_TYPE_F32) ||
      (own_out != nullptr) != (own_lse != nullptr))
    return HS_ERR_INVALID_ARG;
  if (pool->d.row_bytes != ROW_BYTES) return HS_ERR_UNSUPPORTED;
  if (batch == 0) return HS_OK;
  const size_t need = hs_mla_prefix_workspace(pool, batch, max_length);
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || (own_out && (!aligned(own_out, 16) || !aligned(own_lse, 4))) ||
      (prefix_length && !aligned(prefix_length, 4)) || (need && (!aligned(workspace, 256) || workspace_bytes < need)) ||
      !hs_on_device(pool))
    return HS_ERR_INVALID_ARG;
  PrefixArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.rows = static_cast<const uint8_t*>(prefix->rows);
  a.pages = prefix->pages;
  while ((1 << a.page_shift) < prefix->page_rows) ++a.page_shift;
  a.max_length = max_length;
  a.page_limit = prefix->count / prefix->page_rows;
  a.length = prefix_length;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.batch = batch;
  a.nsplit = splits_of(pool, batch, max_length);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)a.nsplit * batch * HEADS * DV);
  a.own_out = own_out;
  a.own_lse = own_lse;
  a.out = out;
  a.out_f32 = out_type == HS_TYPE_F32;
  a.lse = lse;
  if (cudaFuncSetAttribute(hs_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) {
    cudaGetLastError();
    return HS_ERR_UNSUPPORTED;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)batch, HEADS / HG, (unsigned)a.nsplit);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, hs_prefix_kernel, a) != cudaSuccess) return HS_ERR_CUDA;
  cfg.gridDim = dim3((unsigned)batch * HEADS, 1, 1);
  cfg.blockDim = dim3(DV / 4, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, hs_prefix_join_kernel, a) == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}
