// Sparse MLA decode attention over 4-bit rows, sm_103a.
//
// For request b and head h, over the rows that the request's list names:
//     s[i] = sm_scale * q[b][h] . row_i,   out = sum softmax(s)[i] row_i[0:512],   lse = ln sum e^s[i],
// the rows' latents being number times scale (hs_rows.cuh). One block takes eight heads of one request and walks the list
// eight rows at a time, all in 32 bits on the CUDA cores.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/hs.h"
#include "hs_internal.hpp"
#include "hs_load.cuh"
#include "hs_rows.cuh"
#include "hs_source.hpp"

namespace {

using namespace hs;

constexpr int HEADS = 128, GH = 8, KEYS = 8, THREADS = 128;

struct Decode4Args {
  const uint16_t* q;   // bf16 [batch][HEADS][WIDTH]
  const int32_t* idx;  // [batch][k]
  int32_t k;
  RowSource src;
  float scale_log2;
  void* out;
  int32_t out_f32;
  float* lse;
};

__global__ void __launch_bounds__(THREADS) hs_decode4_kernel(const Decode4Args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ float q[GH][WIDTH], row[KEYS][WIDTH], score[KEYS][GH];
  __shared__ const uint8_t* at[KEYS];
  const int b = blockIdx.x / (HEADS / GH), h0 = (blockIdx.x % (HEADS / GH)) * GH, t = threadIdx.x;
  for (int i = t; i < GH * WIDTH; i += THREADS)
    q[i / WIDTH][i % WIDTH] = __uint_as_float((uint32_t)a.q[((size_t)b * HEADS + h0) * WIDTH + i] << 16);
  float m[GH], l[GH], o[GH][4] = {};
  for (int h = 0; h < GH; ++h) m[h] = -INFINITY, l[h] = 0.f;
  for (int i0 = 0; i0 < a.k; i0 += KEYS) {
    __syncthreads();
    if (t < KEYS) at[t] = i0 + t < a.k ? row_at(a.src, b, ld_fresh(a.idx + (size_t)b * a.k + i0 + t), ROW_INT4) : nullptr;
    __syncthreads();
    for (int i = t; i < KEYS * WIDTH; i += THREADS) {
      const int j = i / WIDTH, c = i % WIDTH;
      float v = 0.f;
      if (at[j]) {
        if (c < LATENT) {
          const uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(at[j]) + c / 8);
          const int e = c & 7;
          v = (float)((int)(w >> (16 * (e & 1) + 4 * (e >> 1)) & 15u) - 8) * int4_scale(__ldcg(at[j] + INT4_SCALES + c / INT4_BLOCK));
        } else {
          v = __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const uint16_t*>(at[j] + INT4_ROPE) + c - LATENT) << 16);
        }
      }
      row[j][c] = v;
    }
    __syncthreads();
    if (t < KEYS * GH) {
      const int j = t / GH, h = t % GH;
      float s = 0.f;
      for (int c = 0; c < WIDTH; ++c) s = fmaf(q[h][c], row[j][c], s);
      score[j][h] = at[j] ? s * a.scale_log2 : -INFINITY;
    }
    __syncthreads();
    for (int h = 0; h < GH; ++h) {
      float top = m[h];
      for (int j = 0; j < KEYS; ++j)
        if (at[j]) top = fmaxf(top, score[j][h]);
      const float ref = top == -INFINITY ? 0.f : top, f = exp2f(m[h] - ref);
      m[h] = top;
      l[h] *= f;
      for (int e = 0; e < 4; ++e) o[h][e] *= f;
      for (int j = 0; j < KEYS; ++j) {
        if (!at[j]) continue;
        const float p = exp2f(score[j][h] - ref);
        l[h] += p;
        for (int e = 0; e < 4; ++e) o[h][e] = fmaf(p, row[j][4 * t + e], o[h][e]);
      }
    }
  }
  for (int h = 0; h < GH; ++h) {
    const size_t bh = (size_t)b * HEADS + h0 + h;
    const float inv = l[h] != 0.f ? 1.f / l[h] : 0.f;
    for (int e = 0; e < 4; ++e) {
      if (a.out_f32)
        static_cast<float*>(a.out)[bh * LATENT + 4 * t + e] = o[h][e] * inv;
      else
        static_cast<__nv_bfloat16*>(a.out)[bh * LATENT + 4 * t + e] = __float2bfloat16(o[h][e] * inv);
    }
    if (t == 0) a.lse[bh] = l[h] != 0.f ? ((m[h] == -INFINITY ? 0.f : m[h]) + log2f(l[h])) * 0.6931471805599453f : -INFINITY;
  }
}

int launch(hs_pool* p, int32_t batch, const void* q, const int32_t* idx, int32_t k, const RowSource& src, float sm_scale,
           void* out, int32_t out_type, float* lse, hs_stream_t stream) {
  Decode4Args a;
  std::memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.idx = idx;
  a.k = k;
  a.src = src;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = out;
  a.out_f32 = out_type == HS_TYPE_F32;
  a.lse = lse;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)batch * (HEADS / GH), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return hs_launched(cudaLaunchKernelEx(&cfg, hs_decode4_kernel, a));
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
