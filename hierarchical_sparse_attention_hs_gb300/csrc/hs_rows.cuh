// The formats of a KV row, and the arithmetic of the 4-bit one: what writes such rows, reads them back and attends to them.
//
// A row of 416 bytes: 512 latents as whole numbers q from -7 to 7 in 4 bits each, 32 scales s of 8 bits, one for each 16
// latents, and 64 bf16 values of the rotary key; a latent is q s. A scale is 5 bits of exponent and 3 of fraction, the upper
// bits of a half without its sign. The 32-bit word i holds latents 8 i .. 8 i + 7, each as q + 8: the even ones at bits 0, 4,
// 8, 12, the odd ones 16 bits above them, so that one mask takes two neighbours out, as the low bits of two halves.
//
// Why whole numbers, and not a 4-bit float: on normed latents either is about as far off (0.086 of N(0, 1) against 0.095 for
// e2m1 and the same scales; 0.100 against 0.093 where channels differ by exp(0.4 N)), but e2m1's conversion instruction took
// 2.8 cycles an SM for a warp's pairs (measured), ten times the two instructions below. q has 3 bits and s 4: the product
// is exact in bf16 and in f16, so all readers of a row see the same numbers, none of them rounded.
//
// In halves, at 2^-6 of the value (so that nothing below leaves their range): two numbers at bits 0 and 16 under the exponent
// of 16 are 16 + (q + 8) / 64, at bits 4 and 20 under that of 1 they are 1 + (q + 8) / 64; fma(x, s, -16.125 s) and fma(x, s,
// -1.125 s) leave q s / 64. Every term is exact: 16.125 = 129 / 8 and 1.125 = 9 / 8, with four bits of s at most 11 bits; s <=
// 3840 keeps 16.125 s below 65504, and the smallest, 2^-17 * 2^-6, is a multiple of 2^-24. In bf16, at the value itself: under
// the exponent of 128 they are 128 + q + 8 (the four bits have to lie at bits 0 and 16), and fma(x, s, -136 s) leaves q s; 136
// = 17 * 8, and 17 times four bits of s has 8.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace hs {

constexpr int LATENT = 512, ROPE = 64, WIDTH = LATENT + ROPE;
constexpr int ROW_BF16 = WIDTH * 2;                 // 1152
constexpr int ROW_FP8 = LATENT + 4 * 4 + ROPE * 2;  // 656: e4m3 latents, an fp32 scale for each 128, bf16 key
constexpr int FP8_SCALES = LATENT, FP8_ROPE = LATENT + 4 * 4;
constexpr int INT4_BLOCK = 16;  // latents of a scale
constexpr int INT4_SCALES = LATENT / 2, INT4_ROPE = INT4_SCALES + LATENT / INT4_BLOCK;
constexpr int ROW_INT4 = INT4_ROPE + ROPE * 2;      // 416
constexpr float INT4_SCALE_MIN = 7.62939453125e-06f, INT4_SCALE_MAX = 3840.f;  // 2^-17 and 1.875 * 2^11
constexpr uint32_t INT4_SCALE_NAN = 255;            // a block with a latent that is not finite: it reads back as NaN

// z / d, `inv` being 1 / d to a unit in its last place: the product, corrected once by its residual, which an fma has exactly
// (Markstein). Where z / d is a 32-bit number the result is that number, so that what lies halfway between two codes does.
__device__ __forceinline__ float quotient(float z, float d, float inv) {
  const float y = z * inv;
  return fmaf(fmaf(-y, d, z), inv, y);
}

// The code of the scale for a largest magnitude (a NaN or an infinity: that of NaN): amax / 7 to the nearest scale, ties to
// the even code.
__device__ __forceinline__ uint32_t int4_scale_code(float amax) {
  if (!(amax <= 3.4028234664e38f)) return INT4_SCALE_NAN;
  const float m = fminf(fmaxf(amax, 7.f * INT4_SCALE_MIN), 7.f * INT4_SCALE_MAX);
  const float a = quotient(m, 7.f, 1.f / 7.f);
  if (a < 6.103515625e-05f) return (uint32_t)__float2int_rn(a * 131072.f);  // below 2^-14: multiples of 2^-17
  uint32_t b = __float_as_uint(a);
  b += 0x7ffffu + (b >> 20 & 1u);
  return (b >> 20) - (112u << 3);
}
__device__ __forceinline__ float int4_scale(uint32_t code) {
  return __half2float(__ushort_as_half((unsigned short)(code << 7)));
}

// (w & mask) | magic in one instruction, which takes one of the two from a register: written out as an expression it became
// two, and the unpacking of a row a third slower.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w), "r"(mask), "r"(magic));
  return x;
}
// A scale in both halves of a register, and what takes the numbers' offsets out.
struct Int4Half {
  __half2 s, c0, c1;
  __device__ __forceinline__ void set(uint32_t code) {
    const uint32_t two = code * 0x00800080u;
    s = *reinterpret_cast<const __half2*>(&two);
    c0 = __hmul2(s, __float2half2_rn(-16.125f));
    c1 = __hmul2(s, __float2half2_rn(-1.125f));
  }
};
// Latents 2p and 2p + 1 of a word, p = 0 or 1 (2 and 3: of the word shifted right by 8), at 2^-6 of their value.
template <int P>
__device__ __forceinline__ __half2 int4_pair(uint32_t w, const Int4Half& k) {
  const uint32_t x = P == 0 ? and_or(w, 0x000f000fu, 0x4c004c00u) : and_or(w, 0x00f000f0u, 0x3c003c00u);
  return __hfma2(*reinterpret_cast<const __half2*>(&x), k.s, P == 0 ? k.c0 : k.c1);
}
struct Int4Bf16 {
  __nv_bfloat162 s, c;
  __device__ __forceinline__ void set(uint32_t code) {
    s = __float2bfloat162_rn(int4_scale(code));
    c = __hmul2(s, __float2bfloat162_rn(-136.f));
  }
};
// Latents 2p and 2p + 1 of a word shifted right by 4 p.
__device__ __forceinline__ __nv_bfloat162 int4_pair(uint32_t w, const Int4Bf16& k) {
  const uint32_t x = and_or(w, 0x000f000fu, 0x43004300u);
  return __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), k.s, k.c);
}

}  // namespace hs
