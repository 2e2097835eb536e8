// A cache in 4 bits: its cells and how a row goes into one (not part of the ABI).
//
// A cell is 16 tokens of one head: 64 bytes of codes a token, then a word a group and token
// (step s in the low half, centre z in the high half, both bf16); x^ = s (c - 8) + z.
// The order of a row's bytes -- byte 8 i + u at 8 u + i -- is the tensor cores' own: the 16
// bytes that start at 16 t hold, for every span of 16 entries, the four entries that lane t of
// a quad takes as its part of an operand's row, and the 8 bytes at 8 g the pair of entries that
// lanes g of the quads take as their two rows of a transposed one.
#pragma once

#include "skv_internal.cuh"

namespace skv {

constexpr int kCellTokens = 16;
constexpr int kCodeBytes = 64;  // of a token
__host__ __device__ constexpr int kv4_cell(int ng) { return kCellTokens * (kCodeBytes + 4 * ng); }

// min and max that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A group's word from its least and largest entry, and the entry's code under it.  The range is
// an fp32 difference: one that passes fp32, or a NaN, makes both halves NaN.
__device__ __forceinline__ uint32_t kv4_word(float lo, float hi, float* s, float* z) {
  const float range = hi - lo;
  if (!(range <= 3.402823466e38f)) {
    *s = *z = 0.f;
    return 0x7fc07fc0u;
  }
  const __nv_bfloat16 sb = __float2bfloat16_rn(range / 15.f);
  *s = __bfloat162float(sb);
  // (halves first: a sum of two large entries stays in range)
  const __nv_bfloat16 zb = __float2bfloat16_rn(fmaf(0.5f, hi, 0.5f * lo) + 0.5f * *s);
  *z = __bfloat162float(zb);
  return (uint32_t)__bfloat16_as_ushort(sb) | ((uint32_t)__bfloat16_as_ushort(zb) << 16);
}
// The whole number next to (x - z) / s, ties to even, held to [-8, 7], and 8 more; 8 where s is 0.
__device__ __forceinline__ uint32_t kv4_code(float x, float s, float z) {
  return (uint32_t)((s > 0.f ? (int)fminf(fmaxf(rintf((x - z) / s), -8.f), 7.f) : 0) + 8);
}
// The same of many entries by s's reciprocal: a product with it, corrected by its own remainder, is the
// quotient as a division rounds it (Markstein's correction), borders and all; the whole number is in the low
// bits of its sum with 1.5 * 2^23 (entries lie within 2^18 steps of z).  For steps from 2^-100 up.
__device__ __forceinline__ uint32_t kv4_code(float x, float s, float z, float inv) {
  const float d = x - z, q = d * inv, y = fmaf(fmaf(-q, s, d), inv, q) + 12582912.f;
  const int c = __float_as_int(y) - (0x4b400000 - 8);
  return (uint32_t)(c < 0 ? 0 : c > 15 ? 15 : c);
}

}  // namespace skv
