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
__device__ __forceinline__ uint32_t kv4_code(float x, float s, float z) {
  const float c = s > 0.f ? rintf((x - z) / s) : 0.f;
  return (uint32_t)((int)fminf(fmaxf(c, -8.f), 7.f) + 8);
}

}  // namespace skv
