// The 8-bit cache format: E4M3 codes with one fp32 scale for each block of 16 tokens of a KV head.
//
// A pool is [num_pages][Hkv][page_tokens][D] of codes, its scales [num_pages][Hkv][page_tokens / 16].  An element
// is scale * code; a code has 4 significant bits and lies in 2^-9 .. 448 or is 0, so fp16 holds it exactly.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dkv_internal.cuh"

namespace dkv {
namespace e4m3 {

constexpr int kBlock = 16;
// The scales that the append writes: 448 times the smallest is 2^-55, and the largest holds every bf16 number.
constexpr int kMinExp = -64, kMaxExp = 120;

// The smallest power of two, in that range, that brings the number with these bits (not negative) to at most
// 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(uint32_t top) {
  const int k = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)(min(max(k, kMinExp), kMaxExp) + 127) << 23);
}

// Two codes (the low 16 bits of `w`) as an fp16 pair, the first in its low half.
__device__ __forceinline__ uint32_t lo_to_h2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// The two in the high 16 bits.
__device__ __forceinline__ uint32_t hi_to_h2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// log2 of a positive normal number: its exponent, exactly, and its significand's to 2^-22.
__device__ __forceinline__ float log2_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return (float)((int)(u >> 23) - 127) + __log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
}

// Codes of four numbers, to nearest even; a NaN gives NaN, what is above 448 gives 448.
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

}  // namespace e4m3
}  // namespace dkv
