// The 4-bit cache format: E2M1 codes with one E4M3 scale for 16 elements.
//
// A page of one KV head is one run of bytes: page_tokens rows of D/2 code bytes
// (element 2i in the low four bits of byte i), then page_tokens rows of D/16
// scale bytes.  A pool is [num_pages][Hkv][page_tokens * D * 9 / 16].
// An element is scale * code, which has at most 6 significant bits (4 of the
// scale, 2 of the code) and lies in 2^-10 .. 2688 or is 0: fp16 and bf16 hold it
// exactly, so reading the cache rounds nothing.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "dkv_internal.cuh"

namespace dkv {
namespace e2m1 {

constexpr int kMinPageTokens = 16;  // a 16-row step of the attention stays inside a page

__host__ __device__ constexpr int code_bytes(int D) { return D / 2; }
__host__ __device__ constexpr int scale_bytes(int D) { return D / 16; }
__host__ __device__ constexpr size_t page_bytes(int D, int page_tokens) {
  return (size_t)page_tokens * (code_bytes(D) + scale_bytes(D));
}

// Two codes (the low byte of `b`) as two fp16 numbers, the low code in the low half.
__device__ __forceinline__ uint32_t codes_to_h2(uint32_t b) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)b, __NV_E2M1);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

// Two E4M3 scales (the low 16 bits of `s`) as two fp16 numbers.
__device__ __forceinline__ uint32_t scales_to_h2(uint32_t s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)s, __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

}  // namespace e2m1
}  // namespace dkv
