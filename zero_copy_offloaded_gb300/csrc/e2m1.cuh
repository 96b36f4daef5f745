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

// The eight codes of a word as four fp16 pairs; pair i holds byte i's two codes, the
// low one in its low half.  One conversion instruction a pair, straight from the byte.
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t (&x)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
      : "r"(w));
}

// Two E4M3 scales (the low 16 bits of `s`) as two fp16 numbers.
__device__ __forceinline__ uint32_t scales_to_h2(uint32_t s) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(s));
  return r;
}

}  // namespace e2m1
}  // namespace dkv
