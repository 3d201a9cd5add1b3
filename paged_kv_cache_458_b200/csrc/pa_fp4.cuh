// pa_fp4.cuh -- the E2M1 (4-bit) cache: layout of its pools and conversions.
//
// A pool is [num_blocks][num_kv_heads] runs of block_size * D * 9 / 16 bytes:
// first the codes [block_size][D / 2] (two E2M1 codes a byte, the even
// dim in the low nibble), then the scales [block_size][D / 16] (one E4M3 code
// per 16 dims).  Everything one (block, kv head) holds is one contiguous,
// 16-byte aligned run, so a kernel that reads a head's tokens reads whole
// lines, and a copy of a block is one copy.  The stored value of a dim is
// code * block scale * head scale (the head scale one fp32 per kv head).
#pragma once

#include <cuda_fp8.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "pa_common.cuh"

namespace pa {

// Bytes of one (block, kv head) run, and of its codes.
__host__ __device__ constexpr long long fp4_head_bytes(int block_size, int head_dim) {
  return (long long)block_size * head_dim * 9 / 16;
}
__host__ __device__ constexpr long long fp4_code_bytes(int block_size, int head_dim) {
  return (long long)block_size * head_dim / 2;
}

// Eight E2M1 codes (low nibble first) -> eight f16 values, exact.  For words
// loaded whole: unpacking a zero-extended byte this way gave zeros (nvcc 12.9).
__device__ __forceinline__ void e2m1x8_to_h2(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Two E4M3 codes (low byte first) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint16_t u) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

__device__ __forceinline__ float e4m3_to_f(uint8_t u) { return e4m3x2_to_f2((uint16_t)u).x; }

__device__ __forceinline__ float2 h2_to_f2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace pa
