// Definitions shared by the operators of the target model's side of a cycle
// (block tables, 4-bit cache, attention over it, log probabilities).
#pragma once

#include <cuda_fp16.h>

#include "spec_internal.cuh"

namespace spec {

// ---------------------------------------------------------------- 4-bit cache
// A block of 16 tokens of one key-value head: K codes [16][D/2], K scales
// [16][D/16], V codes [16][D/2], V scales [16][D/16] -- 18 D bytes.
constexpr int CACHE_BLOCK = 16;
__host__ __device__ constexpr int cache_block_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int cache_k_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int cache_v_codes(int D) { return 9 * D; }
__host__ __device__ constexpr int cache_v_scales(int D) { return 17 * D; }

// Block `blk` of page `page`, head h.  64-bit: a cache passes 2^32 bytes.
__device__ __forceinline__ size_t cache_block_at(long long page, int h, int blk, int Hkv, int blocks_per_page,
                                                 int D) {
  return (size_t)((page * Hkv + h) * blocks_per_page + blk) * cache_block_bytes(D);
}

// The two elements of byte I of a word of codes as 16-bit floats (the low half
// of the byte in the low half of the result).
template <int I>
__device__ __forceinline__ uint32_t decode_pair(uint32_t w) {
  uint32_t r;
  if (I == 0) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(r) : "r"(w));
  if (I == 1) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(r) : "r"(w));
  if (I == 2) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(r) : "r"(w));
  if (I == 3) asm("{.reg .b8 a,b,c,d; mov.b32 {a,b,c,d}, %1; cvt.rn.f16x2.e2m1x2 %0, d;}" : "=r"(r) : "r"(w));
  return r;
}
// Two scale bytes as 16-bit floats.
__device__ __forceinline__ uint32_t decode_scales(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two fp32 numbers in one operand; additions and products of both in one
// instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

}  // namespace spec
