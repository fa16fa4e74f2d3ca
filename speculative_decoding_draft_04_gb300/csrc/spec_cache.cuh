// Rounding of 16 elements of a head to 4 bits, shared by the kernels that write the
// paged cache: the scale is the 8-bit float (four exponent bits, three mantissa
// bits) nearest max|x| / (6 g), each code the 4-bit level nearest x / (s g).
//
// The quotients are those of IEEE division, from the rounded reciprocal y of
// r = s g: q = x y, q - (q r - x) y with fused multiply-adds is the rounded quotient
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", IBM J. Res. Dev. 34, 1990).  That holds while nothing over- or
// underflows: |x| <= 8 r here, and where x - q r is below the normal numbers, x / r
// is below 2^-30 and the code is 0 either way.  Groups whose scale saturates, or
// with an element that is not finite, are divided by the plain division.
#pragma once

#include "spec_serve.cuh"

namespace spec {

__device__ __forceinline__ void load16(const bf16* p, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + h);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
      x[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void load16(const float* p, float* x) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + h);
    x[4 * h] = v.x; x[4 * h + 1] = v.y; x[4 * h + 2] = v.z; x[4 * h + 3] = v.w;
  }
}
__device__ __forceinline__ void store16(bf16* p, const float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(x[8 * h + 2 * i], x[8 * h + 2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&t);
    }
    reinterpret_cast<uint4*>(p)[h] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void store16(float* p, const float* x) {
#pragma unroll
  for (int h = 0; h < 4; ++h)
    reinterpret_cast<float4*>(p)[h] = make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
}

// Codes of four pairs of numbers already divided by the scale.
__device__ __forceinline__ uint32_t encode8(const float* y) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// Sixteen elements as stored: codes, and the scale's byte and value.
struct Group4 {
  uint32_t code[2];
  uint16_t scale;
  float s;
};

// Rounds x (which it overwrites) under the cache's scale g.  True: an element was
// not finite.
__device__ __forceinline__ bool round_group(float (&x)[16], float g, Group4& out) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(x[e])));
  const bool odd = !(amax <= 3.402823466e38f);
  if (amax != amax) {                                    // of the numbers: a NaN is passed over
    amax = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
  }
  const float tq = __fdiv_rn(amax, __fmul_rn(6.f, g));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out.scale) : "f"(0.f), "f"(tq));
  out.s = half2_floats(decode_scales(out.scale)).x;
  const float r = __fmul_rn(out.s, g);
  out.code[0] = out.code[1] = 0;
  if (!odd && amax <= 8.f * r) {
    if (r > 0.f) {
      const float y = __frcp_rn(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float q = __fmul_rn(x[e], y);
        x[e] = __fmaf_rn(-__fmaf_rn(q, r, -x[e]), y, q);   // this way round, -0 / r stays -0
      }
      out.code[0] = encode8(x);
      out.code[1] = encode8(x + 8);
    }
  } else if (r > 0.f) {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = x[e] != x[e] ? 0.f : __fdiv_rn(x[e], r);
    out.code[0] = encode8(x);
    out.code[1] = encode8(x + 8);
  }
  return odd;                                            // r = 0: a NaN among zeros
}

// What the codes stand for.
__device__ __forceinline__ void stored_group(const Group4& y, float g, float (&x)[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t d[4] = {decode_pair<0>(y.code[q]), decode_pair<1>(y.code[q]), decode_pair<2>(y.code[q]),
                           decode_pair<3>(y.code[q])};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = half2_floats(d[e]);
      x[8 * q + 2 * e] = __fmul_rn(__fmul_rn(v.x, y.s), g);
      x[8 * q + 2 * e + 1] = __fmul_rn(__fmul_rn(v.y, y.s), g);
    }
  }
}

}  // namespace spec
