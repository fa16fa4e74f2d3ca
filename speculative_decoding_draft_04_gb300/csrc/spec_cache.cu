// Keys and values rounded to 4 bits and written into the paged cache.
//
// Per 16 consecutive elements of a head: the scale s is the 8-bit float (four
// exponent bits, three mantissa bits) nearest max|x| / (6 g), and each code the
// 4-bit level nearest x / (s g), so the largest element takes the largest level
// (6) up to the scale's rounding.
//
// One thread a group; a warp covers consecutive tokens of one head, so codes and
// scales of neighbouring slots leave in whole sectors.  The quotients are those
// of IEEE division, from the rounded reciprocal y of r = s g: q = x y,
// q - (q r - x) y with fused multiply-adds is the rounded quotient (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34, 1990).  That holds while nothing over- or underflows:
// |x| <= 8 r here, and where x - q r is below the normal numbers, x / r is below
// 2^-30 and the code is 0 either way.  Groups whose scale saturates, or with an
// element that is not finite, are divided by the plain division.
//
// Bound by memory on long runs: 65553 tokens of 8 heads of 128 bf16 elements move
// 613 MB in 119 us, 5.1 TB/s of the 6.8 of a copy; 1024 tokens take 3.1 us in a
// graph (1.4 us of copying, 5.4 us a call from Python).  Without the values as
// stored the long run moves 344 MB in 101 us.  With a division an element it took
// 168 us.
#include "spec_serve.cuh"

namespace spec {

struct AppendParams {
  int T, Hkv, D, P, bpp;                 // bpp: blocks of 16 tokens a page
  int gbits;                             // log2 of the groups a head
  uint64_t head_magic;                   // ceil(2^40 / Hkv): i / Hkv = i * magic >> 40 for i < 2^28
  int num_slots;
  const void* x[2];
  long long row_stride[2], head_stride[2];
  const int* slots;
  float g[2];
  uint8_t* cache;
  void* stored[2];
  uint32_t* status;
};

constexpr int APPEND_THREADS = 256;

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

template <class DT>
__global__ void __launch_bounds__(APPEND_THREADS) cache_append_kernel(const __grid_constant__ AppendParams p) {
  // (16 tokens, head, token, group), the last fastest
  const uint32_t i = blockIdx.x * APPEND_THREADS + threadIdx.x;
  const int grp = i & ((1 << p.gbits) - 1), rest = i >> (p.gbits + 4);
  const int t16 = (int)((uint64_t)rest * p.head_magic >> 40), h = rest - t16 * p.Hkv;
  const int t = t16 * 16 + ((i >> p.gbits) & 15);
  if (t >= p.T) return;
  const int which = blockIdx.y;                          // keys, values
  const float g = p.g[which];
  const int slot = __ldg(p.slots + t);
  float x[16];
  DT* stored = static_cast<DT*>(p.stored[which]);
  if (stored) stored += ((size_t)t * p.Hkv + h) * p.D + grp * 16;
  if (slot < 0 || slot >= p.num_slots) {
    if (slot != -1) set_status(p.status, SPEC_DEV_BAD_SLOT);
    if (stored) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
      store16(stored, x);
    }
    return;
  }
  load16(static_cast<const DT*>(p.x[which]) + t * p.row_stride[which] + h * p.head_stride[which] + grp * 16, x);
  float amax = 0.f;                                      // of the numbers: a NaN is passed over
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    amax = fmaxf(amax, fabsf(x[e]));
    odd |= !(fabsf(x[e]) <= 3.402823466e38f);
  }
  uint16_t sb;
  const float tq = __fdiv_rn(amax, __fmul_rn(6.f, g));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.f), "f"(tq));
  const float s = half2_floats(decode_scales(sb)).x;
  const float r = __fmul_rn(s, g);
  uint32_t w[2] = {0, 0};
  if (!odd && amax <= 8.f * r) {
    if (r > 0.f) {
      const float y = __frcp_rn(r);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float q = __fmul_rn(x[e], y);
        x[e] = __fmaf_rn(-__fmaf_rn(q, r, -x[e]), y, q);   // this way round, -0 / r stays -0
      }
      w[0] = encode8(x);
      w[1] = encode8(x + 8);
    }
  } else if (r > 0.f) {
    if (odd) set_status(p.status, SPEC_DEV_BAD_KV);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = x[e] != x[e] ? 0.f : __fdiv_rn(x[e], r);
    w[0] = encode8(x);
    w[1] = encode8(x + 8);
  } else if (odd) {
    set_status(p.status, SPEC_DEV_BAD_KV);               // a NaN among zeros
  }
  const int page = slot / p.P, tok = slot - page * p.P;
  uint8_t* blk = p.cache + cache_block_at(page, h, tok >> 4, p.Hkv, p.bpp, p.D) + (which ? cache_v_codes(p.D) : 0);
  *reinterpret_cast<uint2*>(blk + (tok & 15) * (p.D / 2) + grp * 8) = make_uint2(w[0], w[1]);
  blk[cache_k_scales(p.D) + (tok & 15) * (p.D / 16) + grp] = (uint8_t)sb;
  if (stored) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t d[4] = {decode_pair<0>(w[q]), decode_pair<1>(w[q]), decode_pair<2>(w[q]), decode_pair<3>(w[q])};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = half2_floats(d[e]);
        x[8 * q + 2 * e] = __fmul_rn(__fmul_rn(v.x, s), g);
        x[8 * q + 2 * e + 1] = __fmul_rn(__fmul_rn(v.y, s), g);
      }
    }
    store16(stored, x);
  }
}

cudaError_t launch_cache_append(const spec_cache_append_args& a, cudaStream_t st) {
  AppendParams p{};
  p.T = a.T; p.Hkv = a.Hkv; p.D = a.D; p.P = a.page_size; p.bpp = a.page_size / CACHE_BLOCK;
  p.num_slots = a.num_pages * a.page_size;
  p.x[0] = a.k; p.x[1] = a.v;
  p.row_stride[0] = a.k_row_stride; p.row_stride[1] = a.v_row_stride;
  p.head_stride[0] = a.k_head_stride; p.head_stride[1] = a.v_head_stride;
  p.slots = a.slots;
  p.g[0] = a.k_scale; p.g[1] = a.v_scale;
  p.cache = a.cache;
  p.stored[0] = a.k_stored; p.stored[1] = a.v_stored;
  p.status = a.dev_status;
  if (a.T == 0) return cudaSuccess;
  p.gbits = a.D == 64 ? 2 : a.D == 128 ? 3 : 4;
  p.head_magic = ((1ull << 40) + a.Hkv - 1) / a.Hkv;
  const long long n = (long long)((a.T + 15) / 16) * a.Hkv << (p.gbits + 4);   // below 2^32
  const dim3 grid((unsigned)((n + APPEND_THREADS - 1) / APPEND_THREADS), 2);
  if (a.dtype == SPEC_BF16) cache_append_kernel<bf16><<<grid, APPEND_THREADS, 0, st>>>(p);
  else cache_append_kernel<float><<<grid, APPEND_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace spec
