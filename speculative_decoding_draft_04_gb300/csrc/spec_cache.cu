// Keys and values rounded to 4 bits and written into the paged cache.
//
// Per 16 consecutive elements of a head: the scale s is the 8-bit float (four
// exponent bits, three mantissa bits) nearest max|x| / (6 g), and each code the
// 4-bit level nearest x / (s g), so the largest element takes the largest level
// (6) up to the scale's rounding.  One thread a group.
#include "spec_serve.cuh"

namespace spec {

struct AppendParams {
  int T, Hkv, D, P, bpp;                 // bpp: blocks of 16 tokens a page
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

// Codes of two numbers already divided by the scale (lo in the low half).
__device__ __forceinline__ uint32_t encode_pair(float lo, float hi) {
  uint32_t r;
  asm("{.reg .b8 b; cvt.rn.satfinite.e2m1x2.f32 b, %1, %2; mov.b32 %0, {b, b, b, b};}" : "=r"(r) : "f"(hi), "f"(lo));
  return r & 0xffu;
}

template <class DT>
__global__ void __launch_bounds__(APPEND_THREADS) cache_append_kernel(AppendParams p) {
  const int gpr = p.Hkv * (p.D / 16);                    // groups a row
  const long long n = (long long)p.T * gpr;
  const int which = blockIdx.y;                          // keys, values
  const float g = p.g[which], g6 = __fmul_rn(6.f, g);
  uint32_t flags = 0;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int t = (int)(i / gpr), in_row = (int)(i - (long long)t * gpr);
    const int h = in_row / (p.D / 16), grp = in_row - h * (p.D / 16);
    const int slot = __ldg(p.slots + t);
    float x[16];
    DT* stored = static_cast<DT*>(p.stored[which]);
    if (stored) stored += (size_t)i * 16;
    if (slot < 0 || slot >= p.num_slots) {
      if (slot != -1) flags |= SPEC_DEV_BAD_SLOT;
      if (stored) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = 0.f;
        store16(stored, x);
      }
      continue;
    }
    load16(static_cast<const DT*>(p.x[which]) + t * p.row_stride[which] + h * p.head_stride[which] + grp * 16, x);
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (!(fabsf(x[e]) <= 3.402823466e38f)) {
        flags |= SPEC_DEV_BAD_KV;
        if (x[e] != x[e]) x[e] = 0.f;
      }
      amax = fmaxf(amax, fabsf(x[e]));
    }
    uint16_t sb;
    const float tq = __fdiv_rn(amax, g6);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(sb) : "f"(0.f), "f"(tq));
    const float s = half2_floats(decode_scales(sb)).x;
    const float r = __fmul_rn(s, g);
    uint32_t w[2] = {0, 0};
    if (r > 0.f) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e >> 2] |= encode_pair(__fdiv_rn(x[2 * e], r), __fdiv_rn(x[2 * e + 1], r)) << (8 * (e & 3));
    }
    const int page = slot / p.P, tok = slot - page * p.P;
    uint8_t* blk = p.cache + cache_block_at(page, h, tok >> 4, p.Hkv, p.bpp, p.D) + (which ? cache_v_codes(p.D) : 0);
    *reinterpret_cast<uint2*>(blk + (tok & 15) * (p.D / 2) + grp * 8) = make_uint2(w[0], w[1]);
    blk[8 * p.D + (tok & 15) * (p.D / 16) + grp] = (uint8_t)sb;
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
  if (flags) set_status(p.status, flags);
}

cudaError_t launch_cache_append(const spec_cache_append_args& a, int sms, cudaStream_t st) {
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
  const long long n = (long long)a.T * a.Hkv * (a.D / 16);
  if (n == 0) return cudaSuccess;
  long long ctas = (n + APPEND_THREADS - 1) / APPEND_THREADS;
  if (ctas > 8LL * sms) ctas = 8LL * sms;
  const dim3 grid((unsigned)ctas, 2);
  if (a.dtype == SPEC_BF16) cache_append_kernel<bf16><<<grid, APPEND_THREADS, 0, st>>>(p);
  else cache_append_kernel<float><<<grid, APPEND_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace spec
