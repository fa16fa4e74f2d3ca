// Keys and values rounded to 4 bits and written into the paged cache.
//
// Per 16 consecutive elements of a head: the scale s is the 8-bit float (four
// exponent bits, three mantissa bits) nearest max|x| / (6 g), and each code the
// 4-bit level nearest x / (s g), so the largest element takes the largest level
// (6) up to the scale's rounding.
//
// One thread a group; a warp covers consecutive tokens of one head, so codes and
// scales of neighbouring slots leave in whole sectors.
//
// Bound by memory on long runs: 65553 tokens of 8 heads of 128 bf16 elements move
// 613 MB in 119 us, 5.1 TB/s of the 6.8 of a copy; 1024 tokens take 3.1 us in a
// graph (1.4 us of copying, 5.4 us a call from Python).  Without the values as
// stored the long run moves 344 MB in 101 us.  With a division an element it took
// 168 us.
#include "spec_cache.cuh"

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
  Group4 y;
  if (round_group(x, g, y)) set_status(p.status, SPEC_DEV_BAD_KV);
  const int page = slot / p.P, tok = slot - page * p.P;
  uint8_t* blk = p.cache + cache_block_at(page, h, tok >> 4, p.Hkv, p.bpp, p.D) + (which ? cache_v_codes(p.D) : 0);
  *reinterpret_cast<uint2*>(blk + (tok & 15) * (p.D / 2) + grp * 8) = make_uint2(y.code[0], y.code[1]);
  blk[cache_k_scales(p.D) + (tok & 15) * (p.D / 16) + grp] = (uint8_t)y.scale;
  if (stored) {
    stored_group(y, g, x);
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
