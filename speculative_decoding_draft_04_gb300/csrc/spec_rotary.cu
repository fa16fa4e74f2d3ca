// Queries, keys and values of new tokens made ready for attention in one pass over
// a fused projection's rows: norm of each query and key head, rotation by the
// token's position, queries written out, keys and values rounded to 4 bits into
// the paged cache.
//
//   inv = 1 / sqrt(mean x^2 + eps),  y = (x inv) w
//   y_a' = y_a c - y_b s,  y_b' = y_b c + y_a s
//
// The sum of squares is kept to about 2^-48 of itself and inv is its reciprocal root by one Newton
// step, so that inv is the nearest fp32 number unless the exact one lies within 2^-19 of a unit in the last
// place of a midpoint (4 of 12.8 million random heads): a 4-bit code is decided by the last bit of a key
// that lies next to a border.
//
// A thread has 32 elements of a head, two groups of 16 that one scale each
// describes in the cache: groups g and g + R / 32 where pairs are halves apart, so
// that both elements of a pair are its own, neighbouring groups elsewhere.  D / 32
// lanes share a head, a warp has 1024 / D heads of one token, and a warp that goes
// on to more heads of its token keeps the cosines and sines and requests the next
// heads before it works on the ones that it has.
//
// Long runs are bound by instructions and memory alike: 30011 tokens of 32 + 8 + 8 heads
// of 128 bf16 elements move 787 MB in 166 us, 4.7 TB/s of the 6.8 of a copy, with 65 % of
// the issue slots taken (22 instructions an element; 252 us with the sums of squares by
// TwoSum, one group of heads a warp and nothing ahead).  1024 tokens take 12.6 us a call
// (4.0 us of reading and writing): the heads are requested first, slot and position beside them, and
// only the rotation's row waits for the position; small CTAs in two and a half waves.  fp32 has no
// registers for heads ahead, so a warp has nothing in flight while it computes: 4099 tokens of
// 16 + 4 + 4 heads of 256, 207 MB, take 64 us (with heads ahead in registers 67, with five CTAs an SM
// 74, spilling); 1024 tokens of 32 + 8 + 8 heads of 128 23 us, 15000 of them 205, of 7.7 and 112.
#include "spec_cache.cuh"
#include "spec_df.cuh"

namespace spec {

struct RotaryParams {
  int T, Hq, Hkv, R, P, bpp;              // bpp: blocks of 16 tokens a page
  int num_slots, rope_rows, interleaved;
  int chunks, per_warp;                   // groups of heads a token, and of them a warp's
  const void* x[3];                       // queries, keys, values
  long long row[3], head[3];
  const void* weight[2];
  const int* positions;
  const int* slots;
  const float* rope;
  float eps, g[2];
  void* q_out;
  long long out_row, out_head;
  uint8_t* cache;
  void* stored[2];
  uint32_t* status;
};

constexpr int ROTARY_THREADS = 128;

__device__ __forceinline__ float rounded_to(const bf16*, float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
__device__ __forceinline__ float rounded_to(const float*, float x) { return x; }

// 1 / sqrt(v), from the approximate root by one Newton step whose residual 1 - v r^2 is formed in
// double-float: off by 1.5 d^2 (d at most 2^-22, the root's error) before its rounding.
__device__ __forceinline__ float root_reciprocal(df v) {
  const float r = rsqrtf(v.hi);
  const df p = dd_mul(v, two_prod_df(r, r));
  const float e = rn_sub(rn_sub(1.f, p.hi), p.lo);
  return rn_fma(r, rn_mul(0.5f, e), r);
}

// The sum of a head's squares over its LANES lanes, 32 elements each, in double-float.
// A plain sum first gives a power of two s0 above twice the sum.  Added to s0, every
// partial sum stays within [s0, 2 s0): what an addition rounds away, fma(x, x, s - s'), is itself
// rounded to about 2^-48 of the sum, and the partial sums less s0 add up without rounding.
template <int LANES>
__device__ __forceinline__ df sum_of_squares(const float (&a)[16], const float (&b)[16]) {
  float pa = 0.f, pb = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    pa = fmaf(a[i], a[i], pa);
    pb = fmaf(b[i], b[i], pb);
  }
  float plain = pa + pb;
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) plain += __shfl_xor_sync(0xffffffffu, plain, o);
  const float s0 = __uint_as_float((__float_as_uint(plain) & 0x7f800000u) + (2u << 23));
  float sa = s0, sb = s0, ca = 0.f, cb = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float ta = rn_fma(a[i], a[i], sa), tb = rn_fma(b[i], b[i], sb);
    ca = rn_add(ca, rn_fma(a[i], a[i], rn_sub(sa, ta)));
    cb = rn_add(cb, rn_fma(b[i], b[i], rn_sub(sb, tb)));
    sa = ta;
    sb = tb;
  }
  float hi = rn_add(rn_sub(sa, s0), rn_sub(sb, s0)), lo = rn_add(ca, cb);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    hi = rn_add(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = rn_add(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  return two_sum_df(hi, lo);
}

// Sixteen elements as they are in memory.
template <class DT>
struct Raw16 {
  uint4 v[sizeof(DT)];
  __device__ __forceinline__ void load(const DT* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(DT); ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void read(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(DT); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (sizeof(DT) == 2) {
          x[8 * (i & 1) + 2 * k] = __uint_as_float(w[k] << 16);
          x[8 * (i & 1) + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
          x[4 * i + k] = __uint_as_float(w[k]);
        }
      }
    }
  }
};

template <int D, class DT>
__global__ void __launch_bounds__(ROTARY_THREADS, sizeof(DT) == 2 ? 4 : 3) rotary_append_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int LANES = D / 32, HEADS = 32 / LANES;          // lanes a head, heads a warp
  const int lane = threadIdx.x & 31, j = lane % LANES;
  const long long item = (long long)blockIdx.x * (ROTARY_THREADS / 32) + (threadIdx.x >> 5);
  const int runs = (p.chunks + p.per_warp - 1) / p.per_warp;
  const int t = (int)(item / runs), c0 = (int)(item - (long long)t * runs) * p.per_warp;
  if (t >= p.T) return;
  const int total = p.Hq + 2 * p.Hkv;
  const bool apart = !p.interleaved && 32 * j < p.R, turn = 32 * j < p.R;
  // the thread's two groups of elements, and its pairs of the rotation
  const int ea = apart ? 16 * j : 32 * j, eb = apart ? p.R / 2 + 16 * j : 32 * j + 16;
  // of the heads that come next: the first ones are requested before slot and position
  // are known, later ones (bf16: fp32 has no registers for them) while others are worked on
  constexpr bool AHEAD = sizeof(DT) == 2;
  Raw16<DT> ra, rb;
  auto request = [&](int c) {
    const int head = c * HEADS + lane / LANES;
    if (head >= total) return;
    const int kind = head < p.Hq ? 0 : head < p.Hq + p.Hkv ? 1 : 2;
    const int h = kind == 0 ? head : kind == 1 ? head - p.Hq : head - p.Hq - p.Hkv;
    const DT* src = static_cast<const DT*>(p.x[kind]) + t * p.row[kind] + h * p.head[kind];
    ra.load(src + ea);
    rb.load(src + eb);
  };
  const int c1 = min(c0 + p.per_warp, p.chunks);
  request(c0);
  const int slot = __ldg(p.slots + t), position = __ldg(p.positions + t);
  const bool skip = slot == -1;
  const bool bad_slot = !skip && (slot < 0 || slot >= p.num_slots);
  const bool bad_position = !skip && (position < 0 || position >= p.rope_rows);
  if (c0 == 0 && lane == 0 && (bad_slot || bad_position))
    set_status(p.status, (bad_slot ? SPEC_DEV_BAD_SLOT : 0) | (bad_position ? SPEC_DEV_BAD_POSITION : 0));
  const bool bad = bad_slot || bad_position;

  float cs[32];
  if (turn && !skip && !bad) {
    const float4* r = reinterpret_cast<const float4*>(p.rope + (long long)position * p.R + 32 * j);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = __ldg(r + i);
      cs[4 * i] = v.x; cs[4 * i + 1] = v.y; cs[4 * i + 2] = v.z; cs[4 * i + 3] = v.w;
    }
  }

  for (int c = c0; c < c1; ++c) {
    const int head = c * HEADS + lane / LANES;
    const int kind = head < p.Hq ? 0 : head < p.Hq + p.Hkv ? 1 : 2;
    const int h = kind == 0 ? head : kind == 1 ? head - p.Hq : head - p.Hq - p.Hkv;
    const bool live = head < total;
    if (!AHEAD && c > c0) request(c);
    float a[16], b[16];
    if (skip || bad) {                                       // the whole warp
      if (!live) continue;
      if (kind == 0) {
        if (bad) {
          DT* out = static_cast<DT*>(p.q_out) + t * p.out_row + h * p.out_head;
#pragma unroll
          for (int i = 0; i < 16; ++i) a[i] = quiet_nan();
          store16(out + ea, a);
          store16(out + eb, a);
        }
      } else if (p.stored[kind - 1]) {
        DT* out = static_cast<DT*>(p.stored[kind - 1]) + ((size_t)t * p.Hkv + h) * D;
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = 0.f;
        store16(out + ea, a);
        store16(out + eb, a);
      }
      continue;
    }
    if (live) {
      ra.read(a);
      rb.read(b);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i] = b[i] = 1.f;
    }
    if (AHEAD && c + 1 < c1) request(c + 1);
    // ---- norm
    const void* weight = kind == 2 ? nullptr : p.weight[kind];
    if (__any_sync(0xffffffffu, weight != nullptr)) {
      df v = sum_of_squares<LANES>(a, b);
      v = dd_add_f(df{v.hi * (1.f / D), v.lo * (1.f / D)}, p.eps);
      float inv = root_reciprocal(v);
      // squares that leave the range of fp32: the sum in 64 bits
      if (__any_sync(0xffffffffu, weight && !(v.hi >= 1e-20f && v.hi <= 1e35f))) {
        double wide = 0.;
#pragma unroll
        for (int i = 0; i < 16; ++i) wide += (double)a[i] * a[i] + (double)b[i] * b[i];
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) wide += __shfl_xor_sync(0xffffffffu, wide, o);
        if (!(v.hi >= 1e-20f && v.hi <= 1e35f)) inv = (float)(1. / sqrt(wide / D + (double)p.eps));
      }
      if (weight) {
        float w[16];
        load16(static_cast<const DT*>(weight) + ea, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = rn_mul(rn_mul(a[i], inv), w[i]);
        load16(static_cast<const DT*>(weight) + eb, w);
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = rn_mul(rn_mul(b[i], inv), w[i]);
      }
    }
    if (!live) continue;
    // ---- rotation
    if (kind < 2 && turn) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = a[2 * i], y = a[2 * i + 1], z = b[2 * i], w = b[2 * i + 1];
          a[2 * i] = rn_sub(rn_mul(x, cs[2 * i]), rn_mul(y, cs[2 * i + 1]));
          a[2 * i + 1] = rn_add(rn_mul(y, cs[2 * i]), rn_mul(x, cs[2 * i + 1]));
          b[2 * i] = rn_sub(rn_mul(z, cs[16 + 2 * i]), rn_mul(w, cs[17 + 2 * i]));
          b[2 * i + 1] = rn_add(rn_mul(w, cs[16 + 2 * i]), rn_mul(z, cs[17 + 2 * i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x = a[i], y = b[i];
          a[i] = rn_sub(rn_mul(x, cs[2 * i]), rn_mul(y, cs[2 * i + 1]));
          b[i] = rn_add(rn_mul(y, cs[2 * i]), rn_mul(x, cs[2 * i + 1]));
        }
      }
    }
    if (kind == 0) {
      DT* out = static_cast<DT*>(p.q_out) + t * p.out_row + h * p.out_head;
      store16(out + ea, a);
      store16(out + eb, b);
      continue;
    }
    // ---- keys (rounded to their type first) and values into the cache
    const int which = kind - 1;
    const float g = p.g[which];
    const int page = slot / p.P, tok = slot - page * p.P;
    uint8_t* blk = p.cache + cache_block_at(page, h, tok >> 4, p.Hkv, p.bpp, D) + (which ? cache_v_codes(D) : 0);
    uint8_t* codes = blk + (tok & 15) * (D / 2);
    uint8_t* scales = blk + cache_k_scales(D) + (tok & 15) * (D / 16);
    DT* stored = p.stored[which] ? static_cast<DT*>(p.stored[which]) + ((size_t)t * p.Hkv + h) * D : nullptr;
    bool odd = false;
    auto store = [&](float (&x)[16], int e0) {
      if (kind == 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = rounded_to(static_cast<const DT*>(nullptr), x[i]);
      }
      Group4 y;
      odd |= round_group(x, g, y);
      *reinterpret_cast<uint2*>(codes + e0 / 2) = make_uint2(y.code[0], y.code[1]);
      scales[e0 / 16] = (uint8_t)y.scale;
      if (stored) {
        stored_group(y, g, x);
        store16(stored + e0, x);
      }
    };
    store(a, ea);
    store(b, eb);
    if (odd) set_status(p.status, SPEC_DEV_BAD_KV);
  }
}

namespace {
template <int D, class DT>
cudaError_t launch_rotary(RotaryParams p, int sms, cudaStream_t st) {
  constexpr int HEADS = 1024 / D;
  p.chunks = (p.Hq + 2 * p.Hkv + HEADS - 1) / HEADS;
  // a bf16 warp goes on to further heads of its token where there are warps enough
  int parts = p.chunks;
  while (sizeof(DT) == 2 && parts > 1 && (long long)p.T * (parts - 1) >= 32LL * sms) --parts;
  p.per_warp = (p.chunks + parts - 1) / parts;
  const long long runs = (p.chunks + p.per_warp - 1) / p.per_warp;
  const long long warps = runs * p.T;
  const long long ctas = (warps + ROTARY_THREADS / 32 - 1) / (ROTARY_THREADS / 32);
  rotary_append_kernel<D, DT><<<(unsigned)ctas, ROTARY_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_rotary_append(const spec_rotary_append_args& a, int sms, cudaStream_t st) {
  RotaryParams p{};
  p.T = a.T; p.Hq = a.Hq; p.Hkv = a.Hkv; p.R = a.R; p.P = a.page_size; p.bpp = a.page_size / CACHE_BLOCK;
  p.num_slots = a.num_pages * a.page_size;
  p.rope_rows = a.rope_rows;
  p.interleaved = a.interleaved;
  p.x[0] = a.q; p.x[1] = a.k; p.x[2] = a.v;
  p.row[0] = a.q_row_stride; p.row[1] = a.k_row_stride; p.row[2] = a.v_row_stride;
  p.head[0] = a.q_head_stride; p.head[1] = a.k_head_stride; p.head[2] = a.v_head_stride;
  p.weight[0] = a.q_weight; p.weight[1] = a.k_weight;
  p.positions = a.positions;
  p.slots = a.slots;
  p.rope = a.rope;
  p.eps = a.eps;
  p.g[0] = a.k_scale; p.g[1] = a.v_scale;
  p.q_out = a.q_out;
  p.out_row = a.q_out_row_stride; p.out_head = a.q_out_head_stride;
  p.cache = a.cache;
  p.stored[0] = a.k_stored; p.stored[1] = a.v_stored;
  p.status = a.dev_status;
  if (a.dtype == SPEC_BF16)
    return a.D == 64    ? launch_rotary<64, bf16>(p, sms, st)
           : a.D == 128 ? launch_rotary<128, bf16>(p, sms, st)
                        : launch_rotary<256, bf16>(p, sms, st);
  return a.D == 64    ? launch_rotary<64, float>(p, sms, st)
         : a.D == 128 ? launch_rotary<128, float>(p, sms, st)
                      : launch_rotary<256, float>(p, sms, st);
}

}  // namespace spec
