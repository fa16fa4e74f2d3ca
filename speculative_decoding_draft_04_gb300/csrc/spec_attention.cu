// Attention of each request's new tokens over its 4-bit paged cache.
//
//   y_ij = log2(e) softmax_scale k_scale (q_i . k_j),  p_ij = 2^(y_ij - m_i)
//   out_i = v_scale sum_j p_ij v_j / sum_j p_ij,       lse_i = ln 2 (m_i + log2 sum_j p_ij)
//
// with k_j, v_j = code * scale, exact in 16-bit floats.  The query heads of one
// key-value head and the new tokens are the rows of one product: row r of
// request b is new token r / G, query head h G + r % G (G = Hq / Hkv).
//
// cache_attention_kernel: every warp works alone on a run of 32-token units.
// All units of all (request, key-value head, row tile) segments are numbered in
// order, and warp w takes the w-th equal share of them, so ragged lengths are
// balanced to one unit and a long context is split as far as the machine goes.
// A unit of a head is contiguous in the cache (two blocks of 16 tokens, 36 D
// bytes) and comes by bulk copies into the warp's own ring in shared memory; no
// barrier joins the warps.  Codes go from shared memory to the operands of the
// warp's 16x8x16 products in registers: the order of a product's inner index is
// free as long as both operands agree, so each lane takes contiguous bytes --
// of K one run of D/4 elements of one token, of V D/8 elements (one or two
// scales) of four tokens -- and the queries are laid out in that order once a
// segment.  Scores stay in registers: the layout of the first product's result
// is the layout of the second product's operand.
//
// The running maximum follows lazily: m is the maximum last taken less 7, and
// the sums are rescaled when a score passes it by 15.  So p stays below 2^15 in
// a 16-bit float, rescaling is rare, and p keeps 11 bits down to 2^-21 of the
// row's largest and an absolute error of 2^-32 of it below that.
// p is rounded to 11 bits (two terms: 22) for the second product only; its sum
// is of the unrounded p, so lse keeps 32-bit precision.
//
// A segment inside one warp's share is written at once.  Otherwise each part is
// kept as (m, sum, unnormalised out) in the workspace and
// cache_attention_join_kernel adds the parts in the order of their warps.
#include "spec_serve.cuh"
#include "spec_tc.cuh"

namespace spec {

struct AttnParams {
  int B, T, Hq, Hkv, G, P, num_pages, stride, mask_words;
  const void* q;
  long long q_row, q_head;
  const uint8_t* cache;
  const int* table;
  const int* kv_len;
  const int* row_ptr;
  const uint32_t* mask;
  float scale;                            // softmax_scale * k_scale * log2(e)
  float v_scale;
  void* out;
  float* lse;
  uint32_t* status;
  void* ws;
};

constexpr int AT_WARPS = 8;               // warps a CTA at most
constexpr int AT_UNIT = 32;               // tokens
constexpr int AT_MAX_CTAS = 2 * 160;      // workspace slots: two CTAs an SM at most
constexpr float AT_SLACK = 8.f;           // rows are rescaled once p passes 2^(AT_SHIFT + AT_SLACK) ..
constexpr float AT_SHIFT = 7.f;           // .. which is 2^15, of the 16-bit float's 2^16

// One split segment: the warps first .. last hold its parts.
struct AttnSplit {
  int first, last;                        // last < first: no segment is split after this warp
  int b, h, tile;
  int n, r0;
};

// Geometry of a kernel: head size, row tiles of 16, terms of a 16-bit split.
template <int D_, int M_, int NT_>
struct AttnCfg {
  static constexpr int D = D_, M = M_, NT = NT_;
  static constexpr int ROWS = 16 * M;
  static constexpr int KSTEPS = D / 16;
  static constexpr int KW = D / 32;                     // K code words a lane and token
  static constexpr int KG = D / 64;                     // K scales a lane and token
  static constexpr int NV = D / 8;                      // V columns a lane and token = output tiles
  static constexpr int VW = D >= 128 ? D / 64 : 1;      // V code words a lane and token (D = 64: 4 bytes)
  static constexpr int UNIT_BYTES = 2 * 18 * D;
  static constexpr int Q_BYTES = NT * M * KSTEPS * 512;
  static constexpr int MIN_CTAS = (M == 1 && NT == 1 && D <= 128) ? 2 : 1;
  static constexpr int WARPS = D == 256 && NT == 2 ? 4 : AT_WARPS;
  static constexpr int WARP_BUDGET = (MIN_CTAS == 2 ? 110 : 220) * 1024 / WARPS;
  static constexpr int FIT = (WARP_BUDGET - Q_BYTES) / UNIT_BYTES;
  static constexpr int DEPTH = FIT > 6 ? 6 : FIT;
  static constexpr int WARP_BYTES = Q_BYTES + DEPTH * UNIT_BYTES;
  static constexpr int SMEM = WARPS * WARP_BYTES;
  // floats of a part: the accumulators lane by lane, then (m, sum) a row
  static constexpr int PART = ROWS * D + 2 * ROWS;
  static_assert(DEPTH >= 2, "ring");
};

// What a segment is: request b's units over key-value head h for one row tile.
struct AttnSeg {
  int b, h, tile, u, nu;                  // units u .. nu - 1 are left
  int n, r0, L;
  bool bad;
};

// Units of request b over all heads and row tiles (0: nothing to do).
template <int ROWS>
__device__ __forceinline__ long long attn_work(const AttnParams& p, int b, int& n, int& r0, int& L, int& tiles,
                                               int& nu, bool& bad, bool& outside) {
  r0 = __ldg(p.row_ptr + b);
  const int r1 = __ldg(p.row_ptr + b + 1);
  L = __ldg(p.kv_len + b);
  n = r1 - r0;
  outside = r0 < 0 || r1 < r0 || r1 > p.T;
  bad = false;
  if (outside || n == 0) {
    n = 0;
    tiles = nu = 0;
    return 0;
  }
  bad = L < n || L > (1 << 30) || L > (long long)p.stride * p.P;
  tiles = (n * p.G + ROWS - 1) / ROWS;
  nu = bad ? 1 : (L + AT_UNIT - 1) / AT_UNIT;
  return (long long)p.Hkv * tiles * nu;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive1(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mma_f16(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Byte i (a compile-time constant) of a word array as two 16-bit floats.
__device__ __forceinline__ uint32_t decode_byte(const uint32_t* w, int i) {
  switch (i & 3) {
    case 0: return decode_pair<0>(w[i >> 2]);
    case 1: return decode_pair<1>(w[i >> 2]);
    case 2: return decode_pair<2>(w[i >> 2]);
    default: return decode_pair<3>(w[i >> 2]);
  }
}

__device__ __forceinline__ void load4(const bf16* p, float* x) {
  const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 v = __ldg(reinterpret_cast<const float4*>(p));
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void store4(bf16* p, const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// First head element of lane part t in inner step s of the first product.
template <int D>
__device__ __forceinline__ int k_order(int t, int s) {
  return D == 256 ? (s >> 3) * 128 + 32 * t + 4 * (s & 7) : (D / 4) * t + 4 * s;
}

// The queries of a row tile in the order of the first product's operand, in
// NT 16-bit terms; rows are scaled by powers of two so that their largest
// element is in [2^14, 2^15), which makes bf16 queries exact (elements 2^38
// below their row's largest aside).  c: what scores are multiplied by, a row.
template <class C, class DT>
__device__ __forceinline__ void load_queries(const AttnParams& p, const AttnSeg& sg, uint4* s_q, int lane,
                                             float (&c)[2 * C::M]) {
  const int g = lane >> 2, t = lane & 3;
  const int rows = sg.n * p.G;
#pragma unroll
  for (int m = 0; m < C::M; ++m) {
    float f[2];
    const DT* src[2];
    bool live[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = sg.tile * C::ROWS + 16 * m + 8 * e + g;
      live[e] = r < rows;
      const int i = live[e] ? r / p.G : 0, hq = sg.h * p.G + (live[e] ? r - i * p.G : 0);
      src[e] = static_cast<const DT*>(p.q) + (long long)(sg.r0 + i) * p.q_row + hq * p.q_head;
      float mx = 0.f;
#pragma unroll
      for (int s = 0; s < C::KSTEPS; ++s) {
        float x[4];
        load4(src[e] + k_order<C::D>(t, s), x);
        mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x[0]), fabsf(x[1]))), fmaxf(fabsf(x[2]), fabsf(x[3])));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int ex = 0;                                        // mx in [2^(ex-1), 2^ex)
      if (mx > 0.f && mx <= 3.402823466e38f) frexpf(mx, &ex);
      ex = 15 - ex;
      ex = ex > 120 ? 120 : ex;
      const float up = ldexpf(1.f, ex);
      float cc = fabsf(p.scale) * ldexpf(1.f, -ex);
      f[e] = p.scale < 0.f ? -up : up;
      if (!(cc > 0.f)) {                                 // scores of 0
        f[e] = 0.f;
        cc = 1.f;
      }
      if (!live[e]) f[e] = 0.f;
      c[2 * m + e] = cc;
    }
#pragma unroll
    for (int s = 0; s < C::KSTEPS; ++s) {
      float x[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        load4(src[e] + k_order<C::D>(t, s), x[e]);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[e][k] = live[e] ? x[e][k] * f[e] : 0.f;
      }
#pragma unroll
      for (int term = 0; term < C::NT; ++term) {
        uint4 a;
        a.x = pack_h2(x[0][0], x[0][1]);
        a.y = pack_h2(x[1][0], x[1][1]);
        a.z = pack_h2(x[0][2], x[0][3]);
        a.w = pack_h2(x[1][2], x[1][3]);
        s_q[((term * C::M + m) * C::KSTEPS + s) * 32 + lane] = a;
        if (term + 1 < C::NT) {
          const uint32_t h[2][2] = {{a.x, a.z}, {a.y, a.w}};
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 v = half2_floats(h[e][k]);
              x[e][2 * k] -= v.x;
              x[e][2 * k + 1] -= v.y;
            }
        }
      }
    }
  }
  __syncwarp();
}

template <class C, class DT>
__global__ void __launch_bounds__(32 * C::WARPS, C::MIN_CTAS) cache_attention_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_bar[C::WARPS][C::DEPTH];
  __shared__ long long s_pre[32 * C::WARPS + 1];         // units before each group of requests
  __shared__ long long s_scan[C::WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  uint64_t* bar = s_bar[warp];

  // ---- units before each group of `items` requests
  const int items = (p.B + 32 * C::WARPS - 1) / (32 * C::WARPS);
  long long total;
  {
    long long mine = 0;
    bool flag = false;
    for (int i = 0; i < items; ++i) {
      const int b = tid * items + i;
      if (b >= p.B) break;
      int n, r0, L, tiles, nu;
      bool bad, outside;
      mine += attn_work<C::ROWS>(p, b, n, r0, L, tiles, nu, bad, outside);
      flag |= bad || outside;
    }
    long long v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) s_scan[warp] = v;
    if (lane < C::DEPTH) mbar_init(bar + lane, 1);
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      if (w < warp) before += s_scan[w];
      all += s_scan[w];
    }
    s_pre[tid] = before + v - mine;
    if (tid == 0) s_pre[32 * C::WARPS] = all;
    total = all;
    if (flag && blockIdx.x == 0) set_status(p.status, SPEC_DEV_BAD_LEN);
    __syncthreads();
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  const int workers = gridDim.x * C::WARPS, me = warp * gridDim.x + blockIdx.x;
  const long long share = (total + workers - 1) / workers;
  const long long begin = me * share;
  const long long end = begin + share < total ? begin + share : total;
  float* parts = reinterpret_cast<float*>(static_cast<char*>(p.ws) + AT_MAX_CTAS * AT_WARPS * sizeof(AttnSplit));
  AttnSplit* splits = static_cast<AttnSplit*>(p.ws);
  AttnSplit split{0, -1, 0, 0, 0, 0, 0};
  uint8_t* ring = smem + warp * C::WARP_BYTES;
  uint4* s_q = reinterpret_cast<uint4*>(ring + C::DEPTH * C::UNIT_BYTES);

  if (begin < end) {
    // The segment that holds unit `pos`.
    auto locate = [&](long long pos) {
      int lo = 0, hi = 32 * C::WARPS;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid] <= pos) lo = mid; else hi = mid;
      }
      long long left = pos - s_pre[lo];
      AttnSeg s;
      int tiles;
      for (int b = lo * items;; ++b) {
        bool outside;
        const long long w = attn_work<C::ROWS>(p, b, s.n, s.r0, s.L, tiles, s.nu, s.bad, outside);
        if (left < w) {
          s.b = b;
          break;
        }
        left -= w;
      }
      const long long seg = left / s.nu;
      s.u = (int)(left - seg * s.nu);
      s.h = (int)(seg / tiles);
      s.tile = (int)(seg - (long long)s.h * tiles);
      return s;
    };
    const int bpp = p.P / CACHE_BLOCK;

    // ---- producer: copies of the units ahead
    AttnSeg ps = locate(begin);
    long long ppos = begin;
    int issued = 0, consumed = 0, drain = 0;             // units
    uint32_t bad_stage = 0;
    bool timed_out = false;
    auto pages_of = [&](const AttnSeg& s) {              // lane i < 2: page of the unit's block i
      const int tok = s.u * AT_UNIT + (lane & 1) * CACHE_BLOCK;
      int page = -1;
      if (lane < 2 && !s.bad && tok < s.L) page = __ldg(p.table + (size_t)s.b * p.stride + tok / p.P);
      return page;
    };
    int page = pages_of(ps);
    auto issue = [&]() {
      const int st = issued % C::DEPTH;
      const int tok = ps.u * AT_UNIT;
      const bool second = tok + CACHE_BLOCK < ps.L;
      const bool ok_mine = page >= 0 && page < p.num_pages;
      const uint32_t okm = __ballot_sync(0xffffffffu, ok_mine);
      const bool ok = !ps.bad && (okm & 1u) && (!second || (okm & 2u));
      if (!ok) {
        bad_stage |= 1u << st;
        if (lane == 0) {
          if (!ps.bad) set_status(p.status, SPEC_DEV_BAD_SLOT);
          mbar_arrive1(bar + st);
        }
      } else {
        bad_stage &= ~(1u << st);
        uint8_t* dst = ring + st * C::UNIT_BYTES;
        const int blk = (tok % p.P) / CACHE_BLOCK;
        if (p.P >= AT_UNIT) {
          if (lane == 0) {
            expect_bytes(bar + st, C::UNIT_BYTES);
            bulk_load(dst, p.cache + cache_block_at(page, ps.h, blk, p.Hkv, bpp, C::D), C::UNIT_BYTES, bar + st);
          }
        } else {
          if (lane == 0) expect_bytes(bar + st, second ? C::UNIT_BYTES : C::UNIT_BYTES / 2);
          __syncwarp();
          if (lane == 0 || (lane == 1 && second))
            bulk_load(dst + lane * (C::UNIT_BYTES / 2), p.cache + cache_block_at(page, ps.h, 0, p.Hkv, bpp, C::D),
                      C::UNIT_BYTES / 2, bar + st);
        }
      }
      ++issued;
      ++ppos;
      if (ppos < end) {
        if (++ps.u >= ps.nu) ps = locate(ppos);
        page = pages_of(ps);
      }
    };
    while (issued < C::DEPTH && ppos < end) issue();

    long long pos = begin;
    while (pos < end) {
      AttnSeg sg = locate(pos);
      const int u_first = sg.u;
      const int u_end = sg.nu - sg.u < end - pos ? sg.nu : sg.u + (int)(end - pos);
      const int rows = sg.n * p.G, ctx = sg.L - sg.n;
      float c[2 * C::M], mref[2 * C::M], O[C::M][C::NV][4], l[2 * C::M];   // l: this lane's columns
      load_queries<C, DT>(p, sg, s_q, lane, c);
      int lim[2 * C::M];                                 // tokens a row sees (causal), its packed row
#pragma unroll
      for (int i = 0; i < 2 * C::M; ++i) {
        mref[i] = -INFINITY;
        l[i] = 0.f;
        const int r = sg.tile * C::ROWS + 16 * (i >> 1) + 8 * (i & 1) + g;
        lim[i] = r < rows ? (p.mask ? sg.r0 + r / p.G : ctx + r / p.G + 1) : -1;
      }
#pragma unroll
      for (int m = 0; m < C::M; ++m)
#pragma unroll
        for (int j = 0; j < C::NV; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) O[m][j][k] = 0.f;
      bool poison = false;

      for (int u = u_first; u < u_end; ++u) {
        const int st = consumed % C::DEPTH;
        if (!timed_out && !mbar_wait(bar + st, (uint32_t)(consumed / C::DEPTH) & 1u, 1u << 22)) {
          timed_out = true;
          drain = consumed;
          if (lane == 0) set_status(p.status, SPEC_DEV_TIMEOUT);
        }
        if (__any_sync(0xffffffffu, timed_out) && !timed_out) {
          timed_out = true;
          drain = consumed;
        }
        const bool skip = ((bad_stage >> st) & 1u) || timed_out;
        if (skip) {
          poison = true;
        } else {
          const uint8_t* unit = ring + st * C::UNIT_BYTES;
          // ---- first product: scores of 4 x 8 tokens
          float S[C::M][4][4];
#pragma unroll
          for (int m = 0; m < C::M; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k) S[m][j][k] = 0.f;
          uint32_t kc[4][C::KW], ks[4][C::KG];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int tok = (g >> 1) + 4 * (g & 1) + 8 * (j & 1);
            const uint8_t* blk = unit + (j >> 1) * (18 * C::D);
            const uint8_t* row = blk + tok * (C::D / 2);
            if (C::D == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * t);
              kc[j][0] = v.x; kc[j][1] = v.y;
            } else {
#pragma unroll
              for (int h = 0; h < C::D / 128; ++h) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + 64 * h + 16 * t);
                kc[j][4 * h] = v.x; kc[j][4 * h + 1] = v.y; kc[j][4 * h + 2] = v.z; kc[j][4 * h + 3] = v.w;
              }
            }
            const uint8_t* sc = blk + cache_k_scales(C::D) + tok * (C::D / 16);
            if (C::D == 64) {
              const uint32_t two = decode_scales(sc[t]);
              ks[j][0] = __byte_perm(two, two, 0x1010);
            } else {
#pragma unroll
              for (int h = 0; h < C::D / 128; ++h) {
                const uint32_t two = decode_scales(*reinterpret_cast<const uint16_t*>(sc + 8 * h + 2 * t));
                ks[j][2 * h] = __byte_perm(two, two, 0x1010);
                ks[j][2 * h + 1] = __byte_perm(two, two, 0x3232);
              }
            }
          }
#pragma unroll
          for (int s = 0; s < C::KSTEPS; ++s) {
            uint4 a[C::NT][C::M];
#pragma unroll
            for (int term = 0; term < C::NT; ++term)
#pragma unroll
              for (int m = 0; m < C::M; ++m) a[term][m] = s_q[((term * C::M + m) * C::KSTEPS + s) * 32 + lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t b0 = mul_h2(decode_byte(kc[j], 2 * s), ks[j][s >> 2]);
              const uint32_t b1 = mul_h2(decode_byte(kc[j], 2 * s + 1), ks[j][s >> 2]);
#pragma unroll
              for (int term = 0; term < C::NT; ++term)
#pragma unroll
                for (int m = 0; m < C::M; ++m) mma_f16(S[m][j], a[term][m], b0, b1);
            }
          }
          // ---- masks, where the unit reaches the new tokens
          const int tok0 = u * AT_UNIT;
          const bool edge = tok0 + AT_UNIT > ctx;
          if (edge) {
#pragma unroll
            for (int i = 0; i < 2 * C::M; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int tok = tok0 + 16 * (j >> 1) + 8 * (j & 1) + t + 4 * e;
                  bool seen = tok < lim[i];
                  if (p.mask) {
                    const int d = tok - ctx;
                    seen = lim[i] >= 0 && tok < sg.L;
                    if (seen && d >= 0)
                      seen = (d >> 5) < p.mask_words &&
                             ((__ldg(p.mask + (size_t)lim[i] * p.mask_words + (d >> 5)) >> (d & 31)) & 1u);
                  }
                  if (!seen) S[i >> 1][j][2 * (i & 1) + e] = -INFINITY;
                }
          }
          // ---- probabilities
          float top[2 * C::M];
          bool far = false;
#pragma unroll
          for (int i = 0; i < 2 * C::M; ++i) {
            const int m = i >> 1, e = 2 * (i & 1);
            float x = fmaxf(S[m][0][e], S[m][0][e + 1]);
#pragma unroll
            for (int j = 1; j < 4; ++j) x = fmaxf(x, fmaxf(S[m][j][e], S[m][j][e + 1]));
            top[i] = x;
            far |= c[i] * (x - mref[i]) > AT_SLACK;
          }
          if (__any_sync(0xffffffffu, far)) {
#pragma unroll
            for (int i = 0; i < 2 * C::M; ++i) {
              float x = top[i];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              x = fmaxf(x, mref[i]);
              const float f = x == mref[i] ? 1.f : exp2_approx(c[i] * (mref[i] - x));
              mref[i] = x;
              const int m = i >> 1, e = 2 * (i & 1);
              l[i] *= f;
#pragma unroll
              for (int j = 0; j < C::NV; ++j) {
                O[m][j][e] *= f;
                O[m][j][e + 1] *= f;
              }
            }
          }
          uint4 pa[C::NT][C::M][2];
#pragma unroll
          for (int i = 0; i < 2 * C::M; ++i) {
            const int m = i >> 1, e = 2 * (i & 1);
            const float base = mref[i] == -INFINITY ? 0.f : AT_SHIFT - c[i] * mref[i];
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                S[m][j][e + k] = exp2_approx(fmaf(S[m][j][e + k], c[i], base));
                sum += S[m][j][e + k];
              }
            l[i] += sum;
          }
#pragma unroll
          for (int term = 0; term < C::NT; ++term)
#pragma unroll
            for (int m = 0; m < C::M; ++m)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint4 a;
                a.x = pack_h2(S[m][2 * k][0], S[m][2 * k][1]);
                a.y = pack_h2(S[m][2 * k][2], S[m][2 * k][3]);
                a.z = pack_h2(S[m][2 * k + 1][0], S[m][2 * k + 1][1]);
                a.w = pack_h2(S[m][2 * k + 1][2], S[m][2 * k + 1][3]);
                pa[term][m][k] = a;
                if (term + 1 < C::NT) {
                  const uint32_t h[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const float2 v = half2_floats(h[q]);
                    S[m][2 * k + (q >> 1)][2 * (q & 1)] -= v.x;
                    S[m][2 * k + (q >> 1)][2 * (q & 1) + 1] -= v.y;
                  }
                }
              }
          // ---- second product, 16 tokens a step
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint8_t* blk = unit + k * (18 * C::D);
            uint32_t vc[4][C::VW], vs[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = t + 4 * i;
              const uint8_t* row = blk + cache_v_codes(C::D) + tok * (C::D / 2) + g * (C::D / 16);
              if (C::D == 64) {
                vc[i][0] = *reinterpret_cast<const uint32_t*>(row);
              } else if (C::D == 128) {
                const uint2 v = *reinterpret_cast<const uint2*>(row);
                vc[i][0] = v.x; vc[i][C::VW - 1] = v.y;
              } else {
                const uint4 v = *reinterpret_cast<const uint4*>(row);
                vc[i][0] = v.x; vc[i][1 % C::VW] = v.y; vc[i][2 % C::VW] = v.z; vc[i][3 % C::VW] = v.w;
              }
              const uint8_t* sc = blk + cache_v_scales(C::D) + tok * (C::D / 16);
              uint32_t two = C::D == 256 ? *reinterpret_cast<const uint16_t*>(sc + 2 * g)
                                         : (uint32_t)sc[C::D == 128 ? g : g >> 1];
              if (edge && tok0 + 16 * k + tok >= sg.L) two = 0;   // bytes that nobody wrote
              two = decode_scales(two);
              vs[i][0] = __byte_perm(two, two, 0x1010);
              vs[i][1] = C::D == 256 ? __byte_perm(two, two, 0x3232) : vs[i][0];
            }
#pragma unroll
            for (int jj = 0; jj < C::NV / 2; ++jj) {
              uint32_t v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = mul_h2(decode_byte(vc[i], jj), vs[i][C::D == 256 ? jj >> 3 : 0]);
              const uint32_t b0 = __byte_perm(v[0], v[1], 0x5410), b1 = __byte_perm(v[2], v[3], 0x5410);
              const uint32_t d0 = __byte_perm(v[0], v[1], 0x7632), d1 = __byte_perm(v[2], v[3], 0x7632);
#pragma unroll
              for (int term = 0; term < C::NT; ++term)
#pragma unroll
                for (int m = 0; m < C::M; ++m) {
                  mma_f16(O[m][2 * jj], pa[term][m][k], b0, b1);
                  mma_f16(O[m][2 * jj + 1], pa[term][m][k], d0, d1);
                }
            }
          }
        }
        ++consumed;
        __syncwarp();                                    // all lanes have read the stage
        if (ppos < end && !timed_out) issue();
      }

      // ---- the segment's end in this share
      const bool whole = u_first == 0 && u_end == sg.nu;
#pragma unroll
      for (int i = 0; i < 2 * C::M; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (poison) l[i] = quiet_nan();
      }
      if (whole) {
#pragma unroll
        for (int i = 0; i < 2 * C::M; ++i) {
          const int m = i >> 1, e = 2 * (i & 1);
          const int r = sg.tile * C::ROWS + 16 * m + 8 * (i & 1) + g;
          if (r >= rows) continue;
          const int tok = r / p.G, hq = sg.h * p.G + r - tok * p.G;
          const float sum = l[i];
          const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
          const size_t at = (size_t)(sg.r0 + tok) * p.Hq + hq;
          DT* o = static_cast<DT*>(p.out) + at * C::D;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < C::NV; j += 4) {
              const float x[4] = {O[m][j][e + k] * inv, O[m][j + 1][e + k] * inv, O[m][j + 2][e + k] * inv,
                                  O[m][j + 3][e + k] * inv};
              store4(o + (2 * t + k) * C::NV + j, x);
            }
          if (t == 0 && p.lse)
            p.lse[at] = sum == 0.f ? -INFINITY : 0.69314718056f * (c[i] * mref[i] - AT_SHIFT + log2f(sum));
        }
      } else {
        // slot 0: the segment began before this share; slot 1: it begins here
        const int slot = u_first == 0 ? 1 : 0;
        float* part = parts + (size_t)(2 * me + slot) * C::PART;
#pragma unroll
        for (int i = 0; i < 2 * C::M; ++i) {
          const int m = i >> 1, e = 2 * (i & 1);
          const int rl = 16 * m + 8 * (i & 1) + g;
          if (sg.tile * C::ROWS + rl >= rows) continue;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < C::NV; j += 4)
              *reinterpret_cast<float4*>(part + (((i * 2 + k) * (C::NV / 4) + j / 4) * 32 + lane) * 4) =
                  make_float4(O[m][j][e + k], O[m][j + 1][e + k], O[m][j + 2][e + k], O[m][j + 3][e + k]);
          if (t == 0)
            *reinterpret_cast<float2*>(part + C::ROWS * C::D + 2 * rl) =
                make_float2(mref[i] == -INFINITY ? -INFINITY : c[i] * mref[i] - AT_SHIFT, l[i]);
        }
        if (slot == 1) {
          const long long seg_last = pos + (sg.nu - 1);  // the segment's last unit
          split = AttnSplit{me, (int)(seg_last / share), sg.b, sg.h, sg.tile, sg.n, sg.r0};
        }
      }
      pos += u_end - u_first;
    }
    if (timed_out)                                       // leave no copy in flight
      for (int i = drain; i < issued; ++i) mbar_wait(bar + i % C::DEPTH, (uint32_t)(i / C::DEPTH) & 1u, 1u << 22);
  }
  if (lane == 0) splits[me] = split;
}

// Adds the parts of one split segment: CTA (x, y) takes the segments that begin
// in warps x, x + gridDim.x, ..; y is one of 2 M groups of eight rows.
constexpr int JOIN_THREADS = 256;
template <class C, class DT>
__global__ void __launch_bounds__(JOIN_THREADS) cache_attention_join_kernel(const __grid_constant__ AttnParams p, int workers) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const float* parts = reinterpret_cast<const float*>(static_cast<char*>(p.ws) + AT_MAX_CTAS * AT_WARPS * sizeof(AttnSplit));
  const AttnSplit* splits = static_cast<const AttnSplit*>(p.ws);
  const int i = blockIdx.y, tid = threadIdx.x;
  constexpr int ITEMS = 2 * C::D;                        // float4 of eight rows
  for (int w = blockIdx.x; w < workers; w += gridDim.x) {
    const AttnSplit s = splits[w];
    if (s.last < s.first) continue;
    const int rows = s.n * p.G;
    if (s.tile * C::ROWS + 8 * i >= rows) continue;      // uniform over the CTA
    auto part_of = [&](int x) { return parts + (size_t)(2 * x + (x == s.first ? 1 : 0)) * C::PART; };
    for (int it = tid; it < ITEMS; it += JOIN_THREADS) {
      const int lane = it & 31, q = it >> 5;             // q: k * (NV / 4) + j / 4
      const int g = lane >> 2, t = lane & 3;
      const int r = s.tile * C::ROWS + 8 * i + g;
      if (r >= rows) continue;
      const int ml = C::ROWS * C::D + 2 * (8 * i + g);
      float m = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int x = s.first; x <= s.last; ++x) {
        const float* part = part_of(x);
        const float2 v = __ldg(reinterpret_cast<const float2*>(part + ml));
        const float4 o = __ldg(reinterpret_cast<const float4*>(part + ((i * 2 * (C::NV / 4) + q) * 32 + lane) * 4));
        const float mn = fmaxf(m, v.x);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float fa = exp2f(m - ref), fb = exp2f(v.x - ref);
        m = mn;
        sum = sum * fa + v.y * fb;
        acc.x = acc.x * fa + o.x * fb;
        acc.y = acc.y * fa + o.y * fb;
        acc.z = acc.z * fa + o.z * fb;
        acc.w = acc.w * fa + o.w * fb;
      }
      const int tok = r / p.G, hq = s.h * p.G + r - tok * p.G;
      const size_t at = (size_t)(s.r0 + tok) * p.Hq + hq;
      const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
      const int k = q / (C::NV / 4), j = 4 * (q - k * (C::NV / 4));
      const float x[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
      store4(static_cast<DT*>(p.out) + at * C::D + (2 * t + k) * C::NV + j, x);
      if (q == 0 && t == 0 && p.lse)
        p.lse[at] = sum == 0.f ? -INFINITY : 0.69314718056f * (m + log2f(sum));
    }
  }
}

namespace {
template <class C, class DT>
cudaError_t launch_cfg(const AttnParams& p, int sms, cudaStream_t st) {
  static_assert(C::SMEM <= 227 * 1024 - 4096, "shared memory");
  cudaError_t e = cudaFuncSetAttribute(cache_attention_kernel<C, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // one wave at most, and no more warps than there can be units
  long long ctas = (long long)sms * C::MIN_CTAS;
  if (ctas > C::MIN_CTAS * (AT_MAX_CTAS / 2)) ctas = C::MIN_CTAS * (AT_MAX_CTAS / 2);
  const long long tiles = (long long)p.T * p.G / C::ROWS + (p.T < p.B ? p.T : p.B);
  const long long units = tiles * p.Hkv * (((long long)p.stride * p.P + AT_UNIT - 1) / AT_UNIT);
  if (ctas > units) ctas = units;
  cache_attention_kernel<C, DT><<<(int)ctas, 32 * C::WARPS, C::SMEM, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int workers = (int)ctas * C::WARPS;
  cfg.gridDim = dim3(workers < 2 * sms ? workers : 2 * sms, 2 * C::M);
  cfg.blockDim = dim3(JOIN_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attention_join_kernel<C, DT>, p, workers);
}
}  // namespace

size_t cache_attention_workspace_bytes(int Hq, int Hkv, int D) {
  const size_t rows = D == 256 ? 16 : 32;
  const size_t part = (rows * D + 2 * rows) * sizeof(float);
  // 32-row tiles run one CTA an SM, 16-row tiles two
  const size_t parts = D == 256 ? (size_t)AT_MAX_CTAS : (size_t)AT_MAX_CTAS / 2;
  return (size_t)AT_MAX_CTAS * AT_WARPS * sizeof(AttnSplit) + parts * AT_WARPS * 2 * part + 256;
}

cudaError_t launch_cache_attention(const spec_cache_attention_args& a, int sms, cudaStream_t st) {
  const int G = a.Hq / a.Hkv;
  AttnParams p{a.B, a.T, a.Hq, a.Hkv, G, a.page_size, a.num_pages, a.table_stride, a.mask_words, a.q, a.q_row_stride,
               a.q_head_stride, a.cache, a.block_table, a.kv_len, a.row_ptr, a.tree_mask,
               a.softmax_scale * a.k_scale * 1.4426950408889634f, a.v_scale, a.out, a.lse, a.dev_status, a.workspace};
  if (a.dtype == SPEC_F32) {
    if (a.D == 64) return launch_cfg<AttnCfg<64, 1, 2>, float>(p, sms, st);
    if (a.D == 128) return launch_cfg<AttnCfg<128, 1, 2>, float>(p, sms, st);
    return launch_cfg<AttnCfg<256, 1, 2>, float>(p, sms, st);
  }
  // 16-row tiles where the mean request has no more rows than that
  const bool few = (long long)a.T * G <= 16LL * a.B;
  if (a.D == 64) return few ? launch_cfg<AttnCfg<64, 1, 1>, bf16>(p, sms, st) : launch_cfg<AttnCfg<64, 2, 1>, bf16>(p, sms, st);
  if (a.D == 128) return few ? launch_cfg<AttnCfg<128, 1, 1>, bf16>(p, sms, st) : launch_cfg<AttnCfg<128, 2, 1>, bf16>(p, sms, st);
  return launch_cfg<AttnCfg<256, 1, 1>, bf16>(p, sms, st);
}

}  // namespace spec
