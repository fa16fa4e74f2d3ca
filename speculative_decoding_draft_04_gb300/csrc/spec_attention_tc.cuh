// Attention over the 4-bit cache for requests of many new rows (trees, prompts):
// bf16 heads of 64 or 128 elements, tiles of 128 query rows on the fifth-
// generation tensor cores.
//
// With r rows a key-value head the products are 4 D r operations a token against
// 18 D / 16 bytes of cache, and decoding a token costs the same for one row as
// for 128.  So here a token is decoded once for 128 rows:
//
//   S[128 x 64] = Q K'          Q and decoded K in shared memory, S in tensor memory
//   O[128 x D] += P V           P (16-bit floats) written over S, V in shared memory
//
//   warps 0-3   softmax: a thread holds one row, so its maximum and sum need no
//               exchange (the same lazy maximum as the other kernels)
//   warps 4-7   decode: codes requested a unit of 64 tokens ahead into registers,
//               decoded into two buffers of 16-bit floats; keys' and values'
//               buffers are taken and given back apart
//   warp 8      issues the products, the next unit's first one ahead of this
//               unit's second one
//
// Two CTAs an SM, each with half of the tensor memory, cover each other's waits.
// The units are numbered and shared, and split segments joined, as in the
// kernels of smaller tiles, but a segment counts four units more: beginning and
// ending one (queries in, outputs out, an empty pipeline) takes as long as that,
// and short requests' segments would otherwise meet in one CTA (trees of 100 rows
// over 32 requests of 25 to 4096 tokens: 119 us without it and with keys' and
// values' buffers taken together, 75 now).
//
// Bound by the chain of waits from step to step of a unit: 3500 cycles a unit
// and CTA, two CTAs at a time, of which the products are some 500 a unit.  The
// trees keep 42 % of the issue slots, 27 % of the tensor pipe and 19 % of the
// memory busy.  100 of 128 rows reach 0.4 PFLOP/s (72 to 80 us a call, by the
// trees' lengths); 16-row tiles of mma.sync take 211 us for as many rows, decoding
// every token seven times.  Eight prompts of 512 tokens take 102 us, of 2048 777.
#pragma once

#include <atomic>

#include "spec_attention.cuh"

namespace spec {

constexpr int TA_UNIT = 64;                                  // tokens
constexpr int TA_ROWS = 128;
constexpr int TA_LEAD = 4;                                   // units that beginning and ending a segment costs
constexpr int TA_PREFIX = 256;                               // threads of the prefix sums
constexpr int TA_THREADS = 9 * 32;
constexpr uint32_t TA_COLS = 256;                            // two buffers of scores, outputs
constexpr uint32_t TA_O = 128, TA_P = 32;                    // outputs; P, from its scores' first column on

// Shared memory: queries [D / 64][128 rows][128 bytes], two buffers of keys
// [D / 64][64 tokens][128 bytes] and of values alike, all swizzled by 128 bytes.
template <int D>
struct TaLayout {
  static constexpr int K = TA_ROWS * D * 2, HALF = TA_UNIT * D * 2;
  static constexpr int V = K + 2 * HALF;
  static constexpr int TOTAL = V + 2 * HALF + 1024;          // slack to align the base
  static constexpr int PART = TA_ROWS * D + 2 * TA_ROWS;
};

enum { TB_K = 0, TB_V = 2, TB_S = 4, TB_P = 6, TB_DONE = 8, TB_Q = 10, TB_BARS = 11 };

// Operand kinds: A, B 16-bit floats, D fp32, M = 128.
template <int N>
__device__ __forceinline__ constexpr uint32_t ta_idesc(uint32_t b_mn) {
  return (1u << 4) | (b_mn << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
// One lane of the (converged) warp.  The products are executed by the whole warp
// under its predicate, not inside a branch of one lane: descriptors then stay in
// uniform registers.
__device__ __forceinline__ uint32_t ta_elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
  return r;
}
// A from tensor memory, and A from shared memory.
__device__ __forceinline__ void ta_mma_ts(uint32_t el, uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accum), "r"(el)
      : "memory");
}
__device__ __forceinline__ void ta_mma_ss(uint32_t el, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum), "r"(el)
      : "memory");
}
__device__ __forceinline__ void ta_commit(uint32_t el, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}
template <class T>
__device__ __forceinline__ void ta_st16(uint32_t taddr, const T (&v)[16]) {
  auto u = [&](int i) { return *reinterpret_cast<const uint32_t*>(&v[i]); };
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(u(0)), "r"(u(1)), "r"(u(2)), "r"(u(3)), "r"(u(4)), "r"(u(5)), "r"(u(6)), "r"(u(7)), "r"(u(8)), "r"(u(9)), "r"(u(10)),
      "r"(u(11)), "r"(u(12)), "r"(u(13)), "r"(u(14)), "r"(u(15))
      : "memory");
}
__device__ __forceinline__ void ta_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
        "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
  tc_wait_ld();
}
__device__ __forceinline__ void ta_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Loads that are issued where they stand (not moved down to the first use).
__device__ __forceinline__ uint4 load_now(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_now(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}

// 32 bytes a lane: a whole sector of memory, where the address allows.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8], bool sector) {
  if (sector) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Whether phase `parity` of a barrier is complete, suspended for up to 10 us; the
// other warps issue meanwhile.
__device__ __forceinline__ bool bar_suspend(uint64_t* b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(b)), "r"(parity), "r"(10000)
      : "memory");
  return done != 0;
}

// Which of the new tokens d .. d + 31 (before them: context) a row sees.
__device__ __forceinline__ uint32_t seen_word(const AttnParams& p, int d, int lim, int ctx, int L) {
  auto first = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
  if (lim < 0) return 0;
  if (!p.mask) return first(lim - ctx - d);
  auto word = [&](int i) {
    return i < 0 ? ~0u : i < p.mask_words ? __ldg(p.mask + (size_t)lim * p.mask_words + i) : 0u;
  };
  return __funnelshift_r(word(d >> 5), word((d >> 5) + 1), d & 31) & first(L - ctx - d);
}

// The segments of a CTA's share [pos, end), each with the units u .. u_end - 1 of
// it that are the CTA's.  A share that ends inside a segment's lead has none of
// its units, and one that begins there has it from its first unit on.
template <int PASS>
struct TaWalk {
  AttnSeg sg;
  int u_end;
  long long pos, end;
  __device__ __forceinline__ TaWalk(const AttnParams& p, const long long* s_pre, long long begin, long long end_)
      : pos(begin), end(end_) {
    if (pos < end) {
      sg = attn_locate<PASS, TA_ROWS, TA_UNIT, TA_PREFIX, TA_LEAD>(p, s_pre, pos);
      pos -= sg.u;                                           // where the segment begins
      sg.u = max(sg.u - TA_LEAD, 0);
      cut();
    }
  }
  __device__ __forceinline__ void cut() {
    const long long units = end - pos - TA_LEAD;
    u_end = units < sg.nu ? (int)units : sg.nu;
    if (u_end <= sg.u) pos = end;
  }
  __device__ __forceinline__ bool done() const { return pos >= end; }
  __device__ __forceinline__ void next(const AttnParams& p, const long long* s_pre) {
    pos += TA_LEAD + sg.nu;
    if (pos < end) {
      sg = attn_next<PASS, TA_ROWS, TA_UNIT, TA_PREFIX, TA_LEAD>(p, s_pre, sg, pos);
      cut();
    }
  }
};

template <int PASS, int D>
__global__ void __launch_bounds__(TA_THREADS, 2) cache_attention_tc_kernel(const __grid_constant__ AttnParams p) {
  using L = TaLayout<D>;
  constexpr int KSTEPS = D / 16, TASKS = D / 64;             // 64 elements each: a decoding thread's of a unit
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar[TB_BARS];
  __shared__ long long s_pre[TA_PREFIX + 1];
  __shared__ long long s_scan[TA_PREFIX / 32];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  __shared__ __align__(16) int s_bad[4][4];                                // a unit's pages outside the cache, a decode warp each
  uint8_t* sm = align1k(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    s_fail = 0;
    const int counts[TB_BARS / 2 + 1] = {D / 32, D / 32, 1, 4, 1, 4};   // arriving warps
    for (int i = 0; i < TB_BARS; ++i) mbar_init(bar + i, counts[i / 2]);
    for (int i = 0; i < 16; ++i) s_bad[i >> 2][i & 3] = 0;
  }
  if (warp == 8) tc_alloc(&s_tmem, TA_COLS);
  if (tid < TA_PREFIX)
    attn_prefix<PASS, TA_ROWS, TA_UNIT, TA_PREFIX, TA_LEAD>(p, s_pre, s_scan,
                                                      [] { asm volatile("barrier.cta.sync.aligned 3, 256;\n" ::: "memory"); });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (PASS == PASS_OWN) asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const long long total = s_pre[TA_PREFIX];
  const uint32_t tmem = s_tmem;
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  const int me = blockIdx.x;
  const long long begin = me * share;
  const long long end = begin + share < total ? begin + share : total;

  // Bounded wait for unit (or segment) x; after one wait gives up, none waits
  // long any more and the results are NaN.
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (!bar_suspend(b, parity)) {
      uint32_t tries = *(volatile int*)&s_fail ? 1u : 1u << 16;
      while (tries && !bar_suspend(b, parity)) --tries;
      if (!tries && !*(volatile int*)&s_fail) {
        *(volatile int*)&s_fail = 1;
        set_status(p.status, SPEC_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  };
  auto wait2 = [&](int pair, uint32_t x) { wait(bar + pair + (x & 1), (x >> 1) & 1); };
  auto arrive = [&](uint64_t* b) {
    __syncwarp();
    if (lane == 0) mbar_arrive1(b);
  };
  AttnSplit split{0, -1, 0, 0, 0, 0, 0};

  TaWalk<PASS> walk(p, s_pre, begin, end);
  if (walk.done()) {
  } else if (warp < 4) {
    // ------------------------------------------------ softmax
    const uint32_t trow = tmem + ((uint32_t)(32 * warp) << 16);
    uint32_t i = 0;
    const int rl = 32 * warp + lane;                         // this thread's row
    uint8_t* const qrow = sm + rl * 128;
    int ntok = 0, nhq = 0;                                   // the row's new token and query head; < 0: none
    // Copies the warp's queries of the walk's segment to their place, D / 8 lanes a
    // row: once the last products of the segment before have read that.
    auto copy_queries = [&]() {
      constexpr int LANES = D / 8, PER = 32 / LANES;         // rows an instruction
      const int r = walk.sg.tile * TA_ROWS + rl;
      const bool there = r < walk.sg.n * p.G;
      ntok = there ? r / p.G : -1;
      nhq = walk.sg.h * p.G + (there ? r - ntok * p.G : 0);
      const long long off = there ? (long long)(walk.sg.r0 + ntok) * p.q_row + nhq * p.q_head : -1;
      const int ch = lane % LANES;
#pragma unroll
      for (int k = 0; k < LANES; ++k) {
        const int j = k * PER + lane / LANES, rw = 32 * warp + j;
        const long long from = __shfl_sync(0xffffffffu, off, j);
        cp_async16(sm + (ch >> 3) * (TA_ROWS * 128) + rw * 128 + (((ch & 7) ^ (rw & 7)) << 4),
                   static_cast<const bf16*>(p.q) + (from < 0 ? 0 : from) + 8 * ch, from >= 0);
      }
      cp_async_commit();
    };
    copy_queries();
    for (bool more = true; more;) {
      const AttnSeg sg = walk.sg;
      const int u_first = sg.u, u_end = walk.u_end;
      const long long last = walk.pos + TA_LEAD + sg.nu - 1;   // the segment's last unit
      const int ctx = sg.template context<PASS>();
      const bool live = ntok >= 0;
      const int tok = live ? ntok : 0, hq = nhq;
      // ---- this thread's query as 16-bit floats, scaled by a power of two so that
      // its largest element is in [2^14, 2^15), which makes bf16 exact (elements
      // 2^38 below it aside)
      cp_async_wait_all();
      __syncwarp();
      float c;
      {
        float mx = 0.f;
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(qrow + (k >> 3) * (TA_ROWS * 128) + (((k & 7) ^ (rl & 7)) << 4));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx = max3(mx, fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u)));
        }
        const int ex = query_exponent(mx);
        float f = p.scale < 0.f ? -power_of_2(ex) : power_of_2(ex);
        c = fabsf(p.scale) * power_of_2(-ex);
        if (!(c > 0.f)) {                                    // scores of 0
          f = 0.f;
          c = 1.f;
        }
#pragma unroll 4
        for (int k = 0; k < D / 8; ++k) {
          uint4* at = reinterpret_cast<uint4*>(qrow + (k >> 3) * (TA_ROWS * 128) + (((k & 7) ^ (rl & 7)) << 4));
          const uint4 v = *at;
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pack_h2(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
          *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      fence_async_shared();
      arrive(bar + TB_Q);
      bool poison = sg.bad;                                  // a page outside the cache in this part
      const int lim = live ? (PASS == PASS_PREFIX ? sg.L : p.mask ? sg.r0 + tok : ctx + tok + 1) : -1;   // tokens it sees (causal), its packed row
      const bool some = __any_sync(0xffffffffu, live);
      float mref = -INFINITY, l = 0.f;
      for (int u = u_first; u < u_end; ++u, ++i) {
        wait2(TB_S, i);
        tc_fence_after();
        if (u + 1 == u_end) {                                // the segment's last first product is done
          walk.next(p, s_pre);
          more = !walk.done();
          if (more) copy_queries();
        }
        const int4 bad = *reinterpret_cast<const int4*>(s_bad[i & 3]);
        poison |= (bad.x | bad.y | bad.z | bad.w) != 0;
        const uint32_t at = trow + (i & 1) * TA_UNIT;
        if (some) {
          // 32 tokens at a time, the first ones read twice: fewer registers
          const int tok0 = u * TA_UNIT;
          const bool edge = tok0 + TA_UNIT > ctx;
          uint32_t seen[2] = {~0u, ~0u};
          if (edge)
            for (int h = 0; h < 2; ++h) seen[h] = seen_word(p, tok0 + 32 * h - ctx, lim, ctx, sg.L);
          float s[32], x = -INFINITY;
          auto read = [&](int h) {
            tc_ld32_issue(at + 32 * h, s);
            tc_wait_ld();
            if (edge) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (!(seen[h] >> k & 1)) s[k] = -INFINITY;
            }
          };
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            read(h);
#pragma unroll
            for (int k = 0; k < 32; k += 2) x = max3(x, s[k], s[k + 1]);
          }
          if (__any_sync(0xffffffffu, c * (x - mref) > AT_SLACK)) {
            x = fmaxf(x, mref);
            const float f = x == mref ? 1.f : exp2_approx(c * (mref - x));
            mref = x;
            l *= f;
            if (u > u_first) {                               // (in the first unit O is not written yet)
              wait2(TB_DONE, i - 1);                         // no product adds to O meanwhile
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < D; q += 16) {
                float o[16];
                ta_ld16(trow + TA_O + q, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= f;
                ta_st16(trow + TA_O + q, o);
              }
            }
          }
          const float base = mref == -INFINITY ? 0.f : AT_SHIFT - c * mref;
          const uint64_t c2 = pair(c, c), b2 = pair(base, base);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int h = 1; h >= 0; --h) {                     // over the scores' second half, which is read by now
            if (h == 0) read(0);
            uint32_t y[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 d = unpair(fma2(pair(s[2 * k], s[2 * k + 1]), c2, b2));
              const float e0 = exp2_approx(d.x), e1 = exp2_approx(d.y);
              sum[k & 1] = add2(sum[k & 1], pair(e0, e1));
              y[k] = pack_h2(e0, e1);
            }
            ta_st16(at + TA_P + 16 * h, y);
          }
          const float2 z = unpair(add2(sum[0], sum[1]));
          l += z.x + z.y;
          ta_wait_st();
        }
        tc_fence_before();
        arrive(bar + TB_P + (i & 1));
      }
      // ---- the segment's end in this share
      wait2(TB_DONE, i - 1);
      tc_fence_after();
      const bool whole = u_first == 0 && u_end == sg.nu;
      const int slot = u_first == 0 ? 1 : 0;                 // 0: the segment began before this share
      if (poison || *(volatile int*)&s_fail) l = quiet_nan();
      const float m = mref == -INFINITY ? -INFINITY : c * mref - AT_SHIFT;
      float* part = attn_parts(p) + (size_t)(2 * me + slot) * L::PART;
      if (some) {
        const size_t at = (size_t)(sg.r0 + tok) * p.Hq + hq;
        AttnRow f{};
        if (live && whole && PASS != PASS_PREFIX) f = attn_row<PASS>(p, at, m, l);
        float* const sums = PASS == PASS_PREFIX && whole ? p.raw + at * D : part + rl * D;   // where they are kept as they are
        const bool sector = ((whole && PASS != PASS_PREFIX ? (uintptr_t)p.out : (uintptr_t)sums) & 31) == 0;
#pragma unroll 1
        for (int q = 0; q < D; q += 32) {
          float o[32];
          tc_ld32_issue(trow + TA_O + q, o);
          tc_wait_ld();
          if (live && whole && PASS != PASS_PREFIX) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= f.own;
            if (PASS == PASS_OWN) {
              float4 before[8];                              // the prefix's sums of these columns
#pragma unroll
              for (int k = 0; k < 8; ++k) before[k] = __ldcg(reinterpret_cast<const float4*>(p.prefix + at * D + q) + k);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                float x[4] = {o[k], o[k + 1], o[k + 2], o[k + 3]};
                add_prefix4(before[k / 4], f.prefix, x);
                o[k] = x[0]; o[k + 1] = x[1]; o[k + 2] = x[2]; o[k + 3] = x[3];
              }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = pack_bf16(o[16 * h + 2 * k], o[16 * h + 2 * k + 1]);
              store32(static_cast<bf16*>(p.out) + at * D + q + 16 * h, y, sector);
            }
          } else if (live) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t y[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(o[8 * h + k]);
              store32(sums + q + 8 * h, y, sector);
            }
          }
        }
        if (live && whole && PASS != PASS_PREFIX && p.lse) p.lse[at] = f.lse;
        if (live && whole && PASS == PASS_PREFIX) p.raw_ml[at] = make_float2(m, l);
        if (live && !whole) *reinterpret_cast<float2*>(part + TA_ROWS * D + 2 * rl) = make_float2(m, l);
      }
      tc_fence_before();                                     // before the next segment's first P
      if (!whole && slot == 1)
        split = AttnSplit{me, (int)(last / share), sg.b, sg.h, sg.tile, sg.n, sg.r0};
    }
  } else if (warp < 8) {
    // ------------------------------------------------ decode
    // a thread has 64 elements of one token: of its K and of its V (D = 128), or
    // of one of them
    const int w = tid - 128, tok = w & 63;
    const int bpp = p.P / CACHE_BLOCK, page_bits = 31 - __clz(p.P);
    const AttnSeg& ps = walk.sg;
    int u = ps.u;                                            // the unit to request next
    int page;                                                // its page of that unit
    auto pages = [&]() {
      const int at = ps.bad ? 0 : max(min(u * TA_UNIT + tok, ps.L - 1), 0);
      page = (int)load_now(reinterpret_cast<const uint32_t*>(p.table) + (size_t)ps.b * p.stride + (at >> page_bits));
    };
    struct Codes {
      uint4 code[TASKS][2];
      uint32_t scale[TASKS];                                 // of sixteen elements each
      bool there, bad;                                       // the token exists; and its page does not
    } even, odds;
    const uint32_t head_bytes = (uint32_t)(bpp * cache_block_bytes(D)), page_bytes = head_bytes * (uint32_t)p.Hkv;
    const int half = D == 128 ? w >> 6 : 0;
    auto is_v = [&](int k) { return D == 128 ? k == 1 : w >= 64; };
    // no branch around the loads, and none that keeps a value instead: what is
    // loaded stays in flight until it is decoded (past the end: the last unit again)
    auto request = [&](Codes& x) {
      const int at = u * TA_UNIT + tok;
      x.there = at < ps.L;
      x.bad = x.there && (uint32_t)page >= (uint32_t)p.num_pages;
      const uint8_t* blk = p.cache + (size_t)ps.h * head_bytes +
                           (uint64_t)((uint32_t)page < (uint32_t)p.num_pages ? (uint32_t)page : 0u) * page_bytes +
                           ((at & (p.P - 1)) >> 4) * cache_block_bytes(D);
#pragma unroll
      for (int k = 0; k < TASKS; ++k) {
        const uint4* code = reinterpret_cast<const uint4*>(blk + (is_v(k) ? cache_v_codes(D) : 0) + (tok & 15) * (D / 2) + half * 32);
        x.code[k][0] = load_now(code);
        x.code[k][1] = load_now(code + 1);
        x.scale[k] = load_now(reinterpret_cast<const uint32_t*>(blk + (is_v(k) ? cache_v_scales(D) : cache_k_scales(D)) +
                                                                (tok & 15) * (D / 16) + half * 4));
      }
      if (u + 1 < walk.u_end) {
        ++u;
      } else {
        walk.next(p, s_pre);
        if (!walk.done()) u = ps.u; else walk.pos = end;
      }
      pages();
    };
    auto spread = [&](uint8_t* half0, const uint4 (&code)[2], uint32_t scale) {
      uint8_t* dst = half0 + half * (TA_UNIT * 128) + tok * 128;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t two = decode_scales(scale >> (16 * q));
        const uint32_t f[2] = {__byte_perm(two, two, 0x1010), __byte_perm(two, two, 0x3232)};
        const uint32_t c[4] = {code[q].x, code[q].y, code[q].z, code[q].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = mul_h2(decode_byte(c, 4 * j + e), f[j >> 1]);
          *reinterpret_cast<uint4*>(dst + (((4 * q + j) ^ (tok & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      fence_async_shared();
    };
    auto unit = [&](uint32_t i, const Codes& x) {
      // keys: their buffer is free once the first product of two units ago is done
      if (D == 128 || w < 64) {
        const bool bad = __any_sync(0xffffffffu, x.bad);
        if (i >= 2) wait2(TB_S, i - 2);
        if (lane == 0) {
          s_bad[i & 3][warp & 3] = bad;
          if (bad) set_status(p.status, SPEC_DEV_BAD_SLOT);
        }
        spread(sm + L::K + (i & 1) * L::HALF, x.code[0], x.scale[0]);
        arrive(bar + TB_K + (i & 1));
      }
      // values: once the second one is; 0 for tokens that nobody wrote
      if (D == 128 || w >= 64) {
        if (i >= 2) wait2(TB_DONE, i - 2);
        uint4 code[2] = {x.code[TASKS - 1][0], x.code[TASKS - 1][1]};
        spread(sm + L::V + (i & 1) * L::HALF, code, x.there ? x.scale[TASKS - 1] : 0u);
        arrive(bar + TB_V + (i & 1));
      }
    };
    pages();
    request(even);
    for (uint32_t i = 0;; i += 2) {
      const bool last = walk.done();
      request(odds);
      unit(i, even);
      if (last) break;
      const bool last2 = walk.done();
      request(even);
      unit(i + 1, odds);
      if (last2) break;
    }
  } else {
    // ------------------------------------------------ products
    const uint32_t el = ta_elect();
    const uint32_t q0 = smem_u32(sm), k0 = q0 + L::K, v0 = q0 + L::V;
    bool first_prev = false;
    auto second = [&](uint32_t i, bool first) {
      wait2(TB_V, i);
      wait2(TB_P, i);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < TA_UNIT / 16; ++k)
        ta_mma_ts(el, tmem + TA_O, tmem + (i & 1) * TA_UNIT + TA_P + 8 * k,
                  tc_sdesc(v0 + (i & 1) * L::HALF + k * 2048, TA_UNIT * 128, 1024), ta_idesc<D>(1), first && k == 0 ? 0u : 1u);
      ta_commit(el, bar + TB_DONE + (i & 1));
    };
    uint32_t i = 0;
    for (uint32_t segs = 0; !walk.done(); walk.next(p, s_pre), ++segs)
      for (int u = walk.sg.u; u < walk.u_end; ++u, ++i) {
        const bool first = u == walk.sg.u;
        if (first) {
          if (i > 0) second(i - 1, first_prev);              // the softmax warps end the segment after it
          wait(bar + TB_Q, segs & 1);
        }
        wait2(TB_K, i);
        tc_fence_after();
#pragma unroll
        for (int s = 0; s < KSTEPS; ++s)
          ta_mma_ss(el, tmem + (i & 1) * TA_UNIT, tc_sdesc(q0 + (s >> 2) * (TA_ROWS * 128) + (s & 3) * 32, 16, 1024),
                    tc_sdesc(k0 + (i & 1) * L::HALF + (s >> 2) * (TA_UNIT * 128) + (s & 3) * 32, 16, 1024), ta_idesc<TA_UNIT>(0),
                    s > 0 ? 1u : 0u);
        ta_commit(el, bar + TB_S + (i & 1));
        if (!first) second(i - 1, first_prev);
        first_prev = first;
      }
    second(i - 1, first_prev);
    wait2(TB_DONE, i - 1);                                   // nothing in flight when tensor memory goes
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tc_dealloc(tmem, TA_COLS);
  if (tid == 0) static_cast<AttnSplit*>(p.ws)[me] = split;
}

namespace {
template <int PASS, int D>
cudaError_t launch_tc(const AttnParams& p, int sms, cudaStream_t st) {
  using L = TaLayout<D>;
  static_assert(2 * (L::TOTAL + 5 * 1024) <= 227 * 1024, "two CTAs an SM");
  // once a device: the attribute stays with the function
  static std::atomic<uint64_t> sized{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((sized.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(cache_attention_tc_kernel<PASS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::TOTAL);
    if (e != cudaSuccess) return e;
    if (dev < 64) sized.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  const long long tiles = (long long)p.T * p.G / TA_ROWS + (p.T < p.B ? p.T : p.B);
  const long long units = tiles * p.Hkv * (((long long)p.stride * p.P + TA_UNIT - 1) / TA_UNIT);
  long long ctas = 2LL * sms;
  if (ctas > AT_MAX_CTAS) ctas = AT_MAX_CTAS;
  if (ctas > units) ctas = units;
  e = launch_main<PASS>(cache_attention_tc_kernel<PASS, D>, p, (int)ctas, TA_THREADS, L::TOTAL, st);
  if (e != cudaSuccess) return e;
  return launch_attention_join<PASS, D, TA_ROWS, bf16>(p, (int)ctas, sms, st);
}
}  // namespace

template <int PASS>
cudaError_t launch_cache_attention_tc(const AttnParams& p, int D, int sms, cudaStream_t st) {
  return D == 64 ? launch_tc<PASS, 64>(p, sms, st) : launch_tc<PASS, 128>(p, sms, st);
}

}  // namespace spec
