// Shared by the kernels of the attention over the 4-bit cache: parameters, the
// numbering of the work, operand helpers, and the kernel that joins the parts
// of segments that more than one worker computed.
#pragma once

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

constexpr int AT_WARPS = 8;               // workspace slots: AT_MAX_CTAS * AT_WARPS workers at most
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

// The parts follow one AttnSplit a worker.
__device__ __forceinline__ float* attn_parts(const AttnParams& p) {
  return reinterpret_cast<float*>(static_cast<char*>(p.ws) + AT_MAX_CTAS * AT_WARPS * sizeof(AttnSplit));
}

// What a segment is: request b's units over key-value head h for one row tile.
struct AttnSeg {
  int b, h, tile, u, nu;                  // units u .. nu - 1 are left
  int n, r0, L;
  bool bad;
};

// Units of request b over all heads and row tiles (0: nothing to do).  LEAD: what
// a segment costs besides its units, counted as units ahead of them.
template <int ROWS, int UNIT, int LEAD>
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
  nu = bad ? 1 : (L + UNIT - 1) / UNIT;
  return (long long)p.Hkv * tiles * (nu + LEAD);
}

// Units before each group of requests, by the first THREADS threads of a CTA
// (whole warps; the caller synchronises them before and after): s_pre[THREADS + 1],
// s_scan[THREADS / 32].  A group is ceil(B / THREADS) requests.
template <int ROWS, int UNIT, int THREADS, int LEAD = 0, class Sync>
__device__ __forceinline__ long long attn_prefix(const AttnParams& p, long long* s_pre, long long* s_scan, Sync sync) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int items = (p.B + THREADS - 1) / THREADS;
  long long mine = 0;
  bool flag = false;
  for (int i = 0; i < items; ++i) {
    const int b = tid * items + i;
    if (b >= p.B) break;
    int n, r0, L, tiles, nu;
    bool bad, outside;
    mine += attn_work<ROWS, UNIT, LEAD>(p, b, n, r0, L, tiles, nu, bad, outside);
    flag |= bad || outside;
  }
  long long v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) s_scan[warp] = v;
  sync();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s_scan[w];
    all += s_scan[w];
  }
  s_pre[tid] = before + v - mine;
  if (tid == 0) s_pre[THREADS] = all;
  if (flag && blockIdx.x == 0) set_status(p.status, SPEC_DEV_BAD_LEN);
  return all;
}

// The segment that holds unit `pos` (below the total); LEAD more units to `u`.
template <int ROWS, int UNIT, int THREADS, int LEAD = 0>
__device__ __forceinline__ AttnSeg attn_locate(const AttnParams& p, const long long* s_pre, long long pos) {
  const int items = (p.B + THREADS - 1) / THREADS;
  int lo = 0, hi = THREADS;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_pre[mid] <= pos) lo = mid; else hi = mid;
  }
  long long left = pos - s_pre[lo];
  AttnSeg s;
  int tiles;
  for (int b = lo * items;; ++b) {
    bool outside;
    const long long w = attn_work<ROWS, UNIT, LEAD>(p, b, s.n, s.r0, s.L, tiles, s.nu, s.bad, outside);
    if (left < w) {
      s.b = b;
      break;
    }
    left -= w;
  }
  const long long seg = left / (s.nu + LEAD);
  s.u = (int)(left - seg * (s.nu + LEAD));
  s.h = (int)(seg / tiles);
  s.tile = (int)(seg - (long long)s.h * tiles);
  return s;
}

// Whether phase `parity` of a barrier is complete; what the phase publishes is
// read after it.
__device__ __forceinline__ bool bar_try(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// Bounded wait; false if it gave up.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint32_t tries = 1u << 24) {
  for (uint32_t it = 0; it < tries; ++it)
    if (bar_try(bar, parity)) return true;
  return false;
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
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// The first product of a sum: no accumulator to clear.
__device__ __forceinline__ void mma_f16_first(float* c, const uint4& a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
}
// An 8x8 matrix of 16-bit floats, a row's pair a lane, to its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// The segment after one that ended, whose first unit is `pos`: most often the
// same request's.
template <int ROWS, int UNIT, int THREADS, int LEAD = 0>
__device__ __forceinline__ AttnSeg attn_next(const AttnParams& p, const long long* s_pre, const AttnSeg& seg, long long pos) {
  AttnSeg s = seg;
  s.u = 0;
  if (++s.tile * ROWS < s.n * p.G) return s;
  s.tile = 0;
  if (++s.h < p.Hkv) return s;
  return attn_locate<ROWS, UNIT, THREADS, LEAD>(p, s_pre, pos);
}

// The power of two that takes mx into [2^14, 2^15) (at most 2^120; 2^15 for 0,
// infinities and NaN), as its exponent.
__device__ __forceinline__ int query_exponent(float mx) {
  const uint32_t u = __float_as_uint(mx);
  if (!(mx > 0.f && mx <= 3.402823466e38f)) return 15;
  return min(15 + 126 - (int)(u >> 23), 120);
}
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 .. 127

// The kernel of 128-row tiles (bf16, D = 64 or 128).
cudaError_t launch_cache_attention_tc(const AttnParams& p, int D, int sms, cudaStream_t st);

// Adds the parts of the split segments: CTA (x, y) takes the segments that
// begin at workers x, x + gridDim.x, .. and 1024 / D rows of each.  A part is
// [ROWS][D] unnormalised outputs and (m, sum) a row; worker w has slot 0 for a
// segment that began before its share and slot 1 for one that begins in it.
// Threads that the rows leave over share the parts, and each requests JOIN_BATCH
// of them before it adds the first, so a long context's 30 parts cost a few round
// trips; the order of every sum depends on the numbers of rows and parts alone.
// Its launch overlaps the main kernel's end; 10 to 25 us by itself with cold
// caches (two rows a CTA: 24 us where 14 are kept, for 1824 workers of 2 parts).
constexpr int JOIN_THREADS = 256, JOIN_BATCH = 4;
template <int D, int ROWS, class DT>
__global__ void __launch_bounds__(JOIN_THREADS) cache_attention_join_kernel(const __grid_constant__ AttnParams p, int workers) {
  __shared__ float4 s_acc[JOIN_THREADS];
  __shared__ float2 s_ml[JOIN_THREADS];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  constexpr int PART = ROWS * D + 2 * ROWS, RQ = D / 4;      // float4 a row
  constexpr int JOIN_ROWS = JOIN_THREADS / RQ < ROWS ? JOIN_THREADS / RQ : ROWS;
  const float* parts = attn_parts(p);
  const AttnSplit* splits = static_cast<const AttnSplit*>(p.ws);
  for (int w = blockIdx.x; w < workers; w += gridDim.x) {
    const AttnSplit s = splits[w];
    if (s.last < s.first) continue;
    const int rows = s.n * p.G;
    const int live = min(JOIN_ROWS, rows - s.tile * ROWS - JOIN_ROWS * (int)blockIdx.y);
    if (live <= 0) continue;                               // uniform over the CTA
    const int items = live * RQ;
    // `shares` threads an item: each adds the parts first + own, + shares, ..
    int shares = JOIN_THREADS / items;
    if (shares > s.last - s.first + 1) shares = s.last - s.first + 1;
    if (shares < 1) shares = 1;
    auto add = [](float2& ml, float4& acc, const float2& v, const float4& o) {
      const float mn = fmaxf(ml.x, v.x);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float fa = exp2f(ml.x - ref), fb = exp2f(v.x - ref);
      ml.x = mn;
      ml.y = ml.y * fa + v.y * fb;
      acc.x = acc.x * fa + o.x * fb;
      acc.y = acc.y * fa + o.y * fb;
      acc.z = acc.z * fa + o.z * fb;
      acc.w = acc.w * fa + o.w * fb;
    };
    {
      const int own = threadIdx.x / items, it = threadIdx.x - own * items;
      const bool mine = own < shares;
      const int rl = JOIN_ROWS * blockIdx.y + it / RQ, d = 4 * (it % RQ);
      float2 ml = make_float2(-INFINITY, 0.f);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (mine) {
        // JOIN_BATCH parts requested before the first is added
        for (int x0 = s.first + own; x0 <= s.last; x0 += JOIN_BATCH * shares) {
          float2 v[JOIN_BATCH];
          float4 o[JOIN_BATCH];
#pragma unroll
          for (int k = 0; k < JOIN_BATCH; ++k) {
            const int x = x0 + k * shares;
            v[k] = make_float2(-INFINITY, 0.f);
            o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x <= s.last) {
              const float* part = parts + (size_t)(2 * x + (x == s.first ? 1 : 0)) * PART;
              // not by the read-only path: the parts were written while this kernel was there
              v[k] = __ldcg(reinterpret_cast<const float2*>(part + ROWS * D + 2 * rl));
              o[k] = __ldcg(reinterpret_cast<const float4*>(part + rl * D + d));
            }
          }
#pragma unroll
          for (int k = 0; k < JOIN_BATCH; ++k)
            if (x0 + k * shares <= s.last) add(ml, acc, v[k], o[k]);
        }
      }
      if (shares > 1) {
        __syncthreads();
        s_acc[threadIdx.x] = acc;
        s_ml[threadIdx.x] = ml;
        __syncthreads();
        if (own == 0)
          for (int k = 1; k < shares; ++k) add(ml, acc, s_ml[k * items + it], s_acc[k * items + it]);
      }
      if (own > 0) continue;
      const int r = s.tile * ROWS + rl;
      const int tok = r / p.G, hq = s.h * p.G + r - tok * p.G;
      const size_t at = (size_t)(s.r0 + tok) * p.Hq + hq;
      const float inv = ml.y == 0.f ? 0.f : p.v_scale / ml.y;
      const float x[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
      store4(static_cast<DT*>(p.out) + at * D + d, x);
      if (d == 0 && p.lse) p.lse[at] = ml.y == 0.f ? -INFINITY : 0.69314718056f * (ml.x + log2f(ml.y));
    }
  }
}

// Launches the join after the main kernel of `ctas` CTAs x `per_cta` workers;
// its launch overlaps the main kernel's end.
template <int D, int ROWS, class DT>
cudaError_t launch_attention_join(const AttnParams& p, int workers, int sms, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(workers < 4 * sms ? workers : 4 * sms, (ROWS * D / 4 + JOIN_THREADS - 1) / JOIN_THREADS);
  cfg.blockDim = dim3(JOIN_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_attention_join_kernel<D, ROWS, DT>, p, workers);
}

}  // namespace spec
