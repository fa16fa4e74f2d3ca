// Log probabilities of given tokens, entropy and the top K alternatives of rows
// of logits x (divided by a temperature):
//
//   d = (x - m) log2(e) / T,  Z = sum 2^d,  lse = m / T + ln Z
//   logprob = (x_token - m) / T - ln Z,     H = ln 2 (log2 Z - sum 2^d d / Z)
//
// d is one fused multiply-add of x against the rounded m log2(e) / T; what the
// rounding adds to every d of a warp is known exactly and leaves its sums again.
//
// One read of each row.  logprobs_kernel: a CTA takes one segment of one row,
// 256 threads x 16 vectors of 16 bytes, all requested at once and kept in
// registers, so that maximum, sums and candidates come from one load.
//
// The K largest: a thread's maximum is at hand, so the K-th largest of 64
// group maxima (4 threads each) is a bound that at least K entries reach and,
// for values in no particular order, some 10 to 50 of 32768 do.  Those are
// collected and ranked by counting.  Equal values beyond the list's size (a
// row of few different values) are found one by one instead.
//
// Bound by latency between its phases (load, maxima, sums, bound, candidates), not
// by bytes: 128 requests of 1 to 8 tokens and 32000 bf16 logits (37 MB) take
// 18.5 us, 256 of 128256 (296 MB) 90 us, 3.3 TB/s of the 6.8 of a copy.  Two CTAs
// of 64 KB in registers an SM overlap each other's phases; half the vectors and
// four CTAs took 27 and 90 us (rows of two segments to join), three CTAs spilled.
// Warps with an entry of -inf or of the type's lowest value sum entry by entry:
// with nine tenths of the 128256 masked 285 us.  Rows little longer than a segment
// pay for a second one that has fewer entries than groups: 33000 entries 94 us.
//
// Rows of more than one segment are joined by logprobs_join_kernel, a warp a
// row, from each segment's (m, Z, sum 2^d d) and its K sorted candidates; its
// launch overlaps the first kernel's end.
#include "spec_serve.cuh"

namespace spec {

struct LogprobParams {
  int B, n, V, K, segments;
  float inv_n;                            // 1 / n: row / n without a division
  const void* logits;
  long long b_stride, row_stride;
  const int* tokens;
  const float* temperature;
  float* logprob;
  float* entropy;
  int* top_ids;
  float* top_lp;
  uint32_t* status;
  float4* part;                           // [rows][segments]: m, Z, sum 2^d d
  unsigned long long* keys;               // [rows][segments][K], descending
};

constexpr int LP_THREADS = 256, LP_WARPS = LP_THREADS / 32, LP_VECS = 16, LP_GROUPS = 64, LP_LIST = 256;
constexpr float LP_LN2 = 0.69314718056f;

template <class DT>
struct LpVec {
  static constexpr int E = 16 / sizeof(DT);                  // elements a vector
  static constexpr int SEG = LP_THREADS * LP_VECS * E;       // elements a segment: 32768 bf16, 16384 fp32
};

// Whole numbers in the order of the floats (-0 counts as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// Value descending, then index ascending; no entry's key is 0.
__device__ __forceinline__ unsigned long long entry_key(float x, int v) {
  return (unsigned long long)ordered(x) << 32 | (uint32_t)~v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest element of a vector, NaN if one is.
__device__ __forceinline__ float vec_max(const uint4& v, const bf16*) {
  const uint32_t m = max_nan2(max_nan2(v.x, v.y), max_nan2(v.z, v.w));
  return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}
__device__ __forceinline__ float vec_max(const uint4& v, const float*) {
  return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}
// Element e (a compile-time constant).
__device__ __forceinline__ float vec_get(const uint4& v, int e, const bf16*) {
  const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
  return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float vec_get(const uint4& v, int e, const float*) {
  return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
}
__device__ __forceinline__ uint32_t neg_inf_word(const bf16*) { return 0xff80ff80u; }
__device__ __forceinline__ uint32_t neg_inf_word(const float*) { return 0xff800000u; }
// What fills vectors without an entry: about -1e30, far below the entries of most
// rows, and finite so that 0 times its distance is 0.
__device__ __forceinline__ uint32_t low_word(const bf16*) { return 0xf14af14au; }
__device__ __forceinline__ uint32_t low_word(const float*) { return 0xf149f2cau; }
__device__ __forceinline__ float low_value(const bf16*) { return __uint_as_float(0xf14a0000u); }
__device__ __forceinline__ float low_value(const float*) { return __uint_as_float(0xf149f2cau); }
// Bits of an element.
__device__ __forceinline__ uint32_t bits_of(bf16 x) { return *reinterpret_cast<const uint16_t*>(&x); }
__device__ __forceinline__ uint32_t bits_of(float x) { return __float_as_uint(x); }
// The vector of elements [at, at + E) of a row of V, -inf where there is none.
template <class DT>
__device__ __noinline__ uint4 edge_vector(const DT* x, int at, int V) {
  constexpr int PER = 4 / sizeof(DT);
  const uint32_t w = neg_inf_word(static_cast<const DT*>(nullptr));
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = w;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int v = at + i * PER + e;
      if (v >= 0 && v < V) o[i] = PER == 1 ? bits_of(x[v]) : e ? (o[i] & 0xffffu) | bits_of(x[v]) << 16 : (o[i] & 0xffff0000u) | bits_of(x[v]);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Distances below a maximum as multiples of T / log2(e), not under -200 (where 2^d
// is 0): differences times `up`, then times c.  up = 1 but for a T below the normal
// numbers, whose own quotient would be infinite.
struct Distance {
  float up, c;
  __device__ __forceinline__ explicit Distance(float T) {
    up = T < 1.17549435e-38f ? 0x1p24f : 1.f;
    c = 1.4426950408889634f / (T * up);
  }
  __device__ __forceinline__ float operator()(float below) const { return fmaxf(below * up * c, -200.f); }
};

// What of a row can be said before its entries are read: bits of dev_status, or
// ~0 for a padding row.
__device__ __forceinline__ uint32_t row_flag(const LogprobParams& p, int token, float T) {
  if (token == -1) return ~0u;
  if (token < 0 || token >= p.V) return SPEC_DEV_BAD_TOKEN;
  if (!(T > 0.f) || !(T <= 3.402823466e38f)) return SPEC_DEV_BAD_TEMP;
  return 0;
}
__device__ __forceinline__ void write_nothing(const LogprobParams& p, int row, int lane, int lanes, uint32_t flag) {
  if (lane == 0) {
    p.logprob[row] = p.entropy[row] = quiet_nan();
    if (flag != ~0u) set_status(p.status, flag);
  }
  for (int k = lane; k < p.K; k += lanes) {
    p.top_ids[(size_t)row * p.K + k] = -1;
    p.top_lp[(size_t)row * p.K + k] = quiet_nan();
  }
}
// Request of a row: rows < 2^20, so the product is off by less than 0.125 / n.
__device__ __forceinline__ int request_of(const LogprobParams& p, int row) { return (int)(((float)row + 0.5f) * p.inv_n); }
template <class DT>
__device__ __forceinline__ const DT* row_at(const LogprobParams& p, int row) {
  const int b = request_of(p, row);
  return static_cast<const DT*>(p.logits) + b * p.b_stride + (row - b * p.n) * p.row_stride;
}

template <class DT>
__global__ void __launch_bounds__(LP_THREADS, 2) logprobs_kernel(const __grid_constant__ LogprobParams p) {
  constexpr int E = LpVec<DT>::E, SEG = LpVec<DT>::SEG;
  const DT* const tag = nullptr;
  __shared__ __align__(16) float s_group[LP_GROUPS];
  __shared__ float4 s_warp[LP_WARPS];
  __shared__ unsigned long long s_list[LP_LIST];
  __shared__ uint32_t s_bound;
  __shared__ int s_count;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int row = blockIdx.x, seg = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int token = __ldg(p.tokens + row);
  const float T = p.temperature ? __ldg(p.temperature + request_of(p, row)) : 1.f;
  const uint32_t flag = row_flag(p, token, T);
  if (flag) {
    if (p.segments == 1) write_nothing(p, row, tid, LP_THREADS, flag);
    return;
  }
  // vector i of the row holds elements [E i - lead, E i - lead + E): 16-byte aligned
  const DT* x = row_at<DT>(p, row);
  const int lead = (int)(((uintptr_t)x & 15) / sizeof(DT));
  const int i0 = seg * (SEG / E) + tid;
  uint4 v[LP_VECS];
  float vm[LP_VECS], tm;
  const bool full = seg * SEG >= lead && (seg + 1) * SEG - lead <= p.V;   // uniform: a segment that the row fills
  if (full) {
    const uint4* at = reinterpret_cast<const uint4*>(x + (i0 * E - lead));
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) v[j] = __ldcs(at + j * LP_THREADS);
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) vm[j] = vec_max(v[j], tag);
  } else {
    uint32_t edges = 0;                                      // this thread's vectors that the row fills in part:
                                                             // its first and its last may be one thread's
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) {
      const int at = (i0 + j * LP_THREADS) * E - lead;
      const uint32_t w = low_word(tag);
      v[j] = make_uint4(w, w, w, w);
      if (at >= 0 && at + E <= p.V) v[j] = __ldcs(reinterpret_cast<const uint4*>(x + at));
      else if (at + E > 0 && at < p.V) edges |= 1u << j;
    }
    while (edges) {
      const int edge = __ffs(edges) - 1;
      edges &= edges - 1;
      const uint4 q = edge_vector(x, (i0 + edge * LP_THREADS) * E - lead, p.V);
#pragma unroll
      for (int j = 0; j < LP_VECS; ++j)
        if (j == edge) v[j] = q;
    }
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) {
      const int at = (i0 + j * LP_THREADS) * E - lead;
      vm[j] = at + E > 0 && at < p.V ? vec_max(v[j], tag) : -INFINITY;
    }
  }
  if (tid == 0) {
    s_count = 0;
    s_bound = 0;
  }
  // ---- maxima: thread, group of 4 threads, warp
  tm = vm[0];
#pragma unroll
  for (int j = 1; j < LP_VECS; ++j) tm = max_nan(tm, vm[j]);
  float gm = tm;
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) gm = max_nan(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  if ((lane & 3) == 0) s_group[tid >> 2] = gm;
  float m = gm;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  // ---- sums against the warp's maximum; an entry of -inf adds nothing
  const Distance distance(T);
  const float c = distance.c;
  const float base = m == -INFINITY ? 0.f : -m * c;
  // the distance that the maximum gets: the rounding of m c, exactly.  Every
  // distance of the warp holds it, so Z and sum 2^d d are cleared of it below.
  float off = m == -INFINITY ? 0.f : fmaf(m, c, base);
  float z = 0.f, w1 = 0.f;
  {
    const uint64_t c2 = pair(c, c), b2 = pair(base, base);
    uint64_t z2[2] = {0, 0}, w2[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j)
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint64_t d2 = fma2(pair(vec_get(v[j], e, tag), vec_get(v[j], e + 1, tag)), c2, b2);
        const float2 d = unpair(d2);
        const uint64_t y2 = pair(ex2(d.x), ex2(d.y));
        z2[j & 1] = add2(z2[j & 1], y2);
        w2[j & 1] = fma2(y2, d2, w2[j & 1]);
      }
    const float2 zs = unpair(add2(z2[0], z2[1])), ws = unpair(add2(w2[0], w2[1]));
    z = zs.x + zs.y;
    w1 = ws.x + ws.y;
  }
  // a filler whose exponential is not 0: entries as low as it, or a temperature
  // beside which it is near them
  const bool filler = !full && fmaf(low_value(tag), c, base) > -127.f;
  if (__any_sync(0xffffffffu, !(fabsf(w1) <= 3.4e38f)) || !(fabsf(off) <= 1.f) || filler || distance.up != 1.f) {
    // an entry of -inf (0 times its distance), numbers near the floats' end, |m c|
    // beyond 2^24, where `off` would cost the distances their last bits, a filler
    // that counts, or a subnormal T: once more, distances first and bounded
    z = w1 = off = 0.f;
    for (int j = 0; j < LP_VECS; ++j) {
      const int at = (i0 + j * LP_THREADS) * E - lead;
      float zz = 0.f, ww = 0.f;
      for (int e = max(0, -at); e < E && at + e < p.V; ++e) {
        const float y = tof(x[at + e]);
        const float d = y == -INFINITY ? -200.f : distance(y - m);
        const float q = ex2(d);
        zz += q;
        ww = fmaf(q, d, ww);
      }
      z += zz;
      w1 += ww;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    w1 += __shfl_xor_sync(0xffffffffu, w1, o);
  }
  if (lane == 0) {
    // the maximum itself counts 1, whatever 2^off 2^-off is rounded to
    const float f = ex2(-off);
    w1 = f * fmaf(-off, z, w1);
    z = fmaxf(z * f, 1.f);
    s_warp[warp] = make_float4(m, m == -INFINITY ? 0.f : z, m == -INFINITY ? 0.f : w1, 0.f);
  }
  __syncthreads();
  // ---- bound of the candidates: the K-th largest group maximum
  if (p.K > 0) {
    // the largest group maximum that K groups reach; with a NaN none may, and
    // the row has no distribution
    if (tid < LP_GROUPS) {
      const float g = s_group[tid];
      int reach = 0;
#pragma unroll 4
      for (int i = 0; i < LP_GROUPS; i += 4) {
        const float4 h = *reinterpret_cast<const float4*>(s_group + i);
        reach += (h.x >= g) + (h.y >= g) + (h.z >= g) + (h.w >= g);
      }
      const uint32_t best = __reduce_max_sync(0xffffffffu, reach >= p.K ? ordered(g) : 0u);
      if (lane == 0) atomicMax(&s_bound, best);
    }
    __syncthreads();
    const float bound = s_bound ? from_ordered(s_bound) : INFINITY;
    uint32_t hit = 0;
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) hit |= (vm[j] >= bound ? 1u : 0u) << j;
    // few vectors: read again rather than picked out of the registers, which
    // would take the code of every vector (it is bound by instruction fetches then)
    while (hit) {
      const int j = __ffs(hit) - 1, at = (i0 + j * LP_THREADS) * E - lead;
      hit &= hit - 1;
      const uint4 q = at >= 0 && at + E <= p.V ? __ldg(reinterpret_cast<const uint4*>(x + at)) : edge_vector(x, at, p.V);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float y = vec_get(q, e, tag);
        // entries of -inf count only where the lowest indexes may be needed
        if (y >= bound && (y > -INFINITY || (at + e >= 0 && at + e < p.V && at + e < seg * SEG - lead + 64))) {
          const int k = atomicAdd(&s_count, 1);
          if (k < LP_LIST) s_list[k] = entry_key(y, at + e);
        }
      }
    }
    __syncthreads();
  }
  // ---- this segment's part, warp by warp in order, and its K largest: the
  // first warp's work, unless the list overflowed
  const bool single = p.segments == 1;
  const int count = p.K > 0 ? s_count : 0;
  if (warp > 0 && count <= LP_LIST) return;
  float pm = s_warp[0].x;
#pragma unroll
  for (int i = 1; i < LP_WARPS; ++i) pm = max_nan(pm, s_warp[i].x);
  float pz = 0.f, pw = 0.f;
#pragma unroll
  for (int i = 0; i < LP_WARPS; ++i) {
    const float4 q = s_warp[i];
    const float d = q.x == -INFINITY ? 0.f : distance(q.x - pm), f = ex2(d);
    pz += q.y * f;
    pw += f * fmaf(q.y, d, q.z);
  }
  const bool bad = !(pm < INFINITY) || (single && pm == -INFINITY);
  const size_t at_part = (size_t)row * p.segments + seg;
  if (!single && tid == 0) p.part[at_part] = make_float4(pm, pz, pw, 0.f);
  float lz = 0.f;
  if (single) {
    if (bad) {
      write_nothing(p, row, tid, 32, SPEC_DEV_BAD_LOGIT);
      return;
    }
    lz = LP_LN2 * log2f(pz);
    if (tid == 0) {
      p.logprob[row] = (tof(x[token]) - pm) / T - lz;
      p.entropy[row] = lz - LP_LN2 * pw / pz;
    }
  }
  if (p.K == 0 || bad) return;
  auto put = [&](int rank, unsigned long long key) {
    if (single) {
      p.top_ids[(size_t)row * p.K + rank] = (int)~(uint32_t)key;
      p.top_lp[(size_t)row * p.K + rank] = (from_ordered((uint32_t)(key >> 32)) - pm) / T - lz;
    } else {
      p.keys[at_part * p.K + rank] = key;
    }
  };
  if (count <= LP_LIST) {
    for (int k = lane; k < count; k += 32) {
      const unsigned long long mine = s_list[k];
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < count; ++i) rank += s_list[i] > mine;
      if (rank < p.K) put(rank, mine);
    }
    if (!single && lane >= count && lane < p.K) put(lane, 0);   // a segment of fewer entries
  } else {
    // too many equal values: the largest below the last one found, K times
    unsigned long long last = ~0ull;
    const int lo = max(seg * SEG - lead, 0), hi = min((seg + 1) * SEG - lead, p.V);
    for (int k = 0; k < p.K; ++k) {
      unsigned long long best = 0;
      for (int i = lo + tid; i < hi; i += LP_THREADS) {
        const unsigned long long key = entry_key(tof(x[i]), i);
        if (key < last && key > best) best = key;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const unsigned long long u = __shfl_xor_sync(0xffffffffu, best, o);
        if (u > best) best = u;
      }
      __syncthreads();
      if (lane == 0) s_list[warp] = best;
      __syncthreads();
      for (int i = 0; i < LP_WARPS; ++i)
        if (s_list[i] > best) best = s_list[i];
      last = best;
      if (tid == 0) put(k, best);
    }
  }
}

// A warp a row: the parts' sums joined in order, and K times the largest of the
// segments' next candidates.
constexpr int LPJ_WARPS = 4;
template <class DT>
__global__ void __launch_bounds__(32 * LPJ_WARPS) logprobs_join_kernel(const __grid_constant__ LogprobParams p) {
  extern __shared__ unsigned long long s_lists[];            // [warps][33][K]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * LPJ_WARPS + warp;
  if (row < p.B * p.n) {
    const int token = __ldg(p.tokens + row);
    const float T = p.temperature ? __ldg(p.temperature + request_of(p, row)) : 1.f;
    const uint32_t flag = row_flag(p, token, T);
    const float xt = flag ? 0.f : tof(row_at<DT>(p, row)[token]);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (flag) {
      write_nothing(p, row, lane, 32, flag);
      return;
    }
    const float4* part = p.part + (size_t)row * p.segments;
    float m = -INFINITY;
    for (int s = lane; s < p.segments; s += 32) m = max_nan(m, part[s].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!(m < INFINITY) || m == -INFINITY) {
      write_nothing(p, row, lane, 32, SPEC_DEV_BAD_LOGIT);
      return;
    }
    const Distance distance(T);
    float z = 0.f, w1 = 0.f;
    for (int s = lane; s < p.segments; s += 32) {
      const float4 q = part[s];
      const float d = q.x == -INFINITY ? 0.f : distance(q.x - m), f = ex2(d);
      z += q.y * f;
      w1 += f * fmaf(q.y, d, q.z);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, o);
      w1 += __shfl_xor_sync(0xffffffffu, w1, o);
    }
    const float lz = LP_LN2 * log2f(z);
    if (lane == 0) {
      p.logprob[row] = (xt - m) / T - lz;
      p.entropy[row] = lz - LP_LN2 * w1 / z;
    }
    if (p.K == 0) return;
    const unsigned long long* keys = p.keys + (size_t)row * p.segments * p.K;
    unsigned long long mine = 0;                             // lane k keeps the k-th
    unsigned long long* s_keys = s_lists + warp * (33 * p.K);
    if (p.segments <= 4) {
      // few lists: every entry's rank is its place in its own list and, by
      // bisection, in the others
      const int total = p.segments * p.K;
      for (int i = lane; i < total; i += 32) s_keys[i] = keys[i];
      __syncwarp();
      for (int i = lane; i < total; i += 32) {
        const unsigned long long key = s_keys[i];
        if (key == 0) continue;                              // no entry
        const int own = i / p.K;
        int rank = i - own * p.K;
        for (int s = 0; s < p.segments; ++s)
          if (s != own) {
            int lo = 0, hi = p.K;                            // entries of list s above key
            while (lo < hi) {
              const int mid = (lo + hi) >> 1;
              if (s_keys[s * p.K + mid] > key) lo = mid + 1; else hi = mid;
            }
            rank += lo;
          }
        if (rank < p.K) {
          p.top_ids[(size_t)row * p.K + rank] = (int)~(uint32_t)key;
          p.top_lp[(size_t)row * p.K + rank] = (from_ordered((uint32_t)(key >> 32)) - m) / T - lz;
        }
      }
      return;
    }
    // 32 segments at a time: their sorted lists and the best so far in shared
    // memory, and K times the largest of the lists' heads
    for (int s0 = 0; s0 < p.segments; s0 += 32) {
      const int lists = min(32, p.segments - s0);
      __syncwarp();
      for (int i = lane; i < lists * p.K; i += 32) s_keys[i] = keys[(size_t)s0 * p.K + i];
      if (lane < p.K) s_keys[32 * p.K + lane] = mine;        // the best so far
      __syncwarp();
      int at = 0, at_best = 0;
      unsigned long long head = lane < lists ? s_keys[lane * p.K] : 0, kept = s0 ? s_keys[32 * p.K] : 0;
      unsigned long long out = 0;
      for (int k = 0; k < p.K; ++k) {
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32) == hi ? (uint32_t)head : 0u);
        unsigned long long best = (unsigned long long)hi << 32 | lo;
        if (kept > best) {                                   // uniform
          best = kept;
          kept = ++at_best < p.K ? s_keys[32 * p.K + at_best] : 0;
        } else if (head == best && best) {
          head = ++at < p.K ? s_keys[lane * p.K + at] : 0;
        }
        if (lane == k) out = best;
      }
      mine = out;
    }
    if (lane < p.K) {
      p.top_ids[(size_t)row * p.K + lane] = (int)~(uint32_t)mine;
      p.top_lp[(size_t)row * p.K + lane] = (from_ordered((uint32_t)(mine >> 32)) - m) / T - lz;
    }
  }
}

namespace {
// Segments of the longest layout of a row: V elements after up to E - 1 others.
int segments_of(int V, int dtype) {
  const int E = dtype == SPEC_BF16 ? 8 : 4;
  const int seg = LP_THREADS * LP_VECS * E;
  return (V + E - 1 + seg - 1) / seg;
}
}  // namespace

size_t logprobs_workspace_bytes(int rows, int V, int K) {
  const size_t n = (size_t)rows * segments_of(V, SPEC_F32);
  return n * sizeof(float4) + n * K * sizeof(unsigned long long) + 256;
}

template <class DT>
static cudaError_t launch(LogprobParams p, const spec_logprobs_args& a, cudaStream_t st) {
  // rows that all start on 16 bytes need no room for others' elements before them
  const int E = LpVec<DT>::E;
  const bool even = a.b_stride % E == 0 && a.row_stride % E == 0;
  const int rows = a.B * a.n;
  p.segments = (a.V + (even ? 0 : E - 1) + LpVec<DT>::SEG - 1) / LpVec<DT>::SEG;
  p.part = static_cast<float4*>(a.workspace);
  p.keys = reinterpret_cast<unsigned long long*>(p.part + (size_t)rows * p.segments);
  p.inv_n = 1.f / (float)a.n;
  logprobs_kernel<DT><<<dim3(rows, p.segments), LP_THREADS, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.segments == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + LPJ_WARPS - 1) / LPJ_WARPS);
  cfg.blockDim = dim3(32 * LPJ_WARPS);
  cfg.dynamicSmemBytes = (size_t)LPJ_WARPS * 33 * p.K * sizeof(unsigned long long);   // at most 33 KB
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_join_kernel<DT>, p);
}

cudaError_t launch_logprobs(const spec_logprobs_args& a, cudaStream_t st) {
  LogprobParams p{a.B, a.n, a.V, a.K, 0, 0.f, a.logits, a.b_stride, a.row_stride, a.tokens, a.temperature, a.logprob,
                  a.entropy, a.top_ids, a.top_logprobs, a.dev_status, nullptr, nullptr};
  return a.dtype == SPEC_BF16 ? launch<bf16>(p, a, st) : launch<float>(p, a, st);
}

}  // namespace spec
