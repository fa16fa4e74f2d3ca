// Sampling with temperature, top-k, top-p and min-p from given uniform numbers.
//
//   w_v = exp((x_v - max x) / T); kept: the first n entries in descending order;
//   token: the smallest v (vocabulary order) with F(v) > u F(V), F over kept w.
//
// Weights are whole numbers of 2^-frac of the largest, so sums are exact in any
// order and every border -- the k-th entry, the mass of top-p, the drawn token -- is
// decided on exact sums of them (Weigh says how near a weight is to its value).
//
// A cluster of CTAs takes a row, each CTA a slice of the vocabulary, a warp a tile of
// it at a time:
//
//   1  the largest entry; of each thread the largest of groups of its entries
//   2  what is certainly kept and what has to be looked at: with top-k, a bound that
//      at least k of the groups' maxima reach; with top-p alone, from the whole mass and
//      a histogram of counts over (max x - x), which bounds the running mass at the
//      bins' edges from both sides
//   3  certainly kept entries add to their tile's sum, the others go to a list
//   4  the list sorted by (value, index): its kept entries add to their tiles' sums
//   5  the tile that holds the drawn token, then the token
//
// Rows whose list overflows (thousands of entries next to a border: wide ties) find
// their borders by histograms over the row itself, 2048 bins of keys a pass.
#include <cooperative_groups.h>

#include <atomic>

#include "spec_df.cuh"
#include "spec_serve.cuh"

namespace spec {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

struct SampleParams {
  int n, V;
  const void* logits;
  long long b_stride, row_stride;
  const float* u;
  const float* temperature;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  int* tokens;
  float* logprob;
  int* kept;
  uint32_t* status;
  int idx_bits, frac;                     // bits of an index; a weight's unit is 2^-frac
  int slice, tile_vectors;                // entries a CTA, vectors a lane of a tile
};

constexpr int SA_THREADS = 512, SA_WARPS = SA_THREADS / 32, SA_BINS = 2048;
constexpr int SA_STEP_BITS = 10;           // of a key, a pass of a search
constexpr int SA_LIST = 2048;             // entries of a row's list
constexpr int SA_TILES = 512;             // tiles a CTA
constexpr int SA_GROUPS = 8;              // groups of entries a thread, each with its maximum
constexpr float SA_LOWEST = -3.402823466e38f;

// Order of a logit, descending: smaller for larger values, -0 as 0; 16 bits hold bf16's.
template <class DT>
__device__ __forceinline__ uint32_t descending(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t d = (b & 0x80000000u) ? b : ~(b | 0x80000000u);
  return sizeof(DT) == 2 ? d >> 16 : d;
}
// x of descending(x).
template <class DT>
__device__ __forceinline__ float of_descending(uint32_t d) {
  if (sizeof(DT) == 2) d = (d << 16) | ((d & 0x8000u) ? 0u : 0xffffu);
  return __uint_as_float((d & 0x80000000u) ? d : ~d & 0x7fffffffu);
}

// 2^(j/1024) as sums of two fp32 numbers, from 64-bit products of 2^(2^i/1024).
constexpr int SA_TABLE = 1024;
struct alignas(16) PowerTable {           // copied 16 bytes at a time
  float2 at[SA_TABLE];
};
constexpr PowerTable power_table() {
  // square roots of 2, 2^(1/2), .. by Newton's iteration
  double root[10] = {};
  double x = 2.;
  for (int i = 0; i < 10; ++i) {
    double y = 1. + (x - 1.) / 2.;
    for (int k = 0; k < 60; ++k) y = (y + x / y) / 2.;
    root[9 - i] = x = y;
  }
  PowerTable t{};
  for (int j = 0; j < SA_TABLE; ++j) {
    double v = 1.;
    for (int i = 0; i < 10; ++i)
      if (j >> i & 1) v *= root[i];
    const float hi = (float)v;
    t.at[j].x = hi;
    t.at[j].y = (float)(v - (double)hi);
  }
  return t;
}
__device__ const PowerTable g_powers = power_table();

// Weights of a row: 2^t, t = (x - m) log2(e) / T, in whole units of 2^-frac.  In
// 1024ths of an octave t is formed in double-float, k the nearest whole number and
// y = t - k, and 2^(t/1024) = 2^(k/1024) (1 + s + s^2 / 2), s = y ln 2 / 1024, whose
// next term is 2^-37 at most; with the table's two terms that leaves a relative error
// below 2^-34.5, of either sign.  Entries below 2^-44 count as nothing.  T is taken as
// f times a number whose reciprocal is ordinary.
struct Weigh {
  float m, f, least, unit;
  u64 step;                               // units a 2^-22
  df c, inv;                              // 1024 log2(e) f / T, 1 / (T f)
  const float2* tab;
  __device__ __forceinline__ Weigh(float m_, float T, int frac, const float2* tab_) : m(m_), tab(tab_) {
    const int e = max(-100, min(100, -ilogbf(T)));
    f = ldexpf(1.f, e);
    inv = dd_recip(rn_mul(T, f));
    c = dd_mul(inv, octaves());
    least = -44.f * 1024.f / c.hi;
    unit = ldexpf(1.f, frac);
    step = 1ull << (frac - 22);
  }
  __device__ __forceinline__ static df octaves() { return {1477.31970f, 1.97218615e-05f}; }   // 1024 log2(e)
  // 2^((t + te) / 1024) as hi + lo, t in the range of fp32's exponents.
  __device__ __forceinline__ static df power(float t, float te, const float2* tab) {
    const float k = rn_add(t, 12582912.f);                   // 1.5 2^23: k in the low bits
    const float y = rn_add(rn_sub(t, rn_sub(k, 12582912.f)), te);
    const float s = rn_mul(y, 6.76901552e-04f);
    const float s2 = rn_fma(rn_mul(s, 0.5f), s, s);
    const int ki = __float_as_int(k) - 0x4b400000;
    const float2 p = tab[ki & (SA_TABLE - 1)];
    const float scale = __int_as_float(((ki >> 10) << 23) + 0x3f800000);
    return {rn_mul(p.x, scale), rn_mul(rn_fma(p.x, s2, p.y), scale)};
  }
  // (x - m) / T
  __device__ __forceinline__ df argument(float x) const {
    const df d = two_sum_df(x, -m);
    return dd_mul(df{rn_mul(d.hi, f), rn_mul(d.lo, f)}, inv);
  }
  __device__ __forceinline__ u64 operator()(float x) const { return of(two_sum_df(x, -m)); }
  // Of an entry that lies d below the largest.
  __device__ __forceinline__ u64 of(df d) const {
    const float h = rn_mul(d.hi, f);
    const bool in = h > least;
    const float dh = in ? h : least, dl = in ? rn_mul(d.lo, f) : 0.f;
    const float t = rn_mul(dh, c.hi);
    const df w = power(t, rn_fma(dl, c.hi, rn_fma(dh, c.lo, rn_fma(dh, c.hi, -t))), tab);
    const float a = rn_add(w.hi, 3.f);                       // hi to a whole number of 2^-22
    const float rest = rn_add(rn_sub(w.hi, rn_sub(a, 3.f)), w.lo);
    return (u64)(uint32_t)(__float_as_int(a) - 0x40400000) * step + (u64)(long long)__float2int_rn(rn_mul(rest, unit));
  }
  // The natural logarithm of z > 0: the fp32 one and a Newton step.
  __device__ __forceinline__ df log(df z) const {
    const float y = logf(z.hi);
    if (!(fabsf(y) < 87.f)) return {y, 0.f};
    const float t = rn_mul(-y, octaves().hi);
    const df e = power(t, rn_fma(-y, octaves().lo, rn_fma(-y, octaves().hi, -t)), tab);   // 1 / z, nearly
    const df q = two_prod_df(z.hi, e.hi);
    return {y, rn_add(rn_sub(q.hi, 1.f), rn_fma(z.hi, e.lo, rn_fma(z.lo, e.hi, q.lo)))};
  }
};

// A number of [0, 1) in units of 2^-64 (below 2^-40 rounded down).
__device__ __forceinline__ u64 fraction64(float x) { return __float2ull_rz(x * 18446744073709551616.f); }

struct SampleShared {
  u64 sorted[SA_LIST];                    // the row's list
  u64 key[SA_LIST];                       // this CTA's list
  u64 hist[SA_BINS / 2];                  // counts of 32 bits; 64-bit sums of half as many bins in a search
  u64 tile[SA_TILES];                     // kept mass
  u64 scan[2][SA_WARPS];
  u64 before;                             // of the bin that a search goes on in
  u64 sum[2];                             // of one CTA, read by the cluster: mass, entries
  alignas(16) float2 tab[SA_TABLE];
  int bin[2], listed, at;
  uint32_t top, low, bad;                 // of one CTA
};
static_assert(offsetof(SampleShared, tab) % 16 == 0, "copied 16 bytes at a time");

template <class DT>
struct Sampler {
  static constexpr int W = 16 / sizeof(DT), BATCH = 4;
  const SampleParams& p;
  SampleShared& s;
  cg::cluster_group cl;
  const int tid, lane, warp, C, rank;
  const DT* row;
  int first, last;                        // this CTA's entries
  int begin;                              // where its first vector begins: `first`, or before it in the first CTA
  int tile_len, tiles;
  u64 mask;                               // of an index in a key

  __device__ __forceinline__ Sampler(const SampleParams& p_, SampleShared& s_)
      : p(p_), s(s_), cl(cg::this_cluster()), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        C((int)cl.num_blocks()), rank((int)cl.block_rank()) {
    mask = (1ull << p.idx_bits) - 1;
  }

  __device__ __forceinline__ u64 key_of(float x, int v) const { return ((u64)descending<DT>(x) << p.idx_bits) | (u64)v; }
  __device__ __forceinline__ float value_of(u64 key) const { return of_descending<DT>((uint32_t)(key >> p.idx_bits)); }

  // The vector that begins at entry v, as it is in memory; entries that are not this
  // CTA's are -inf.
  __device__ __forceinline__ uint4 load(int v) const {
    if (v >= first && v + W <= last) return __ldg(reinterpret_cast<const uint4*>(row + v));
    uint32_t w[4];
    const uint32_t none = sizeof(DT) == 2 ? 0xff80u : 0xff800000u;
    const auto* bits = reinterpret_cast<const typename std::conditional<sizeof(DT) == 2, uint16_t, uint32_t>::type*>(row);
    auto one = [&](int i) { return i >= first && i < last ? (uint32_t)bits[i] : none; };
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = sizeof(DT) == 2 ? one(v + 2 * i) | one(v + 2 * i + 1) << 16 : one(v + i);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ static float entry(const uint4& q, int e) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if (sizeof(DT) == 4) return __uint_as_float(w[e & 3]);
    return __uint_as_float(e & 1 ? w[(e >> 1) & 3] & 0xffff0000u : w[(e >> 1) & 3] << 16);
  }
  // f(x, index, place in two vectors) of the CTA's entries, done(tile) after each tile.
  template <class F, class Done>
  __device__ __forceinline__ void each_entry(F f, Done done) const {
    for (int t = warp; t < tiles; t += SA_WARPS) {
      for (int i0 = 0; i0 < p.tile_vectors; i0 += BATCH) {
        uint4 q[BATCH];
        const int v = begin + t * tile_len + (i0 * 32 + lane) * W;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (i0 + i < p.tile_vectors) q[i] = load(v + i * 32 * W);
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (i0 + i < p.tile_vectors)
#pragma unroll
            for (int e = 0; e < W; ++e) f(entry(q[i], e), v + i * 32 * W + e, (i & 1) * W + e);
      }
      done(t);
    }
  }
  template <class F>
  __device__ __forceinline__ void each_entry(F f) const { each_entry(f, [](int) {}); }

  __device__ __forceinline__ static u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ u64 warp_upto(u64 v) const {    // sum of the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  }
  // Sums of the threads before this one and of all (of one CTA).
  __device__ __forceinline__ u64 block_before(u64 v, u64& all, int slot = 0) {
    const u64 upto = warp_upto(v);
    __syncthreads();
    if (lane == 31) s.scan[slot][warp] = upto;
    __syncthreads();
    u64 ahead = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < SA_WARPS; ++w) {
      const u64 x = s.scan[slot][w];
      if (w < warp) ahead += x;
      all += x;
    }
    return ahead + upto - v;
  }

  __device__ __forceinline__ void clear_bins() {
    for (int i = tid; i < SA_BINS / 2; i += SA_THREADS) s.hist[i] = 0;
    __syncthreads();
  }
  // Counts of the thread's bins tid * 4 .. + 3 over the cluster.
  __device__ __forceinline__ uint4 counts() const {
    uint4 c = make_uint4(0, 0, 0, 0);
    for (int r = 0; r < C; ++r) {
      const uint4 x = reinterpret_cast<const uint4*>(cl.map_shared_rank(s.hist, r))[tid];
      c.x += x.x; c.y += x.y; c.z += x.z; c.w += x.w;
    }
    return c;
  }

  // The smallest key of [lo, hi] whose running sum, from `base` on, passes `goal`, over
  // the row, adding weight(x) of its entries.  False: no key does.
  template <class Weight>
  __device__ __forceinline__ bool search(u64 lo, u64 hi, u64 base, u64 goal, Weight weight, u64& found) {
    for (;;) {
      const int bits = 64 - __clzll((long long)(hi - lo));
      const int shift = bits > SA_STEP_BITS ? bits - SA_STEP_BITS : 0;
      cl.sync();                                             // the bins have been read
      clear_bins();
      each_entry([&](float x, int v, int) {
        const u64 k = key_of(x, v);
        if (k >= lo && k <= hi) {
          const u64 w = weight(x);
          if (w) atomicAdd(&s.hist[(k - lo) >> shift], w);
        }
      });
      cl.sync();
      constexpr int PER = (1 << SA_STEP_BITS) / SA_THREADS;
      u64 h[PER] = {}, mine = 0, all;
      for (int r = 0; r < C; ++r) {
        const u64* o = cl.map_shared_rank(s.hist, r) + tid * PER;
#pragma unroll
        for (int j = 0; j < PER; ++j) h[j] += o[j];
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) mine += h[j];
      u64 at = base + block_before(mine, all);
      if (base + all <= goal) return false;
      if (at <= goal && goal < at + mine) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          if (at <= goal && goal < at + h[j]) {
            s.bin[0] = tid * PER + j;
            s.before = at;
          }
          at += h[j];
        }
      }
      __syncthreads();
      lo += (u64)s.bin[0] << shift;
      base = s.before;
      const u64 end = lo + ((1ull << shift) - 1);
      hi = end < hi ? end : hi;
      if (shift == 0) {
        found = lo;
        return true;
      }
    }
  }

  __device__ __forceinline__ void refuse(size_t at, uint32_t bit) {
    if (tid == 0 && rank == 0) {
      if (bit) set_status(p.status, bit);
      p.tokens[at] = -1;
      if (p.logprob) p.logprob[at] = quiet_nan();
      if (p.kept) p.kept[at] = 0;
    }
  }

  // The list of all CTAs, n entries, sorted.
  __device__ __forceinline__ void sort_list(int n) {
    int size = 32;
    while (size < n) size *= 2;
    int at = 0;
    for (int r = 0; r < C; ++r) {
      const SampleShared* o = cl.map_shared_rank(&s, r);
      const int m = o->listed;
      for (int i = tid; i < m; i += SA_THREADS) s.sorted[at + i] = o->key[i];
      at += m;
    }
    for (int i = n + tid; i < size; i += SA_THREADS) s.sorted[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int i = tid; i < size / 2; i += SA_THREADS) {
          const int a = 2 * i - (i & (j - 1)), b = a + j;
          const u64 x = s.sorted[a], y = s.sorted[b];
          if ((x > y) == ((a & k) == 0)) {
            s.sorted[a] = y;
            s.sorted[b] = x;
          }
        }
        __syncthreads();
      }
  }

  __device__ __forceinline__ void run() {
    const size_t at = blockIdx.x / C;
    const int b = (int)(at / p.n), j = (int)(at - (size_t)b * p.n);
    const float u = __ldg(p.u + at), T = p.temperature ? __ldg(p.temperature + b) : 1.f;
    const float top_p = p.top_p ? __ldg(p.top_p + b) : 1.f, min_p = p.min_p ? __ldg(p.min_p + b) : 0.f;
    const int top_k = p.top_k ? __ldg(p.top_k + b) : 0;
    if (u == -1.f) return refuse(at, 0);
    if (!(u >= 0.f && u < 1.f && top_p >= 0.f && top_p <= 1.f && min_p >= 0.f && min_p <= 1.f))
      return refuse(at, SPEC_DEV_BAD_FILTER);
    if (!temp_ok(T)) return refuse(at, SPEC_DEV_BAD_TEMP);
    const bool by_k = top_k > 0 && top_k < p.V, by_p = top_p < 1.f;

    // slices begin where vectors do (no slice is empty: the launch sees to that)
    row = static_cast<const DT*>(p.logits) + b * p.b_stride + j * p.row_stride;
    const int skew = (int)(((uintptr_t)row & 15) / sizeof(DT));
    first = rank > 0 ? rank * p.slice - skew : 0;
    last = rank + 1 < C ? (rank + 1) * p.slice - skew : p.V;
    begin = rank * p.slice - skew;
    tile_len = 32 * W * p.tile_vectors;
    tiles = (last - begin + tile_len - 1) / tile_len;

    static_assert(SA_TABLE / 2 == SA_THREADS, "16 bytes of the table a thread");
    const float4 powers = __ldg(reinterpret_cast<const float4*>(g_powers.at) + tid);
    if (tid == 0) {
      s.top = 0xffffffffu;
      s.low = 0;
      s.bad = 0;
      s.listed = 0;
    }

    // ---- 1: the largest logit, and the largest of each group
    float group[SA_GROUPS];
#pragma unroll
    for (int g = 0; g < SA_GROUPS; ++g) group[g] = -INFINITY;
    bool bad = false;
    each_entry([&](float x, int, int e) {
      bad |= !(x <= -SA_LOWEST);
      group[e & 7] = fmaxf(group[e & 7], x);
    });
    float m = group[0], low = INFINITY;
#pragma unroll
    for (int g = 0; g < SA_GROUPS; ++g) {
      m = fmaxf(m, group[g]);
      if (group[g] > -INFINITY) low = fminf(low, group[g]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    __syncthreads();
    if (lane == 0 && m > -INFINITY) {
      atomicMin(&s.top, descending<DT>(m));
      atomicMax(&s.low, descending<DT>(low));
    }
    if (bad) s.bad = 1;
    reinterpret_cast<float4*>(s.tab)[tid] = powers;
    clear_bins();
    cl.sync();
    uint32_t top = 0xffffffffu, far = 0, any = 0;
    for (int r = 0; r < C; ++r) {
      const SampleShared* o = cl.map_shared_rank(&s, r);
      top = min(top, o->top);
      far = max(far, o->low);
      any |= o->bad;
    }
    if (any || top == 0xffffffffu) {
      cl.sync();
      return refuse(at, SPEC_DEV_BAD_LOGIT);
    }
    m = of_descending<DT>(top);
    const Weigh weigh(m, T, p.frac, s.tab);

    // the smallest logit that min-p keeps
    float least = SA_LOWEST;
    if (min_p > 0.f) {
      const df edge = dd_add_f(dd_mul_f(weigh.log(df{min_p, 0.f}), T), m);
      if (edge.hi > least) least = edge.lo > 0.f ? nextafterf(edge.hi, INFINITY) : edge.hi;
    }
    if (sizeof(DT) == 2) least = __bfloat162float(__float2bfloat16_ru(least));
    const u64 floor_key = key_of(least, 0) | mask;
    const u64 every = key_of(SA_LOWEST, 0) | mask;
    auto mass_goal = [&](u64 z) {                            // what a running sum has to pass for top-p to be full
      const u64 pf = fraction64(top_p), g = __umul64hi(pf, z) + (pf * z != 0);
      return g > 0 ? g - 1 : 0;
    };

    // ---- 2: entries above `sure` are kept (if min-p keeps them), from there to `low_x` listed
    float sure = INFINITY, low_x = SA_LOWEST, bin_scale;
    u64 all_mass = 0;
    bool fits = !by_k || top_k <= SA_LIST;
    auto bin_of = [&](float x) { return min(__float2int_rz(rn_mul(rn_sub(m, x), bin_scale)), SA_BINS - 1); };
    const bool listing = by_k || by_p;
    if (listing && fits && p.V > SA_LIST) {
      uint32_t* bins = reinterpret_cast<uint32_t*>(s.hist);
      float range = m - of_descending<DT>(far);
      if (!by_k) range = fminf(-weigh.least / weigh.f, 2.5f * range);   // down to the smallest weight, or well below the maxima
      bin_scale = (float)SA_BINS / fmaxf(range, 1e-30f);
      u64 sum = 0;
      if (!by_k) {
        each_entry([&](float x, int, int) {
          const u64 w = weigh(x);
          sum += w;
          if (w) atomicAdd(&bins[bin_of(x)], 1u);
        });
        block_before(sum, all_mass);
        if (tid == 0) s.sum[0] = all_mass;
      } else if (top_k <= C * (SA_THREADS / 4)) {            // enough threads: their maxima
        float g = group[0];
#pragma unroll
        for (int i = 1; i < SA_GROUPS; ++i) g = fmaxf(g, group[i]);
        if (g > -INFINITY) atomicAdd(&bins[bin_of(g)], 1u);
      } else {
#pragma unroll
        for (int i = 0; i < SA_GROUPS; ++i)
          if (group[i] > -INFINITY) atomicAdd(&bins[bin_of(group[i])], 1u);
      }
      if (tid < 2) s.bin[tid] = SA_BINS;
      cl.sync();
      const uint4 c = counts();
      const uint32_t n[4] = {c.x, c.y, c.z, c.w};
      const float step = 1.f / bin_scale;
      if (by_k) {
        u64 all, at = block_before((u64)c.x + c.y + c.z + c.w, all);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (at < (u64)top_k && (u64)top_k <= at + n[i]) s.bin[1] = 4 * tid + i;
          at += n[i];
        }
        __syncthreads();
      } else {
        all_mass = 0;
        for (int r = 0; r < C; ++r) all_mass += *cl.map_shared_rank(&s.sum[0], r);
        const u64 goal = mass_goal(all_mass);
        // a bin's mass lies between its count times the weights of its edges, moved outwards
        // by more than the edges' rounding
        u64 most[4], fewest[4], most_4 = 0, fewest_4 = 0, most_all, fewest_all;
        u64 edge = weigh.of(df{-(float)(4 * tid) * step, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          most[i] = n[i] * (edge + (edge >> 14));
          edge = 4 * tid + i + 1 < SA_BINS ? weigh.of(df{-(float)(4 * tid + i + 1) * step, 0.f}) : 0;
          fewest[i] = n[i] * (edge - (edge >> 14));
          most_4 += most[i];
          fewest_4 += fewest[i];
        }
        u64 above = block_before(most_4, most_all, 0), below = block_before(fewest_4, fewest_all, 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // the running mass after the bin, from the front or from the end
          above += most[i];
          below += fewest[i];
          const u64 rest = fewest_all - below, rest_most = most_all - above;
          if (above > goal && all_mass - rest > goal) atomicMin(&s.bin[0], 4 * tid + i);
          if (below > goal || (all_mass > rest_most && all_mass - rest_most > goal)) atomicMin(&s.bin[1], 4 * tid + i);
        }
        __syncthreads();
        // above every entry of the first bin in which the mass can run full
        const int first_bin = s.bin[0];
        for (float o = 0x1p-10f; first_bin > 0 && o < 0x1p12f && sure == INFINITY; o *= 2.f) {
          const float x = m - ((float)first_bin - o) * step;
          if (bin_of(x) < first_bin) sure = x;
        }
      }
      const int last_bin = s.bin[1];
      // below every entry of the last one; with fewer groups than k, below all
      for (float o = 0x1p-10f; last_bin < SA_BINS - 1 && o < 0x1p12f && low_x == SA_LOWEST; o *= 2.f) {
        const float x = m - ((float)(last_bin + 1) + o) * step;
        if (bin_of(x) > last_bin && x > SA_LOWEST) low_x = x;
      }
    }

    // ---- 3: sums of the tiles, list
    u64 limit = floor_key, mine = 0, count = 0, sum = 0, above_sum = 0;
    auto close_tile = [&](int t) {
      const u64 z = warp_sum(sum);
      if (lane == 0) s.tile[t] = z;
      above_sum += sum;
      sum = 0;
    };
    if (!listing) {
      each_entry(
          [&](float x, int, int) {
            if (x >= least) {
              sum += weigh(x);
              ++count;
            }
          },
          close_tile);
    } else if (fits) {
      u64 floor_sum = 0;                                     // what min-p takes away above `sure`
      each_entry(
          [&](float x, int v, int) {
            if (x > sure) {
              const u64 w = weigh(x);
              const bool in = x >= least;
              sum += in ? w : 0;
              floor_sum += in ? 0 : w;
              count += in;
            } else if (x >= low_x) {
              const int i = atomicAdd(&s.listed, 1);
              if (i < SA_LIST) s.key[i] = key_of(x, v);
            }
          },
          close_tile);
      u64 base;
      block_before(above_sum + floor_sum, base);
      if (tid == 0) s.sum[1] = base;
      cl.sync();
      int n = 0;
      base = 0;
      for (int r = 0; r < C; ++r) {
        const SampleShared* o = cl.map_shared_rank(&s, r);
        n += o->listed;
        base += o->sum[1];
      }
      fits = n <= SA_LIST;
      if (fits) {
        // ---- 4: the last kept entry of the list
        sort_list(n);
        constexpr int PER = SA_LIST / SA_THREADS;
        u64 w[PER], own = 0, all;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int k = tid * PER + i;
          w[i] = k < n && !(by_k && k >= top_k) ? weigh(value_of(s.sorted[k])) : 0;
          own += w[i];
        }
        int keep = by_k ? min(top_k, n) : n;
        if (by_p) {
          u64 ahead = base + block_before(own, all);
          const u64 goal = mass_goal(by_k || p.V <= SA_LIST ? all : all_mass);
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if (ahead <= goal && goal < ahead + w[i]) s.at = tid * PER + i;
            ahead += w[i];
          }
          __syncthreads();
          keep = min(keep, s.at + 1);
        }
        limit = s.sorted[keep - 1];
        limit = floor_key < limit ? floor_key : limit;
        for (int i = tid; i < s.listed; i += SA_THREADS) {
          const u64 k = s.key[i];
          if (k <= limit) {
            atomicAdd(&s.tile[((int)(k & mask) - begin) / tile_len], weigh(value_of(k)));
            ++count;
          }
        }
      }
    }
    if (listing && !fits) {
      // ---- 2 to 4 by searches over the row
      limit = every;
      const u64 most = (u64)top << p.idx_bits;
      u64 k;
      if (by_k && search(most, every, 0, (u64)(top_k - 1), [](float) { return 1ull; }, k)) limit = k;
      if (by_p) {
        u64 all, z = 0;
        sum = 0;
        each_entry([&](float x, int v, int) { sum += key_of(x, v) <= limit ? weigh(x) : 0; });
        block_before(sum, all);
        cl.sync();                                           // the sums before it have been read
        if (tid == 0) s.sum[0] = all;
        cl.sync();
        for (int r = 0; r < C; ++r) z += *cl.map_shared_rank(&s.sum[0], r);
        if (search(most, limit, 0, mass_goal(z), [&](float x) { return weigh(x); }, k)) limit = k;
      }
      limit = floor_key < limit ? floor_key : limit;
      sum = count = 0;
      each_entry(
          [&](float x, int v, int) {
            if (key_of(x, v) <= limit) {
              sum += weigh(x);
              ++count;
            }
          },
          close_tile);
    }

    // ---- 5: the CTA, the tile, the token
    u64 entries;
    block_before(count, entries);                            // and the tiles' sums are written
    constexpr int PER_TILE = SA_TILES / SA_THREADS;
    static_assert(PER_TILE == 1, "a thread a tile");
    const u64 in_tile = tid < tiles ? s.tile[tid] : 0;
    const u64 before_tile = block_before(in_tile, mine);
    if (listing) cl.sync();                                  // the sums before these have been read
    if (tid == 0) {
      s.sum[0] = mine;
      s.sum[1] = entries;
    }
    cl.sync();
    u64 z = 0, ahead = 0, total = 0;
    for (int r = 0; r < C; ++r) {
      const SampleShared* o = cl.map_shared_rank(&s, r);
      const u64 x = o->sum[0];
      if (r < rank) ahead += x;
      z += x;
      total += o->sum[1];
    }
    cl.sync();                                               // nothing of another CTA is read after this
    const u64 goal = __umul64hi(fraction64(u), z);
    if (goal < ahead || goal >= ahead + mine) return;
    if (tid == 0) s.at = 0;
    __syncthreads();
    if (in_tile && ahead + before_tile <= goal && goal < ahead + before_tile + in_tile) {
      s.at = tid;
      s.before = ahead + before_tile;
    }
    __syncthreads();
    if (warp != 0) return;
    u64 done = s.before;
    for (int i = 0; i < p.tile_vectors; ++i) {
      const int v = begin + s.at * tile_len + (i * 32 + lane) * W;
      const uint4 q = load(v);
      u64 sum = 0, w[W];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float x = entry(q, e);
        w[e] = key_of(x, v + e) <= limit ? weigh(x) : 0;
        sum += w[e];
      }
      const u64 upto = done + warp_upto(sum);
      const u64 before = upto - sum;
      if (before <= goal && goal < upto) {
        u64 f = before;
        int token = -1;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if (f <= goal && goal < f + w[e]) {
            token = v + e;
            x = entry(q, e);
          }
          f += w[e];
        }
        p.tokens[at] = token;
        if (p.logprob) {
          const float scale = ldexpf(1.f, -p.frac), zh = __ull2float_rn(z);
          const df l = weigh.log(df{zh * scale, __ll2float_rn((long long)(z - __float2ull_rn(zh))) * scale});
          const df a = weigh.argument(x), d = two_sum_df(a.hi, -l.hi);
          p.logprob[at] = d.hi + (d.lo + (a.lo - l.lo));
        }
        if (p.kept) p.kept[at] = (int)total;
      }
      done = __shfl_sync(0xffffffffu, upto, 31);
    }
  }
};

template <class DT>
__global__ void __launch_bounds__(SA_THREADS, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Sampler<DT>(p, *reinterpret_cast<SampleShared*>(smem)).run();
}

namespace {
template <class DT>
cudaError_t launch(const cudaLaunchConfig_t& cfg, const SampleParams& p) {
  // once a device: the attribute stays with the function
  static std::atomic<uint64_t> sized{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((sized.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SampleShared));
    if (e != cudaSuccess) return e;
    if (dev < 64) sized.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return cudaLaunchKernelEx(&cfg, sample_kernel<DT>, p);
}
}  // namespace

cudaError_t launch_sample(const spec_sample_args& a, int sms, cudaStream_t st) {
  SampleParams p{a.n,     a.V,     a.logits, a.b_stride, a.row_stride, a.u, a.temperature, a.top_k,
                 a.top_p, a.min_p, a.tokens, a.logprob,  a.kept,       a.dev_status};
  int bits = 1;
  while ((1 << bits) < a.V) ++bits;
  p.idx_bits = bits;
  p.frac = bits > 21 ? 62 - bits : 41;
  const long long rows = (long long)a.B * a.n;
  const int W = a.dtype == SPEC_BF16 ? 8 : 4;
  int C = 1;
  while (C < 8 && 2 * C * rows <= 4LL * sms && a.V / (2 * C) >= 4096) C *= 2;
  p.slice = ((a.V + C - 1) / C + 32 * W - 1) / (32 * W) * (32 * W);
  while ((long long)(C - 1) * p.slice >= a.V) --C;           // no empty slice
  p.tile_vectors = 1;
  while ((p.slice + 32 * W * p.tile_vectors) / (32 * W * p.tile_vectors) > SA_TILES ||
         (p.tile_vectors < 4 && p.slice > 32 * W * p.tile_vectors * 4 * SA_WARPS))
    p.tile_vectors *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(SA_THREADS);
  cfg.dynamicSmemBytes = sizeof(SampleShared);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return a.dtype == SPEC_BF16 ? launch<bf16>(cfg, p) : launch<float>(cfg, p);
}

}  // namespace spec
