// Sampling with temperature, top-k, top-p and min-p from given uniform numbers.
//
//   w_v = exp((x_v - max x) / T); kept: the first n entries in descending order;
//   token: the smallest v (vocabulary order) with F(v) > u F(V), F over kept w.
//
// Weights are whole numbers of 2^-frac of the largest (double-float exponentials,
// rounded once), so sums are exact in any order and every border -- the k-th
// entry, the mass of top-p, the drawn token -- is decided on exact sums.
//
// A cluster of CTAs takes a row, each CTA a slice of the vocabulary.  Every border
// is found by the same search: the smallest key whose running sum passes a target,
// by a histogram of 2048 bins over the keys' range, then over the bin that holds
// the border, until a bin is one key.  The keys are (descending value, index) for
// the filters, and the index for the draw.  The searches run over a list of the
// entries that can be kept, gathered by a lower bound from the maxima of groups of
// entries; where the list does not fit, over the row itself.
#include <cooperative_groups.h>

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
};

constexpr int SA_THREADS = 512, SA_BIN_BITS = 11, SA_BINS = 1 << SA_BIN_BITS, SA_LIST = 1536;
constexpr int SA_GROUPS = 8;              // groups of entries a thread, each with its maximum

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

// Weights of a row.  T is taken as f times a number whose reciprocal is ordinary.
struct Weigh {
  float m, f, unit;
  u64 one;
  df inv;
  const df* tab;
  __device__ __forceinline__ Weigh(float m_, float T, int frac, const df* tab_) : m(m_), tab(tab_) {
    const int e = max(-100, min(100, -ilogbf(T)));
    f = ldexpf(1.f, e);
    inv = dd_recip(rn_mul(T, f));
    unit = ldexpf(1.f, frac);
    one = 1ull << frac;
  }
  // (x - m) / T
  __device__ __forceinline__ df argument(float x) const {
    const df d = two_sum_df(x, -m);
    return dd_mul(df{rn_mul(d.hi, f), rn_mul(d.lo, f)}, inv);
  }
  __device__ __forceinline__ u64 operator()(float x) const {
    if (x == m) return one;
    if (!(rn_mul(rn_mul(rn_sub(x, m), f), inv.hi) > -44.f)) return 0;      // below 2^-63
    const df e = dd_exp(argument(x), tab);
    return (u64)(__float2ll_rn(rn_mul(e.hi, unit)) + __float2ll_rn(rn_mul(e.lo, unit)));
  }
};

// A number of [0, 1) in units of 2^-64 (below 2^-40 rounded down).
__device__ __forceinline__ u64 fraction64(float x) { return __float2ull_rz(x * 18446744073709551616.f); }

struct SampleShared {
  u64 hist[SA_BINS];
  u64 key[SA_LIST], weight[SA_LIST];
  u64 scan[SA_THREADS / 32];
  u64 before;                             // of the bin that a search goes on in
  u64 sum[2];                             // of one CTA, read by the cluster
  df tab[DD_EXP_TAB];
  int bin, listed;
  uint32_t top, low, bad;                 // of one CTA
  float wmax[SA_THREADS / 32];
};

template <class DT>
struct Sampler {
  const SampleParams& p;
  SampleShared& s;
  cg::cluster_group cl;
  const int tid, lane, warp;
  const DT* row;
  int first, last;                        // this CTA's entries
  int begin;                              // where its first vector begins: `first`, or before it in the first CTA
  u64 mask;                               // of an index in a key

  __device__ __forceinline__ Sampler(const SampleParams& p_, SampleShared& s_)
      : p(p_), s(s_), cl(cg::this_cluster()), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {
    mask = (1ull << p.idx_bits) - 1;
  }

  // f(x, index, place in the vector) of the CTA's entries, 16 bytes at a time where they are whole.
  template <class F>
  __device__ __forceinline__ void each_entry(F f) const {
    constexpr int W = 16 / sizeof(DT);
    for (int v = begin + tid * W; v < last; v += SA_THREADS * W) {
      float x[W];
      if (v >= first && v + W <= last) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + v));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < W; ++e)
          x[e] = sizeof(DT) == 4 ? __uint_as_float(w[e & 3])
                                 : __uint_as_float(e & 1 ? w[(e >> 1) & 3] & 0xffff0000u : w[(e >> 1) & 3] << 16);
#pragma unroll
        for (int e = 0; e < W; ++e) f(x[e], v + e, e);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (v + e >= first && v + e < last) f((float)row[v + e], v + e, e);
      }
    }
  }

  // f(key, weigh) of the entries whose key is at most `limit`: of the list, or of the row.
  template <class F>
  __device__ __forceinline__ void each_kept(bool list, u64 limit, const Weigh& weigh, F f) const {
    if (list) {
      for (int i = tid; i < s.listed; i += SA_THREADS) {
        const u64 k = s.key[i];
        if (k <= limit) f(k, [&] { return s.weight[i]; });
      }
    } else {
      each_entry([&](float x, int v, int) {
        const u64 k = ((u64)descending<DT>(x) << p.idx_bits) | (u64)v;
        if (k <= limit && x > -INFINITY) f(k, [&] { return weigh(x); });
      });
    }
  }

  // Sum over the cluster of one number a thread.
  __device__ __forceinline__ u64 total(u64 v, int slot) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) s.scan[warp] = v;
    __syncthreads();
    if (tid == 0) {
      u64 t = 0;
      for (int w = 0; w < SA_THREADS / 32; ++w) t += s.scan[w];
      s.sum[slot] = t;
    }
    cl.sync();
    u64 t = 0;
    for (unsigned r = 0; r < cl.num_blocks(); ++r) t += *cl.map_shared_rank(&s.sum[slot], r);
    cl.sync();
    return t;
  }

  // The smallest key of [lo, hi] whose running sum passes `target(sum of all)`,
  // from add(lo, hi, shift), which adds its entries to the histogram.  levels: stop
  // after so many, with the last key of the bin.  False: no key does.
  template <class Add, class Target>
  __device__ __forceinline__ bool search(u64 lo, u64 hi, int levels, Add add, Target target, u64& found) {
    u64 base = 0, goal = 0;
    for (int level = 0;; ++level) {
      const int bits = 64 - __clzll((long long)(hi - lo));
      const int shift = bits > SA_BIN_BITS ? bits - SA_BIN_BITS : 0;
      for (int i = tid; i < SA_BINS; i += SA_THREADS) s.hist[i] = 0;
      __syncthreads();
      add(lo, hi, shift);
      cl.sync();
      constexpr int PER = SA_BINS / SA_THREADS;
      u64 h[PER], mine = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        h[j] = 0;
        for (unsigned r = 0; r < cl.num_blocks(); ++r) h[j] += cl.map_shared_rank(s.hist, r)[tid * PER + j];
        mine += h[j];
      }
      u64 upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
      }
      if (lane == 31) s.scan[warp] = upto;
      __syncthreads();
      u64 all = 0, ahead = 0;
      for (int w = 0; w < SA_THREADS / 32; ++w) {
        if (w < warp) ahead += s.scan[w];
        all += s.scan[w];
      }
      if (level == 0) {
        goal = target(all);
        if (all <= goal) {
          cl.sync();
          return false;
        }
      }
      u64 at = base + ahead + upto - mine;
      if (at <= goal && goal < at + mine) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          if (at <= goal && goal < at + h[j]) {
            s.bin = tid * PER + j;
            s.before = at;
          }
          at += h[j];
        }
      }
      __syncthreads();
      const u64 bin = (u64)s.bin;
      base = s.before;
      cl.sync();
      lo += bin << shift;
      const u64 end = lo + ((1ull << shift) - 1);
      hi = end < hi ? end : hi;
      if (shift == 0 || level + 1 == levels) {
        found = hi;
        return true;
      }
    }
  }

  __device__ __forceinline__ void refuse(size_t at, uint32_t bit) {
    if (tid == 0 && cl.block_rank() == 0) {
      if (bit) set_status(p.status, bit);
      p.tokens[at] = -1;
      if (p.logprob) p.logprob[at] = quiet_nan();
      if (p.kept) p.kept[at] = 0;
    }
  }

  __device__ __forceinline__ void run() {
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
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

    row = static_cast<const DT*>(p.logits) + b * p.b_stride + j * p.row_stride;
    const int W = 16 / sizeof(DT);
    const int slice = ((p.V + C - 1) / C + W - 1) / W * W;
    first = min(rank * slice, p.V);
    last = min(first + slice, p.V);
    // slices begin where vectors do (no slice is empty: the launch sees to that)
    const int skew = (int)(((uintptr_t)row & 15) / sizeof(DT));
    if (rank > 0) first -= skew;
    if (rank + 1 < C) last -= skew;
    begin = rank > 0 ? first : -skew;

    // ---- the largest logit, and the largest of each group
    if (tid < DD_EXP_TAB) dd_exp_table_entry(s.tab, tid);
    float group[SA_GROUPS];
#pragma unroll
    for (int g = 0; g < SA_GROUPS; ++g) group[g] = -INFINITY;
    bool bad = false;
    {
      int turn = 0;
      each_entry([&](float x, int, int e) {
        bad |= !(x <= 3.402823466e38f);
        if (sizeof(DT) == 2) {
          group[e & 7] = fmaxf(group[e & 7], x);
        } else if (turn & 1) {
          group[4 + (e & 3)] = fmaxf(group[4 + (e & 3)], x);
        } else {
          group[e & 3] = fmaxf(group[e & 3], x);
        }
        if ((e & 3) == 3) ++turn;
      });
    }
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
    if (tid == 0) {
      s.top = 0xffffffffu;
      s.low = 0;
      s.bad = 0;
      s.listed = 0;
    }
    __syncthreads();
    if (lane == 0 && m > -INFINITY) {
      atomicMin(&s.top, descending<DT>(m));
      atomicMax(&s.low, descending<DT>(low));
    }
    if (bad) s.bad = 1;
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

    // ---- the smallest logit that min-p keeps
    float least = -3.402823466e38f;
    if (min_p > 0.f) {
      const double edge = (double)m + (double)T * log((double)min_p);
      if (edge > (double)least) {
        least = (float)edge;
        if ((double)least < edge) least = nextafterf(least, INFINITY);
      }
    }
    if (sizeof(DT) == 2) least = __bfloat162float(__float2bfloat16_ru(least));
    const u64 floor_key = ((u64)descending<DT>(least) << p.idx_bits) | mask;
    const u64 top_key = (u64)top << p.idx_bits;
    const u64 every = ((u64)descending<DT>(-3.402823466e38f) << p.idx_bits) | mask;

    // ---- the mass of all entries, where top-p is of that
    u64 all_mass = 0;
    if (by_p && !by_k) {
      u64 sum = 0;
      each_entry([&](float x, int, int) { sum += weigh(x); });
      all_mass = total(sum, 0);
    }
    auto mass_goal = [&](u64 z) {                            // what a running sum has to pass for top-p to be full
      const u64 pf = fraction64(top_p), g = __umul64hi(pf, z) + (pf * z != 0);
      return g > 0 ? g - 1 : 0;
    };

    // ---- a list of what can be kept
    u64 bound = every;
    if (by_k || by_p) {
      u64 edge;
      const bool known = search(
          top, far, 1,
          [&](u64 lo, u64 hi, int shift) {
#pragma unroll
            for (int g = 0; g < SA_GROUPS; ++g) {
              const u64 d = descending<DT>(group[g]);
              if (group[g] > -INFINITY && d >= lo && d <= hi)
                atomicAdd(&s.hist[(d - lo) >> shift], by_k ? 1ull : weigh(group[g]));
            }
          },
          [&](u64) { return by_k ? (u64)(top_k - 1) : mass_goal(all_mass); }, edge);
      if (known) bound = (edge << p.idx_bits) | mask;
    }
    if (!(by_k && by_p) && floor_key < bound) bound = floor_key;
    bool list = bound < every;
    if (list) {
      each_entry([&](float x, int v, int) {
        const u64 k = ((u64)descending<DT>(x) << p.idx_bits) | (u64)v;
        if (k <= bound && x > -INFINITY) {
          const int i = atomicAdd(&s.listed, 1);
          if (i < SA_LIST) {
            s.key[i] = k;
            s.weight[i] = weigh(x);
          }
        }
      });
      cl.sync();
      for (int r = 0; r < C; ++r) list &= *cl.map_shared_rank(&s.listed, r) <= SA_LIST;
      cl.sync();
    }

    // ---- the last kept entry
    u64 limit = every;
    if (by_k) {
      u64 k;
      if (search(
              top_key, bound, 99,
              [&](u64 lo, u64 hi, int shift) {
                each_kept(list, hi, weigh, [&](u64 key, auto) {
                  if (key >= lo) atomicAdd(&s.hist[(key - lo) >> shift], 1ull);
                });
              },
              [&](u64) { return (u64)(top_k - 1); }, k))
        limit = k;
    }
    if (by_p) {
      u64 z = all_mass, k;
      if (by_k) {
        u64 sum = 0;
        each_kept(list, limit, weigh, [&](u64, auto w) { sum += w(); });
        z = total(sum, 0);
      }
      const u64 within = limit < bound ? limit : bound;
      if (search(
              top_key, within, 99,
              [&](u64 lo, u64 hi, int shift) {
                each_kept(list, hi, weigh, [&](u64 key, auto w) {
                  if (key >= lo) atomicAdd(&s.hist[(key - lo) >> shift], w());
                });
              },
              [&](u64) { return mass_goal(z); }, k))
        limit = k;
    }
    limit = floor_key < limit ? floor_key : limit;

    // ---- how many, and the draw
    u64 count = 0;
    each_kept(list, limit, weigh, [&](u64, auto) { ++count; });
    count = total(count, 1);
    u64 token = 0, z = 0;
    search(
        0, (u64)(p.V - 1), 99,
        [&](u64 lo, u64 hi, int shift) {
          each_kept(list, limit, weigh, [&](u64 key, auto w) {
            const u64 v = key & mask;
            if (v >= lo && v <= hi) atomicAdd(&s.hist[(v - lo) >> shift], w());
          });
        },
        [&](u64 sum) {
          z = sum;
          return __umul64hi(fraction64(u), sum);
        },
        token);
    if (tid == 0 && rank == 0) {
      p.tokens[at] = (int)token;
      if (p.logprob)
        p.logprob[at] = (float)(dd_to_double(weigh.argument((float)row[token])) -
                                (log((double)z) - p.frac * 0.69314718055994530942));
      if (p.kept) p.kept[at] = (int)count;
    }
  }
};

template <class DT>
__global__ void __launch_bounds__(SA_THREADS) sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Sampler<DT>(p, *reinterpret_cast<SampleShared*>(smem)).run();
}

cudaError_t launch_sample(const spec_sample_args& a, int sms, cudaStream_t st) {
  SampleParams p{a.n,     a.V,     a.logits, a.b_stride, a.row_stride, a.u, a.temperature, a.top_k,
                 a.top_p, a.min_p, a.tokens, a.logprob,  a.kept,       a.dev_status};
  int bits = 1;
  while ((1 << bits) < a.V) ++bits;
  p.idx_bits = bits;
  p.frac = bits > 17 ? 62 - bits : 45;
  const long long rows = (long long)a.B * a.n;
  int C = 1;
  while (C < 8 && 2 * C * rows <= 2LL * sms && a.V / (2 * C) >= 4096) C *= 2;
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
  static_assert(sizeof(SampleShared) <= 48 * 1024, "shared memory without an opt-in");
  return a.dtype == SPEC_BF16 ? cudaLaunchKernelEx(&cfg, sample_kernel<bf16>, p)
                              : cudaLaunchKernelEx(&cfg, sample_kernel<float>, p);
}

}  // namespace spec
