// Sampling with temperature, top-k, top-p and min-p from given uniform numbers.
//
//   w_v = exp((x_v - max x) / T); kept: the first n entries in descending order;
//   token: the smallest v (vocabulary order) with F(v) > u F(V), F over kept w.
//
// Weights are whole numbers of 2^-43 of the largest, so sums are exact in any order
// and every border -- the k-th entry, the mass of top-p, the drawn token -- is
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
// A slice that fits stays in shared memory: it is read from memory once (a pass over a
// slice in L2 cost about as much as reading it from memory).  Larger ones are staged
// anew in every pass, the next vectors on their way while some are worked on.
//
// Rows whose list overflows (2048 entries next to a border: wide ties, flat rows of few values) and those
// with top_k from 2048 on find their borders by histograms over the row itself, 1024 bins of keys a pass.
//
// Bound by instructions where every weight is needed (no filter, or top-p alone: some
// 40 slots an entry, of which the weight's double-float argument, table and two numbers
// are 30), by the chain of steps elsewhere: 16 rows of 128256 take 19 us with min-p
// 0.05, 25 with top-k 50, 56 with top-p 0.9, 23 without a filter.  256 rows of
// 128256 bf16 of mixed settings take 117 us (10 us of reading), 128 of 32000 39 us, 64 of
// 151936 fp32 at temperatures alone 41 us, 4 of 1000 13 to 22 us.  By one kind of filter,
// 256 rows of 128256: none 91 us, top-k 50 68, min-p 0.05 52, top-p 0.9 175 (fp32 111, 89, 72, 195);
// by searches over the row 539 with top-k 5000, and 588 with top-p 0.9 of logits around -10, whose lists
// overflow.
#include <cooperative_groups.h>

#include <atomic>

#include "spec_df.cuh"
#include "spec_gemm.cuh"
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
  int idx_bits, less;                     // bits of an index; weights are 2^-less of what they are called
  int slice, tile_vectors;                // entries a CTA, vectors a lane of a tile
  int resident;                           // slices stay in shared memory
};

constexpr int SA_THREADS = 512, SA_WARPS = SA_THREADS / 32, SA_BINS = 2048;
constexpr int SA_STEP_BITS = 10;          // of a key, a pass of a search
constexpr int SA_LIST = 2048;             // entries of a row's list
constexpr int SA_TILES = 256;             // tiles a CTA
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

// Weights of a row: 2^t, t = (x - m) log2(e) / T, in whole units of 2^-43 (times
// 2^-less).  In 1024ths of an octave t is formed in double-float, k is the nearest
// whole number and y = t - k, and 2^(t/1024) = 2^(k/1024) (1 + s + s^2 / 2),
// s = y ln 2 / 1024, whose next term is 2^-37 at most; with the table's two terms that
// leaves a relative error below 2^-34, of either sign (it averages out: 1e-14 of the
// sum of two million random weights).  Entries below 2^-44.1 count as nothing: less than half a unit.
//
// A weight comes as two 32-bit numbers, of units 2^-22 and 2^-43 (signed), that adding
// 3 and 1.5 2^-20 leaves in the low bits of fp32 numbers: the second one is at most 2^20 in
// size, so up to 2047 weights add up in 32 bits without their offsets.  Two weights at a time, by instructions of two numbers.
struct Weights2 {
  uint32_t a[2], b[2];                    // offset by WEIGHT_A and WEIGHT_B
};
constexpr uint32_t WEIGHT_A = 0x40400000u, WEIGHT_B = 0x35c00000u;   // 3 and 1.5 2^-20
__device__ __forceinline__ u64 weight_sum(uint32_t a, uint32_t b) {  // of sums without their offsets
  return ((u64)a << 21) + (u64)(long long)(int32_t)b;
}
__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) { return fma2(b, both(-1.f), a); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) { return fma2(a, b, both(-0.f)); }

struct Weigh {
  float m, low;                           // the largest entry; below `low` nothing counts
  uint32_t one;                           // 2^-less as fp32 bits
  df c, inv;                              // 1024 log2(e) / T, 1 / T
  const float2* tab;
  __device__ __forceinline__ Weigh(float m_, float T, int less, const float2* tab_) : m(m_), tab(tab_) {
    inv = dd_recip(T);
    c = dd_mul(inv, octaves());
    one = 0x3f800000u - ((uint32_t)less << 23);
    // rounded away from m: whatever lies lower is given the weight of `low`, which has to be 0
    low = fmaxf(__fsub_rd(m, fminf(44.1f * 1024.f / c.hi, -SA_LOWEST)), SA_LOWEST);
    // A distance that leaves the exponents' range: `low` is the number next to m (T is below the
    // logits' resolution), or m = -(2^k - 1 unit in the last place) and the number between them, of 0.4
    // to 2 units, gets 2.
    const float most = (float)(126 - less) * 1024.f;
    if ((m - low) * c.hi > most) c = {most / (m - low), 0.f};
  }
  __device__ __forceinline__ static df octaves() { return {1477.31970f, 1.97218615e-05f}; }   // 1024 log2(e)
  // (x - m) / T
  __device__ __forceinline__ df argument(float x) const { return dd_mul(two_sum_df(x, -m), inv); }

  // Weights of entries that lie s + e (<= 0, not far below low - m) from the largest.
  __device__ __forceinline__ Weights2 of(uint64_t s, uint64_t e) const {
    const uint64_t ch = both(c.hi), magic = both(12582912.f);                  // 1.5 2^23
    const uint64_t nt = mul2(s, both(-c.hi));                                  // -t
    const uint64_t te = fma2(e, ch, fma2(s, both(c.lo), fma2(s, ch, nt)));
    const uint64_t k = sub2(magic, nt);                                        // k in the low bits
    const uint64_t y = sub2(te, add2(nt, sub2(k, magic)));
    const uint64_t q = mul2(y, both(6.76901552e-04f));
    const float2 s2 = unpair(fma2(mul2(q, both(0.5f)), q, q)), kf = unpair(k);
    float hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t bits = __float_as_uint(i ? kf.y : kf.x);
      const float2 p = tab[bits & (SA_TABLE - 1)];
      const float scale = __uint_as_float(((bits & ~(uint32_t)(SA_TABLE - 1)) << 13) + one);
      hi[i] = rn_mul(p.x, scale);
      lo[i] = rn_mul(rn_fma(p.x, i ? s2.y : s2.x, p.y), scale);
    }
    const uint64_t h = pair(hi[0], hi[1]), l = pair(lo[0], lo[1]);
    const uint64_t sum = add2(h, l), rest = sub2(l, sub2(sum, h));
    const uint64_t a = add2(sum, both(3.f));
    const uint64_t b = add2(add2(sub2(sum, sub2(a, both(3.f))), rest), both(0x1.8p-20f));
    const float2 af = unpair(a), bf = unpair(b);
    return {{__float_as_uint(af.x), __float_as_uint(af.y)}, {__float_as_uint(bf.x), __float_as_uint(bf.y)}};
  }
  __device__ __forceinline__ Weights2 two(float x0, float x1) const {
    const uint64_t x = pair(fmaxf(x0, low), fmaxf(x1, low)), nm = both(-m);
    const uint64_t s = add2(x, nm), bb = sub2(s, x);
    return of(s, add2(sub2(x, sub2(s, bb)), sub2(nm, bb)));
  }
};
// Of one entry.
__device__ __noinline__ u64 weight_of(const Weigh weigh, float x) {
  const Weights2 w = weigh.two(x, x);
  return x > -INFINITY ? weight_sum(w.a[0] - WEIGHT_A, w.b[0] - WEIGHT_B) : 0;
}
// The natural logarithm of z > 0: the fp32 one and a Newton step.
__device__ __noinline__ df log_of(df z, const float2* tab) {
  const float y = logf(z.hi);
  if (!(fabsf(y) < 87.f)) return {y, 0.f};
  const float t = rn_mul(-y, Weigh::octaves().hi);
  const float te = rn_fma(-y, Weigh::octaves().lo, rn_fma(-y, Weigh::octaves().hi, -t));
  const float k = rn_add(t, 12582912.f);
  const float q = rn_mul(rn_add(rn_sub(t, rn_sub(k, 12582912.f)), te), 6.76901552e-04f);
  const float2 p = tab[__float_as_uint(k) & (SA_TABLE - 1)];
  const float scale = __uint_as_float(((__float_as_uint(k) & ~(uint32_t)(SA_TABLE - 1)) << 13) + 0x3f800000u);
  const float hi = rn_mul(p.x, scale), lo = rn_mul(rn_fma(p.x, rn_fma(rn_mul(q, 0.5f), q, q), p.y), scale);   // 1 / z, nearly
  const df v = two_prod_df(z.hi, hi);
  return {y, rn_add(rn_sub(v.hi, 1.f), rn_fma(z.hi, lo, rn_fma(z.lo, hi, v.lo)))};
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_upto64(u64 v) {          // sum of the lanes up to this one
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
// Sums of the threads before this one and of all (of one CTA); scan[SA_WARPS].
struct Before {
  u64 before, all;
};
__device__ __noinline__ Before block_before(u64 v, u64* scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 upto = warp_upto64(v);
  __syncthreads();
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  const u64 sums = warp_upto64(lane < SA_WARPS ? scan[lane] : 0);
  return {(warp ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0) + upto - v, __shfl_sync(0xffffffffu, sums, 31)};
}

// A number of [0, 1) in units of 2^-64 (below 2^-40 rounded down).
__device__ __forceinline__ u64 fraction64(float x) { return __float2ull_rz(x * 18446744073709551616.f); }

struct SampleShared {
  u64 sorted[SA_LIST];                    // the row's list
  u64 hist[SA_BINS / 2];                  // counts of 32 bits; 64-bit sums of half as many bins in a search
  u64 tile[SA_TILES];                     // kept mass
  alignas(16) float2 tab[SA_TABLE];
  u64 scan[SA_WARPS], ends[2][SA_WARPS];
  u64 before;                             // of the bin or tile that a search goes on in
  u64 sum[3];                             // of one CTA, read by the cluster: all, certainly kept, kept
  int bin[2], listed, at;
  int lists[8];                           // entries of the CTAs' lists before each
  uint32_t top, low, bad, entries;        // of one CTA, read by the cluster
  uint32_t count[SA_WARPS];
  int index[SA_LIST];                     // this CTA's list
};
constexpr int SA_STAGE = 4;               // vectors a lane at a time; two such stages a warp where slices do not stay
constexpr int SA_SLICE = 69 * 1024;       // bytes of a slice that stays: two CTAs an SM
static_assert(offsetof(SampleShared, tab) % 16 == 0 && SA_LIST % 2 == 0 && sizeof(SampleShared) % 16 == 0,
              "16 bytes at a time");
static_assert(2 * (sizeof(SampleShared) + SA_SLICE + 1024) <= 227 * 1024, "two CTAs an SM");

template <class DT>
struct Sampler {
  static constexpr int W = 16 / sizeof(DT);
  const SampleParams& p;
  SampleShared& s;
  uint8_t* const data;                    // the slice, or the warps' stages
  cg::cluster_group cl;
  const int tid, lane, warp, C, rank;
  const DT* row;
  int first, last;                        // this CTA's entries
  int begin;                              // where its first vector begins: `first`, or before it in the first CTA
  int tile_len, tiles;
  u64 mask;                               // of an index in a key

  __device__ __forceinline__ Sampler(const SampleParams& p_, SampleShared& s_)
      : p(p_), s(s_), data(reinterpret_cast<uint8_t*>(&s_ + 1)), cl(cg::this_cluster()), tid(threadIdx.x), lane(threadIdx.x & 31), warp(threadIdx.x >> 5),
        C((int)cl.num_blocks()), rank((int)cl.block_rank()) {
    mask = (1ull << p.idx_bits) - 1;
  }

  __device__ __forceinline__ u64 key_of(float x, int v) const { return ((u64)descending<DT>(x) << p.idx_bits) | (u64)v; }
  __device__ __forceinline__ float value_of(u64 key) const { return of_descending<DT>((uint32_t)(key >> p.idx_bits)); }

  // ---- vectors of 16 bytes, as they are in memory
  // The one that begins at entry v; entries that are not this CTA's are -inf.
  __device__ __forceinline__ uint4 load_part(int v) const { return load_entries(row, v, first, last); }
  __device__ __noinline__ static uint4 load_entries(const DT* row, int v, int first, int last) {
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
  // The larger of two words of a vector, entry by entry; a NaN stays one.
  __device__ __forceinline__ static uint32_t word_max(uint32_t a, uint32_t b) {
    uint32_t r;
    if (sizeof(DT) == 2) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ __forceinline__ static float vector_max(const uint4& q) {
    const uint4 w = make_uint4(word_max(word_max(q.x, q.y), word_max(q.z, q.w)), 0, 0, 0);
    return sizeof(DT) == 2 ? fmaxf(entry(w, 0), entry(w, 1)) : __uint_as_float(w.x);
  }
  __device__ __forceinline__ static uint32_t group_word(const uint4& q, int g) {   // the word of entry g
    const int w = sizeof(DT) == 2 ? g >> 1 : g;
    return w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
  }
  // Entry v, which is CTA r's.
  __device__ __forceinline__ float value_at(int v, int r) const {
    if (!p.resident) return (float)row[v];
    const int own = v - (begin + (r - rank) * p.slice);
    return (float)reinterpret_cast<const DT*>(cl.map_shared_rank(data, r))[own];
  }
  // Requests the vectors [i0, i0 + n) a lane of tile t, to `to`.
  __device__ __forceinline__ void request(uint8_t* to, int t, int i0, int n) const {
    to += lane * 16;
    int v = begin + t * tile_len + (i0 * 32 + lane) * W;
#pragma unroll 1
    for (int i = 0; i < n; ++i, v += 32 * W, to += 512) {
      if (v >= first && v + W <= last) cp_async16(to, row + v, true);
      else *reinterpret_cast<uint4*>(to) = load_part(v);
    }
  }
  // f(vector, its first entry) of the CTA's entries, SA_STAGE vectors a lane at a time;
  // done(tile) after each tile.  Where the slice does not stay, the next vectors are on
  // their way while some are worked on.
  template <class F, class Done>
  __device__ __forceinline__ void each_vector(F f, Done done) const {
    const int most = min(SA_STAGE, p.tile_vectors);
    auto stage = [&](int turn) { return data + ((turn & 1) * SA_WARPS + warp) * (SA_STAGE * 512); };
    if (!p.resident && warp < tiles) {
      request(stage(0), warp, 0, most);
      cp_async_commit();
    }
    int turn = 0;
#pragma unroll 1
    for (int t = warp; t < tiles; t += SA_WARPS) {
#pragma unroll 1
      for (int i0 = 0; i0 < p.tile_vectors; i0 += SA_STAGE, ++turn) {
        const int n = min(SA_STAGE, p.tile_vectors - i0);
        const uint8_t* at = data + (t * p.tile_vectors + i0) * 512;
        if (!p.resident) {
          const bool same = i0 + SA_STAGE < p.tile_vectors;
          const int next = same ? t : t + SA_WARPS, from = same ? i0 + SA_STAGE : 0;
          __syncwarp();                                      // the buffer has been read
          if (next < tiles) request(stage(turn + 1), next, from, min(SA_STAGE, p.tile_vectors - from));
          cp_async_commit();
          asm volatile("cp.async.wait_group 1;\n" ::: "memory");   // each lane reads what it requested
          at = stage(turn);
        }
        at += lane * 16;
        int v = begin + t * tile_len + (i0 * 32 + lane) * W;
        if (n == SA_STAGE) {
          uint4 q[SA_STAGE];
#pragma unroll
          for (int i = 0; i < SA_STAGE; ++i) q[i] = *reinterpret_cast<const uint4*>(at + i * 512);
#pragma unroll
          for (int i = 0; i < SA_STAGE; ++i) f(q[i], v + i * 32 * W, at + i * 512);
        } else {
#pragma unroll 1
          for (int i = 0; i < n; ++i, v += 32 * W, at += 512) f(*reinterpret_cast<const uint4*>(at), v, at);
        }
      }
      done(t);
    }
  }
  // f(x, index) of each entry.
  template <class F, class Done>
  __device__ __forceinline__ void each_entry(F f, Done done) const {
    each_vector(
        [&](const uint4&, int v, const uint8_t* at) {
#pragma unroll 1
          for (int e = 0; e < W; ++e) f((float)reinterpret_cast<const DT*>(at)[e], v + e);
        },
        done);
  }

  // Weights of a vector's entries that are at least x.
  struct Sum {
    uint32_t a = 0, b = 0, n = 0;         // units of 2^-22, of 2^-43, entries
  };
  __device__ __forceinline__ static void add(Sum& to, const Weigh& weigh, const uint4& q, float x) {
#pragma unroll
    for (int e = 0; e < W; e += 2) {
      const float x0 = entry(q, e), x1 = entry(q, e + 1);
      const Weights2 w = weigh.two(x0, x1);
      const bool in0 = x0 >= x, in1 = x1 >= x;
      to.a += (in0 ? w.a[0] - WEIGHT_A : 0u) + (in1 ? w.a[1] - WEIGHT_A : 0u);
      to.b += (in0 ? w.b[0] - WEIGHT_B : 0u) + (in1 ? w.b[1] - WEIGHT_B : 0u);
      to.n += in0 + in1;
    }
  }

  // ---- sums over the CTA and the cluster
  __device__ __forceinline__ void sync() {
    if (C == 1) __syncthreads();
    else cl.sync();
  }
  // f(shared memory of CTA r) by lane r of each warp; the others get `none`.
  template <class T, class F>
  __device__ __forceinline__ T of_rank(T none, F f) const {
    return lane < C ? f(cl.map_shared_rank(&s, lane)) : none;
  }

  // Lanes that are `in` add w to a 64-bit bin, once for those that add the same to the same one:
  // 64-bit additions to one address go one after the other, and ties send thousands there.  Called
  // by whole warps: the lanes that match one another are those of the ballot.
  __device__ __forceinline__ void add_to_bin(bool in, int bin, u64 w) const {
    const uint32_t lanes = __ballot_sync(0xffffffffu, in);
    if (!in) return;
    const uint32_t same = __match_any_sync(lanes, ((u64)bin << 44) | w);
    if (__ffs(same) - 1 == lane) atomicAdd(&s.hist[bin], w * __popc(same));
  }
  __device__ __forceinline__ void clear_bins() {
    for (int i = tid; i < SA_BINS / 2; i += SA_THREADS) s.hist[i] = 0;
  }
  // Counts of the thread's bins 4 tid .. 4 tid + 3 over the cluster.
  __device__ __forceinline__ uint4 counts() const {
    uint4 c = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r < C) {
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
      sync();                                             // the bins have been read
      clear_bins();
      __syncthreads();
      each_vector(
          [&](const uint4& q, int v, const uint8_t* at) {
            bool some = false;
#pragma unroll
            for (int e = 0; e < W; ++e) {
              const u64 k = key_of(entry(q, e), v + e);
              some |= k >= lo && k <= hi;
            }
            if (!__any_sync(0xffffffffu, some)) return;
#pragma unroll 1
            for (int e = 0; e < W; ++e) {
              const float x = (float)reinterpret_cast<const DT*>(at)[e];
              const u64 k = key_of(x, v + e);
              u64 w = 0;
              if (k >= lo && k <= hi) w = weight(x);
              add_to_bin(w != 0, (int)((k - lo) >> shift), w);
            }
          },
          [](int) {});
      sync();
      constexpr int PER = (1 << SA_STEP_BITS) / SA_THREADS;
      u64 h[PER] = {}, mine = 0;
      for (int r = 0; r < C; ++r) {
        const u64* o = cl.map_shared_rank(s.hist, r) + tid * PER;
#pragma unroll
        for (int j = 0; j < PER; ++j) h[j] += o[j];
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) mine += h[j];
      const Before scan = block_before(mine, s.scan);
      u64 at = base + scan.before;
      if (base + scan.all <= goal) return false;
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

  // ---- the list
  // k: n keys, one a thread, sorted (and left in s.hist): bitonic merges, within a warp by
  // shuffles, across warps by shared memory.
  __device__ __forceinline__ u64 sort_keys(u64 k, int n) {
    auto keep = [](u64 own, u64 other, bool smaller) { return (own < other) == smaller ? own : other; };
#pragma unroll 1
    for (int len = 2; len < 2 * n; len <<= 1)
#pragma unroll 1
      for (int j = len >> 1; j > 0; j >>= 1) {
        u64 other;
        if (j >= 32) {
          __syncthreads();
          s.hist[tid] = k;
          __syncthreads();
          other = s.hist[tid ^ j];
        } else {
          other = __shfl_xor_sync(0xffffffffu, k, j);
        }
        k = keep(k, other, ((tid & j) == 0) == ((tid & len) == 0));
      }
    __syncthreads();
    s.hist[tid] = k;
    __syncthreads();
    return k;
  }
  // Of the list's n keys up to `most`: the first whose running sum, of weights after `base`
  // or of ones, passes `goal`; `most` where none does (fewer entries than k, or min-p's
  // floor above the list).
  __device__ __forceinline__ u64 pick(const Weigh& weigh, int n, u64 most, bool weights, u64 base, u64 goal) {
    constexpr int PER = SA_LIST / SA_THREADS, BINS = SA_BINS / 2;
    u64 k[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + i * SA_THREADS;
      k[i] = at < n && s.sorted[at] <= most ? s.sorted[at] : ~0ull;
    }
    // while there are more than threads: the bin of their range in which the sum passes the
    // goal, by values first, then (equal values, or values of one bin) by whole keys
    int left = n;
    for (int round = 0; left > SA_THREADS; ++round) {
      u64 lo = ~0ull, hi = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        lo = k[i] < lo ? k[i] : lo;
        hi = k[i] != ~0ull && k[i] > hi ? k[i] : hi;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const u64 a = __shfl_xor_sync(0xffffffffu, lo, o), b = __shfl_xor_sync(0xffffffffu, hi, o);
        lo = a < lo ? a : lo;
        hi = b > hi ? b : hi;
      }
      __syncthreads();
      if (lane == 0) {
        s.ends[0][warp] = lo;
        s.ends[1][warp] = hi;
      }
      clear_bins();
      __syncthreads();
#pragma unroll 1
      for (int w = 0; w < SA_WARPS; ++w) {
        lo = s.ends[0][w] < lo ? s.ends[0][w] : lo;
        hi = s.ends[1][w] > hi ? s.ends[1][w] : hi;
      }
      const float top = value_of(lo), scale = (float)BINS / fminf(fmaxf(top - value_of(hi), 1e-30f), -SA_LOWEST);
      const int bits = 64 - __clzll((long long)(hi - lo)), shift = bits > 10 ? bits - 10 : 0;
      static_assert(BINS == 1 << 10, "ten bits of a key");
      auto bin_of = [&](u64 key) {
        return round == 0 ? min(__float2int_rz(rn_mul(rn_sub(top, value_of(key)), scale)), BINS - 1) : (int)((key - lo) >> shift);
      };
#pragma unroll
      for (int i = 0; i < PER; ++i)
        add_to_bin(k[i] != ~0ull, bin_of(k[i]), k[i] == ~0ull ? 0 : weights ? weight_of(weigh, value_of(k[i])) : 1ull);
      if (tid == 0) {
        s.bin[0] = -1;
        s.bin[1] = 0;
      }
      __syncthreads();
      const u64 h0 = s.hist[2 * tid], h1 = s.hist[2 * tid + 1];
      const u64 at0 = base + block_before(h0 + h1, s.scan).before, at1 = at0 + h0;
      if (at0 <= goal && goal < at1) {
        s.bin[0] = 2 * tid;
        s.before = at0;
      }
      if (at1 <= goal && goal < at1 + h1) {
        s.bin[0] = 2 * tid + 1;
        s.before = at1;
      }
      __syncthreads();
      const int bin = s.bin[0];
      if (bin < 0) break;                                    // the sum does not pass it here: min-p's floor lies above
      base = s.before;
      int in_bin = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (k[i] != ~0ull && bin_of(k[i]) != bin) k[i] = ~0ull;
        in_bin += k[i] != ~0ull;
      }
      if (in_bin) atomicAdd(&s.bin[1], in_bin);
      __syncthreads();
      left = s.bin[1];
    }
    // one a thread
    __syncthreads();
    if (tid == 0) s.bin[1] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (k[i] != ~0ull) {
        const int to = atomicAdd(&s.bin[1], 1);
        if (to < SA_THREADS) s.hist[to] = k[i];
      }
    __syncthreads();
    left = min(s.bin[1], SA_THREADS);
    u64 own = tid < left ? s.hist[tid] : ~0ull;
    if (tid == 0) s.at = -1;
    own = sort_keys(own, left);
    const u64 w = own == ~0ull ? 0 : weights ? weight_of(weigh, value_of(own)) : 1;
    const u64 at = base + block_before(w, s.scan).before;
    if (at <= goal && goal < at + w) s.at = tid;
    __syncthreads();
    const u64 found = s.at >= 0 ? s.hist[s.at] : most;
    __syncthreads();
    return found;
  }

  __device__ __forceinline__ void refuse(size_t at, uint32_t bit) {
    if (tid == 0 && rank == 0) {
      if (bit) set_status(p.status, bit);
      p.tokens[at] = -1;
      if (p.logprob) p.logprob[at] = quiet_nan();
      if (p.kept) p.kept[at] = 0;
    }
  }

  __device__ __forceinline__ void run() {
    const size_t at = blockIdx.x / C;
    const int b = (int)(at / p.n), j = (int)(at - (size_t)b * p.n);
    // slices begin where vectors do (no slice is empty: the launch sees to that)
    row = static_cast<const DT*>(p.logits) + b * p.b_stride + j * p.row_stride;
    const int skew = (int)(((uintptr_t)row & 15) / sizeof(DT));
    first = rank > 0 ? rank * p.slice - skew : 0;
    last = rank + 1 < C ? (rank + 1) * p.slice - skew : p.V;
    begin = rank * p.slice - skew;
    tile_len = 32 * W * p.tile_vectors;
    tiles = (last - begin + tile_len - 1) / tile_len;

    const float u = __ldg(p.u + at), T = p.temperature ? __ldg(p.temperature + b) : 1.f;
    const float top_p = p.top_p ? __ldg(p.top_p + b) : 1.f, min_p = p.min_p ? __ldg(p.min_p + b) : 0.f;
    const int top_k = p.top_k ? __ldg(p.top_k + b) : 0;
    if (p.resident) {                                        // (a row that is refused is not waited for)
      if (u != -1.f)
        for (int t = warp; t < tiles; t += SA_WARPS) request(data + t * p.tile_vectors * 512, t, 0, p.tile_vectors);
      cp_async_commit();
    }
    static_assert(SA_TABLE / 2 == SA_THREADS, "16 bytes of the table a thread");
    const float4 powers = __ldg(reinterpret_cast<const float4*>(g_powers.at) + tid);
    if (tid == 0) {
      s.top = 0xffffffffu;
      s.low = 0;
      s.bad = 0;
      s.listed = 0;
      s.at = 0;
    }
    const uint32_t fault = u == -1.f ? 0u
                           : !(u >= 0.f && u < 1.f && top_p >= 0.f && top_p <= 1.f && min_p >= 0.f && min_p <= 1.f)
                               ? (uint32_t)SPEC_DEV_BAD_FILTER
                               : (uint32_t)SPEC_DEV_BAD_TEMP;
    cp_async_wait_all();                                     // each lane reads what it requested, for the most part
    __syncwarp();
    if (u == -1.f || fault == SPEC_DEV_BAD_FILTER || !temp_ok(T)) return refuse(at, fault);
    const bool by_k = top_k > 0 && top_k < p.V, by_p = top_p < 1.f;

    // ---- 1: the largest logit, and the largest of each group: entry e of a vector's words
    const uint32_t none = sizeof(DT) == 2 ? 0xff80ff80u : 0xff800000u;
    uint32_t group[4] = {none, none, none, none};
    each_vector(
        [&](const uint4& q, int, const uint8_t*) {
          group[0] = word_max(group[0], q.x);
          group[1] = word_max(group[1], q.y);
          group[2] = word_max(group[2], q.z);
          group[3] = word_max(group[3], q.w);
        },
        [](int) {});
    const uint4 groups = make_uint4(group[0], group[1], group[2], group[3]);
    float m = -INFINITY, low = INFINITY;
    bool bad = false;
#pragma unroll
    for (int g = 0; g < W; ++g) {
      const float x = entry(groups, g);
      bad |= !(x <= -SA_LOWEST);
      m = fmaxf(m, x);
      if (x > -INFINITY) low = fminf(low, x);
    }
    const uint32_t top_here = __reduce_min_sync(0xffffffffu, m > -INFINITY ? descending<DT>(m) : 0xffffffffu);
    const uint32_t low_here = __reduce_max_sync(0xffffffffu, low < INFINITY ? descending<DT>(low) : 0u);
    reinterpret_cast<float4*>(s.tab)[tid] = powers;
    clear_bins();
    __syncthreads();
    if (lane == 0) {
      atomicMin(&s.top, top_here);
      atomicMax(&s.low, low_here);
    }
    if (bad) s.bad = 1;
    sync();
    const uint32_t top = __reduce_min_sync(0xffffffffu, of_rank(0xffffffffu, [](const SampleShared* o) { return o->top; }));
    const uint32_t far = __reduce_max_sync(0xffffffffu, of_rank(0u, [](const SampleShared* o) { return o->low; }));
    if (__reduce_or_sync(0xffffffffu, of_rank(0u, [](const SampleShared* o) { return o->bad; })) || top == 0xffffffffu) {
      sync();
      return refuse(at, SPEC_DEV_BAD_LOGIT);
    }
    m = of_descending<DT>(top);
    // Above 2^104 the second term of 1 / T would lose bits below the smallest numbers (a weight's 2^-34 needs
    // 18 of them), and from 2^123 on the cut-off, 31 T below the largest logit, would leave the type.
    const float temp = fminf(fmaxf(T, 0x1p-100f), 0x1p104f);
    const Weigh weigh(m, temp, p.less, s.tab);

    // the smallest logit that min-p keeps
    float least = SA_LOWEST;
    if (min_p > 0.f) {
      // (log_of takes numbers whose reciprocal is one: smaller ones times 2^60, and 60 ln 2 off again)
      const bool tiny = min_p < 0x1p-100f;
      df l = log_of(df{tiny ? rn_mul(min_p, 0x1p60f) : min_p, 0.f}, s.tab);
      if (tiny) l = dd_add(l, df{-41.58883f, -1.7930694e-06f});
      const df edge = dd_add_f(dd_mul_f(l, temp), m);
      if (edge.hi > least) least = edge.lo > 0.f ? nextafterf(edge.hi, INFINITY) : edge.hi;
    }
    if (sizeof(DT) == 2) least = __bfloat162float(__float2bfloat16_ru(least));
    const u64 floor_key = key_of(least, 0) | mask;
    const u64 every = key_of(SA_LOWEST, 0) | mask;
    auto mass_goal = [&](u64 z) {                            // what a running sum has to pass for top-p to be full
      const u64 pf = fraction64(top_p), g = __umul64hi(pf, z) + (pf * z != 0);
      return g > 0 ? g - 1 : 0;
    };

    // ---- 2 and 3: entries from `from` on are kept and add to their tile's sum, those of
    // [low_x, sure] are listed; sure < from.  Where the mass of all has to be known first,
    // a first pass sums everything and counts the bins.
    float from = least, sure = -INFINITY, low_x = SA_LOWEST, bin_scale = 0.f;
    u64 all_mass = 0, base = 0, limit = floor_key, kept = 0;   // kept: this thread's mass, in the end
    uint32_t count = 0;
    const bool listing = by_k || by_p, small = p.V < SA_LIST;
    bool fits = !by_k || top_k < SA_LIST;
    auto bin_of = [&](float x) { return min(__float2int_rz(rn_mul(rn_sub(m, x), bin_scale)), SA_BINS - 1); };
    uint32_t* bins = reinterpret_cast<uint32_t*>(s.hist);
    bool counting = by_p && !by_k && !small;
    if (listing) {
      from = sure = INFINITY;
      float range = m - of_descending<DT>(far);
      if (!by_k) range = fminf(m - weigh.low, 2.5f * range);   // down to the smallest weight, or well below the maxima
      bin_scale = (float)SA_BINS / fminf(fmaxf(range, 1e-30f), -SA_LOWEST);
      if (counting) {
        from = SA_LOWEST;
      } else if (!small) {
        // groups: the threads' maxima where those are enough
        const bool threads = top_k <= C * (SA_THREADS / 4);
#pragma unroll 1
        for (int g = 0; g < (threads ? 1 : W); ++g) {
          const uint32_t word = group_word(groups, g) >> (sizeof(DT) == 2 ? 16 * (g & 1) : 0);
          const float x = threads ? vector_max(groups) : entry(make_uint4(word, 0, 0, 0), 0);
          if (x > -INFINITY) atomicAdd(&bins[bin_of(x)], 1u);
        }
      }
    }
    for (bool again = listing && fits && !small;;) {
      if (listing && small && fits) {                        // every entry is listed, in its place
        for (int i = tid; i < p.V; i += SA_THREADS) s.index[i] = i;
        if (tid < tiles) s.tile[tid] = 0;
        if (tid == 0) s.listed = p.V;
      } else if (!listing || (fits && (counting || !again))) {
        Sum part;
        each_vector(
            [&](const uint4& q, int v, const uint8_t*) {
              const float largest = vector_max(q);
              if (largest >= from) add(part, weigh, q, from);
              if (counting) {
                if (largest > weigh.low)
#pragma unroll
                  for (int e = 0; e < W; ++e)
                    if (entry(q, e) > weigh.low) atomicAdd(&bins[bin_of(entry(q, e))], 1u);
              } else if (listing && largest >= low_x) {
                uint32_t hits = 0;
#pragma unroll
                for (int e = 0; e < W; ++e) hits |= (entry(q, e) >= low_x && entry(q, e) <= sure ? 1u : 0u) << e;
                while (hits) {
                  const int e = __ffs(hits) - 1;
                  hits &= hits - 1;
                  const int to = atomicAdd(&s.listed, 1);
                  if (to < SA_LIST) s.index[to] = v + e;
                }
              }
            },
            [&](int t) {
              u64 tile = 0;
              if (__any_sync(0xffffffffu, part.n != 0)) {
                const u64 z = weight_sum(part.a, part.b);
                tile = warp_sum64(z);
                kept += z;
                count += part.n;
                part = Sum{};
              }
              if (lane == 0) s.tile[t] = tile;
            });
      }
      if (!again) break;
      again = false;
      if (counting) {
        const Before scan = block_before(kept, s.scan);
        if (tid == 0) s.sum[0] = scan.all;
        kept = count = 0;
      }
      if (tid < 2) s.bin[tid] = SA_BINS;
      sync();
      const uint4 c = counts();
      const uint32_t n[4] = {c.x, c.y, c.z, c.w};
      const float step = 1.f / bin_scale;
      if (by_k) {
        u64 at = block_before((u64)c.x + c.y + c.z + c.w, s.scan).before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (at < (u64)top_k && (u64)top_k <= at + n[i]) s.bin[1] = 4 * tid + i;
          at += n[i];
        }
        __syncthreads();
      } else {
        counting = false;
        all_mass = warp_sum64(of_rank((u64)0, [](const SampleShared* o) { return o->sum[0]; }));
        const u64 goal = mass_goal(all_mass);
        // a bin's mass lies between its count times the weights of its edges, moved outwards
        // by more than the edges' and the weights' rounding
        const float per_bin = -step * weigh.c.hi * (1.f / SA_TABLE), one = ldexpf(1.f, 43 - p.less);
        auto edge_of = [&](int i) { return __float2ull_rn(exp2f((float)i * per_bin) * one); };
        u64 most[4], fewest[4], most_4 = 0, fewest_4 = 0;
        u64 edge = edge_of(4 * tid);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          most[i] = n[i] * (edge + (edge >> 14) + 1);
          edge = 4 * tid + i + 1 < SA_BINS ? edge_of(4 * tid + i + 1) : 0;
          const u64 slack = (edge >> 14) + 1;
          fewest[i] = n[i] * (edge > slack ? edge - slack : 0);
          most_4 += most[i];
          fewest_4 += fewest[i];
        }
        const Before a = block_before(most_4, s.scan), f = block_before(fewest_4, s.scan);
        u64 above = a.before, below = f.before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // the running mass after the bin, from the front or from the end
          above += most[i];
          below += fewest[i];
          const u64 rest = f.all - below, rest_most = a.all - above;
          if (above > goal && all_mass - rest > goal) atomicMin(&s.bin[0], 4 * tid + i);
          if (below > goal || (all_mass > rest_most && all_mass - rest_most > goal)) atomicMin(&s.bin[1], 4 * tid + i);
        }
        __syncthreads();
        // above every entry of the first bin in which the mass can run full
        const int first_bin = s.bin[0];
#pragma unroll 1
        for (float o = 0x1p-10f; first_bin > 0 && o < 0x1p12f && sure == INFINITY; o *= 2.f) {
          const float x = m - ((float)first_bin - o) * step;
          if (bin_of(x) < first_bin) sure = x;
        }
        // down to the type's next number: the same entries lie above it, and its key (of 16 bits) is its own,
        // which a search begins with
        if (sizeof(DT) == 2) sure = __bfloat162float(__float2bfloat16_rd(sure));
        from = least > sure ? least : nextafterf(sure, INFINITY);   // (where min-p takes some away, its floor is the limit)
      }
      const int last_bin = s.bin[1];
      // below every entry of the last one; with fewer groups than k, below all
#pragma unroll 1
      for (float o = 0x1p-10f; last_bin < SA_BINS - 1 && o < 0x1p12f && low_x == SA_LOWEST; o *= 2.f) {
        const float x = m - ((float)(last_bin + 1) + o) * step;
        if (bin_of(x) > last_bin && x > SA_LOWEST) low_x = x;
      }
    }
    if (listing && fits) {
      base = block_before(kept, s.scan).all;                 // the mass above `sure`
      if (tid == 0) s.sum[1] = base;
      sync();
      const u64 list_here = of_rank((u64)0, [](const SampleShared* o) { return (u64)o->listed; }), lists = warp_upto64(list_here);
      const int n = (int)__shfl_sync(0xffffffffu, lists, 31);
      if (warp == 0 && lane < 8) s.lists[lane] = (int)(lists - list_here);
      base = warp_sum64(of_rank((u64)0, [](const SampleShared* o) { return o->sum[1]; }));
      fits = n < SA_LIST;
      if (fits) {
        // ---- 4: the last kept entry of the list
        __syncthreads();
        for (int i = tid; i < n; i += SA_THREADS) {
          int r = 0;
          for (int k = 1; k < C; ++k) r = i >= s.lists[k] ? k : r;
          const int v = cl.map_shared_rank(s.index, r)[i - s.lists[r]];
          s.sorted[i] = key_of(value_at(v, r), v);
        }
        __syncthreads();
        limit = every;                                       // (-inf, in small lists, comes behind)
        if (by_k) limit = pick(weigh, n, every, false, 0, (u64)(top_k - 1));
        if (by_p) {
          u64 mass = all_mass;
          if (by_k || small) {
            u64 sum = 0;
            for (int i = tid; i < n; i += SA_THREADS)
              if (s.sorted[i] <= limit) sum += weight_of(weigh, value_of(s.sorted[i]));
            mass = block_before(sum, s.scan).all;
          }
          limit = pick(weigh, n, limit, true, base, mass_goal(mass));
        }
        limit = floor_key < limit ? floor_key : limit;
        for (int i = tid; i < s.listed; i += SA_THREADS) {
          const int v = s.index[i];
          const float x = value_at(v, rank);
          if (key_of(x, v) <= limit) {
            const u64 w = weight_of(weigh, x);
            atomicAdd(&s.tile[(v - begin) / tile_len], w);
            kept += w;
            ++count;
          }
        }
      }
    }
    if (listing && !fits) {
      // ---- 2 to 4 by searches over the row; with top-p alone among the keys of the window
      const bool window = all_mass != 0;
      limit = every;
      for (int filter = by_k ? 0 : 1; filter < 3; ++filter) {  // the k-th entry, the mass of top-p, the tiles' sums
        u64 lo = (u64)top << p.idx_bits, from_mass = 0, goal = (u64)(top_k - 1), k;
        if (filter == 1 && !by_p) continue;
        if (filter == 2) limit = floor_key < limit ? floor_key : limit;
        if (filter == 1 && window) {
          if (sure < INFINITY) lo = key_of(sure, 0);
          from_mass = base;
          goal = mass_goal(all_mass);
        } else if (filter > 0) {
          kept = count = 0;
          u64 sum = 0;
          each_entry(
              [&](float x, int v) {
                if (key_of(x, v) <= limit) {
                  sum += weight_of(weigh, x);
                  ++count;
                }
              },
              [&](int t) {
                const u64 tile = warp_sum64(sum);
                if (lane == 0) s.tile[t] = tile;
                kept += sum;
                sum = 0;
              });
          if (filter == 2) break;
          const u64 here = block_before(kept, s.scan).all;
          sync();                                            // the sums before it have been read
          if (tid == 0) s.sum[0] = here;
          sync();
          goal = mass_goal(warp_sum64(of_rank((u64)0, [](const SampleShared* o) { return o->sum[0]; })));
        }
        const u64 hi = filter == 1 && window ? key_of(low_x, 0) | mask : limit;
        if (search(lo, hi, from_mass, goal, [&](float x) { return filter == 0 ? 1ull : weight_of(weigh, x); }, k)) limit = k;
      }
    }

    // ---- 5: the CTA, the tile, the token
    const u64 kept_here = warp_sum64(kept);
    const uint32_t count_here = __reduce_add_sync(0xffffffffu, count);
    __syncthreads();
    if (lane == 0) {
      s.scan[warp] = kept_here;
      s.count[warp] = count_here;
    }
    __syncthreads();
    if (warp == 0) {
      const u64 sum = warp_sum64(lane < SA_WARPS ? s.scan[lane] : 0);
      const uint32_t entries = __reduce_add_sync(0xffffffffu, lane < SA_WARPS ? s.count[lane] : 0u);
      if (lane == 0) {
        s.sum[2] = sum;
        s.entries = entries;
      }
    }
    sync();
    const u64 share = of_rank((u64)0, [](const SampleShared* o) { return o->sum[2]; });
    const uint32_t total = __reduce_add_sync(0xffffffffu, of_rank(0u, [](const SampleShared* o) { return o->entries; }));
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");   // nothing of another CTA is read after this
    const u64 upto = warp_upto64(share), z = __shfl_sync(0xffffffffu, upto, 31);
    const u64 ahead = __shfl_sync(0xffffffffu, upto - share, rank), mine = __shfl_sync(0xffffffffu, share, rank);
    const u64 goal = __umul64hi(fraction64(u), z);
    if (goal >= ahead && goal < ahead + mine) draw(at, goal, ahead, z, total, limit, weigh);
    __syncwarp();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");   // none of this one is read any more
  }

  // The token, by the CTA that holds it.
  __device__ __forceinline__ void draw(size_t at, u64 goal, u64 ahead, u64 z, uint32_t total, u64 limit, const Weigh& weigh) {
    static_assert(SA_TILES <= SA_THREADS, "a thread a tile");
    const u64 in_tile = tid < tiles ? s.tile[tid] : 0;
    const u64 before = ahead + block_before(in_tile, s.scan).before;
    if (before <= goal && goal < before + in_tile) {
      s.at = tid;
      s.before = before;
    }
    __syncthreads();
    // two entries a thread at a time
    const int tile = s.at;
    u64 done = s.before;
#pragma unroll 1
    for (int i = 0; i < tile_len; i += 2 * SA_THREADS) {
      const int o = i + 2 * tid, v = begin + tile * tile_len + o;
      float x[2];
      bool in[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool there = o + e < tile_len && v + e >= first && v + e < last;
        x[e] = there ? value_at(v + e, rank) : -INFINITY;
        in[e] = there && key_of(x[e], v + e) <= limit;
      }
      const Weights2 w = weigh.two(x[0], x[1]);
      u64 f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) f[e] = in[e] ? weight_sum(w.a[e] - WEIGHT_A, w.b[e] - WEIGHT_B) : 0;
      const Before scan = block_before(f[0] + f[1], s.scan);
      const u64 at_pair = done + scan.before;
      if (at_pair <= goal && goal < at_pair + f[0] + f[1]) {
        const int e = goal >= at_pair + f[0];
        p.tokens[at] = v + e;
        if (p.logprob) {
          const float unit = ldexpf(1.f, p.less - 43), zh = __ull2float_rn(z);
          const df l = log_of(df{zh * unit, __ll2float_rn((long long)(z - __float2ull_rn(zh))) * unit}, s.tab);
          const df a = weigh.argument(x[e]), d = two_sum_df(a.hi, -l.hi);
          p.logprob[at] = d.hi + (d.lo + (a.lo - l.lo));
        }
        if (p.kept) p.kept[at] = (int)total;
      }
      done += scan.all;
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
    e = cudaFuncSetAttribute(sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(SampleShared) + SA_SLICE);
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
  p.less = bits > 19 ? bits - 19 : 0;
  const long long rows = (long long)a.B * a.n;
  const int size = a.dtype == SPEC_BF16 ? 2 : 4, W = 16 / size;
  // CTAs a row: more of them while all are on the GPU at once, two an SM, and have 16384
  // entries each.  us a call, cold caches, with 1, 2, 4 and 8: 128 rows of 32000 bf16,
  // top-k 50: 22, 27, 45, 96; 16 rows of 128256 bf16, top-p 0.9: 86, 57, 39, 39; 64 rows of
  // 151936 fp32, top-p 0.9: 123, 78, 70, 94.
  int C = 1;
  auto slice = [&] { return ((a.V + C - 1) / C + 32 * W - 1) / (32 * W) * (32 * W); };
  while (C < 8 && 2 * C * rows <= 2LL * sms && a.V / (2 * C) >= 16384) C *= 2;
  // two a row also where that is a second wave, but the rows of one are long ones: 256 rows of
  // 128256 bf16 of mixed settings 117 us, with one CTA a row 135 to 158
  if (C == 1 && 2 * rows <= 4LL * sms && a.V >= 65536) C = 2;
  // a lane of a tile adds at most 1024 weights, whose low parts (to 2^20 each) fit 32 bits
  while (slice() > 1 << 22) C *= 2;
  while ((long long)(C - 1) * slice() >= a.V) --C;           // no empty slice
  p.slice = slice();
  // tiles of four vectors a lane where every warp has some
  p.tile_vectors = p.slice >= 32 * W * SA_STAGE * SA_WARPS / 2 ? SA_STAGE : 1;
  while ((p.slice + 32 * W * p.tile_vectors) / (32 * W * p.tile_vectors) > SA_TILES) p.tile_vectors *= 2;
  const long long whole = (long long)(p.slice + W + 32 * W * p.tile_vectors - 1) / (32 * W * p.tile_vectors) * p.tile_vectors * 512;
  p.resident = whole <= SA_SLICE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(SA_THREADS);
  cfg.dynamicSmemBytes = sizeof(SampleShared) + (size_t)(p.resident ? whole : 2 * SA_WARPS * SA_STAGE * 512);
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
