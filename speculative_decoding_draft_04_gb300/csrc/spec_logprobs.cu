// Log probabilities of given tokens, entropy and the top K alternatives of rows
// of logits x (divided by a temperature):
//
//   d = (x - m) log2(e) / T,  Z = sum 2^d,  lse = m / T + ln Z
//   logprob = (x_token - m) / T - ln Z,     H = ln 2 (log2 Z - sum 2^d d / Z)
//
// One read of each row.  logprobs_kernel: a CTA takes one segment of one row,
// 256 threads x 8 vectors of 16 bytes, all requested at once and kept in
// registers, so that maximum, sums and candidates come from one load.
//
// The K largest: a thread's maximum is at hand, so the K-th largest of 32
// group maxima (8 threads each) is a bound that at least K entries reach and,
// for values in no particular order, some 30 to 130 of 16384 do.  Those are
// collected and ranked by counting.  Equal values beyond the list's size (a
// row of few different values) are found one by one instead.
//
// Rows of more than one segment are joined by logprobs_join_kernel, a warp a
// row, from each segment's (m, Z, sum 2^d d) and its K sorted candidates; its
// launch overlaps the first kernel's end.
#include "spec_serve.cuh"

namespace spec {

struct LogprobParams {
  int B, n, V, K, segments;
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

constexpr int LP_THREADS = 256, LP_WARPS = LP_THREADS / 32, LP_VECS = 8, LP_GROUPS = 32, LP_LIST = 256;
constexpr float LP_LN2 = 0.69314718056f;

template <class DT>
struct LpVec {
  static constexpr int E = 16 / sizeof(DT);                  // elements a vector
  static constexpr int SEG = LP_THREADS * LP_VECS * E;       // elements a segment: 16384 bf16, 8192 fp32
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
__device__ __forceinline__ void vec_set(uint4& v, int e, bf16 x) {
  const uint32_t b = *reinterpret_cast<const uint16_t*>(&x);
  uint32_t& w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
  w = e & 1 ? (w & 0xffffu) | b << 16 : (w & 0xffff0000u) | b;
}
__device__ __forceinline__ void vec_set(uint4& v, int e, float x) {
  uint32_t& w = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
  w = __float_as_uint(x);
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

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
template <class DT>
__device__ __forceinline__ const DT* row_at(const LogprobParams& p, int row) {
  const int b = row / p.n;
  return static_cast<const DT*>(p.logits) + b * p.b_stride + (row - b * p.n) * p.row_stride;
}

template <class DT>
__global__ void __launch_bounds__(LP_THREADS, 4) logprobs_kernel(const __grid_constant__ LogprobParams p) {
  constexpr int E = LpVec<DT>::E, SEG = LpVec<DT>::SEG;
  const DT* const tag = nullptr;
  __shared__ float s_group[LP_GROUPS];
  __shared__ float4 s_warp[LP_WARPS];
  __shared__ unsigned long long s_list[LP_LIST];
  __shared__ float s_bound;
  __shared__ int s_count;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int row = blockIdx.x / p.segments, seg = blockIdx.x - row * p.segments;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int token = __ldg(p.tokens + row);
  const float T = p.temperature ? __ldg(p.temperature + row / p.n) : 1.f;
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
#pragma unroll
  for (int j = 0; j < LP_VECS; ++j) {
    const int at = (i0 + j * LP_THREADS) * E - lead;
    if (at >= 0 && at + E <= p.V) {
      v[j] = __ldcs(reinterpret_cast<const uint4*>(x + at));
    } else {
      const uint32_t w = neg_inf_word(tag);
      v[j] = make_uint4(w, w, w, w);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (at + e >= 0 && at + e < p.V) vec_set(v[j], e, x[at + e]);
    }
  }
  if (tid == 0) s_count = 0;
  // ---- maxima: vector, thread, group of 8 threads, warp
  float vm[LP_VECS], tm;
#pragma unroll
  for (int j = 0; j < LP_VECS; ++j) vm[j] = vec_max(v[j], tag);
  tm = max_nan(max_nan(max_nan(vm[0], vm[1]), max_nan(vm[2], vm[3])), max_nan(max_nan(vm[4], vm[5]), max_nan(vm[6], vm[7])));
  float gm = tm;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) gm = max_nan(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  if ((lane & 7) == 0) s_group[tid >> 3] = gm;
  float m = gm;
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  // ---- sums against the warp's maximum; an entry of -inf adds nothing
  const float c = 1.4426950408889634f / T;
  const float base = m == -INFINITY ? 0.f : -m * c;
  float z = 0.f, w1 = 0.f;
  auto sums = [&](auto dist) {
#pragma unroll
    for (int j = 0; j < LP_VECS; ++j) {
      float zz = 0.f, ww = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = fmaxf(dist(vec_get(v[j], e, tag)), -200.f);
        const float y = ex2(d);
        zz += y;
        ww = fmaf(y, d, ww);
      }
      z += zz;
      w1 += ww;
    }
  };
  if (fabsf(base) < 3.0e38f) sums([&](float y) { return fmaf(y, c, base); });
  else sums([&](float y) { return (y - m) * c; });           // m / T beyond the floats
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    w1 += __shfl_xor_sync(0xffffffffu, w1, o);
  }
  if (lane == 0) s_warp[warp] = make_float4(m, m == -INFINITY ? 0.f : z, m == -INFINITY ? 0.f : w1, 0.f);
  __syncthreads();
  // ---- bound of the candidates: the K-th largest group maximum
  if (p.K > 0) {
    if (warp == 0) {
      const float g = s_group[lane];
      int above = 0;
#pragma unroll
      for (int i = 0; i < LP_GROUPS; ++i) {
        const float h = s_group[i];
        above += h > g || (h == g && i < lane);
      }
      if (above == p.K - 1) s_bound = g;                     // NaN: the row has no distribution
      if (lane == 0 && !(s_group[0] == s_group[0])) s_bound = -INFINITY;
    }
    __syncthreads();
    const float bound = s_bound;
    if (tm >= bound) {
#pragma unroll
      for (int j = 0; j < LP_VECS; ++j)
        if (vm[j] >= bound) {
          const int at = (i0 + j * LP_THREADS) * E - lead;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float y = vec_get(v[j], e, tag);
            // entries of -inf count only where the lowest indexes may be needed
            if (y >= bound && (y > -INFINITY || (at + e >= 0 && at + e < p.V && at + e < seg * SEG - lead + 64))) {
              const int k = atomicAdd(&s_count, 1);
              if (k < LP_LIST) s_list[k] = entry_key(y, at + e);
            }
          }
        }
    }
    __syncthreads();
  }
  // ---- this segment's part: every thread has it, warp by warp in order
  float pm = s_warp[0].x;
#pragma unroll
  for (int i = 1; i < LP_WARPS; ++i) pm = max_nan(pm, s_warp[i].x);
  float pz = 0.f, pw = 0.f;
#pragma unroll
  for (int i = 0; i < LP_WARPS; ++i) {
    const float4 q = s_warp[i];
    const float d = q.x == -INFINITY ? 0.f : fmaxf((q.x - pm) * c, -200.f), f = ex2(d);
    pz += q.y * f;
    pw += f * fmaf(q.y, d, q.z);
  }
  const bool single = p.segments == 1;
  const bool bad = !(pm < INFINITY) || (single && pm == -INFINITY);
  if (!single && tid == 0) p.part[blockIdx.x] = make_float4(pm, pz, pw, 0.f);
  const float lz = LP_LN2 * log2f(pz);
  if (single) {
    if (bad) {
      write_nothing(p, row, tid, LP_THREADS, SPEC_DEV_BAD_LOGIT);
      return;
    }
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
      p.keys[(size_t)blockIdx.x * p.K + rank] = key;
    }
  };
  const int count = s_count;
  if (count <= LP_LIST) {
    if (tid < count) {
      const unsigned long long mine = s_list[tid];
      int rank = 0;
      for (int i = 0; i < count; ++i) rank += s_list[i] > mine;
      if (rank < p.K) put(rank, mine);
    }
    if (!single && tid >= count && tid < p.K) put(tid, 0);   // a segment of fewer entries
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
  extern __shared__ uint8_t s_next[];                        // [warps][segments] candidates taken (multi-pass rows)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * LPJ_WARPS + warp;
  if (row < p.B * p.n) {
    const int token = __ldg(p.tokens + row);
    const float T = p.temperature ? __ldg(p.temperature + row / p.n) : 1.f;
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
    const float c = 1.4426950408889634f / T;
    float z = 0.f, w1 = 0.f;
    for (int s = lane; s < p.segments; s += 32) {
      const float4 q = part[s];
      const float d = q.x == -INFINITY ? 0.f : fmaxf((q.x - m) * c, -200.f), f = ex2(d);
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
    uint8_t* next = s_next + warp * p.segments;
    const unsigned long long* keys = p.keys + (size_t)row * p.segments * p.K;
    // the best of this lane's lists and where it is
    unsigned long long head = 0;
    int from = -1;
    auto look = [&]() {
      head = 0;
      for (int s = lane; s < p.segments; s += 32) {
        const int at = next[s];
        const unsigned long long key = at < p.K ? keys[(size_t)s * p.K + at] : 0;
        if (key > head) {
          head = key;
          from = s;
        }
      }
    };
    for (int s = lane; s < p.segments; s += 32) next[s] = 0;
    __syncwarp();
    look();
    unsigned long long mine = 0;                             // lane k keeps the k-th
    for (int k = 0; k < p.K; ++k) {
      const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32));
      const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(head >> 32) == hi ? (uint32_t)head : 0u);
      const unsigned long long best = (unsigned long long)hi << 32 | lo;
      if (lane == k) mine = best;
      if (head == best && best) {
        ++next[from];
        look();
      }
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
  if ((long long)rows * p.segments > 0x7fffffff) return cudaErrorInvalidValue;
  logprobs_kernel<DT><<<rows * p.segments, LP_THREADS, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.segments == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + LPJ_WARPS - 1) / LPJ_WARPS);
  cfg.blockDim = dim3(32 * LPJ_WARPS);
  cfg.dynamicSmemBytes = (size_t)LPJ_WARPS * p.segments;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_join_kernel<DT>, p);
}

cudaError_t launch_logprobs(const spec_logprobs_args& a, int sms, cudaStream_t st) {
  LogprobParams p{a.B, a.n, a.V, a.K, 0, a.logits, a.b_stride, a.row_stride, a.tokens, a.temperature, a.logprob,
                  a.entropy, a.top_ids, a.top_logprobs, a.dev_status, nullptr, nullptr};
  return a.dtype == SPEC_BF16 ? launch<bf16>(p, a, st) : launch<float>(p, a, st);
}

}  // namespace spec
