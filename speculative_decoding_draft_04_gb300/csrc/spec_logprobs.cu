// Log probabilities of given tokens, entropy and the top K alternatives of rows
// of logits x (divided by a temperature):
//
//   lse = m + log Z,  Z = sum e^(x - m),  logprob = x_token - lse,
//   H = log Z - sum e^(x - m) (x - m) / Z
//
// One CTA a row: the maximum, then the sums, then K rounds that each find the
// largest entry below the last one found (value descending, index ascending).
#include "spec_serve.cuh"

namespace spec {

struct LogprobParams {
  int B, n, V, K;
  const void* logits;
  long long b_stride, row_stride;
  const int* tokens;
  const float* temperature;
  float* logprob;
  float* entropy;
  int* top_ids;
  float* top_lp;
  uint32_t* status;
};

constexpr int LPT = 256;

// Whole numbers in the order of the floats (-0 counts as 0).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <class DT>
__global__ void __launch_bounds__(LPT) logprobs_kernel(LogprobParams p) {
  __shared__ float s_a[LPT / 32], s_b[LPT / 32];
  __shared__ unsigned long long s_k[LPT / 32];
  const int row = blockIdx.x, b = row / p.n, j = row - b * p.n, tid = threadIdx.x;
  const int token = p.tokens[row];
  const float T = p.temperature ? p.temperature[b] : 1.f;
  uint32_t flag = 0;
  if (token < -1 || token >= p.V) flag = SPEC_DEV_BAD_TOKEN;
  else if (!(T > 0.f) || !isfinite(T)) flag = SPEC_DEV_BAD_TEMP;
  const DT* x = static_cast<const DT*>(p.logits) + b * p.b_stride + j * p.row_stride;
  float m = -INFINITY;
  int odd = 0;
  if (token >= 0 && !flag)
    for (int v = tid; v < p.V; v += LPT) {
      const float u = tof(x[v]);
      odd |= !(u < INFINITY);
      m = fmaxf(m, u);
    }
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) s_a[tid >> 5] = m;
  odd = __syncthreads_or(odd);
  for (int w = 0; w < LPT / 32; ++w) m = fmaxf(m, s_a[w]);
  if (token >= 0 && !flag && (odd || m == -INFINITY)) flag = SPEC_DEV_BAD_LOGIT;
  if (token < 0 || flag) {
    if (tid == 0) {
      p.logprob[row] = p.entropy[row] = quiet_nan();
      if (flag) set_status(p.status, flag);
    }
    if (tid < p.K) {
      p.top_ids[(size_t)row * p.K + tid] = -1;
      p.top_lp[(size_t)row * p.K + tid] = quiet_nan();
    }
    return;
  }
  __syncthreads();
  float z = 0.f, w1 = 0.f;
  const float mt = m / T;
  // sums of 32 terms, then their sums: the rounding of a long row stays small
  for (int v0 = tid; v0 < p.V; v0 += 32 * LPT) {
    float zz = 0.f, ww = 0.f;
    for (int v = v0; v < p.V && v < v0 + 32 * LPT; v += LPT) {
      const float d = tof(x[v]) / T - mt;
      const float e = expf(d);
      zz += e;
      if (e > 0.f) ww += e * d;
    }
    z += zz;
    w1 += ww;
  }
  for (int o = 16; o; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    w1 += __shfl_xor_sync(0xffffffffu, w1, o);
  }
  if ((tid & 31) == 0) {
    s_a[tid >> 5] = z;
    s_b[tid >> 5] = w1;
  }
  __syncthreads();
  z = w1 = 0.f;
  for (int w = 0; w < LPT / 32; ++w) {
    z += s_a[w];
    w1 += s_b[w];
  }
  const float lz = logf(z);
  if (tid == 0) {
    p.logprob[row] = tof(x[token]) / T - mt - lz;
    p.entropy[row] = lz - w1 / z;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < p.K; ++k) {
    unsigned long long best = 0;
    for (int v = tid; v < p.V; v += LPT) {
      const unsigned long long key = (unsigned long long)ordered(tof(x[v])) << 24 | (0xffffff - v);
      if (key < last && key > best) best = key;
    }
    for (int o = 16; o; o >>= 1) {
      const unsigned long long u = __shfl_xor_sync(0xffffffffu, best, o);
      if (u > best) best = u;
    }
    __syncthreads();
    if ((tid & 31) == 0) s_k[tid >> 5] = best;
    __syncthreads();
    for (int w = 0; w < LPT / 32; ++w)
      if (s_k[w] > best) best = s_k[w];
    last = best;
    if (tid == 0) {
      const int v = 0xffffff - (int)(best & 0xffffff);
      p.top_ids[(size_t)row * p.K + k] = v;
      p.top_lp[(size_t)row * p.K + k] = tof(x[v]) / T - mt - lz;
    }
  }
}

size_t logprobs_workspace_bytes(int rows, int V, int K) { return 256; }

cudaError_t launch_logprobs(const spec_logprobs_args& a, int sms, cudaStream_t st) {
  LogprobParams p{a.B, a.n, a.V, a.K, a.logits, a.b_stride, a.row_stride, a.tokens, a.temperature, a.logprob,
                  a.entropy, a.top_ids, a.top_logprobs, a.dev_status};
  if (a.dtype == SPEC_BF16) logprobs_kernel<bf16><<<a.B * a.n, LPT, 0, st>>>(p);
  else logprobs_kernel<float><<<a.B * a.n, LPT, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace spec
