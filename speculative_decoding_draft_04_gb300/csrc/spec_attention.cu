// Attention of each request's new tokens over its 4-bit paged cache.
//
//   s_ij = softmax_scale k_scale (q_i . k_j),  out_i = v_scale sum_j e^(s_ij - m_i) v_j / sum_j e^(s_ij - m_i)
//
// One CTA a (packed row, query head): 128 tokens a step, each thread one
// token's score, then each thread the output columns d = thread, + 128 over
// the step's tokens, with a running maximum and sum.
#include "spec_serve.cuh"

namespace spec {

struct AttnParams {
  int B, T, Hq, Hkv, D, P, bpp, num_pages, stride, mask_words;
  const void* q;
  long long q_row, q_head;
  const uint8_t* cache;
  const int* table;
  const int* kv_len;
  const int* row_ptr;
  const uint32_t* mask;
  float scale_k, scale_v;                 // softmax_scale * k_scale, v_scale
  void* out;
  float* lse;
  uint32_t* status;
};

constexpr int ATT = 128;

template <class DT>
__global__ void __launch_bounds__(ATT) cache_attention_kernel(AttnParams p) {
  __shared__ float s_q[256];
  __shared__ float s_p[ATT];
  __shared__ float s_red[ATT / 32];
  __shared__ long long s_blk[ATT];
  __shared__ int s_bad;
  const int row = blockIdx.x, hq = blockIdx.y, h = hq / (p.Hq / p.Hkv), tid = threadIdx.x;
  const int first_row = p.row_ptr[0], end_row = p.row_ptr[p.B];
  if (row < first_row || row >= end_row || first_row < 0 || end_row > p.T) {
    if (tid == 0 && (first_row < 0 || end_row > p.T)) set_status(p.status, SPEC_DEV_BAD_LEN);
    return;
  }
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.row_ptr[mid] <= row) lo = mid; else hi = mid;
  }
  const int b = lo, r0 = p.row_ptr[b], n = p.row_ptr[b + 1] - r0, L = p.kv_len[b];
  const bool bad = n <= 0 || row < r0 || row >= r0 + n || L < n || L > (long long)p.stride * p.P || L > (1 << 30);
  if (tid == 0) {
    s_bad = 0;
    if (bad) set_status(p.status, SPEC_DEV_BAD_LEN);
  }
  DT* out = static_cast<DT*>(p.out) + ((size_t)row * p.Hq + hq) * p.D;
  if (bad) {
    for (int d = tid; d < p.D; d += ATT) out[d] = (DT)quiet_nan();
    if (tid == 0 && p.lse) p.lse[(size_t)row * p.Hq + hq] = quiet_nan();
    return;
  }
  const DT* q = static_cast<const DT*>(p.q) + row * p.q_row + hq * p.q_head;
  for (int d = tid; d < p.D; d += ATT) s_q[d] = tof(q[d]);
  const int ctx = L - n, i = row - r0;
  const int last = p.mask ? L : ctx + i + 1;
  float m = -INFINITY, sum = 0.f, acc[2] = {0.f, 0.f};
  __syncthreads();
  for (int t0 = 0; t0 < last; t0 += ATT) {
    const int t = t0 + tid;
    bool seen = t < last;
    if (seen && p.mask && t >= ctx) {
      const int u = t - ctx;
      seen = (u >> 5) < p.mask_words && ((p.mask[(size_t)row * p.mask_words + (u >> 5)] >> (u & 31)) & 1);
    }
    float s = -INFINITY;
    s_blk[tid] = -1;
    if (seen) {
      const int page = p.table[(size_t)b * p.stride + t / p.P], tok = t % p.P;
      if (page < 0 || page >= p.num_pages) {
        s_bad = 1;
      } else {
        const long long at = (long long)cache_block_at(page, h, tok >> 4, p.Hkv, p.bpp, p.D);
        s_blk[tid] = at;
        const uint8_t* codes = p.cache + at + (tok & 15) * (p.D / 2);
        const uint8_t* scales = p.cache + at + cache_k_scales(p.D) + (tok & 15) * (p.D / 16);
        float dot = 0.f;
        for (int g = 0; g < p.D / 16; ++g) {
          const uint2 w = *reinterpret_cast<const uint2*>(codes + g * 8);
          const uint32_t ww[2] = {w.x, w.y};
          float part = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t e[4] = {decode_pair<0>(ww[k]), decode_pair<1>(ww[k]), decode_pair<2>(ww[k]),
                                   decode_pair<3>(ww[k])};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float2 v = half2_floats(e[x]);
              part += v.x * s_q[g * 16 + k * 8 + 2 * x] + v.y * s_q[g * 16 + k * 8 + 2 * x + 1];
            }
          }
          dot += part * half2_floats(decode_scales(scales[g])).x;
        }
        s = dot * p.scale_k;
      }
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    for (int w = 0; w < ATT / 32; ++w) mx = fmaxf(mx, s_red[w]);
    const float mn = fmaxf(m, mx);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float f = expf(m - ref), e = expf(s - ref);
    m = mn;
    s_p[tid] = e;
    sum *= f;
    acc[0] *= f;
    acc[1] *= f;
    __syncthreads();
    const int steps = min(ATT, last - t0);
    for (int u = 0; u < steps; ++u) {
      const float w = s_p[u];
      sum += w;
      if (s_blk[u] < 0) continue;
      const int tok = (t0 + u) % p.P & 15;
      const uint8_t* base = p.cache + s_blk[u];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = tid + k * ATT;
        if (d < p.D) {
          const uint32_t c = base[cache_v_codes(p.D) + tok * (p.D / 2) + d / 2];
          const float2 v = half2_floats(decode_pair<0>(c));
          acc[k] += w * (d & 1 ? v.y : v.x) * half2_floats(decode_scales(base[cache_v_scales(p.D) + tok * (p.D / 16) + d / 16])).x;
        }
      }
    }
    __syncthreads();
  }
  const bool poison = s_bad;
  if (poison && tid == 0) set_status(p.status, SPEC_DEV_BAD_SLOT);
  const float inv = sum > 0.f ? p.scale_v / sum : sum;
  for (int k = 0; k < 2; ++k)
    if (tid + k * ATT < p.D) out[tid + k * ATT] = (DT)(poison ? quiet_nan() : acc[k] * inv);
  if (tid == 0 && p.lse)
    p.lse[(size_t)row * p.Hq + hq] = poison ? quiet_nan() : sum == 0.f ? -INFINITY : m + logf(sum);
}

size_t cache_attention_workspace_bytes(int Hq, int Hkv, int D) { return 256; }

cudaError_t launch_cache_attention(const spec_cache_attention_args& a, int sms, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  AttnParams p{a.B, a.T, a.Hq, a.Hkv, a.D, a.page_size, a.page_size / CACHE_BLOCK, a.num_pages, a.table_stride,
               a.mask_words, a.q, a.q_row_stride, a.q_head_stride, a.cache, a.block_table, a.kv_len, a.row_ptr,
               a.tree_mask, a.softmax_scale * a.k_scale, a.v_scale, a.out, a.lse, a.dev_status};
  const dim3 grid(a.T, a.Hq);
  if (a.dtype == SPEC_BF16) cache_attention_kernel<bf16><<<grid, ATT, 0, st>>>(p);
  else cache_attention_kernel<float><<<grid, ATT, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace spec
