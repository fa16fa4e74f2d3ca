// Attention of requests of which groups share a prefix that is held once.
//
//   out = (sum_prefix 2^(y - m) v + sum_own 2^(y - m) v) / (the same without v)
//
// Two passes of the kernels of spec_attention.cu: the rows of each group over its
// prefix as one request's that see every token, so that a token of it is decoded once
// for 128 rows; then every request's rows over its own tokens, whose end adds the sums
// (unnormalised, 32 bits, with their maximum) that the first pass left.
//
// us a call: trees of 25 nodes of 32 requests behind 32768 tokens 457, nearly all of it
// the first pass: 0.95 PFLOP/s (225 us at the rate of a matrix product), bound as the
// 128-row tiles are by a unit's chain of waits; blocks of 2 to 8 tokens of 128 requests in
// four groups behind up to 8192 tokens 203; one token of 64 requests behind 16384 tokens 79
// (35 and 37 in the two passes, the rest in their joins; 14 us of reading); one token of 4
// requests behind 2000 tokens 23.
#include "spec_attention_rows.cuh"

namespace spec {

// Workspace: that of a pass, a word, the prefixes' sums.
size_t prefix_attention_workspace_bytes(int T, int Hq, int Hkv, int D) {
  return cache_attention_workspace_bytes(Hq, Hkv, D) + 256 + (size_t)T * Hq * (D * sizeof(float) + sizeof(float2));
}

cudaError_t launch_prefix_attention(const spec_prefix_attention_args& a, int sms, cudaStream_t st) {
  const spec_cache_attention_args& o = a.own;
  AttnParams own = own_params(o), shared = own;
  char* ws = static_cast<char*>(o.workspace) + (cache_attention_workspace_bytes(o.Hq, o.Hkv, o.D) + 15) / 16 * 16;
  shared.B = a.groups;
  shared.stride = a.prefix_stride;
  shared.table = a.prefix_table;
  shared.kv_len = a.prefix_len;
  shared.mask = nullptr;
  shared.cut = a.group_ptr;
  shared.members = o.B;
  shared.ranges = reinterpret_cast<int*>(ws);
  shared.raw = reinterpret_cast<float*>(ws + 128);
  shared.raw_ml = reinterpret_cast<float2*>(shared.raw + (size_t)o.T * o.Hq * o.D);
  own.prefix = shared.raw;
  own.prefix_ml = shared.raw_ml;
  own.prefix_ranges = shared.ranges;
  // 128-row tiles, whose segments cost little to begin and end, from 9 rows on: for the
  // prefixes always (4 requests of 4 rows behind 2000 tokens: 34 us a call, 40 with 16-row
  // tiles), for the requests' own tokens where tables have room for few (blocks of 8 to 32
  // rows behind 516 own tokens on average: 212 us, 273 with 16-row tiles; 8 rows and fewer
  // stay with their tiles: one token of 64 requests 99 us, 124 in 128-row tiles).  Tables of
  // more room may hold long contexts; they keep the plain call's border.
  const cudaError_t e = launch_tiles<PASS_PREFIX>(shared, o.D, o.dtype, 8, sms, st);
  if (e != cudaSuccess) return e;
  return launch_tiles<PASS_OWN>(own, o.D, o.dtype, (long long)o.table_stride * o.page_size <= 4096 ? 8 : 32, sms, st);
}

}  // namespace spec
