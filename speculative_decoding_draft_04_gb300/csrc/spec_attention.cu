// Attention of each request's new tokens over its 4-bit paged cache.
//
//   y_ij = log2(e) softmax_scale k_scale (q_i . k_j),  p_ij = 2^(y_ij - m_i)
//   out_i = v_scale sum_j p_ij v_j / sum_j p_ij,       lse_i = ln 2 (m_i + log2 sum_j p_ij)
//
// with k_j, v_j = code * scale, exact in 16-bit floats.  The query heads of one
// key-value head and the new tokens are the rows of one product: row r of
// request b is new token r / G, query head h G + r % G (G = Hq / Hkv).
//
// Requests of at most 32 rows on average (others: spec_attention_tc.cuh).  The kernels
// are in spec_attention_rows.cuh; spec_prefix.cu launches them for shared prefixes.
//
// cache_attention_kernel: every warp works alone on a run of 32-token units.
// All units of all (request, key-value head, row tile) segments are numbered in
// order, and warp w takes the w-th equal share of them, so ragged lengths are
// balanced to one unit and a long context is split as far as the machine goes.
// A unit of a head is contiguous in the cache (two blocks of 16 tokens, 36 D
// bytes) and comes by bulk copies into the warp's own ring in shared memory; no
// barrier joins the warps.  Codes go from shared memory to the operands of the
// warp's 16x8x16 products in registers: the order of a product's inner index is
// free as long as both operands agree, so each lane takes contiguous bytes --
// of K one run of D/4 elements of one token, of V D/8 elements (one or two
// scales) of four tokens -- and the queries are laid out in that order once a
// segment.  Decoded words fit either operand of a product, so the rows may be its
// 16 rows (RowTiles) or its 8 columns (ColumnTile, tiles of up to 8 rows).  Scores
// stay in registers: the layout of the first product's result is the layout of
// the second product's operand, after a transposition of 8x8 tiles for columns.
//
// The running maximum follows lazily: m is the maximum last taken less 7, and
// the sums are rescaled when a score passes it by 15.  So p stays below 2^15 in
// a 16-bit float, rescaling is rare, and p keeps 11 bits down to 2^-21 of the
// row's largest and an absolute error of 2^-32 of it below that.
// p is rounded to 11 bits (two terms: 22) for the second product only; its sum
// is of the unrounded p, so lse keeps 32-bit precision.
//
// Bound by instructions, not bytes: a token of one head (144 bytes at D = 128)
// costs a warp's pass 22 instructions, 12 of them to decode it, at 2.1 a cycle
// and SM.  One token of 32 requests (306 MB) takes 74 us, 4.1 TB/s of the 6.8 of
// a copy; blocks of 2 to 8 tokens and 4 heads for 128 requests (619 MB) 255 to
// 290 us, by their lengths; the same for 4 requests of 50k to 131k tokens (418 MB)
// 131 to 151 us.  Twelve warps of 168 registers were faster than eight of 255 (by
// 7 % on the blocks when they were chosen).
//
// A segment inside one warp's share is written at once.  Otherwise each part is
// kept as (m, sum, unnormalised out) in the workspace and
// cache_attention_join_kernel adds the parts in the order of their warps.
#include "spec_attention_rows.cuh"

namespace spec {

size_t cache_attention_workspace_bytes(int Hq, int Hkv, int D) {
  const size_t rows = D == 256 ? 16 : 32;
  const size_t part = (rows * D + 2 * rows) * sizeof(float);
  // 32-row tiles run one CTA an SM, 16-row tiles two
  const size_t parts = D == 256 ? (size_t)AT_MAX_CTAS : (size_t)AT_MAX_CTAS / 2;
  return (size_t)AT_MAX_CTAS * AT_WARPS * sizeof(AttnSplit) + parts * AT_WARPS * 2 * part + 256;
}

// What scores in codes are multiplied by.
float cache_attention_scale(const spec_cache_attention_args& a) {
  return a.softmax_scale * a.k_scale * 1.4426950408889634f;
}

cudaError_t launch_cache_attention(const spec_cache_attention_args& a, int sms, cudaStream_t st) {
  return launch_tiles<PASS_PLAIN>(own_params(a), a.D, a.dtype, 32, sms, st);
}

}  // namespace spec
