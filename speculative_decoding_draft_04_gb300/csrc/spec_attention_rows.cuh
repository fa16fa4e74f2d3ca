// The kernels of the attention over the 4-bit cache for requests of few new rows, and
// the choice among them and the 128-row tiles; see spec_attention.cu.
#pragma once

#include <atomic>

#include "spec_attention_tc.cuh"

namespace spec {

// A query row of this lane: its D / 4 elements of the order above, and what they
// are multiplied by.  Rows are scaled by powers of two so that their largest
// element is in [2^14, 2^15), which makes bf16 queries exact in 16-bit floats
// (elements 2^38 below their row's largest aside); c is what the scores are
// multiplied by in turn.
template <int D, class DT>
struct QueryRow {
  const DT* src;
  float f, c;
  bool live;
  __device__ __forceinline__ QueryRow(const AttnParams& p, const AttnSeg& sg, int r, int t) {
    live = r < sg.n * p.G;
    const int i = live ? r / p.G : 0, hq = sg.h * p.G + (live ? r - i * p.G : 0);
    src = static_cast<const DT*>(p.q) + (long long)(sg.r0 + i) * p.q_row + hq * p.q_head;
    float mx = 0.f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      float x[4];
      load4(src + k_order<D>(t, s), x);
      mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x[0]), fabsf(x[1]))), fmaxf(fabsf(x[2]), fabsf(x[3])));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int ex = query_exponent(mx);
    const float up = power_of_2(ex);
    f = p.scale < 0.f ? -up : up;
    c = fabsf(p.scale) * power_of_2(-ex);
    if (!(c > 0.f)) {                                    // scores of 0
      f = 0.f;
      c = 1.f;
    }
  }
  // Four elements of inner step s in NT 16-bit terms.
  template <int NT>
  __device__ __forceinline__ void terms(int t, int s, uint2 (&a)[NT]) const {
    float x[4];
    load4(src + k_order<D>(t, s), x);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = live ? x[k] * f : 0.f;
#pragma unroll
    for (int term = 0; term < NT; ++term) {
      a[term] = make_uint2(pack_h2(x[0], x[1]), pack_h2(x[2], x[3]));
      const float2 lo = half2_floats(a[term].x), hi = half2_floats(a[term].y);
      x[0] -= lo.x; x[1] -= lo.y; x[2] -= hi.x; x[3] -= hi.y;
    }
  }
};

// Codes and scales of a unit's K, four tokens a lane: tokens (g / 2) + 4 (g % 2)
// + 8 j of the two blocks, the D / 4 elements of part t.
template <class C>
__device__ __forceinline__ void load_k(const uint8_t* unit, int g, int t, uint32_t (&kc)[4][C::KW], uint32_t (&ks)[4][C::KG]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int tok = (g >> 1) + 4 * (g & 1) + 8 * (j & 1);
    const uint8_t* blk = unit + (j >> 1) * (18 * C::D);
    const uint8_t* row = blk + tok * (C::D / 2);
    if (C::D == 64) {
      const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * t);
      kc[j][0] = v.x; kc[j][1] = v.y;
    } else {
#pragma unroll
      for (int h = 0; h < C::D / 128; ++h) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + 64 * h + 16 * t);
        kc[j][4 * h] = v.x; kc[j][4 * h + 1] = v.y; kc[j][4 * h + 2] = v.z; kc[j][4 * h + 3] = v.w;
      }
    }
    const uint8_t* sc = blk + cache_k_scales(C::D) + tok * (C::D / 16);
    if (C::D == 64) {
      const uint32_t two = decode_scales(sc[t]);
      ks[j][0] = __byte_perm(two, two, 0x1010);
    } else {
#pragma unroll
      for (int h = 0; h < C::D / 128; ++h) {
        const uint32_t two = decode_scales(*reinterpret_cast<const uint16_t*>(sc + 8 * h + 2 * t));
        ks[j][2 * h] = __byte_perm(two, two, 0x1010);
        ks[j][2 * h + 1] = __byte_perm(two, two, 0x3232);
      }
    }
  }
}
// Codes and scales of a block's V, D / 8 elements (from D / 8 g on) of four tokens
// a lane.  tokens t and t + 4 in one word, t + 8 and t + 12 in the other: the
// even elements' codes side by side in `even`, the odd ones' in `odd`
template <class C>
__device__ __forceinline__ void load_v(const uint8_t* blk, int g, int t, uint32_t (&even)[2][C::VW], uint32_t (&odd)[2][C::VW],
                                       uint32_t (&vs)[2][2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t a[C::VW], b[C::VW], sa, sb;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int tok = t + 8 * i + 4 * e;
      const uint8_t* row = blk + cache_v_codes(C::D) + tok * (C::D / 2) + g * (C::D / 16);
      uint32_t* w = e ? b : a;
      if (C::D == 64) {
        w[0] = *reinterpret_cast<const uint32_t*>(row);
      } else if (C::D == 128) {
        const uint2 v = *reinterpret_cast<const uint2*>(row);
        w[0] = v.x; w[C::VW - 1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(row);
        w[0] = v.x; w[1 % C::VW] = v.y; w[2 % C::VW] = v.z; w[3 % C::VW] = v.w;
      }
      const uint8_t* sc = blk + cache_v_scales(C::D) + tok * (C::D / 16);
      uint32_t two = C::D == 256 ? *reinterpret_cast<const uint16_t*>(sc + 2 * g)
                                 : (uint32_t)sc[C::D == 128 ? g : g >> 1];
      if (e) sb = two; else sa = two;
    }
    vs[i][0] = decode_scales(__byte_perm(sa, sb, 0x0040));
    vs[i][1] = C::D == 256 ? decode_scales(__byte_perm(sa, sb, 0x0051)) : vs[i][0];
#pragma unroll
    for (int w = 0; w < C::VW; ++w) {
      even[i][w] = (a[w] & 0x0f0f0f0fu) | ((b[w] << 4) & 0xf0f0f0f0u);
      odd[i][w] = ((a[w] >> 4) & 0x0f0f0f0fu) | (b[w] & 0xf0f0f0f0u);
    }
  }
}
// Bytes of tokens that nobody wrote: V scales of 0 (after the last read of K's).
template <class C>
__device__ __forceinline__ void clear_unwritten(const uint8_t* unit, int tok0, int L, int lane) {
  if (tok0 + lane >= L) {
    uint8_t* sc = const_cast<uint8_t*>(unit) + (lane >> 4) * (18 * C::D) + cache_v_scales(C::D) + (lane & 15) * (C::D / 16);
#pragma unroll
    for (int i = 0; i < C::D / 64; ++i) reinterpret_cast<uint32_t*>(sc)[i] = 0;
  }
  fence_async_shared();                                  // before the stage's next copy
  __syncwarp();
}
// Whether a row sees token tok (>= ctx: a new one).  lim: tokens that it sees
// (causal) or its packed row (tree mask); -1 where there is no row.
__device__ __forceinline__ bool sees(const AttnParams& p, int tok, int lim, int ctx, int L) {
  if (!p.mask) return tok < lim;
  const int d = tok - ctx;
  if (lim < 0 || tok >= L) return false;
  return d < 0 || ((d >> 5) < p.mask_words && ((__ldg(p.mask + (size_t)lim * p.mask_words + (d >> 5)) >> (d & 31)) & 1u));
}

// The tensor cores cut what their sums leave behind 32 bits instead of rounding it: over
// the units of a long part that takes 1e-6 to 3e-6 of the outputs.  For 32-bit storage
// the passes with prefixes therefore form each product of two terms by itself and add it
// with rounding (64 requests of 4 rows behind 16384 tokens: 1.6e-6 of the outputs before, 8e-7 now).
__device__ __forceinline__ void add_fresh(float* sum, const uint4& small, const uint4& large, uint32_t b0, uint32_t b1) {
  float t[4];
  mma_f16_first(t, small, b0, b1);
  mma_f16(t, large, b0, b1);
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] += t[e];
}

// Products with query rows along the operands' 16 rows: M tiles of 16.
template <int PASS_, int D_, int M_, int NT_>
struct RowTiles {
  using C = RowTiles;
  static constexpr bool FRESH = NT_ == 2 && PASS_ != PASS_PLAIN;
  static_assert(PASS_ != PASS_PREFIX || D_ == 256 || NT_ == 2, "bf16 rows of groups: 8-row or 128-row tiles");
  static constexpr int PASS = PASS_, D = D_, M = M_, NT = NT_, ROWS = 16 * M;
  static constexpr int KSTEPS = D / 16, KW = D / 32, KG = D / 64, NV = D / 8, VW = D >= 128 ? D / 64 : 1;
  static constexpr int Q_BYTES = NT * ROWS * KSTEPS * 32;
  // 12 warps of 168 registers where 8 of 255 are not needed; two CTAs of 8 for small heads
  static constexpr int MIN_CTAS = M == 1 && NT == 1 && D == 64 ? 2 : 1;
  static constexpr int WARPS = D == 256 && NT == 2 ? 4 : D == 128 && M == 1 && NT == 1 ? 12 : 8;
  float c[2 * M], mref[2 * M], O[M][NV][4], l[2 * M];    // l: this lane's tokens
  int lim[2 * M];
  bool upper;                                            // rows 8 .. of the tile exist

  template <class DT>
  __device__ __forceinline__ void begin(const AttnParams& p, const AttnSeg& sg, uint4* s_q, int lane) {
    const int g = lane >> 2, t = lane & 3, rows = sg.n * p.G;
    upper = M > 1 || rows - sg.tile * ROWS > 8;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const QueryRow<D, DT> lo(p, sg, sg.tile * ROWS + 16 * m + g, t), hi(p, sg, sg.tile * ROWS + 16 * m + 8 + g, t);
      c[2 * m] = lo.c;
      c[2 * m + 1] = hi.c;
#pragma unroll
      for (int s = 0; s < KSTEPS; ++s) {
        uint2 a[NT], b[NT];
        lo.terms(t, s, a);
        hi.terms(t, s, b);
#pragma unroll
        for (int term = 0; term < NT; ++term)
          s_q[((term * M + m) * KSTEPS + s) * 32 + lane] = make_uint4(a[term].x, b[term].x, a[term].y, b[term].y);
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2 * M; ++i) {
      mref[i] = -INFINITY;
      l[i] = 0.f;
      const int r = sg.tile * ROWS + 16 * (i >> 1) + 8 * (i & 1) + g;
      lim[i] = r < rows ? (PASS == PASS_PREFIX ? sg.L : p.mask ? sg.r0 + r / p.G : sg.L - sg.n + r / p.G + 1) : -1;
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) O[m][j][k] = 0.f;
  }

  __device__ __forceinline__ void pass(const AttnParams& p, const AttnSeg& sg, const uint4* s_q, const uint8_t* unit, int u,
                                       int lane) {
    const int g = lane >> 2, t = lane & 3;
    // ---- first product: scores of 4 x 8 tokens
    float S[M][4][4];
    uint32_t kc[4][KW], ks[4][KG];
    load_k<C>(unit, g, t, kc, ks);
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      uint4 a[NT][M];
#pragma unroll
      for (int term = 0; term < NT; ++term)
#pragma unroll
        for (int m = 0; m < M; ++m) a[term][m] = s_q[((term * M + m) * KSTEPS + s) * 32 + lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b0 = mul_h2(decode_byte(kc[j], 2 * s), ks[j][s >> 2]);
        const uint32_t b1 = mul_h2(decode_byte(kc[j], 2 * s + 1), ks[j][s >> 2]);
#pragma unroll
        for (int term = 0; term < NT; ++term)
#pragma unroll
          for (int m = 0; m < M; ++m) {
            if (s == 0 && term == 0) mma_f16_first(S[m][j], a[term][m], b0, b1);
            else mma_f16(S[m][j], a[term][m], b0, b1);
          }
      }
    }
    // ---- masks, where the unit reaches the new tokens
    const int tok0 = u * AT_UNIT, ctx = sg.template context<PASS>();
    if (tok0 + AT_UNIT > ctx) {
      clear_unwritten<C>(unit, tok0, sg.L, lane);
#pragma unroll
      for (int i = 0; i < 2 * M; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!sees(p, tok0 + 16 * (j >> 1) + 8 * (j & 1) + t + 4 * e, lim[i], ctx, sg.L))
              S[i >> 1][j][2 * (i & 1) + e] = -INFINITY;
    }
    // ---- probabilities
    float top[2 * M];
    bool far = false;
#pragma unroll
    for (int i = 0; i < 2 * M; ++i) {
      const int m = i >> 1, e = 2 * (i & 1);
      float x = fmaxf(S[m][0][e], S[m][0][e + 1]);
#pragma unroll
      for (int j = 1; j < 4; ++j) x = max3(x, S[m][j][e], S[m][j][e + 1]);
      top[i] = x;
      far |= c[i] * (x - mref[i]) > AT_SLACK;
    }
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
      for (int i = 0; i < 2 * M; ++i) {
        float x = top[i];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        x = fmaxf(x, mref[i]);
        const float f = x == mref[i] ? 1.f : exp2_approx(c[i] * (mref[i] - x));
        mref[i] = x;
        const int m = i >> 1, e = 2 * (i & 1);
        l[i] *= f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          O[m][j][e] *= f;
          O[m][j][e + 1] *= f;
        }
      }
    }
    uint4 pa[NT][M][2];
#pragma unroll
    for (int i = 0; i < 2 * M; ++i) {
      const int m = i >> 1, e = 2 * (i & 1);
      if (i == 1 && !upper) {
#pragma unroll
        for (int j = 0; j < 4; ++j) S[m][j][e] = S[m][j][e + 1] = 0.f;
        continue;
      }
      const float base = mref[i] == -INFINITY ? 0.f : AT_SHIFT - c[i] * mref[i];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          S[m][j][e + k] = exp2_approx(fmaf(S[m][j][e + k], c[i], base));
          sum += S[m][j][e + k];
        }
      l[i] += sum;
    }
#pragma unroll
    for (int term = 0; term < NT; ++term)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint4 a;
          a.x = pack_h2(S[m][2 * k][0], S[m][2 * k][1]);
          a.y = pack_h2(S[m][2 * k][2], S[m][2 * k][3]);
          a.z = pack_h2(S[m][2 * k + 1][0], S[m][2 * k + 1][1]);
          a.w = pack_h2(S[m][2 * k + 1][2], S[m][2 * k + 1][3]);
          pa[term][m][k] = a;
          if (term + 1 < NT) {
            const uint32_t h[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 v = half2_floats(h[q]);
              S[m][2 * k + (q >> 1)][2 * (q & 1)] -= v.x;
              S[m][2 * k + (q >> 1)][2 * (q & 1) + 1] -= v.y;
            }
          }
        }
    // ---- second product, 16 tokens a step
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t even[2][VW], odd[2][VW], vs[2][2];
      load_v<C>(unit + k * (18 * D), g, t, even, odd, vs);
#pragma unroll
      for (int jj = 0; jj < NV / 2; ++jj) {
        const int sg2 = C::D == 256 ? jj >> 3 : 0;
        const uint32_t b0 = mul_h2(decode_byte(even[0], jj), vs[0][sg2]), b1 = mul_h2(decode_byte(even[1], jj), vs[1][sg2]);
        const uint32_t d0 = mul_h2(decode_byte(odd[0], jj), vs[0][sg2]), d1 = mul_h2(decode_byte(odd[1], jj), vs[1][sg2]);
        if (FRESH) {
#pragma unroll
          for (int m = 0; m < M; ++m) {
            add_fresh(O[m][2 * jj], pa[NT - 1][m][k], pa[0][m][k], b0, b1);
            add_fresh(O[m][2 * jj + 1], pa[NT - 1][m][k], pa[0][m][k], d0, d1);
          }
        } else {
#pragma unroll
          for (int term = 0; term < NT; ++term)
#pragma unroll
            for (int m = 0; m < M; ++m) {
              mma_f16(O[m][2 * jj], pa[term][m][k], b0, b1);
              mma_f16(O[m][2 * jj + 1], pa[term][m][k], d0, d1);
            }
        }
      }
    }
  }

  // The lanes' sums added up.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < 2 * M; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
  }
  // Sums i, 0 .. 2 M - 1: their row in the tile; four elements at a time of the
  // lane's part of it; and whether the lane writes (m, sum).
  static constexpr int SUMS = 2 * M, QUADS = NV / 2;
  __device__ __forceinline__ static int row(int i, int lane) { return 16 * (i >> 1) + 8 * (i & 1) + (lane >> 2); }
  __device__ __forceinline__ static int column(int q, int lane) {
    return (2 * (lane & 3) + q / (NV / 4)) * NV + 4 * (q % (NV / 4));
  }
  __device__ __forceinline__ void quad(int i, int q, float (&x)[4]) const {
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = O[i >> 1][4 * (q % (NV / 4)) + v][2 * (i & 1) + q / (NV / 4)];
  }
  __device__ __forceinline__ static bool first(int lane) { return (lane & 3) == 0; }
};

// Products with tokens (first) and head elements (second) along the operands' 16
// rows and 8 query rows along their columns, for tiles of no more rows: half the
// products and half the softmax of a 16-row tile.  The first product's result
// becomes the second's operand by transposing 8x8 tiles of it.
template <int PASS_, int D_, int NT_>
struct ColumnTile {
  using C = ColumnTile;
  static constexpr bool FRESH = NT_ == 2 && PASS_ != PASS_PLAIN;
  static constexpr int PASS = PASS_, D = D_, NT = NT_, ROWS = 8;
  static constexpr int KSTEPS = D / 16, KW = D / 32, KG = D / 64, NV = D / 8, VW = D >= 128 ? D / 64 : 1;
  static constexpr int Q_BYTES = NT * ROWS * KSTEPS * 32;
  static constexpr int MIN_CTAS = NT == 1 && D == 64 ? 2 : 1;
  static constexpr int WARPS = D == 128 && NT == 1 ? 12 : 8;
  float c[2], mref[2], O[NV / 2][4], l[2];               // rows 2 t and 2 t + 1; l: this lane's tokens
  int lim[2];

  template <class DT>
  __device__ __forceinline__ void begin(const AttnParams& p, const AttnSeg& sg, uint4* s_q, int lane) {
    const int g = lane >> 2, t = lane & 3, rows = sg.n * p.G;
    const QueryRow<D, DT> q(p, sg, sg.tile * ROWS + g, t);
#pragma unroll
    for (int s = 0; s < KSTEPS; s += 2) {
      uint2 a[NT], b[NT];
      q.terms(t, s, a);
      q.terms(t, s + 1, b);
#pragma unroll
      for (int term = 0; term < NT; ++term)
        s_q[(term * (KSTEPS / 2) + s / 2) * 32 + lane] = make_uint4(a[term].x, a[term].y, b[term].x, b[term].y);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = __shfl_sync(0xffffffffu, q.c, 8 * t + 4 * i);
      mref[i] = -INFINITY;
      l[i] = 0.f;
      const int r = sg.tile * ROWS + 2 * t + i;
      lim[i] = r < rows ? (PASS == PASS_PREFIX ? sg.L : p.mask ? sg.r0 + r / p.G : sg.L - sg.n + r / p.G + 1) : -1;
    }
#pragma unroll
    for (int j = 0; j < NV / 2; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) O[j][k] = 0.f;
  }

  __device__ __forceinline__ void pass(const AttnParams& p, const AttnSeg& sg, const uint4* s_q, const uint8_t* unit, int u,
                                       int lane) {
    const int g = lane >> 2, t = lane & 3;
    // ---- first product: scores of 2 x 16 tokens
    float S[2][4];
    uint32_t kc[4][KW], ks[4][KG];
    load_k<C>(unit, g, t, kc, ks);
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      uint4 a[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i].x = mul_h2(decode_byte(kc[2 * i], 2 * s), ks[2 * i][s >> 2]);
        a[i].y = mul_h2(decode_byte(kc[2 * i + 1], 2 * s), ks[2 * i + 1][s >> 2]);
        a[i].z = mul_h2(decode_byte(kc[2 * i], 2 * s + 1), ks[2 * i][s >> 2]);
        a[i].w = mul_h2(decode_byte(kc[2 * i + 1], 2 * s + 1), ks[2 * i + 1][s >> 2]);
      }
#pragma unroll
      for (int term = 0; term < NT; ++term) {
        const uint2 b = reinterpret_cast<const uint2*>(s_q)[((term * (KSTEPS / 2) + s / 2) * 32 + lane) * 2 + (s & 1)];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (s == 0 && term == 0) mma_f16_first(S[i], a[i], b.x, b.y);
          else mma_f16(S[i], a[i], b.x, b.y);
        }
      }
    }
    // ---- masks, where the unit reaches the new tokens
    const int tok0 = u * AT_UNIT, ctx = sg.template context<PASS>();
    if (tok0 + AT_UNIT > ctx) {
      clear_unwritten<C>(unit, tok0, sg.L, lane);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!sees(p, tok0 + 16 * i + 8 * e + (g >> 1) + 4 * (g & 1), lim[r], ctx, sg.L)) S[i][2 * e + r] = -INFINITY;
    }
    // ---- probabilities
    float top[2];
    bool far = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = max3(fmaxf(S[0][r], S[0][r + 2]), S[1][r], S[1][r + 2]);
      far |= c[r] * (top[r] - mref[r]) > AT_SLACK;
    }
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = top[r];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        x = fmaxf(x, mref[r]);
        const float f = x == mref[r] ? 1.f : exp2_approx(c[r] * (mref[r] - x));
        mref[r] = x;
        l[r] *= f;
#pragma unroll
        for (int j = 0; j < NV / 2; ++j) {
          O[j][r] *= f;
          O[j][r + 2] *= f;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float base = mref[r] == -INFINITY ? 0.f : AT_SHIFT - c[r] * mref[r];
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          S[i][r + 2 * k] = exp2_approx(fmaf(S[i][r + 2 * k], c[r], base));
          sum += S[i][r + 2 * k];
        }
      l[r] += sum;
    }
    uint32_t pb[NT][2][2];
#pragma unroll
    for (int term = 0; term < NT; ++term)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t h = pack_h2(S[i][2 * k], S[i][2 * k + 1]);
          pb[term][i][k] = transpose8(h);
          if (term + 1 < NT) {
            const float2 v = half2_floats(h);
            S[i][2 * k] -= v.x;
            S[i][2 * k + 1] -= v.y;
          }
        }
    // ---- second product, 16 tokens a step
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t even[2][VW], odd[2][VW], vs[2][2];
      load_v<C>(unit + k * (18 * D), g, t, even, odd, vs);
#pragma unroll
      for (int jj = 0; jj < NV / 2; ++jj) {
        const int sg2 = D == 256 ? jj >> 3 : 0;
        uint4 a;
        a.x = mul_h2(decode_byte(even[0], jj), vs[0][sg2]);
        a.y = mul_h2(decode_byte(odd[0], jj), vs[0][sg2]);
        a.z = mul_h2(decode_byte(even[1], jj), vs[1][sg2]);
        a.w = mul_h2(decode_byte(odd[1], jj), vs[1][sg2]);
        if (FRESH) {
          float t[4];
          mma_f16_first(t, a, pb[NT - 1][k][0], pb[NT - 1][k][1]);
          mma_f16(t, a, pb[0][k][0], pb[0][k][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) O[jj][e] += t[e];
        } else {
#pragma unroll
          for (int term = 0; term < NT; ++term) mma_f16(O[jj], a, pb[term][k][0], pb[term][k][1]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  }
  static constexpr int SUMS = 2, QUADS = NV / 4;
  __device__ __forceinline__ static int row(int i, int lane) { return 2 * (lane & 3) + i; }
  __device__ __forceinline__ static int column(int q, int lane) { return (lane >> 2) * NV + 4 * q; }
  __device__ __forceinline__ void quad(int i, int q, float (&x)[4]) const {
#pragma unroll
    for (int v = 0; v < 4; ++v) x[v] = O[2 * q + (v >> 1)][i + 2 * (v & 1)];
  }
  __device__ __forceinline__ static bool first(int lane) { return lane < 4; }
};

// Shared memory of a kernel, and the floats of a part: [ROWS][D] outputs, then
// (m, sum) a row.
template <class C>
struct AttnCfg {
  static constexpr int UNIT_BYTES = 2 * 18 * C::D;
  static constexpr int WARP_BUDGET = (C::MIN_CTAS == 2 ? 110 : 220) * 1024 / C::WARPS;
  static constexpr int FIT = (WARP_BUDGET - C::Q_BYTES) / UNIT_BYTES;
  static constexpr int DEPTH = FIT > 6 ? 6 : FIT;
  static constexpr int WARP_BYTES = C::Q_BYTES + DEPTH * UNIT_BYTES;
  static constexpr int SMEM = C::WARPS * WARP_BYTES;
  static constexpr int PART = C::ROWS * C::D + 2 * C::ROWS;
  static_assert(DEPTH >= 2, "ring");
};

template <class C, class DT>
__global__ void __launch_bounds__(32 * C::WARPS, C::MIN_CTAS) cache_attention_kernel(const __grid_constant__ AttnParams p) {
  using F = AttnCfg<C>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_bar[C::WARPS][F::DEPTH];
  __shared__ long long s_pre[32 * C::WARPS + 1];         // units before each group of requests
  __shared__ long long s_scan[C::WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bar = s_bar[warp];

  if (lane < F::DEPTH) mbar_init(bar + lane, 1);
  const long long total = attn_prefix<C::PASS, C::ROWS, AT_UNIT, 32 * C::WARPS>(p, s_pre, s_scan, [] { __syncthreads(); });
  __syncthreads();
  if (C::PASS == PASS_OWN) asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  const int workers = gridDim.x * C::WARPS, me = warp * gridDim.x + blockIdx.x;
  const long long share = (total + workers - 1) / workers;
  const long long begin = me * share;
  const long long end = begin + share < total ? begin + share : total;
  float* parts = attn_parts(p);
  AttnSplit* splits = static_cast<AttnSplit*>(p.ws);
  AttnSplit split{0, -1, 0, 0, 0, 0, 0};
  uint8_t* ring = smem + warp * F::WARP_BYTES;
  uint4* s_q = reinterpret_cast<uint4*>(ring + F::DEPTH * F::UNIT_BYTES);

  if (begin < end) {
    auto locate = [&](long long at) { return attn_locate<C::PASS, C::ROWS, AT_UNIT, 32 * C::WARPS>(p, s_pre, at); };
    auto following = [&](const AttnSeg& s, long long at) {
      return attn_next<C::PASS, C::ROWS, AT_UNIT, 32 * C::WARPS>(p, s_pre, s, at);
    };
    const int bpp = p.P / CACHE_BLOCK, page_bits = 31 - __clz(p.P);
    const size_t head_bytes = (size_t)bpp * cache_block_bytes(C::D);

    // ---- producer: copies of the units ahead.  `run` units from src on lie in
    // one page, one segment and this share; the next page's id is read a page
    // ahead.  A bad page is replaced by page 0 here and found by the consumer.
    AttnSeg ps = locate(begin);
    long long ppos = begin;
    int istage = 0, run = 0;
    const bool big = p.P >= AT_UNIT;
    const uint8_t* src = nullptr;
    bool second = true;                                  // 16-token pages: the unit has a second one
    auto page_id = [&](int tok) {                        // of the page that holds token tok of ps (-1: none)
      return !ps.bad && tok < ps.L ? __ldg(p.table + (size_t)ps.b * p.stride + (tok >> page_bits)) : -1;
    };
    int next = page_id(ps.u * AT_UNIT + (big ? 0 : (lane & 1) * CACHE_BLOCK));
    auto refill = [&]() {
      if (ps.u >= ps.nu) {
        ps = following(ps, ppos);
        next = page_id(ps.u * AT_UNIT + (big ? 0 : (lane & 1) * CACHE_BLOCK));
      }
      const int tok = ps.u * AT_UNIT;
      const int page = next >= 0 && next < p.num_pages ? next : 0;
      src = p.cache + ((size_t)page * p.Hkv + ps.h) * head_bytes;
      if (big) {
        const int in_page = (tok & (p.P - 1)) / AT_UNIT, left = p.P / AT_UNIT - in_page;
        src += (size_t)in_page * F::UNIT_BYTES;
        run = min(min(left, ps.nu - ps.u), end - ppos < left ? (int)(end - ppos) : left);
        next = page_id(tok + left * AT_UNIT);
      } else {
        run = 1;
        second = tok + CACHE_BLOCK < ps.L;
        next = page_id(tok + AT_UNIT + (lane & 1) * CACHE_BLOCK);
      }
    };
    auto issue = [&]() {
      if (run == 0) refill();
      uint64_t* ibar = bar + istage;
      uint8_t* dst = ring + istage * F::UNIT_BYTES;
      if (big) {
        if (lane == 0) {
          expect_bytes(ibar, F::UNIT_BYTES);
          bulk_load(dst, src, F::UNIT_BYTES, ibar);
        }
        src += F::UNIT_BYTES;
      } else {
        if (lane == 0) expect_bytes(ibar, second ? F::UNIT_BYTES : F::UNIT_BYTES / 2);
        __syncwarp();
        if (lane == 0 || (lane == 1 && second))
          bulk_load(dst + lane * (F::UNIT_BYTES / 2), src, F::UNIT_BYTES / 2, ibar);
      }
      if (++istage == F::DEPTH) istage = 0;
      --run;
      ++ps.u;
      ++ppos;
    };
    for (int i = 0; i < F::DEPTH && ppos < end; ++i) issue();
    int cstage = 0;
    uint32_t cphase = 0;
    bool timed_out = false;

    long long pos = begin;
    AttnSeg next_sg = locate(begin);
    while (pos < end) {
      const AttnSeg sg = next_sg;
      const int u_first = sg.u;
      const int u_end = sg.nu - sg.u < end - pos ? sg.nu : sg.u + (int)(end - pos);
      const int rows = sg.n * p.G;
      C tile;
      tile.template begin<DT>(p, sg, s_q, lane);
      // a page outside the cache in this part, or copies that never came: the
      // share's rows are NaN from there on
      bool poison = sg.bad || timed_out;
      if (!poison) {
        const int tok_end = min(sg.L, u_end * AT_UNIT);
        bool bad = false;
        for (int pg = (u_first * AT_UNIT >> page_bits) + lane; pg << page_bits < tok_end; pg += 32) {
          const int id = __ldg(p.table + (size_t)sg.b * p.stride + pg);
          bad |= id < 0 || id >= p.num_pages;
        }
        poison = __any_sync(0xffffffffu, bad);
        if (poison && lane == 0) set_status(p.status, SPEC_DEV_BAD_SLOT);
      }

      for (int u = u_first; u < u_end && !timed_out; ++u) {
        if (!bar_wait(bar + cstage, cphase)) timed_out = true;
        timed_out = __any_sync(0xffffffffu, timed_out);
        if (timed_out) {
          if (lane == 0) set_status(p.status, SPEC_DEV_TIMEOUT);
          poison = true;
          break;
        }
        tile.pass(p, sg, s_q, ring + cstage * F::UNIT_BYTES, u, lane);
        if (++cstage == F::DEPTH) {
          cstage = 0;
          cphase ^= 1u;
        }
        __syncwarp();                                    // all lanes have read the stage
        if (ppos < end) issue();
      }

      // ---- the segment's end in this share
      const bool whole = u_first == 0 && u_end == sg.nu;
      tile.finish();
      const int slot = u_first == 0 ? 1 : 0;             // 0: the segment began before this share
      float* part = parts + (size_t)(2 * me + slot) * F::PART;
#pragma unroll
      for (int i = 0; i < C::SUMS; ++i) {
        const int rl = C::row(i, lane), r = sg.tile * C::ROWS + rl;
        if (r >= rows) continue;
        const float sum = poison ? quiet_nan() : tile.l[i];
        const float m = tile.mref[i] == -INFINITY ? -INFINITY : tile.c[i] * tile.mref[i] - AT_SHIFT;
        if (whole) {
          const int tok = r / p.G, hq = sg.h * p.G + r - tok * p.G;
          const size_t at = (size_t)(sg.r0 + tok) * p.Hq + hq;
          if (C::PASS == PASS_PREFIX) {
#pragma unroll
            for (int q = 0; q < C::QUADS; ++q) {
              float x[4];
              tile.quad(i, q, x);
              store4(p.raw + at * C::D + C::column(q, lane), x);
            }
            if (C::first(lane)) p.raw_ml[at] = make_float2(m, sum);
            continue;
          }
          float4 before[C::QUADS];                       // the prefix's sums, requested before the first store
          if (C::PASS == PASS_OWN)
#pragma unroll
            for (int q = 0; q < C::QUADS; ++q)
              before[q] = __ldcg(reinterpret_cast<const float4*>(p.prefix + at * C::D + C::column(q, lane)));
          const AttnRow f = attn_row<C::PASS>(p, at, m, sum);
#pragma unroll
          for (int q = 0; q < C::QUADS; ++q) {
            float x[4];
            tile.quad(i, q, x);
#pragma unroll
            for (int v = 0; v < 4; ++v) x[v] *= f.own;
            if (C::PASS == PASS_OWN) add_prefix4(before[q], f.prefix, x);
            store4(static_cast<DT*>(p.out) + at * C::D + C::column(q, lane), x);
          }
          if (C::first(lane) && p.lse) p.lse[at] = f.lse;
        } else {
#pragma unroll
          for (int q = 0; q < C::QUADS; ++q) {
            float x[4];
            tile.quad(i, q, x);
            store4(part + rl * C::D + C::column(q, lane), x);
          }
          if (C::first(lane)) *reinterpret_cast<float2*>(part + C::ROWS * C::D + 2 * rl) = make_float2(m, sum);
        }
      }
      if (!whole) {
        if (slot == 1) {
          const long long seg_last = pos + (sg.nu - 1);  // the segment's last unit
          split = AttnSplit{me, (int)(seg_last / share), sg.b, sg.h, sg.tile, sg.n, sg.r0};
        }
      }
      pos += u_end - u_first;
      if (pos < end) next_sg = following(sg, pos);
    }
    if (timed_out)                                       // leave no copy in flight
      for (int i = 0; i < F::DEPTH; ++i) {
        bar_wait(bar + cstage, cphase);
        if (++cstage == F::DEPTH) {
          cstage = 0;
          cphase ^= 1u;
        }
      }
  }
  if (lane == 0) splits[me] = split;
}

namespace {
template <class C, class DT>
cudaError_t launch_cfg(const AttnParams& p, int sms, cudaStream_t st) {
  using F = AttnCfg<C>;
  static_assert(F::SMEM <= 227 * 1024 - 4096, "shared memory");
  // once a device: the attribute stays with the function
  static std::atomic<uint64_t> sized{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((sized.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(cache_attention_kernel<C, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) sized.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  // one wave at most, and no more warps than there can be units
  long long ctas = (long long)sms * C::MIN_CTAS;
  if (ctas > C::MIN_CTAS * (AT_MAX_CTAS / 2)) ctas = C::MIN_CTAS * (AT_MAX_CTAS / 2);
  const long long tiles = (long long)p.T * p.G / C::ROWS + (p.T < p.B ? p.T : p.B);
  const long long units = tiles * p.Hkv * (((long long)p.stride * p.P + AT_UNIT - 1) / AT_UNIT);
  if (ctas > units) ctas = units;
  e = launch_main<C::PASS>(cache_attention_kernel<C, DT>, p, (int)ctas, 32 * C::WARPS, F::SMEM, st);
  if (e != cudaSuccess) return e;
  return launch_attention_join<C::PASS, C::D, C::ROWS, DT>(p, (int)ctas * C::WARPS, sms, st);
}
}  // namespace

float cache_attention_scale(const spec_cache_attention_args& a);
size_t cache_attention_workspace_bytes(int Hq, int Hkv, int D);

inline AttnParams own_params(const spec_cache_attention_args& a) {
  return AttnParams{a.B, a.T, a.Hq, a.Hkv, a.Hq / a.Hkv, a.page_size, a.num_pages, a.table_stride, a.mask_words, a.q,
                    a.q_row_stride, a.q_head_stride, a.cache, a.block_table, a.kv_len, a.row_ptr, a.tree_mask,
                    cache_attention_scale(a), a.v_scale, a.out, a.lse, a.dev_status, a.workspace};
}

// tc_from: 128-row tiles from more rows a request on (PASS_PREFIX: 8).
template <int PASS>
cudaError_t launch_tiles(const AttnParams& p, int D, int dtype, int tc_from, int sms, cudaStream_t st) {
  // The tile by the mean rows a request (finished requests and rows of no request
  // count in it: the host does not see them).  Times are us a call of these
  // kernels, cold caches, D = 128, 4 query heads a key-value head, all requests of
  // one number of rows: (a) 32 requests of 64 to 4096 tokens, (b) 128 of 64 to
  // 8192, (c) 4 of 50k to 131k; D = 64 orders them nearly alike.
  //   8-row tiles up to 8:  8 rows take (a) 44, (b) 141, (c) 105 in them and 48,
  //     174, 115 in 16-row tiles; 12 rows 56, 250, 158 and 52, 188, 118.  fp32 and
  //     D = 256, 4 rows of 32 requests to 16384 tokens: 77 to 95 and 87 to 149.
  //   32-row tiles from a mean above 24 to 32:  28 rows (b) 304, (c) 169 in one
  //     and 350, 196 in two 16-row tiles.  (a) loses, 82 against 77.  Uniform
  //     requests of 20 rows would gain too (280 against 328, 166 against 191), but
  //     blocks of mixed sizes hardly do (b, 8 to 32 rows: 256 against 268) or lose
  //     (c, 8 to 20 rows: 165 against 131).
  const long long rows = (long long)p.T * p.G;
  const bool few = rows <= 8LL * p.B, wide = rows > 24LL * p.B && rows <= 32LL * p.B;
  if (dtype == SPEC_F32) {
    if (D == 64) return few ? launch_cfg<ColumnTile<PASS, 64, 2>, float>(p, sms, st) : launch_cfg<RowTiles<PASS, 64, 1, 2>, float>(p, sms, st);
    if (D == 128)
      return few ? launch_cfg<ColumnTile<PASS, 128, 2>, float>(p, sms, st) : launch_cfg<RowTiles<PASS, 128, 1, 2>, float>(p, sms, st);
    return few ? launch_cfg<ColumnTile<PASS, 256, 2>, float>(p, sms, st) : launch_cfg<RowTiles<PASS, 256, 1, 2>, float>(p, sms, st);
  }
  //   128-row tiles above 32:  36 rows take (a) 66, (b) 357, (c) 224 in them, 97,
  //     492, 274 in 16-row tiles and 122, 533, 286 in 32-row tiles; 100 rows 75,
  //     379, 235 against 211, 1120, 596.  At 32 rows (b) 347, (c) 219 lose to 305
  //     and 170, and only (a) would gain (64 against 83).
  if (D <= 128 && rows > (long long)tc_from * p.B) return launch_cache_attention_tc<PASS>(p, D, sms, st);
  if constexpr (PASS == PASS_PREFIX) {                       // more rows than 8 went to the 128-row tiles
    if (D == 64) return launch_cfg<ColumnTile<PASS, 64, 1>, bf16>(p, sms, st);
    if (D == 128) return launch_cfg<ColumnTile<PASS, 128, 1>, bf16>(p, sms, st);
  } else {
    if (D == 64)
      return few    ? launch_cfg<ColumnTile<PASS, 64, 1>, bf16>(p, sms, st)
             : wide ? launch_cfg<RowTiles<PASS, 64, 2, 1>, bf16>(p, sms, st)
                    : launch_cfg<RowTiles<PASS, 64, 1, 1>, bf16>(p, sms, st);
    if (D == 128)
      return few    ? launch_cfg<ColumnTile<PASS, 128, 1>, bf16>(p, sms, st)
             : wide ? launch_cfg<RowTiles<PASS, 128, 2, 1>, bf16>(p, sms, st)
                    : launch_cfg<RowTiles<PASS, 128, 1, 1>, bf16>(p, sms, st);
  }
  return few ? launch_cfg<ColumnTile<PASS, 256, 1>, bf16>(p, sms, st) : launch_cfg<RowTiles<PASS, 256, 1, 1>, bf16>(p, sms, st);
}

}  // namespace spec
