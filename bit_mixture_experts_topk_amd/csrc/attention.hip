// Attention of a step's queries over the paged 4-bit cache.
//
//   out[t][hq] = sum_p softmax_p(scale * q[t][hq] . k[p]) v[p]
//
// over the positions p the row sees: not past its own, inside its window, on
// a page of the cache; with an optional sink logit per query head in the
// softmax's sum. Keys and values are decoded in registers, the running maximum
// and sum of the softmax make it one pass over the cache (the pages list FP8
// paged decode attention with sliding window, sinks and a custom scale: "MoE
// Training on Consumer GPUs -- Loggetta & Cerin Amroth", Task guides table;
// this is the 4-bit form of it on this library's formats).
//
// Tiling. The query heads that share a cache head, for all new tokens of a
// sequence, are the rows of one problem (row = token * G + g), cut into tiles
// of 16 * NQ rows. A workgroup takes one tile, one cache head and a range of
// positions; its four waves take 32 positions in turn (128 a round) and join
// at the end through LDS. Ranges of one tile are joined by a second kernel.
//
// Registers only, no transposes. v_mfma_f32_16x16x32_bf16 takes A rows from
// lanes 0..15 with 8 consecutive k per lane group g = lane / 16, and leaves C
// with its column in the lane and rows 4g..4g+3 in the registers. Computed are
// S^T = K Q^T (rows = positions, columns = query rows) and O^T = V^T P^T. Row r
// of K tile i (of two) is position 8 (r / 4) + 4 i + r % 4 of the 32, so the
// scores that a lane holds after both tiles are those of positions 8g..8g+7,
// which are just the k indices that it has to supply of P^T: the
// probabilities go from one product to the next without leaving their lane,
// and so does the softmax, whose row is the lane's column.
// The k order of S is free as well: MXFP4 lane group g takes values g D/4 ..
// (g+1) D/4 of the head, so that one load brings its codes and (D = 128) they
// share one scale. V^T rows are columns of the cache, so lane c reads its
// D/16 values of every one of 8 positions and pairs of positions are put
// together after decoding.
#include <algorithm>

#include "kvcache.h"

namespace gnf4 {

constexpr int kAttnThreads = 256;
constexpr int kAttnRound = 128;                 // positions per round of the four waves
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float max_xor16_32(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v), __builtin_bit_cast(unsigned, v),
                                            false, false);
  v = fmaxf(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
  auto q = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v), __builtin_bit_cast(unsigned, v),
                                            false, false);
  return fmaxf(__builtin_bit_cast(float, (unsigned)q[0]), __builtin_bit_cast(float, (unsigned)q[1]));
}

__device__ __forceinline__ float sum_xor16_32(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v), __builtin_bit_cast(unsigned, v),
                                            false, false);
  v = __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
  auto q = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v), __builtin_bit_cast(unsigned, v),
                                            false, false);
  return __builtin_bit_cast(float, (unsigned)q[0]) + __builtin_bit_cast(float, (unsigned)q[1]);
}

__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

__device__ __forceinline__ bf16x8_t op8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, make_uint4(a, b, c, d));
}

// What a row tile sees, from the step's arrays; the same in every kernel.
struct AttnRange {
  int r0, rows;                   // first token row, query rows (tokens * G)
  int start;                      // position of the sequence's first new token
  int q_first, q_last;            // positions of the tile's first and last token
  int lo, hi;                     // positions any of its rows may see, lo on a round's border
};

__device__ __forceinline__ AttnRange attn_range(const KvAttnArgs &a, int b, int row0, int M) {
  const KvView &kv = a.kv;
  AttnRange x;
  const int o0 = kv.offsets[b], o1 = kv.offsets[b + 1], len = kv.lens[b];
  const int e = min(max(o1, 0), kv.n_tokens);
  x.r0 = min(max(o0, 0), e);
  const int n = e - x.r0;
  x.rows = n * a.G;
  x.start = len - n;
  const int last = min(row0 + M, x.rows) - 1;
  x.q_first = x.start + row0 / a.G;
  x.q_last = x.start + (last < 0 ? 0 : last / a.G);
  const int64_t cap = (int64_t)kv.max_pages << kv.page_shift;
  x.hi = (int)min((int64_t)x.q_last + 1, cap);
  x.lo = a.window > 0 ? max(0, x.q_first - a.window + 1) & ~(kAttnRound - 1) : 0;
  if (row0 >= x.rows) x.hi = x.lo;
  return x;
}

// One wave's 32 positions: raw codes and scales in registers.
template <int FMT, int D>
struct AttnTile {
  static constexpr bool MX = FMT == GNF4_MXFP4;
  static constexpr int KW = D / 32;                          // code dwords per lane and K tile
  static constexpr int VW = MX ? (D == 256 ? 2 : 1) : D / 64;  // code pieces per lane and position
  static constexpr int SW = MX ? (D == 256 ? 4 : D / 64) : D / 8 / 4;  // 16-byte pieces of 8 positions' scales
  uint32_t kc[2][KW];
  uint32_t ks[2];                                            // MXFP4: the lane's scale byte(s)
  uint32_t vc[8][VW];
  uint4 ksv[MX ? 1 : SW];                                    // NF4: absmax of positions 8g..8g+7
  uint4 vsv[SW];
  bool bad;                                                  // positions 8g..8g+7 lie on no page
};

template <int FMT, int D>
__device__ __forceinline__ int attn_page(const KvView &kv, int b, int pos) {
  return kv.pages[(int64_t)b * kv.max_pages + min(pos >> kv.page_shift, kv.max_pages - 1)];
}

// Page ids of the wave's tile at position t: the lane's K rows and V rows.
struct AttnPages {
  int k, v;
};

template <int FMT, int D>
__device__ __forceinline__ AttnPages attn_pages(const KvView &kv, int b, int t, int lane) {
  AttnPages p;
  p.k = attn_page<FMT, D>(kv, b, t + ((lane & 15) >> 2) * 8);
  p.v = attn_page<FMT, D>(kv, b, t + (lane >> 4) * 8);
  return p;
}

template <int FMT, int D>
__device__ __forceinline__ void attn_load(AttnTile<FMT, D> &x, const KvView &kv, int h, int t, AttnPages p,
                                          int lane) {
  typedef AttnTile<FMT, D> T;
  const int r = lane & 15, g = lane >> 4, mask = (1 << kv.page_shift) - 1;
  x.bad = (uint32_t)p.v >= (uint32_t)kv.n_pages;
  // an id outside the cache reads page 0 and is masked
  const int pk = (uint32_t)p.k >= (uint32_t)kv.n_pages ? 0 : p.k, pv = x.bad ? 0 : p.v;
  const int kt = t + (r >> 2) * 8 + (r & 3), vt = t + g * 8;
  const int64_t krow = (((int64_t)pk * kv.H + h) << kv.page_shift) + (kt & mask);
  const int64_t vrow = (((int64_t)pv * kv.H + h) << kv.page_shift) + (vt & mask);
  const uint8_t *kp = kv.k_codes + krow * (D / 2), *vp = kv.v_codes + vrow * (D / 2);
  if constexpr (T::MX) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t *s = kp + i * 4 * (D / 2) + g * (D / 8);
      if constexpr (D == 64) {
        const uint2 v = *reinterpret_cast<const uint2 *>(s);
        x.kc[i][0] = v.x;
        x.kc[i][1] = v.y;
      } else {
#pragma unroll
        for (int w = 0; w < T::KW; w += 4) {
          const uint4 v = *reinterpret_cast<const uint4 *>(s + 4 * w);
          x.kc[i][w] = v.x;
          x.kc[i][w + 1] = v.y;
          x.kc[i][w + 2] = v.z;
          x.kc[i][w + 3] = v.w;
        }
      }
      const uint8_t *sc = static_cast<const uint8_t *>(kv.k_scales) + (krow + i * 4) * (D / 32);
      if constexpr (D == 64) x.ks[i] = sc[g >> 1];
      else if constexpr (D == 128) x.ks[i] = sc[g];
      else x.ks[i] = *reinterpret_cast<const uint16_t *>(sc + 2 * g);
    }
    const uint4 *vs = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(kv.v_scales) + vrow * (D / 32));
#pragma unroll
    for (int w = 0; w < T::SW; ++w) x.vsv[w] = vs[w];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t *s = vp + j * (D / 2) + r * (D / 32);
      if constexpr (D == 64) x.vc[j][0] = *reinterpret_cast<const uint16_t *>(s);
      else if constexpr (D == 128) x.vc[j][0] = *reinterpret_cast<const uint32_t *>(s);
      else {
        const uint2 v = *reinterpret_cast<const uint2 *>(s);
        x.vc[j][0] = v.x;
        x.vc[j][1] = v.y;
      }
    }
  } else {
    // block b of 64: lane group g takes values 16 g .. 16 g + 15 of it (K),
    // lane c values 4 c .. 4 c + 3 (V)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        const uint2 v = *reinterpret_cast<const uint2 *>(kp + i * 4 * (D / 2) + b * 32 + g * 8);
        x.kc[i][2 * b] = v.x;
        x.kc[i][2 * b + 1] = v.y;
      }
    const int64_t srow = (((int64_t)pv * kv.H + h) << kv.page_shift) + (vt & mask);
    const uint4 *ks = reinterpret_cast<const uint4 *>(static_cast<const float *>(kv.k_scales) + srow * (D / 64));
    const uint4 *vs = reinterpret_cast<const uint4 *>(static_cast<const float *>(kv.v_scales) + srow * (D / 64));
#pragma unroll
    for (int w = 0; w < T::SW; ++w) {
      x.ksv[w] = ks[w];
      x.vsv[w] = vs[w];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
        x.vc[j][b] = *reinterpret_cast<const uint16_t *>(vp + j * (D / 2) + b * 32 + r * 2);
  }
}

// Word w of an array of 16-byte pieces (indices are compile-time constants).
template <int N>
__device__ __forceinline__ uint32_t word_of(const uint4 (&v)[N], int w) {
  const uint4 &x = v[w >> 2];
  return (w & 3) == 0 ? x.x : (w & 3) == 1 ? x.y : (w & 3) == 2 ? x.z : x.w;
}

// Copies of the NF4 byte table: one per lane of half a wave.
constexpr int kAttnLutCopies = 32;

__device__ __forceinline__ uint32_t nf4_lut32(const uint32_t *lut, uint32_t byte, int lane) {
  return lut[byte * kAttnLutCopies + (lane & 31)];
}

// NQ * 16 query rows of one wave: Q operand, running statistics, O^T.
template <int FMT, int D, int NQ>
struct AttnWave {
  static constexpr bool MX = FMT == GNF4_MXFP4;
  static constexpr bool QLDS = NQ >= 4;
  static constexpr int KS = D / 32, ND = D / 16;
  bf16x8_t q[QLDS ? 1 : NQ][QLDS ? 1 : KS];
  f32x4_t o[NQ][ND];
  float m[NQ], l[NQ];
  int qpos[NQ];                                              // position of the lane's query row
};

// The scales of values j = 0..7 (positions 8g + j) for the lane's V values.
template <int D>
__device__ __forceinline__ uint32_t mx_vscale(const AttnTile<GNF4_MXFP4, D> &x, int j, int c) {
  // position j's D/32 scale bytes start at byte j * D/32 of vsv
  if constexpr (D == 64) return (word_of(x.vsv, j >> 1) >> ((j & 1) * 16 + ((c >> 3) << 3))) & 0xffu;
  else if constexpr (D == 128) return (word_of(x.vsv, j) >> ((c >> 2) << 3)) & 0xffu;
  else {
    const uint32_t w = (c >> 1) < 4 ? word_of(x.vsv, 2 * j) : word_of(x.vsv, 2 * j + 1);
    return (w >> (((c >> 1) & 3) << 3)) & 0xffu;
  }
}

template <int FMT, int D, int NQ, bool MASKED>
__device__ __forceinline__ void attn_tile(AttnWave<FMT, D, NQ> &w, AttnTile<FMT, D> &x, const KvAttnArgs &a,
                                          const uint32_t *lut, const uint4 *qlds, int t, int lane) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  constexpr int KS = D / 32, ND = D / 16;
  const int c = lane & 15, g = lane >> 4;
  float s[NQ][8];
  // ---- scores of positions 8g..8g+7 for the lane's query row
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f32x4_t acc[NQ];
    f32x4_t blk[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) acc[n] = blk[n] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      bf16x8_t ka;
      const uint32_t kw = x.kc[i][k];
      if constexpr (MX) {
        const uint32_t sb = D == 256 ? (k < KS / 2 ? x.ks[i] & 0xffu : x.ks[i] >> 8) : x.ks[i];
        const float sc = e8m0_to_f32(sb);
        ka = op8(fp4_pair<0>(kw, sc), fp4_pair<1>(kw, sc), fp4_pair<2>(kw, sc), fp4_pair<3>(kw, sc));
      } else {
        ka = op8(nf4_lut32(lut, kw & 0xffu, lane), nf4_lut32(lut, (kw >> 8) & 0xffu, lane),
                 nf4_lut32(lut, (kw >> 16) & 0xffu, lane), nf4_lut32(lut, kw >> 24, lane));
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        bf16x8_t qv;
        if constexpr (AttnWave<FMT, D, NQ>::QLDS) qv = __builtin_bit_cast(bf16x8_t, qlds[(n * KS + k) * 64 + lane]);
        else qv = w.q[n][k];
        if constexpr (MX) acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, qv, acc[n], 0, 0, 0);
        else blk[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, qv, blk[n], 0, 0, 0);
      }
      if constexpr (!MX) {
        if (k & 1) {                                         // a block of 64 is complete
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float ab = __builtin_bit_cast(float, word_of(x.ksv, (4 * i + j) * (D / 64) + k / 2)) * kNF4InvScale;
#pragma unroll
            for (int n = 0; n < NQ; ++n) acc[n][j] = fmaf(blk[n][j], ab, acc[n][j]);
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n) blk[n] = f32x4_t{0, 0, 0, 0};
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[n][4 * i + j] = acc[n][j] * a.scale_log2;
  }
  // ---- mask, running maximum, probabilities
  uint32_t see[NQ];
  bf16x8_t pb[MX ? NQ : 1];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if constexpr (MASKED) {
      see[n] = 0;
      const int lo = a.window > 0 ? w.qpos[n] - a.window + 1 : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int pos = t + g * 8 + j;
        const bool ok = pos <= w.qpos[n] && pos >= lo && !x.bad;
        see[n] |= ok ? 1u << j : 0u;
        s[n][j] = ok ? s[n][j] : kNegInf;
      }
    }
    float mx = s[n][0];
#pragma unroll
    for (int j = 1; j < 8; ++j) mx = fmaxf(mx, s[n][j]);
    mx = fmaxf(max_xor16_32(mx), w.m[n]);
    const float ms = mx == kNegInf ? 0.0f : mx;              // nothing seen yet: exp2(-inf - 0) = 0
    const float alpha = __builtin_amdgcn_exp2f(w.m[n] - ms);
    w.m[n] = mx;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[n][j] = __builtin_amdgcn_exp2f(s[n][j] - ms);
      sum += s[n][j];
    }
    w.l[n] = w.l[n] * alpha + sum;
#pragma unroll
    for (int d = 0; d < ND; ++d) w.o[n][d] *= alpha;
    if constexpr (MX)
      pb[n] = op8(pk_bf16(s[n][0], s[n][1]), pk_bf16(s[n][2], s[n][3]), pk_bf16(s[n][4], s[n][5]),
                  pk_bf16(s[n][6], s[n][7]));
  }
  // ---- O^T += V^T P^T
  if constexpr (MX) {
    uint32_t sb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sb[j] = mx_vscale<D>(x, j, c);
    if constexpr (MASKED) {
      // A NaN scale in a place that some row does not see: 0 * NaN must not
      // reach that row. Such values are taken out of the product and their NaN
      // is given to the rows that do see them (a product of 0/1 operands).
      uint32_t nan = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) nan |= sb[j] == 255u ? 1u << j : 0u;
      if (__any(nan != 0)) {
        uint32_t u[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          u[j] = ((nan >> (2 * j)) & 1u ? 0x3f80u : 0u) | ((nan >> (2 * j + 1)) & 1u ? 0x3f800000u : 0u);
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = ((see[n] >> (2 * j)) & 1u ? 0x3f80u : 0u) | ((see[n] >> (2 * j + 1)) & 1u ? 0x3f800000u : 0u);
          const f32x4_t hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              op8(u[0], u[1], u[2], u[3]), op8(v[0], v[1], v[2], v[3]), f32x4_t{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) w.o[n][d][i] = hit[i] > 0.0f ? __builtin_nanf("") : w.o[n][d][i];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sb[j] = sb[j] == 255u ? 127u : sb[j];
      }
    }
    float sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sc[j] = e8m0_to_f32(sb[j]);
    // byte y of a lane's codes holds its values 2y and 2y+1
#pragma unroll
    for (int y = 0; y < ND / 2; ++y) {
      uint32_t pr[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t cw = x.vc[j][y >> 2];
        pr[j] = (y & 3) == 0 ? fp4_pair<0>(cw, sc[j]) : (y & 3) == 1 ? fp4_pair<1>(cw, sc[j])
              : (y & 3) == 2 ? fp4_pair<2>(cw, sc[j]) : fp4_pair<3>(cw, sc[j]);
      }
      uint32_t e[4], f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = __builtin_amdgcn_perm(pr[2 * j + 1], pr[2 * j], 0x05040100u);
        f[j] = __builtin_amdgcn_perm(pr[2 * j + 1], pr[2 * j], 0x07060302u);
      }
      const bf16x8_t v0 = op8(e[0], e[1], e[2], e[3]), v1 = op8(f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        w.o[n][2 * y] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pb[n], w.o[n][2 * y], 0, 0, 0);
        w.o[n][2 * y + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pb[n], w.o[n][2 * y + 1], 0, 0, 0);
      }
    }
  } else {
    // the absmax of (position, block) goes into the probabilities of that block
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      float ab[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        ab[j] = __builtin_bit_cast(float, word_of(x.vsv, j * (D / 64) + b)) * kNF4InvScale;
      bf16x8_t pq[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = s[n][j] * ab[j];
          if constexpr (MASKED) p[j] = (see[n] >> j) & 1u ? p[j] : 0.0f;
        }
        pq[n] = op8(pk_bf16(p[0], p[1]), pk_bf16(p[2], p[3]), pk_bf16(p[4], p[5]), pk_bf16(p[6], p[7]));
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t pr[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) pr[j] = nf4_lut32(lut, y ? x.vc[j][b] >> 8 : x.vc[j][b] & 0xffu, lane);
        uint32_t e[4], f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = __builtin_amdgcn_perm(pr[2 * j + 1], pr[2 * j], 0x05040100u);
          f[j] = __builtin_amdgcn_perm(pr[2 * j + 1], pr[2 * j], 0x07060302u);
        }
        const bf16x8_t v0 = op8(e[0], e[1], e[2], e[3]), v1 = op8(f[0], f[1], f[2], f[3]);
        const int d = 4 * b + 2 * y;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          w.o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pq[n], w.o[n][d], 0, 0, 0);
          w.o[n][d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pq[n], w.o[n][d + 1], 0, 0, 0);
        }
      }
    }
  }
}

// Result of one row from its unnormalised sum o (scaled by 2^-m), l and m:
// the sink joins the sum, and a row that saw nothing gives 0.
struct AttnScale {
  float mul, lse;
};

__device__ __forceinline__ AttnScale attn_finish(float m, float l, const float *sinks, int hq) {
  AttnScale r;
  float f = 1.0f;
  if (sinks) {
    const float sk = sinks[hq] * 1.44269504088896340736f;
    const float top = fmaxf(m, sk);
    if (top != kNegInf) {
      f = __builtin_amdgcn_exp2f(m - top);
      l = l * f + __builtin_amdgcn_exp2f(sk - top);
      m = top;
    }
  }
  r.mul = l == 0.0f ? 0.0f : f / l;
  r.lse = l == 0.0f ? kNegInf : (m + log2f(l)) * 0.69314718055994530942f;
  return r;
}

template <int FMT, int D, int NQ>
__global__ __launch_bounds__(kAttnThreads, 2) void kv_attn_kernel(KvAttnArgs a) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  constexpr int KS = D / 32, ND = D / 16, M = 16 * NQ;
  constexpr bool QLDS = AttnWave<FMT, D, NQ>::QLDS;
  constexpr int RED = 4 * 16 * (D + 4);                      // words: the four waves' O tile
  constexpr int LUT = MX ? 0 : 256 * kAttnLutCopies;
  constexpr int QW = QLDS ? NQ * KS * 64 * 4 : 0;
  constexpr int WORDS = (LUT + QW) > RED ? (LUT + QW) : RED;
  __shared__ __attribute__((aligned(16))) uint32_t lds[WORDS];
  __shared__ float sm[4][NQ * 16], sl[4][NQ * 16];
  uint32_t *lut = lds;
  uint4 *qlds = reinterpret_cast<uint4 *>(lds + LUT);
  const KvView &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
  // heads fastest, then row tiles (the last tiles see the most), sequences, splits
  int idx = (int)blockIdx.x;
  const int h = idx % kv.H;
  idx /= kv.H;
  const int mt = a.n_mt - 1 - idx % a.n_mt;
  idx /= a.n_mt;
  const int b = idx % kv.B, split = idx / kv.B;
  const int row0 = mt * M, Hq = kv.H * a.G;
  const AttnRange x = attn_range(a, b, row0, M);
  if (row0 >= x.rows) return;
  const int t0 = x.lo + split * a.chunk;
  const int t1 = split == a.n_split - 1 ? x.hi : min(x.hi, t0 + a.chunk);
  if (t0 >= t1 && split > 0) return;
  const bool whole = split == 0 && t1 >= x.hi;               // the only range of this tile

  AttnWave<FMT, D, NQ> w;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int row = row0 + n * 16 + c, tok = row / a.G;
    const bool ok = row < x.rows;
    w.qpos[n] = ok ? x.start + tok : -1;
    w.m[n] = kNegInf;
    w.l[n] = 0.0f;
    const uint16_t *qp = a.q + (int64_t)(x.r0 + tok) * a.q_stride + (int64_t)(h * a.G + row - tok * a.G) * D;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = MX ? g * (D / 4) + k * 8 : (k >> 1) * 64 + g * 16 + (k & 1) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok && (!QLDS || wave == n)) v = *reinterpret_cast<const uint4 *>(qp + d);
      if constexpr (QLDS) {
        if (wave == n) qlds[(n * KS + k) * 64 + lane] = v;
      } else {
        w.q[n][k] = __builtin_bit_cast(bf16x8_t, v);
      }
    }
#pragma unroll
    for (int d = 0; d < ND; ++d) w.o[n][d] = f32x4_t{0, 0, 0, 0};
  }
  if constexpr (!MX) {
    // entry b, copies 4j..4j+3 as one 16-byte store
#pragma unroll 4
    for (int i = tid; i < 256 * kAttnLutCopies / 4; i += kAttnThreads) {
      const uint32_t e = (uint32_t)i / (kAttnLutCopies / 4);
      const uint32_t v = nf4_bf16(e >> 4) | (nf4_bf16(e & 15u) << 16);
      *reinterpret_cast<uint4 *>(lut + 4 * i) = make_uint4(v, v, v, v);
    }
  }
  if constexpr (!MX || QLDS) __syncthreads();

  const int full_lo = a.window > 0 ? x.q_last - a.window + 1 : 0;   // seen by every row from here ...
  const int full_hi = x.q_first;                                    // ... up to here
  // One round ahead the codes are in flight, two rounds ahead the page ids.
  AttnTile<FMT, D> ta, tb;
  int t = t0 + wave * 32;
  auto tile = [&](AttnTile<FMT, D> &cur, int at) {
    const bool all = at >= full_lo && at + 31 <= full_hi && __ballot(cur.bad) == 0;
    if (all) attn_tile<FMT, D, NQ, false>(w, cur, a, lut, qlds, at, lane);
    else attn_tile<FMT, D, NQ, true>(w, cur, a, lut, qlds, at, lane);
  };
  if (t < t1) {
    AttnPages p = attn_pages<FMT, D>(kv, b, t, lane);
    AttnPages pn = attn_pages<FMT, D>(kv, b, t + kAttnRound, lane);
    attn_load<FMT, D>(ta, kv, h, t, p, lane);
    for (;;) {
      p = attn_pages<FMT, D>(kv, b, t + 2 * kAttnRound, lane);
      if (t + kAttnRound < t1) attn_load<FMT, D>(tb, kv, h, t + kAttnRound, pn, lane);
      tile(ta, t);
      t += kAttnRound;
      if (t >= t1) break;
      pn = attn_pages<FMT, D>(kv, b, t + 2 * kAttnRound, lane);
      if (t + kAttnRound < t1) attn_load<FMT, D>(ta, kv, h, t + kAttnRound, p, lane);
      tile(tb, t);
      t += kAttnRound;
      if (t >= t1) break;
    }
  }

  // ---- join the four waves
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    w.l[n] = sum_xor16_32(w.l[n]);
    if (g == 0) {
      sm[wave][n * 16 + c] = w.m[n];
      sl[wave][n * 16 + c] = w.l[n];
    }
  }
  __syncthreads();
  float *red = reinterpret_cast<float *>(lds);
  const int64_t item = ((int64_t)b * a.n_mt + mt) * kv.H + h;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = n * 16 + c;
    const float top = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
    const float ts = top == kNegInf ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(w.m[n] - ts);
    float *mine = red + (wave * 16 + c) * (D + 4);
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int cc = g * 4 + i;
        const int at = MX ? cc * (D / 16) + d : (d >> 2) * 64 + cc * 4 + (d & 3);
        mine[at] = w.o[n][d][i] * f;
      }
    __syncthreads();
    // 16 rows x D/4 groups of four values over the workgroup
    for (int u = tid; u < 16 * (D / 4); u += kAttnThreads) {
      const int rr = u / (D / 4), d4 = (u - rr * (D / 4)) * 4;
      const int row = row0 + n * 16 + rr;
      if (row < x.rows) {
        float4 s = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float4 o = *reinterpret_cast<const float4 *>(red + (v * 16 + rr) * (D + 4) + d4);
          s.x += o.x;
          s.y += o.y;
          s.z += o.z;
          s.w += o.w;
        }
        const int k = n * 16 + rr;
        const float mr = fmaxf(fmaxf(sm[0][k], sm[1][k]), fmaxf(sm[2][k], sm[3][k]));
        const float mrs = mr == kNegInf ? 0.0f : mr;
        float l = 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) l += sl[v][k] * __builtin_amdgcn_exp2f(sm[v][k] - mrs);
        if (whole) {
          const int tok = row / a.G, hq = h * a.G + row - tok * a.G;
          const AttnScale z = attn_finish(mr, l, a.sinks, hq);
          *reinterpret_cast<uint2 *>(a.out + (int64_t)(x.r0 + tok) * a.out_stride + (int64_t)hq * D + d4) =
              make_uint2(pk_bf16(s.x * z.mul, s.y * z.mul), pk_bf16(s.z * z.mul, s.w * z.mul));
          if (a.lse && d4 == 0) a.lse[(int64_t)(x.r0 + tok) * Hq + hq] = z.lse;
        } else {
          const int64_t pr = (item * a.n_split + split) * M + k;
          *reinterpret_cast<float4 *>(a.part + pr * D + d4) = s;
          if (d4 == 0) *reinterpret_cast<float2 *>(a.part + a.part_rows * D + pr * 2) = make_float2(mr, l);
        }
      }
    }
    __syncthreads();
  }
}

// Joins the ranges of one tile: a thread per four values of a row.
template <int D>
__global__ __launch_bounds__(kAttnThreads) void kv_attn_join_kernel(KvAttnArgs a, int M) {
  const KvView &kv = a.kv;
  int idx = (int)blockIdx.x;
  const int64_t item = idx;
  const int h = idx % kv.H;
  idx /= kv.H;
  const int mt = idx % a.n_mt, b = idx / a.n_mt;
  const int u = (int)blockIdx.y * kAttnThreads + threadIdx.x;
  const int r = u / (D / 4), d4 = (u - r * (D / 4)) * 4, row = mt * M + r;
  const AttnRange x = attn_range(a, b, mt * M, M);
  if (r >= M || row >= x.rows) return;
  const int n = x.hi > x.lo ? min((x.hi - x.lo + a.chunk - 1) / a.chunk, a.n_split) : 1;
  if (n <= 1) return;                                        // written by its only range
  const float2 *ml = reinterpret_cast<const float2 *>(a.part + a.part_rows * D) + item * a.n_split * M + r;
  const float *po = a.part + (item * a.n_split * M + r) * D + d4;
  float top = kNegInf;
#pragma unroll 8
  for (int s = 0; s < n; ++s) top = fmaxf(top, ml[(int64_t)s * M].x);
  const float ts = top == kNegInf ? 0.0f : top;
  float l = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 8
  for (int s = 0; s < n; ++s) {
    const float2 v = ml[(int64_t)s * M];
    const float4 p = *reinterpret_cast<const float4 *>(po + (int64_t)s * M * D);
    const float f = __builtin_amdgcn_exp2f(v.x - ts);
    l = fmaf(v.y, f, l);
    o.x = fmaf(p.x, f, o.x);
    o.y = fmaf(p.y, f, o.y);
    o.z = fmaf(p.z, f, o.z);
    o.w = fmaf(p.w, f, o.w);
  }
  const int tok = row / a.G, hq = h * a.G + row - tok * a.G;
  const AttnScale z = attn_finish(top, l, a.sinks, hq);
  *reinterpret_cast<uint2 *>(a.out + (int64_t)(x.r0 + tok) * a.out_stride + (int64_t)hq * D + d4) =
      make_uint2(pk_bf16(o.x * z.mul, o.y * z.mul), pk_bf16(o.z * z.mul, o.w * z.mul));
  if (a.lse && d4 == 0) a.lse[(int64_t)(x.r0 + tok) * kv.H * a.G + hq] = z.lse;
}

// Rows per tile from the most new tokens of a sequence; enough ranges that a
// few workgroups per compute unit exist, none shorter than two rounds.
bool kv_attention_plan(int32_t D, int32_t H, int32_t G, int32_t B, int64_t n_tokens, int32_t max_new,
                       int64_t max_len, int32_t window, KvAttnPlan *p) {
  const int64_t rows = (int64_t)max_new * G;
  p->nq = rows <= 16 ? 1 : (rows <= 32 || D == 256) ? 2 : 4;
  const int M = 16 * p->nq;
  const int64_t n_mt = (rows + M - 1) / M;
  p->items = (int64_t)B * n_mt * H;
  constexpr int64_t kTarget = 1024;
  const int64_t busy = std::min<int64_t>((int64_t)B * n_mt, (n_tokens * G) / M + B) * H;
  int64_t len = std::max<int64_t>(max_len, 1);
  if (window > 0) len = std::min<int64_t>(len, (int64_t)window + max_new + kAttnRound);
  int64_t split = std::min<int64_t>(std::max<int64_t>(kTarget / std::max<int64_t>(busy, 1), 1),
                                    (len + 2 * kAttnRound - 1) / (2 * kAttnRound));
  int64_t chunk = ((len + split - 1) / split + kAttnRound - 1) / kAttnRound * kAttnRound;
  split = (len + chunk - 1) / chunk;
  if (p->items * split > 0x7fffffffLL || n_mt > 0x7fffffffLL) return false;
  p->n_mt = (int32_t)n_mt;
  p->n_split = (int32_t)split;
  p->chunk = (int32_t)std::min<int64_t>(chunk, 0x40000000LL);
  p->bytes = split > 1 ? (size_t)(p->items * split * M) * (D + 2) * 4 : 0;
  return true;
}

template <int FMT, int D, int NQ>
static hipError_t attn_go(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  hipLaunchKernelGGL((kv_attn_kernel<FMT, D, NQ>), dim3((unsigned)(p.items * p.n_split)), dim3(kAttnThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.n_split == 1) return e;
  const int M = 16 * NQ;
  hipLaunchKernelGGL((kv_attn_join_kernel<D>), dim3((unsigned)p.items, (M * (D / 4) + kAttnThreads - 1) / kAttnThreads),
                     dim3(kAttnThreads), 0, s, a, M);
  return hipGetLastError();
}

template <int FMT, int D>
static hipError_t attn_nq(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  if (p.nq == 1) return attn_go<FMT, D, 1>(a, p, s);
  if constexpr (D != 256) {
    if (p.nq == 4) return attn_go<FMT, D, 4>(a, p, s);
  }
  return attn_go<FMT, D, 2>(a, p, s);
}

hipError_t launch_kv_attention(const KvAttnArgs &args, const KvAttnPlan &p, int32_t format, hipStream_t s) {
  KvAttnArgs a = args;
  a.n_mt = p.n_mt;
  a.n_split = p.n_split;
  a.chunk = p.chunk;
  a.part_rows = p.items * p.n_split * 16 * p.nq;
  if (format == GNF4_MXFP4) {
    if (a.kv.D == 64) return attn_nq<GNF4_MXFP4, 64>(a, p, s);
    if (a.kv.D == 128) return attn_nq<GNF4_MXFP4, 128>(a, p, s);
    return attn_nq<GNF4_MXFP4, 256>(a, p, s);
  }
  if (a.kv.D == 64) return attn_nq<GNF4_NF4, 64>(a, p, s);
  if (a.kv.D == 128) return attn_nq<GNF4_NF4, 128>(a, p, s);
  return attn_nq<GNF4_NF4, 256>(a, p, s);
}

}  // namespace gnf4
