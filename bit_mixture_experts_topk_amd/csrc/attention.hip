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
// of 16 * NQ rows. A workgroup's NW waves take 32 positions each, 32 * NW a
// round, and join at the end of a tile through LDS. NW is 8 where a wave's
// registers allow two waves per SIMD, else 4.
// Sequences differ in length, so the rounds of all (sequence, tile, head)
// problems are numbered through and every workgroup, one per compute unit,
// takes an equal run of them, over the end of one problem into the next. A
// problem that lies in several runs is put together by a second kernel.
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
#include <cmath>
#include <type_traits>

#include "kvcache.h"

namespace gnf4 {

constexpr int kAttnGroups = 256;                // workgroups of a shared launch: the compute units
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

// A sequence as its rows see it, from the step's arrays.
struct AttnSeq {
  int r0, rows;                   // first token row, query rows (tokens * G)
  int start;                      // position of its first new token
  int lo, hi;                     // positions that any row may see, lo a multiple of 32
  int mts, units;                 // row tiles; rounds per tile and head (at least one: it writes the result)
};

__device__ __forceinline__ AttnSeq attn_seq(const KvAttnArgs &a, int b, int M, int round) {
  const KvView &kv = a.kv;
  AttnSeq x;
  const int o0 = kv.offsets[b], o1 = kv.offsets[b + 1], len = kv.lens[b];
  const int e = min(max(o1, 0), kv.n_tokens);
  x.r0 = min(max(o0, 0), e);
  const int n = e - x.r0;
  x.rows = n * a.G;
  x.start = len - n;
  x.hi = (int)min((int64_t)len, (int64_t)kv.max_pages << kv.page_shift);
  x.lo = a.window > 0 ? max(0, x.start - a.window + 1) & ~31 : 0;
  x.mts = min((x.rows + M - 1) / M, a.n_mt);
  x.units = x.hi > x.lo ? (x.hi - x.lo + round - 1) / round : 1;
  return x;
}

__device__ __forceinline__ int64_t attn_units(const KvAttnArgs &a, int b, int M, int round) {
  const AttnSeq x = attn_seq(a, b, M, round);
  return (int64_t)x.mts * a.kv.H * x.units;
}

// One wave's 32 positions: raw codes and scales in registers. The scales of
// positions 8g..8g+7 lie in lane group g's own row of 16 lanes, read there
// with a row broadcast where they are used.
template <int FMT, int D>
struct AttnTile {
  static constexpr bool MX = FMT == GNF4_MXFP4;
  static constexpr int KW = D / 32;                          // code dwords per lane and K tile
  static constexpr int VW = MX ? (D == 256 ? 2 : 1) : D / 64;  // code pieces per lane and position
  static constexpr int SW = MX ? (D == 256 ? 2 : 1) : (D == 256 ? 2 : 1);
  uint32_t kc[2][KW];
  uint32_t ks[2];                 // MXFP4: scale byte(s) of the lane's K rows; NF4: words of absmax
  uint32_t vc[8][VW];
  uint32_t vs[SW];                // MXFP4: scale bytes of position 8g + c % 8; NF4: words of absmax
  bool bad;                       // positions 8g..8g+7 lie on no page
};

// Lane N of the lane's row of 16.
template <int N>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + N, 0xf, 0xf, false);
}

// Pages of the wave's tile at position t: of its first and of its last 16
// positions (pages hold 16 at least).
struct AttnPages {
  int a, b;
};

__device__ __forceinline__ AttnPages attn_pages(const KvView &kv, int b, int t) {
  const int32_t *row = kv.pages + (int64_t)b * kv.max_pages;
  AttnPages p;
  p.a = row[min(t >> kv.page_shift, kv.max_pages - 1)];
  p.b = row[min((t + 16) >> kv.page_shift, kv.max_pages - 1)];
  return p;
}

// The loads of a tile from the addresses of its lanes: krow / vrow are the K
// and V rows of the lane's group (a position 8 (r / 4) and 8 g of the tile).
template <int FMT, int D, class Row>
__device__ __forceinline__ void attn_load_at(AttnTile<FMT, D> &x, const KvView &kv, Row at, int lane) {
  typedef AttnTile<FMT, D> T;
  const int r = lane & 15, g = lane >> 4;
  const uint32_t kt = (uint32_t)((r >> 2) * 8 + (r & 3)), vt = (uint32_t)(g * 8);
  if constexpr (T::MX) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint8_t *s = at(kv.k_codes, D / 2, r >> 2, (kt + i * 4) * (D / 2) + g * (D / 8));
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
      const uint8_t *sc = at(static_cast<const uint8_t *>(kv.k_scales), D / 32, r >> 2,
                             (kt + i * 4) * (D / 32) + (D == 64 ? g >> 1 : D == 128 ? g : 2 * g));
      if constexpr (D == 256) x.ks[i] = *reinterpret_cast<const uint16_t *>(sc);
      else x.ks[i] = *sc;
    }
    const uint8_t *sv = at(static_cast<const uint8_t *>(kv.v_scales), D / 32, g, (vt + (r & 7)) * (D / 32));
    if constexpr (D == 64) x.vs[0] = *reinterpret_cast<const uint16_t *>(sv);
    else if constexpr (D == 128) x.vs[0] = *reinterpret_cast<const uint32_t *>(sv);
    else {
      const uint2 v = *reinterpret_cast<const uint2 *>(sv);
      x.vs[0] = v.x;
      x.vs[1] = v.y;
    }
    const uint8_t *vp = at(kv.v_codes, D / 2, g, vt * (D / 2) + r * (D / 32));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t *s = vp + j * (D / 2);
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
    const uint8_t *kp = at(kv.k_codes, D / 2, r >> 2, kt * (D / 2) + g * 8);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        const uint2 v = *reinterpret_cast<const uint2 *>(kp + i * 4 * (D / 2) + b * 32);
        x.kc[i][2 * b] = v.x;
        x.kc[i][2 * b + 1] = v.y;
      }
    // absmax of positions 8g..8g+7: D/8 words, word w in lane w % 16 of the row
    // (D = 64: lanes 8..15 repeat lanes 0..7)
    const uint32_t w = vt * (D / 16) + 4 * (D == 64 ? r & 7 : r);
    const uint8_t *ks = at(static_cast<const uint8_t *>(kv.k_scales), D / 16, g, w);
    const uint8_t *vs = at(static_cast<const uint8_t *>(kv.v_scales), D / 16, g, w);
    x.ks[0] = *reinterpret_cast<const uint32_t *>(ks);
    x.vs[0] = *reinterpret_cast<const uint32_t *>(vs);
    if constexpr (D == 256) {
      x.ks[1] = *reinterpret_cast<const uint32_t *>(ks + 64);
      x.vs[1] = *reinterpret_cast<const uint32_t *>(vs + 64);
    }
    const uint8_t *vp = at(kv.v_codes, D / 2, g, vt * (D / 2) + r * 2);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
        x.vc[j][b] = *reinterpret_cast<const uint16_t *>(vp + j * (D / 2) + b * 32);
  }
}

// Page ids are the same for the whole wave, so rows are found with scalar
// arithmetic: of both halves of the tile, equal where a page covers it all.
template <int FMT, int D>
__device__ __forceinline__ void attn_load(AttnTile<FMT, D> &x, const KvView &kv, int h, int t, AttnPages p,
                                          int lane) {
  const int mask = (1 << kv.page_shift) - 1;
  int pa = __builtin_amdgcn_readfirstlane(p.a), pb = __builtin_amdgcn_readfirstlane(p.b);
  const bool bada = (uint32_t)pa >= (uint32_t)kv.n_pages, badb = (uint32_t)pb >= (uint32_t)kv.n_pages;
  x.bad = (lane >> 5) ? badb : bada;
  // an id outside the cache reads page 0 and is masked
  pa = bada ? 0 : pa;
  pb = badb ? 0 : pb;
  const int64_t ra = (((int64_t)pa * kv.H + h) << kv.page_shift) + (t & mask);
  if (kv.page_shift > 4) {
    attn_load_at<FMT, D>(x, kv, [&](const uint8_t *base, int size, int, uint32_t off) {
      return base + ra * size + off;
    }, lane);
  } else {
    const int64_t rb = (((int64_t)pb * kv.H + h) << kv.page_shift) + ((t + 16) & mask) - 16;
    attn_load_at<FMT, D>(x, kv, [&](const uint8_t *base, int size, int group, uint32_t off) {
      return base + (group < 2 ? ra : rb) * size + off;
    }, lane);
  }
}

// NF4: the absmax of position 8g + J, block B of the lane's group.
template <int D, int J, int B>
__device__ __forceinline__ float nf4_absmax(const uint32_t *w) {
  constexpr int at = J * (D / 64) + B;
  return __builtin_bit_cast(float, row_bcast<at % 16>(w[at / 16]));
}

// MXFP4: scale of position 8g + J for the lane's V values (block c / (512/D)),
// as a float32 whose exponent is the e8m0 byte (v_cvt_scalef32 reads the
// exponent only: 0 is 2^-127, 255 gives NaN).
template <int D, int J>
__device__ __forceinline__ uint32_t mx_vbyte(const uint32_t *w, int c) {
  const int blk = c / (512 / D);
  uint32_t x = row_bcast<J>(w[0]);
  if constexpr (D == 256) {
    const uint32_t y = row_bcast<J>(w[1]);                   // by every lane: the source lane must be active
    x = blk < 4 ? x : y;
  }
  return (x >> ((blk & 3) * 8)) & 0xffu;
}

template <int I, int N, class F>
__device__ __forceinline__ void static_for(F &&f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

// NQ * 16 query rows of one wave: Q operand, running statistics, O^T.
template <int FMT, int D, int NQ>
struct AttnWave {
  static constexpr int KS = D / 32, ND = D / 16;
  bf16x8_t q[NQ][KS];
  f32x4_t o[NQ][ND];
  float m[NQ], l[NQ];
  int qpos[NQ];                                              // position of the lane's query row
};

__device__ __forceinline__ float e8m0_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

template <int FMT, int D, int NQ, bool MASKED>
__device__ __forceinline__ void attn_tile(AttnWave<FMT, D, NQ> &w, AttnTile<FMT, D> &x, const KvAttnArgs &a,
                                          const uint32_t *lut, int t, int lane) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  constexpr int KS = D / 32, ND = D / 16;
  const int c = lane & 15, g = lane >> 4;
  const uint32_t lane4 = (uint32_t)lane * 4;
  float s[NQ][8];
  if constexpr (!MX) {                                       // absmax over the operand codebook's scale
#pragma unroll
    for (int i = 0; i < AttnTile<FMT, D>::SW; ++i) {
      x.ks[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, x.ks[i]) * kNF4InvScale);
      x.vs[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, x.vs[i]) * kNF4InvScale);
    }
  }
  // ---- scores of positions 8g..8g+7 for the lane's query row
  static_for<0, 2>([&](auto I) {
    constexpr int i = I;
    f32x4_t acc[NQ], blk[NQ];
    static_for<0, KS>([&](auto K) {
      constexpr int k = K;
      bf16x8_t ka;
      const uint32_t kw = x.kc[i][k];
      if constexpr (MX) {
        const float sc = e8m0_scale(D == 256 ? (k < KS / 2 ? x.ks[i] & 0xffu : x.ks[i] >> 8) : x.ks[i]);
        ka = op8(fp4_pair<0>(kw, sc), fp4_pair<1>(kw, sc), fp4_pair<2>(kw, sc), fp4_pair<3>(kw, sc));
      } else {
        ka = op8(lut_read(lut, lut_addr(kw, lane4, 0)), lut_read(lut, lut_addr(kw, lane4, 1)),
                 lut_read(lut, lut_addr(kw, lane4, 2)), lut_read(lut, lut_addr(kw, lane4, 3)));
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        constexpr f32x4_t zero = {0, 0, 0, 0};
        if constexpr (MX)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, w.q[n][k], k == 0 ? zero : acc[n], 0, 0, 0);
        else
          blk[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka, w.q[n][k], (k & 1) == 0 ? zero : blk[n], 0, 0, 0);
      }
      if constexpr (!MX && (k & 1)) {                        // a block of 64 is complete
        static_for<0, 4>([&](auto J) {
          constexpr int j = J;
          const float ab = nf4_absmax<D, 4 * i + j, k / 2>(x.ks);
#pragma unroll
          for (int n = 0; n < NQ; ++n) acc[n][j] = k == 1 ? blk[n][j] * ab : fmaf(blk[n][j], ab, acc[n][j]);
        });
      }
    });
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[n][4 * i + j] = acc[n][j];
  });
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
    mx = max_xor16_32(mx) * a.scale_log2;
    // m is raised only when it has fallen 2^8 behind: until then the
    // probabilities are up to 256 instead of 1, which costs no accuracy in
    // float32 or bf16, and the sums need not be rescaled.
    if (__builtin_expect(__any(mx > w.m[n] + 8.0f), 0)) {
      mx = fmaxf(mx, w.m[n]);
      const float alpha = __builtin_amdgcn_exp2f(w.m[n] - (mx == kNegInf ? 0.0f : mx));
      w.m[n] = mx;
      w.l[n] *= alpha;
#pragma unroll
      for (int d = 0; d < ND; ++d) w.o[n][d] *= alpha;
    }
    const float ms = w.m[n] == kNegInf ? 0.0f : w.m[n];      // nothing seen yet: exp2(-inf - 0) = 0
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[n][j] = __builtin_amdgcn_exp2f(fmaf(s[n][j], a.scale_log2, -ms));
      sum += s[n][j];
    }
    w.l[n] += sum;
    if constexpr (MX)
      pb[n] = op8(pk_bf16(s[n][0], s[n][1]), pk_bf16(s[n][2], s[n][3]), pk_bf16(s[n][4], s[n][5]),
                  pk_bf16(s[n][6], s[n][7]));
  }
  // ---- O^T += V^T P^T
  if constexpr (MX) {
    uint32_t sb[8];
    static_for<0, 8>([&](auto J) { sb[J] = mx_vbyte<D, J>(x.vs, c); });
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
    for (int j = 0; j < 8; ++j) sc[j] = e8m0_scale(sb[j]);
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
    static_for<0, D / 64>([&](auto BL) {
      constexpr int b = BL;
      float ab[8];
      static_for<0, 8>([&](auto J) { ab[J] = nf4_absmax<D, J, b>(x.vs); });
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
        for (int j = 0; j < 8; ++j) pr[j] = lut_read(lut, lut_addr(x.vc[j][b], lane4, y));
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
    });
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

// Shares of the numbered rounds: workgroup w takes [w * share, (w + 1) * share).
__device__ __forceinline__ int64_t attn_share(int64_t total) { return (total + kAttnGroups - 1) / kAttnGroups; }

// Sum over the workgroup of one value per thread, in every thread.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t *lds, int tid, int waves) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if ((tid & 63) == 0) lds[tid >> 6] = v;
  __syncthreads();
  v = 0;
  for (int i = 0; i < waves; ++i) v += lds[i];
  return v;
}

template <int FMT, int D, int NQ, int NW>
__global__ __launch_bounds__(64 * NW, NW / 4) void kv_attn_kernel(KvAttnArgs a) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  constexpr int NT = 64 * NW, ROUND = 32 * NW;
  constexpr int KS = D / 32, ND = D / 16, M = 16 * NQ;
  constexpr int DC = D < 128 ? D : 128;                      // values of a row joined at a time
  constexpr int LUT = MX ? 0 : kLutWords;
  constexpr int DEPTH = D == 256 || NQ > 1 || (!MX && D == 128) ? 2 : 3;          // tiles in registers: one computed, the others in flight
  // one block, so that the table starts at LDS address 0 and a byte's address
  // is what lut_addr forms
  struct Lds {
    uint32_t lut[LUT ? LUT : 4];
    float red[NW * 16 * (DC + 4)];
    float sm[NW][M], sl[NW][M];
    int64_t pre[NT + 1], wsum[NW];
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  uint32_t *lut = lds.lut;
  float *red = lds.red;
  auto &sm = lds.sm, &sl = lds.sl;
  int64_t *pre = lds.pre, *wsum = lds.wsum;
  const KvView &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
  const int Hq = kv.H * a.G;
  if constexpr (!MX) {
    fill_nf4_lut<NT>(lut, tid);
    __syncthreads();
  }

  // ---- the run of rounds: [u, end), from sequence b0 + (an index into pre) on
  int64_t u = 0, end = 0, base = 0;                          // base: rounds before the sequences of pre
  int b = 0, b0 = 0;
  if (a.shared) {
    int64_t v = tid < kv.B ? attn_units(a, tid, M, ROUND) : 0, total = v;
    for (int i = tid + NT; i < kv.B; i += NT) total += attn_units(a, i, M, ROUND);
    total = block_sum(total, wsum, tid, NW);
    const int64_t share = attn_share(total);
    u = blockIdx.x * share;
    end = min(total, u + share);
    if (u >= end) return;
    for (;;) {                                               // the chunk of sequences that holds round u
      int64_t s = v;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(s, d, 64);
        if (lane >= d) s += o;
      }
      __syncthreads();
      if (lane == 63) wsum[wave] = s;
      __syncthreads();
      int64_t before = base;
      for (int i = 0; i < wave; ++i) before += wsum[i];
      pre[tid + 1] = before + s;
      if (tid == 0) pre[0] = base;
      __syncthreads();
      if (u < pre[NT] || b0 + NT >= kv.B) break;
      base = pre[NT];
      b0 += NT;
      v = b0 + tid < kv.B ? attn_units(a, b0 + tid, M, ROUND) : 0;
    }
    for (int lo = 0, n = NT; n > 1;) {             // the last sequence with pre <= u: 64 probes at a time
      const int step = (n + 63) >> 6;
      const bool below = lane * step < n && pre[lo + lane * step] <= u;
      const int k = __popcll(__ballot(below));
      lo += (k - 1) * step;
      n = min(step, n - (k - 1) * step);
      b = lo;
    }
  }

  for (;;) {
    // ---- the next problem: tile mt, head h of sequence bb; its rounds [q0, q1)
    int bb, mt, h, q0 = 0, q1;
    AttnSeq x;
    if (a.shared) {
      if (u >= end) return;
      while (u >= pre[b + 1]) {                              // sequences without rows have no rounds
        if (++b < NT) continue;
        base = pre[NT];
        b0 += NT;
        b = 0;
        int64_t s = b0 + tid < kv.B ? attn_units(a, b0 + tid, M, ROUND) : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int64_t o = __shfl_up(s, d, 64);
          if (lane >= d) s += o;
        }
        __syncthreads();
        if (lane == 63) wsum[wave] = s;
        __syncthreads();
        int64_t before = base;
        for (int i = 0; i < wave; ++i) before += wsum[i];
        pre[tid + 1] = before + s;
        if (tid == 0) pre[0] = base;
        __syncthreads();
      }
      bb = b0 + b;
      x = attn_seq(a, bb, M, ROUND);
      const int64_t rel = u - pre[b], item = rel / x.units;
      q0 = (int)(rel - item * x.units);
      mt = (int)(item / kv.H);
      h = (int)(item - (int64_t)mt * kv.H);
      q1 = (int)min((int64_t)x.units, q0 + (end - u));
      u += q1 - q0;
    } else {
      int idx = (int)blockIdx.x;
      h = idx % kv.H;
      idx /= kv.H;
      mt = idx % a.n_mt;
      bb = idx / a.n_mt;
      x = attn_seq(a, bb, M, ROUND);
      if (mt >= x.mts) return;
      q1 = x.units;
    }
    const bool whole = q0 == 0 && q1 == x.units;
    const int t0 = x.lo + q0 * ROUND, t1 = min(x.hi, x.lo + q1 * ROUND), row0 = mt * M;

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
        if (ok) v = *reinterpret_cast<const uint4 *>(qp + d);
        v.x ^= a.q_sign;
        v.y ^= a.q_sign;
        v.z ^= a.q_sign;
        v.w ^= a.q_sign;
        w.q[n][k] = __builtin_bit_cast(bf16x8_t, v);
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) w.o[n][d] = f32x4_t{0, 0, 0, 0};
    }
    const int last = min(row0 + M, x.rows) - 1;
    const int full_hi = x.start + row0 / a.G;                // every row sees from full_lo to full_hi
    const int full_lo = a.window > 0 ? x.start + last / a.G - a.window + 1 : 0;
    AttnTile<FMT, D> tl[DEPTH];
    AttnPages pg[DEPTH];
    int t = t0 + wave * 32;
    if (t < t1) {
      // DEPTH - 1 rounds ahead the codes are in flight, one more the page ids
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) pg[i] = attn_pages(kv, bb, t + i * ROUND);
#pragma unroll
      for (int i = 0; i < DEPTH - 1; ++i)
        if (t + i * ROUND < t1) attn_load<FMT, D>(tl[i], kv, h, t + i * ROUND, pg[i], lane);
      for (bool more = true; more;) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
          constexpr int A = DEPTH - 1;
          pg[i] = attn_pages(kv, bb, t + DEPTH * ROUND);
          if (t + A * ROUND < t1)
            attn_load<FMT, D>(tl[(i + A) % DEPTH], kv, h, t + A * ROUND, pg[(i + A) % DEPTH], lane);
          const bool all = t >= full_lo && t + 31 <= full_hi && __ballot(tl[i].bad) == 0;
          if (all) attn_tile<FMT, D, NQ, false>(w, tl[i], a, lut, t, lane);
          else attn_tile<FMT, D, NQ, true>(w, tl[i], a, lut, t, lane);
          t += ROUND;
          if (t >= t1) {
            more = false;
            break;
          }
        }
      }
    }

    // ---- join the waves
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      w.l[n] = sum_xor16_32(w.l[n]);
      if (g == 0) {
        sm[wave][n * 16 + c] = w.m[n];
        sl[wave][n * 16 + c] = w.l[n];
      }
    }
    __syncthreads();
    // a problem that goes on from the workgroup before lies in this one's first
    // slot, one that goes on in the next in its second
    const int64_t slot = 2 * (int64_t)blockIdx.x + (q0 == 0 ? 1 : 0);
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = n * 16 + c;
      float top = sm[0][r];
#pragma unroll
      for (int v = 1; v < NW; ++v) top = fmaxf(top, sm[v][r]);
      const float f = __builtin_amdgcn_exp2f(w.m[n] - (top == kNegInf ? 0.0f : top));
#pragma unroll
      for (int dc = 0; dc < D; dc += DC) {
        float *mine = red + (wave * 16 + c) * (DC + 4);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int cc = g * 4 + i;
            const int at = MX ? cc * (D / 16) + d : (d >> 2) * 64 + cc * 4 + (d & 3);
            if (at >= dc && at < dc + DC) mine[at - dc] = w.o[n][d][i] * f;
          }
        __syncthreads();
        for (int k4 = tid; k4 < 16 * (DC / 4); k4 += NT) {
          const int rr = k4 / (DC / 4), d4 = (k4 - rr * (DC / 4)) * 4;
          const int k = n * 16 + rr, row = row0 + k;
          if (row < x.rows) {
            float4 s = make_float4(0, 0, 0, 0);
            float mr = sm[0][k], l = 0.0f;
#pragma unroll
            for (int v = 0; v < NW; ++v) {
              const float4 o = *reinterpret_cast<const float4 *>(red + (v * 16 + rr) * (DC + 4) + d4);
              s.x += o.x;
              s.y += o.y;
              s.z += o.z;
              s.w += o.w;
              mr = fmaxf(mr, sm[v][k]);
            }
            const float mrs = mr == kNegInf ? 0.0f : mr;
#pragma unroll
            for (int v = 0; v < NW; ++v) l += sl[v][k] * __builtin_amdgcn_exp2f(sm[v][k] - mrs);
            if (whole) {
              const int tok = row / a.G, hq = h * a.G + row - tok * a.G;
              const AttnScale z = attn_finish(mr, l, a.sinks, hq);
              *reinterpret_cast<uint2 *>(a.out + (int64_t)(x.r0 + tok) * a.out_stride + (int64_t)hq * D + dc + d4) =
                  make_uint2(pk_bf16(s.x * z.mul, s.y * z.mul), pk_bf16(s.z * z.mul, s.w * z.mul));
              if (a.lse && dc + d4 == 0) a.lse[(int64_t)(x.r0 + tok) * Hq + hq] = z.lse;
            } else {
              const int64_t pr = slot * M + k;
              *reinterpret_cast<float4 *>(a.part + pr * D + dc + d4) = s;
              if (dc + d4 == 0)
                *reinterpret_cast<float2 *>(a.part + 2LL * kAttnGroups * M * D + pr * 2) = make_float2(mr, l);
            }
          }
        }
        __syncthreads();
      }
    }
    if (!a.shared) return;
  }
}

// Puts together the problems that lie in several runs: a workgroup per problem,
// a thread per four values of a row.
constexpr int kJoinThreads = 256;

template <int D>
__global__ __launch_bounds__(kJoinThreads) void kv_attn_join_kernel(KvAttnArgs a, int M, int round) {
  __shared__ int64_t wsum[kJoinThreads / 64];
  const KvView &kv = a.kv;
  const int tid = threadIdx.x;
  int idx = (int)blockIdx.x;
  const int h = idx % kv.H;
  idx /= kv.H;
  const int mt = idx % a.n_mt, b = idx / a.n_mt;
  const AttnSeq x = attn_seq(a, b, M, round);
  int64_t first = 0, total = 0;
  for (int i = tid; i < kv.B; i += kJoinThreads) {
    const int64_t n = attn_units(a, i, M, round);
    total += n;
    first += i < b ? n : 0;
  }
  total = block_sum(total, wsum, tid, kJoinThreads / 64);
  first = block_sum(first, wsum, tid, kJoinThreads / 64);
  if (mt >= x.mts) return;
  const int64_t share = attn_share(total);
  first += ((int64_t)mt * kv.H + h) * x.units;
  const int64_t w0 = first / share, w1 = (first + x.units - 1) / share;
  if (w0 == w1) return;                                      // written by its only workgroup
  const int n = (int)(w1 - w0) + 1;
  const float2 *ml = reinterpret_cast<const float2 *>(a.part + 2LL * kAttnGroups * M * D);
  for (int u = tid; u < M * (D / 4); u += kJoinThreads) {
    const int r = u / (D / 4), d4 = (u - r * (D / 4)) * 4, row = mt * M + r;
    if (row >= x.rows) break;
    // the first workgroup's second slot, the first slots of the others
    auto at = [&](int s) { return (2 * (w0 + s) + (s == 0 ? 1 : 0)) * M + r; };
    float top = kNegInf, l = 0.0f;
    float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const int64_t pr = at(s);
      const float2 v = ml[pr];
      const float4 p = *reinterpret_cast<const float4 *>(a.part + pr * D + d4);
      const float nt = fmaxf(top, v.x), ns = nt == kNegInf ? 0.0f : nt;
      const float f = __builtin_amdgcn_exp2f(top - ns), e = __builtin_amdgcn_exp2f(v.x - ns);
      top = nt;
      l = l * f + v.y * e;
      o.x = o.x * f + p.x * e;
      o.y = o.y * f + p.y * e;
      o.z = o.z * f + p.z * e;
      o.w = o.w * f + p.w * e;
    }
    const int tok = row / a.G, hq = h * a.G + row - tok * a.G;
    const AttnScale z = attn_finish(top, l, a.sinks, hq);
    *reinterpret_cast<uint2 *>(a.out + (int64_t)(x.r0 + tok) * a.out_stride + (int64_t)hq * D + d4) =
        make_uint2(pk_bf16(o.x * z.mul, o.y * z.mul), pk_bf16(o.z * z.mul, o.w * z.mul));
    if (a.lse && d4 == 0) a.lse[(int64_t)(x.r0 + tok) * kv.H * a.G + hq] = z.lse;
  }
}

// Rows per tile from the most new tokens of a sequence. Short contexts, of up
// to four rounds, take a workgroup per problem and one launch; where these are
// at least as many as compute units, of four waves, so that two fit on one.
bool kv_attention_plan(int32_t D, int32_t H, int32_t G, int32_t B, int64_t n_tokens, int32_t max_new,
                       int64_t max_len, int32_t window, KvAttnPlan *p) {
  const int64_t rows = (int64_t)max_new * G;
  p->nq = rows <= 16 || D == 256 ? 1 : 2;                     // D = 256: the registers hold no second tile
  p->waves = p->nq == 1 && D <= 128 ? 8 : 4;
  int round = 32 * p->waves;
  const int M = 16 * p->nq;
  const int64_t n_mt = (rows + M - 1) / M;
  p->items = (int64_t)B * n_mt * H;
  int64_t len = std::max<int64_t>(max_len, 1);
  if (window > 0) len = std::min<int64_t>(len, (int64_t)window + max_new - 1 + 31);
  if (p->items > 0x7fffffffLL) return false;
  p->n_mt = (int32_t)n_mt;
  p->shared = len > 4 * round;
  if (!p->shared && p->items >= kAttnGroups) p->waves = 4;
  p->bytes = p->shared ? (size_t)(2 * kAttnGroups * M) * (D + 2) * 4 : 0;
  return true;
}

template <int FMT, int D, int NQ, int NW>
static hipError_t attn_go(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  hipLaunchKernelGGL((kv_attn_kernel<FMT, D, NQ, NW>), dim3(p.shared ? kAttnGroups : (unsigned)p.items), dim3(64 * NW),
                     0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.shared) return e;
  hipLaunchKernelGGL((kv_attn_join_kernel<D>), dim3((unsigned)p.items), dim3(kJoinThreads), 0, s, a, 16 * NQ, 32 * NW);
  return hipGetLastError();
}

template <int FMT, int D>
static hipError_t attn_nq(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  if constexpr (D <= 128) {
    if (p.nq == 2) return attn_go<FMT, D, 2, 4>(a, p, s);
    if (p.waves == 8) return attn_go<FMT, D, 1, 8>(a, p, s);
  }
  return attn_go<FMT, D, 1, 4>(a, p, s);
}

hipError_t launch_kv_attention(const KvAttnArgs &args, const KvAttnPlan &p, int32_t format, hipStream_t s) {
  KvAttnArgs a = args;
  a.n_mt = p.n_mt;
  a.shared = p.shared;
  // The running maximum is taken before the scale, which therefore must not be
  // negative (the queries change sign instead) nor 0 (0 times the -inf of a
  // masked place; 2^-100 leaves the weights equal).
  a.q_sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
  a.scale_log2 = std::max(std::fabs(a.scale_log2), 0x1p-100f);
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
