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
// of 16 * NQ rows. A workgroup's NW waves take 32 positions each in turn and
// join at the end of a problem through LDS.
// Sequences differ in length, so the runs of 128 positions of all (sequence,
// tile, head) problems are numbered through and every workgroup, one per
// compute unit, takes an equal share of them, over the end of one problem into
// the next. A problem that lies in several shares is put together by a second
// kernel.
//
// With few rows it is bound by the cache's bytes: a wave keeps its next tiles in
// flight straight into LDS (global_load_lds, no registers), S slots of its own,
// so that a compute unit has about 70 KB under way, and two waves per SIMD take
// turns at decoding and multiplying. MXFP4, 16 sequences of 16 to 32 thousand
// positions of 8 heads of 128: 443 MB in 85 us, 5.2 TB/s (a plain read of
// 1 GiB: 5.5), and 5 us to join. With less to read per workgroup its ends
// show: NF4, 32 sequences of 0.8 to 8 thousand positions of 4 heads, 86 MB in
// 34 us, of which a workgroup spends 20 in its tiles (at 5.6 TB/s) and the
// rest in finding its share, in the first pages, queries and tiles of each of
// its problems, and in joining its waves.
// With many rows it is bound by instructions: 2 x 1024 tokens of 32 heads over
// up to 8192 positions, MXFP4: 260 us, 715 TFLOP/s (a large bf16 product of the
// library: 1137). Vector instructions (exponentials, roundings, decoding) take
// about 55 % of a SIMD's cycles and the products 29 %; its two waves overlap
// them in part.
//
// No transposes. v_mfma_f32_16x16x32 (bf16 or f16) takes A rows from lanes 0..15 with 8
// consecutive k per lane group g = lane / 16, and leaves C with its column in
// the lane and rows 4g..4g+3 in the registers. Computed are S^T = K Q^T (rows =
// positions, columns = query rows) and O^T = V^T P^T. Row r of K tile i (of
// two) is position 8 (r / 4) + 4 i + r % 4 of the 32, so the scores that a lane
// holds after both tiles are those of positions 8g..8g+7, which are just the k
// indices that it has to supply of P^T: the probabilities go from one product
// to the next without leaving their lane, and so does the softmax, whose row is
// the lane's column.
// The k order of S is free as well: MXFP4 lane group g takes values g D/4 ..
// (g+1) D/4 of the head (D = 128: one 16-byte piece and one scale), NF4 16 of
// every block of 64. V^T rows are columns of the cache: lane c reads its values
// of each of 8 positions, and pairs of positions are put together after
// decoding.
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

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t pk_f16(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  const f32x2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

// The product type of a format: bf16 holds MXFP4 values exactly at every scale.
// NF4 takes fp16, whose three more bits matter there: a codebook value's
// rounding is the same wherever the code occurs, so it does not average out
// over positions as the values themselves do (bf16 left 6e-3 of a result over
// 4500 positions). Its operands are kept in fp16's range: codes are at most
// s, queries and probabilities are brought there by powers of two.
template <int FMT>
__device__ __forceinline__ f32x4_t mfma_16x16x32(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  if constexpr (FMT == GNF4_MXFP4)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

// The float32 s in [1, 2) with the least mean of (fp16(s c[q]) / s - c[q])^2 over
// the 16 codes (2.5x below s = 1 in the root); results are scaled by 1/s.
constexpr float kNF4HalfScale = 1.6776896715164185f;
constexpr float kNF4HalfInv = 1.0f / kNF4HalfScale;

constexpr uint64_t nf4_f16_bits(int q) {
  return __builtin_bit_cast(uint16_t, (_Float16)(__builtin_bit_cast(float, kNF4Bits[q & 15]) * kNF4HalfScale));
}

__device__ __forceinline__ uint32_t nf4_f16(uint32_t q) {
  constexpr uint64_t w[4] = {
      nf4_f16_bits(0) | nf4_f16_bits(1) << 16 | nf4_f16_bits(2) << 32 | nf4_f16_bits(3) << 48,
      nf4_f16_bits(4) | nf4_f16_bits(5) << 16 | nf4_f16_bits(6) << 32 | nf4_f16_bits(7) << 48,
      nf4_f16_bits(8) | nf4_f16_bits(9) << 16 | nf4_f16_bits(10) << 32 | nf4_f16_bits(11) << 48,
      nf4_f16_bits(12) | nf4_f16_bits(13) << 16 | nf4_f16_bits(14) << 32 | nf4_f16_bits(15) << 48};
  const uint64_t x = q < 8u ? (q < 4u ? w[0] : w[1]) : (q < 12u ? w[2] : w[3]);
  return (uint32_t)(x >> ((q & 3u) * 16u)) & 0xffffu;
}

__device__ __forceinline__ bf16x8_t op8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8_t, make_uint4(a, b, c, d));
}

// A sequence as its rows see it, from the step's arrays.
struct AttnSeq {
  int r0, rows;                   // first token row, query rows (tokens * G)
  int start;                      // position of its first new token
  int hi;                         // end of the positions that any row may see
  int mts, units;                 // row tiles; runs of 128 positions per tile and head, from the first
                                  // that the tile sees on (at least one: it writes the result)
};

constexpr int kAttnUnit = 128;

// Arrays that no kernel writes meanwhile: scalar loads where the index is uniform.
typedef const __attribute__((address_space(4))) int32_t *const_ints;

// What the arrays say of sequence b: first row, rows, length.
struct AttnRaw {
  int r0, n, len;
};

__device__ __forceinline__ AttnRaw attn_raw(const KvView &kv, int b) {
  const const_ints off = (const_ints)(uintptr_t)kv.offsets, lens = (const_ints)(uintptr_t)kv.lens;
  const int o0 = off[b], o1 = off[b + 1];
  const int e = min(max(o1, 0), kv.n_tokens);
  AttnRaw x;
  x.r0 = min(max(o0, 0), e);
  x.n = e - x.r0;
  x.len = lens[b];
  return x;
}

__device__ __forceinline__ AttnSeq attn_seq(const KvAttnArgs &a, const AttnRaw &s, int M) {
  AttnSeq x;
  x.r0 = s.r0;
  x.rows = s.n * a.G;
  x.start = s.len - s.n;
  x.hi = (int)min((int64_t)s.len, (int64_t)a.kv.max_pages << a.kv.page_shift);
  x.mts = min((x.rows + M - 1) / M, a.n_mt);
  int span = x.hi;
  if (a.window > 0) span = (int)min((int64_t)span, (int64_t)a.window + a.tile_tokens - 1 + 31);
  x.units = span > 0 ? (span + kAttnUnit - 1) / kAttnUnit : 1;
  return x;
}

// Sum over the wave's lanes up to and with this one (DPP shifts within rows of
// 16, then the last lanes of the rows before).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

__device__ __forceinline__ int attn_units(const KvAttnArgs &a, const AttnSeq &x) { return x.mts * a.kv.H * x.units; }

// 64 sequences from b0 on, one per lane, and the running sum of their units.
struct AttnChunk {
  AttnRaw s;
  int sum;
};

__device__ __forceinline__ AttnChunk attn_chunk(const KvAttnArgs &a, int b0, int M, int lane) {
  const int b = b0 + lane;
  AttnChunk k;
  k.s = attn_raw(a.kv, min(b, a.kv.B - 1));
  if (b >= a.kv.B) k.s.n = 0;
  k.sum = wave_scan(attn_units(a, attn_seq(a, k.s, M)));
  return k;
}

__device__ __forceinline__ AttnRaw attn_pick(const AttnChunk &k, int l) {
  AttnRaw s;
  s.r0 = __builtin_amdgcn_readlane(k.s.r0, l);
  s.n = __builtin_amdgcn_readlane(k.s.n, l);
  s.len = __builtin_amdgcn_readlane(k.s.len, l);
  return s;
}

// Lane N of the lane's row of 16.
template <int N>
__device__ __forceinline__ uint32_t row_bcast(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x150 + N, 0xf, 0xf, false);
}

// ------------------------------------------------------- a tile's way into LDS

// 16 or 4 bytes per lane from base + off (or p) to LDS address lds + lane * 16
// (4). Counted by vmcnt; nothing is returned to registers.
__device__ __forceinline__ void dma16(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void dma16(const uint8_t *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory", "m0");
}

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A slot: 32 positions' codes of K (in the order the lanes read them), of V
// (row 4j + g holds position 8g + j, so that lane (c, g) reads along a line),
// and the scales of both.
template <int FMT, int D>
struct AttnSlot {
  static constexpr bool MX = FMT == GNF4_MXFP4;
  static constexpr int CH = D / 32;                          // 16-byte pieces per row
  static constexpr int N16 = CH / 2;                         // loads of 1 KB per side
  static constexpr int SC = MX ? D : 2 * D;                  // scale bytes per side
  static constexpr int VOFF = 16 * D, SOFF = 32 * D;
  static constexpr int BYTES = 32 * D + (2 * SC < 256 ? 256 : 2 * SC);
  static constexpr int LOADS = 2 * N16 + (SC == 256 ? 2 : 1);
};

// Where one head's rows lie, and page ids of 64 tiles of the wave, one per lane:
// of the first and the last 16 positions (pages hold 16 at least).
struct AttnPlace {
  const uint8_t *k, *v, *ks, *vs;                            // the head's rows on page 0
  int32_t page_rows, page_shift, n_pages;                    // rows of a page, all heads
  int a, b;
};

__device__ __forceinline__ void attn_pages(AttnPlace &x, const KvView &kv, int bb, int t) {
  const int32_t *row = kv.pages + (int64_t)bb * kv.max_pages;
  x.a = row[min(t >> kv.page_shift, kv.max_pages - 1)];
  x.b = row[min((t + 16) >> kv.page_shift, kv.max_pages - 1)];
  asm volatile("" : "+v"(x.a), "+v"(x.b));                   // here, not at their use among the tiles under way
}

// Sends the tile at position t (page ids in lane l of x) into the slot at LDS
// address lds. Returns which halves of it lie on no page (bit 0, 1): these
// read page 0 and are masked.
template <int FMT, int D>
__device__ __forceinline__ uint32_t attn_send(const AttnPlace &x, int l, int t, uint32_t lds, int lane) {
  typedef AttnSlot<FMT, D> T;
  constexpr int RB = D / 2, SB = T::SC / 32;                 // bytes per row: codes, scales
  int pa = __builtin_amdgcn_readlane(x.a, l), pb = __builtin_amdgcn_readlane(x.b, l);
  const bool bada = (uint32_t)pa >= (uint32_t)x.n_pages, badb = (uint32_t)pb >= (uint32_t)x.n_pages;
  pa = bada ? 0 : pa;
  pb = badb ? 0 : pb;
  const int64_t ra = (int64_t)pa * x.page_rows + (t & ((1 << x.page_shift) - 1));
  // K: LDS piece (i, q, r) = piece q of the row of tile i, lane r
  constexpr int LCH = T::CH == 2 ? 1 : T::CH == 4 ? 2 : 3;
  const int r = lane & 15;
  const int ki = T::CH == 2 ? lane >> 5 : 0, kq = T::CH == 2 ? (lane >> 4) & 1 : lane >> 4;
  const int ktok = (r >> 2) * 8 + ki * 4 + (r & 3);
  // V: LDS row 4j + g; the first load's rows, CH pieces each
  const int vrow = lane >> LCH, vq = lane & (T::CH - 1);
  const int vtok = (vrow & 3) * 8 + (vrow >> 2);
  constexpr int VSTEP = (64 / T::CH) / 4;                    // positions further per load
  // scales: lanes of one load share both sides unless a side takes a load of its own
  constexpr int SW = T::SC == 512 ? 16 : 4;                  // bytes per lane
  constexpr int SL = T::SC / SW;                             // lanes per side
  const int sside = T::SC == 256 ? 0 : (lane / SL) & 1, soff = (T::SC == 256 ? lane : lane % SL) * SW;
  if (x.page_shift > 4) {
    const uint8_t *kb = x.k + ra * RB, *vb = x.v + ra * RB;
#pragma unroll
    for (int n = 0; n < T::N16; ++n) {
      const int step = T::CH == 8 ? (n >> 1) * 4 * RB + (n & 1) * 64 : n * 4 * RB;
      dma16(kb + step, (uint32_t)(ktok * RB + kq * 16), lds + n * 1024);
      dma16(vb + n * VSTEP * RB, (uint32_t)(vtok * RB + vq * 16), lds + T::VOFF + n * 1024);
    }
    if constexpr (T::SC == 256) {
      dma4(x.ks + ra * SB, (uint32_t)soff, lds + T::SOFF);
      dma4(x.vs + ra * SB, (uint32_t)soff, lds + T::SOFF + 256);
    } else {
      const uint8_t *q = (sside ? x.vs : x.ks) + ra * SB + soff;
      if constexpr (SW == 16) dma16(q, lds + T::SOFF);
      else dma4(q, lds + T::SOFF);
    }
  } else {
    // pages of 16: the second half of the tile lies on another one
    const int64_t rb = (int64_t)pb * x.page_rows - 16;
    const int64_t rk = (r >> 2) < 2 ? ra : rb, rv = (vrow & 3) < 2 ? ra : rb;
    const int64_t rs = soff / SB < 16 ? ra : rb;
    const uint8_t *kb = x.k + rk * RB + ktok * RB + kq * 16;
    const uint8_t *vb = x.v + rv * RB + vtok * RB + vq * 16;
#pragma unroll
    for (int n = 0; n < T::N16; ++n) {
      const int step = T::CH == 8 ? (n >> 1) * 4 * RB + (n & 1) * 64 : n * 4 * RB;
      dma16(kb + step, lds + n * 1024);
      dma16(vb + n * VSTEP * RB, lds + T::VOFF + n * 1024);
    }
    if constexpr (T::SC == 256) {
      dma4(x.ks + rs * SB + soff, lds + T::SOFF);
      dma4(x.vs + rs * SB + soff, lds + T::SOFF + 256);
    } else {
      const uint8_t *q = (sside ? x.vs : x.ks) + rs * SB + soff;
      if constexpr (SW == 16) dma16(q, lds + T::SOFF);
      else dma4(q, lds + T::SOFF);
    }
  }
  return (bada ? 1u : 0u) | (badb ? 2u : 0u);
}

// NF4: the absmax of position 8g + J, block B of the lane's group: word w of the
// group's D/8 lies in lane w % 16 of its row of lanes.
template <int D, int J, int B>
__device__ __forceinline__ float nf4_absmax(const float *w) {
  constexpr int at = J * (D / 64) + B;
  return __builtin_bit_cast(float, row_bcast<at % 16>(__builtin_bit_cast(uint32_t, w[at / 16])));
}

// The float32 that v_cvt_scalef32 takes an e8m0 byte from: it reads the
// exponent only, 0 being 2^-127 and 255 giving NaN.
__device__ __forceinline__ float e8m0_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

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
  static constexpr bool QLDS = NQ > 2 || (D == 256 && NQ > 1);  // many results: the queries stay in LDS
  bf16x8_t q[QLDS ? 1 : NQ][QLDS ? 1 : KS];
  f32x4_t o[NQ][ND];
  float m[NQ], l[NQ];
  float sc[NQ];                                              // what a row's scores are multiplied by (base 2)
  int qpos[NQ];                                              // position of the lane's query row
};

// A table like the NF4 byte table of common.h, in fp16, with 64 >> LS copies:
// entry b of copy c at byte (b * 64 + c) * 4 >> LS. With fewer copies a lane's
// address takes one more instruction, and lanes of one copy meet in a bank.
template <int LS>
__device__ __forceinline__ uint32_t attn_lut(const uint32_t *lut, uint32_t w, uint32_t lane4, int byte) {
  return lut_read(lut, lut_addr(w, lane4, byte) >> LS);
}

template <int LS, int NT>
__device__ __forceinline__ void fill_attn_lut(uint32_t *lut, int tid) {
#pragma unroll
  for (int i = 0; i < (4096 >> LS) / NT; ++i) {
    const uint32_t grp = (uint32_t)tid + NT * i, b = grp >> (4 - LS);
    const uint32_t v = nf4_f16(b >> 4) | (nf4_f16(b & 15u) << 16);
    *reinterpret_cast<uint4 *>(lut + grp * 4) = make_uint4(v, v, v, v);
  }
}

// One tile from its slot sl. bad: the lane's positions 8g..8g+7 lie on no page.
template <int FMT, int D, int NQ, bool MASKED, int LS>
__device__ __forceinline__ void attn_tile(AttnWave<FMT, D, NQ> &w, const uint8_t *sl, bool bad, const KvAttnArgs &a,
                                          const uint32_t *lut, const uint4 *ql, int t, int lane) {
  typedef AttnSlot<FMT, D> T;
  constexpr bool MX = FMT == GNF4_MXFP4;
  constexpr int KS = D / 32, ND = D / 16;
  const int c = lane & 15, g = lane >> 4;
  const uint32_t lane4 = (uint32_t)(lane & ((64 >> LS) - 1)) << (2 + LS);
  float s[NQ][8];
  const uint8_t *sc_k = sl + T::SOFF, *sc_v = sc_k + T::SC;
  float ksn[2], vsn[2];                                      // NF4: absmax over the codebook's scale
  if constexpr (!MX) {
#pragma unroll
    for (int i = 0; i < (D == 256 ? 2 : 1); ++i) {
      const int at = g * (D / 8) + (D == 64 ? c & 7 : c) + 16 * i;
      ksn[i] = reinterpret_cast<const float *>(sc_k)[at] * kNF4HalfInv;
      vsn[i] = reinterpret_cast<const float *>(sc_v)[at] * kNF4HalfInv;
    }
  }
  // ---- scores of positions 8g..8g+7 for the lane's query row
  static_for<0, 2>([&](auto I) {
    constexpr int i = I;
    f32x4_t acc[NQ], blk[NQ];
    uint32_t kc[KS];                                         // the lane's codes of its row of this K tile
    uint32_t kb = 0;                                         // MXFP4: its scale byte(s)
    const int tok = (c >> 2) * 8 + i * 4 + (c & 3);
    if constexpr (MX && D == 128) {
      const uint4 v = *reinterpret_cast<const uint4 *>(sl + i * 1024 + lane * 16);
      kc[0] = v.x, kc[1] = v.y, kc[2] = v.z, kc[3] = v.w;
      kb = sc_k[tok * 4 + g];
    } else if constexpr (MX && D == 256) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 v = *reinterpret_cast<const uint4 *>(sl + ((i * 8 + 2 * g + e) * 16 + c) * 16);
        kc[4 * e] = v.x, kc[4 * e + 1] = v.y, kc[4 * e + 2] = v.z, kc[4 * e + 3] = v.w;
      }
      kb = *reinterpret_cast<const uint16_t *>(sc_k + tok * 8 + 2 * g);
    } else {
      // MXFP4, D = 64: 8 bytes at g * 8 of the row; NF4: at b * 32 + g * 8 of block b
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        const uint2 v = *reinterpret_cast<const uint2 *>(sl + ((i * T::CH + 2 * b + (g >> 1)) * 16 + c) * 16 + (g & 1) * 8);
        kc[2 * b] = v.x, kc[2 * b + 1] = v.y;
      }
      if constexpr (MX) kb = sc_k[tok * 2 + (g >> 1)];
    }
    static_for<0, KS>([&](auto K) {
      constexpr int k = K;
      bf16x8_t ka;
      const uint32_t kw = kc[k];
      if constexpr (MX) {
        const float sc = e8m0_scale(D == 256 ? (k < KS / 2 ? kb & 0xffu : kb >> 8) : kb);
        ka = op8(fp4_pair<0>(kw, sc), fp4_pair<1>(kw, sc), fp4_pair<2>(kw, sc), fp4_pair<3>(kw, sc));
      } else {
        ka = op8(attn_lut<LS>(lut, kw, lane4, 0), attn_lut<LS>(lut, kw, lane4, 1),
                 attn_lut<LS>(lut, kw, lane4, 2), attn_lut<LS>(lut, kw, lane4, 3));
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        constexpr f32x4_t zero = {0, 0, 0, 0};
        bf16x8_t qv;
        if constexpr (AttnWave<FMT, D, NQ>::QLDS) qv = __builtin_bit_cast(bf16x8_t, ql[(n * KS + k) * 64 + lane]);
        else qv = w.q[n][k];
        if constexpr (MX) acc[n] = mfma_16x16x32<FMT>(ka, qv, k == 0 ? zero : acc[n]);
        else blk[n] = mfma_16x16x32<FMT>(ka, qv, (k & 1) == 0 ? zero : blk[n]);
      }
      if constexpr (!MX && (k & 1)) {                        // a block of 64 is complete
        static_for<0, 4>([&](auto J) {
          constexpr int j = J;
          const float ab = nf4_absmax<D, 4 * i + j, k / 2>(ksn);
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
  bf16x8_t pb[MX ? NQ : 1], pr[1];
  // NF4: log2 of a position's largest V absmax, in the lanes of its words, less
  // 7. Clamped so that sums of probabilities stay in float32's range.
  float la[D == 256 ? 2 : 1];
  if constexpr (!MX) {
#pragma unroll
    for (int i = 0; i < (D == 256 ? 2 : 1); ++i) {
      float v = fabsf(vsn[i]);
      if constexpr (D >= 128)                                // quad_perm 1,0,3,2
        v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true)));
      if constexpr (D == 256)                                // quad_perm 2,3,0,1
        v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, true)));
      la[i] = fminf(fmaxf(__builtin_amdgcn_logf(v), -60.0f), 60.0f) - 7.0f;
    }
  }
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if constexpr (MASKED) {
      see[n] = 0;
      const int lo = a.window > 0 ? w.qpos[n] - a.window + 1 : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int pos = t + g * 8 + j;
        const bool ok = pos <= w.qpos[n] && pos >= lo && !bad;
        see[n] |= ok ? 1u << j : 0u;
        s[n][j] = ok ? s[n][j] : kNegInf;
      }
    }
    float mx;
    if constexpr (MX) {
      mx = s[n][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = fmaxf(mx, s[n][j]);
      mx = max_xor16_32(mx) * w.sc[n];
    } else {
      // The maximum is that of p times absmax, what enters the second product:
      // its largest term is kept in 2^7 to 2^15, the top of fp16's range, whatever
      // the absmax are.
      mx = kNegInf;
      static_for<0, 8>([&](auto J) {
        constexpr int j = J, at = j * (D / 64);
        s[n][j] *= w.sc[n];
        const float y = s[n][j] + __builtin_bit_cast(float, row_bcast<at % 16>(__builtin_bit_cast(uint32_t, la[at / 16])));
        mx = fmaxf(mx, y);
      });
      mx = max_xor16_32(mx);
    }
    // m is raised only when it has fallen 2^8 behind: until then the terms are up
    // to 256 instead of 1, which costs no accuracy in floating point, and the
    // sums need not be rescaled.
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
      s[n][j] = __builtin_amdgcn_exp2f(MX ? fmaf(s[n][j], w.sc[n], -ms) : s[n][j] - ms);
      sum += s[n][j];
    }
    w.l[n] += sum;
    if constexpr (MX) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = pk_bf16(s[n][2 * j], s[n][2 * j + 1]);
      pb[n] = op8(h[0], h[1], h[2], h[3]);
      if constexpr (NQ == 1) {
        // what the rounding left out, as a second operand: the first product's
        // time is its cache's, not the matrix cores'
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[j] = pk_bf16(s[n][2 * j] - __builtin_bit_cast(float, h[j] << 16),
                         s[n][2 * j + 1] - __builtin_bit_cast(float, h[j] & 0xffff0000u));
        pr[0] = op8(r[0], r[1], r[2], r[3]);
      }
    }
  }
  // ---- O^T += V^T P^T
  if constexpr (MX) {
    uint32_t sb[8];                                          // scales of the lane's values: its block is c / (512/D)
#pragma unroll
    for (int j = 0; j < 8; ++j) sb[j] = sc_v[(g * 8 + j) * (D / 32) + c / (512 / D)];
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
    uint32_t vc[8][D == 256 ? 2 : 1];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t *row = sl + T::VOFF + (4 * j + g) * (D / 2) + c * (D / 32);
      if constexpr (D == 64) vc[j][0] = *reinterpret_cast<const uint16_t *>(row);
      else if constexpr (D == 128) vc[j][0] = *reinterpret_cast<const uint32_t *>(row);
      else {
        const uint2 v = *reinterpret_cast<const uint2 *>(row);
        vc[j][0] = v.x, vc[j][1] = v.y;
      }
    }
    // byte y of a lane's codes holds its values 2y and 2y+1
#pragma unroll
    for (int y = 0; y < ND / 2; ++y) {
      uint32_t pv[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t cw = vc[j][y >> 2];
        pv[j] = (y & 3) == 0 ? fp4_pair<0>(cw, sc[j]) : (y & 3) == 1 ? fp4_pair<1>(cw, sc[j])
              : (y & 3) == 2 ? fp4_pair<2>(cw, sc[j]) : fp4_pair<3>(cw, sc[j]);
      }
      uint32_t e[4], f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = __builtin_amdgcn_perm(pv[2 * j + 1], pv[2 * j], 0x05040100u);
        f[j] = __builtin_amdgcn_perm(pv[2 * j + 1], pv[2 * j], 0x07060302u);
      }
      const bf16x8_t v0 = op8(e[0], e[1], e[2], e[3]), v1 = op8(f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        w.o[n][2 * y] = mfma_16x16x32<FMT>(v0, pb[n], w.o[n][2 * y]);
        w.o[n][2 * y + 1] = mfma_16x16x32<FMT>(v1, pb[n], w.o[n][2 * y + 1]);
        if constexpr (NQ == 1) {
          w.o[n][2 * y] = mfma_16x16x32<FMT>(v0, pr[0], w.o[n][2 * y]);
          w.o[n][2 * y + 1] = mfma_16x16x32<FMT>(v1, pr[0], w.o[n][2 * y + 1]);
        }
      }
    }
  } else {
    // the absmax of (position, block) goes into the probabilities of that block
    static_for<0, D / 64>([&](auto BL) {
      constexpr int b = BL;
      float ab[8];
      uint32_t vc[8];                                        // lane c: values 4c .. 4c + 3 of the block
#pragma unroll
      for (int j = 0; j < 8; ++j)
        vc[j] = *reinterpret_cast<const uint16_t *>(sl + T::VOFF + (4 * j + g) * (D / 2) + b * 32 + c * 2);
      static_for<0, 8>([&](auto J) { ab[J] = nf4_absmax<D, J, b>(vsn); });
      bf16x8_t pq[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          p[j] = s[n][j] * ab[j];
          if constexpr (MASKED) p[j] = (see[n] >> j) & 1u ? p[j] : 0.0f;
        }
        pq[n] = op8(pk_f16(p[0], p[1]), pk_f16(p[2], p[3]), pk_f16(p[4], p[5]), pk_f16(p[6], p[7]));
      }
      // two positions' nibbles side by side: a byte of x holds value 2y of both, of
      // z value 2y + 1, so a table entry is the operand's pair of positions
      uint32_t x[4], z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t p0 = vc[2 * j], p1 = vc[2 * j + 1];
        x[j] = (p0 & 0xf0f0u) | ((p1 >> 4) & 0x0f0fu);
        z[j] = ((p0 << 4) & 0xf0f0u) | (p1 & 0x0f0fu);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const bf16x8_t v0 = op8(attn_lut<LS>(lut, x[0], lane4, y), attn_lut<LS>(lut, x[1], lane4, y),
                                attn_lut<LS>(lut, x[2], lane4, y), attn_lut<LS>(lut, x[3], lane4, y));
        const bf16x8_t v1 = op8(attn_lut<LS>(lut, z[0], lane4, y), attn_lut<LS>(lut, z[1], lane4, y),
                                attn_lut<LS>(lut, z[2], lane4, y), attn_lut<LS>(lut, z[3], lane4, y));
        const int d = 4 * b + 2 * y;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          w.o[n][d] = mfma_16x16x32<FMT>(v0, pq[n], w.o[n][d]);
          w.o[n][d + 1] = mfma_16x16x32<FMT>(v1, pq[n], w.o[n][d + 1]);
        }
      }
    });
  }
}

// A row's queries (its values lie in lanes c, c + 16, c + 32, c + 48) from bf16 to
// fp16, divided by the power of two that brings the largest into [1, 2);
// returns that power. Values 2^-14 and more below it lose bits that are 2^-24 of
// the largest. A row with an infinity or a NaN keeps them.
template <int KS>
__device__ __forceinline__ float nf4_query(uint4 (&v)[KS]) {
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) mag = max(mag, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
  }
  mag = __builtin_bit_cast(uint32_t, max_xor16_32(__builtin_bit_cast(float, mag << 16))) >> 16;
  // the exponent byte, 2^-126 for what lies below; the scale of a finite row
  const int e = min(max((int)(mag >> 7), 1), 254) - 127;
#pragma unroll
  for (int i = 0; i < KS; ++i) {
    uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = pk_f16(ldexpf(__builtin_bit_cast(float, w[j] << 16), -e), ldexpf(__builtin_bit_cast(float, w[j] & 0xffff0000u), -e));
    v[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return ldexpf(1.0f, e);
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

// Shares of the numbered runs: workgroup w takes [w * share, (w + 1) * share).
__device__ __forceinline__ int attn_share(int total) { return (total + kAttnGroups - 1) / kAttnGroups; }

template <int FMT, int D, int NQ, int NW, int S>
__global__ __launch_bounds__(64 * NW, NW == 4 ? (D == 256 ? 1 : NQ == 1 ? 3 : 2) : NW / 4) void kv_attn_kernel(KvAttnArgs a) {
  typedef AttnSlot<FMT, D> T;
  constexpr bool MX = FMT == GNF4_MXFP4;
  constexpr int NT = 64 * NW, ROUND = 32 * NW;
  constexpr int KS = D / 32, ND = D / 16, M = 16 * NQ;
  constexpr bool QLDS = AttnWave<FMT, D, NQ>::QLDS;
  constexpr int LS = NW == 4 && D <= 128 ? 2 : 0;
  // one block, so that the table starts at LDS address 0 and a byte's address
  // is what lut_addr forms
  struct Lds {
    uint32_t lut[MX ? 4 : kLutWords >> LS];
    union {
      uint8_t ring[NW * S * T::BYTES];                       // S slots of every wave
      float red[NW * 16 * (D + 4)];                          // the waves' O tile, when they join
    };
    float sm[NW][M], sl[NW][M];
    float qsc[M];
    uint4 q[QLDS ? NQ * KS * 64 : 1];                        // lane's operand of (tile n, step k) at (n KS + k) 64 + lane
  };
  __shared__ __attribute__((aligned(16))) Lds lds;
  const KvView &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint8_t *ring = lds.ring + wave * S * T::BYTES;
  const uint32_t ring_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)ring;
  const int Hq = kv.H * a.G;
  if constexpr (!MX) fill_attn_lut<LS, NT>(lds.lut, tid);         // read after the barrier below

  // ---- the share [u, end) of the runs, by every wave for itself
  int u = 0, end = 0, b0 = 0, base = 0;                      // base: runs before sequence b0
  AttnChunk k;
  if (a.shared) {
    k = attn_chunk(a, 0, M, lane);
    int total = __builtin_amdgcn_readlane(k.sum, 63);
    for (int i = 64; i < kv.B; i += 64) total += __builtin_amdgcn_readlane(attn_chunk(a, i, M, lane).sum, 63);
    const int share = attn_share(total);
    u = blockIdx.x * share;
    end = min(total, u + share);
  }
  if constexpr (!MX) __syncthreads();

  for (;;) {
    // ---- the next problem: tile mt, head h of sequence bb; its runs [q0, q1)
    int bb, mt, h, q0 = 0, q1;
    AttnSeq x;
    if (a.shared) {
      if (u >= end) return;
      uint64_t past;
      while ((past = __ballot(base + k.sum > u)) == 0) {     // sequences without rows have no runs
        base += __builtin_amdgcn_readlane(k.sum, 63);
        b0 += 64;
        k = attn_chunk(a, b0, M, lane);
      }
      const int l = __builtin_ctzll(past);
      bb = b0 + l;
      x = attn_seq(a, attn_pick(k, l), M);
      const int rel = u - (base + __builtin_amdgcn_readlane(k.sum, l) - attn_units(a, x));
      const int item = rel / x.units;
      q0 = rel - item * x.units;
      mt = item / kv.H;
      h = item - mt * kv.H;
      q1 = min(x.units, q0 + (end - u));
      u += q1 - q0;
    } else {
      int idx = (int)blockIdx.x;
      h = idx % kv.H;
      idx /= kv.H;
      mt = idx % a.n_mt;
      bb = idx / a.n_mt;
      x = attn_seq(a, attn_raw(kv, bb), M);
      if (mt >= x.mts) return;
      q1 = x.units;
    }
    const bool whole = q0 == 0 && q1 == x.units;
    // Tiles of late tokens see more than those of early ones: they alternate, so
    // that shares of several tiles come out alike.
    mt = (mt & 1) ? x.mts - 1 - (mt >> 1) : mt >> 1;
    const int row0 = mt * M, last = min(row0 + M, x.rows) - 1;
    const int full_hi = x.start + row0 / a.G;                // every row sees from full_lo to full_hi
    // (not below 0 - window: a window may be as wide as the type)
    const int full_lo = a.window > 0 ? max(x.start + last / a.G, 0) - a.window + 1 : 0;
    // the run's positions, among those that some row of this tile sees
    const int lo = a.window > 0 ? max(0, max(full_hi, 0) - a.window + 1) & ~31 : 0;
    const int hi = min(x.hi, x.start + last / a.G + 1);
    const int t0 = lo + q0 * kAttnUnit, t1 = q1 == x.units ? hi : min(hi, lo + q1 * kAttnUnit);

    // ---- S - 1 tiles under way, then the queries
    const int first = t0 + wave * 32, tiles = first < t1 ? (t1 - first + ROUND - 1) / ROUND : 0;
    uint32_t bad = 0;                                        // two bits per slot
    const int64_t hr = (int64_t)h << kv.page_shift;
    AttnPlace pl;
    pl.k = kv.k_codes + hr * (D / 2);
    pl.v = kv.v_codes + hr * (D / 2);
    pl.ks = static_cast<const uint8_t *>(kv.k_scales) + hr * (T::SC / 32);
    pl.vs = static_cast<const uint8_t *>(kv.v_scales) + hr * (T::SC / 32);
    pl.page_rows = kv.H << kv.page_shift;
    pl.page_shift = kv.page_shift;
    pl.n_pages = kv.n_pages;
    attn_pages(pl, kv, bb, first + lane * ROUND);
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
      if (i < tiles) bad |= attn_send<FMT, D>(pl, i, first + i * ROUND, ring_at + i * T::BYTES, lane) << (2 * i);
    AttnWave<FMT, D, NQ> w;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = row0 + n * 16 + c, tok = row / a.G;
      const bool ok = row < x.rows;
      w.qpos[n] = ok ? max(x.start + tok, -1) : -1;             // below 0: sees nothing
      w.m[n] = kNegInf;
      w.l[n] = 0.0f;
      const uint16_t *qp = a.q + (int64_t)(x.r0 + tok) * a.q_stride + (int64_t)(h * a.G + row - tok * a.G) * D;
      w.sc[n] = a.scale_log2;
      if (!QLDS || n % NW == wave) {                         // the waves share the loading
        uint4 v[KS];
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          const int d = MX ? g * (D / 4) + i * 8 : (i >> 1) * 64 + g * 16 + (i & 1) * 8;
          v[i] = make_uint4(0, 0, 0, 0);
          if (ok) v[i] = *reinterpret_cast<const uint4 *>(qp + d);
          v[i].x ^= a.q_sign;
          v[i].y ^= a.q_sign;
          v[i].z ^= a.q_sign;
          v[i].w ^= a.q_sign;
        }
        if constexpr (!MX)                                   // not 0 or inf: masked scores are -inf, others may be 0
          w.sc[n] = fminf(fmaxf(w.sc[n] * nf4_query<KS>(v), 1e-37f), 1e38f);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          if constexpr (QLDS) lds.q[(n * KS + i) * 64 + lane] = v[i];
          else w.q[n][i] = __builtin_bit_cast(bf16x8_t, v[i]);
        }
        if constexpr (QLDS) lds.qsc[n * 16 + c] = w.sc[n];
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) w.o[n][d] = f32x4_t{0, 0, 0, 0};
    }
    // The queries are here before the loop: a wait for them inside it would be
    // one for the tiles under way as well.
    if constexpr (QLDS) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NQ; ++n) w.sc[n] = lds.qsc[n * 16 + c];
    } else {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < KS; ++i) asm volatile("" : "+v"(w.q[n][i]));
    }

    int slot = 0, next = S - 1;                              // of this tile, of the one sent now
    // Sends the tile S - 1 further and waits for tile i.
    auto advance = [&](int i) {
      const int ahead = i + S - 1;
      if (ahead < tiles) {
        if ((ahead & 63) == 0) attn_pages(pl, kv, bb, first + (ahead + lane) * ROUND);
        bad &= ~(3u << (2 * next));
        bad |= attn_send<FMT, D>(pl, ahead & 63, first + ahead * ROUND, ring_at + next * T::BYTES, lane) << (2 * next);
        wait_vm<(S - 1) * T::LOADS>();
      } else if (S > 2 && i + 1 < tiles) {
        wait_vm<T::LOADS>();
      } else {
        wait_vm<0>();
      }
    };
    auto done = [&] {
      slot = slot + 1 == S ? 0 : slot + 1;
      next = next + 1 == S ? 0 : next + 1;
    };
    auto full = [&](int i) {
      const int t = first + i * ROUND;
      return t >= full_lo && t + 31 <= full_hi && ((bad >> (2 * slot)) & 3u) == 0;
    };
    // Of the waves of a SIMD the oldest is served first, and would be done a
    // quarter of the time before the last; in turns they end together.
    auto turn = [&](int i) {
      if ((i ^ (wave >> 2)) & 1) __builtin_amdgcn_s_setprio(1);
      else __builtin_amdgcn_s_setprio(0);
    };
    // Two loops, so that the accumulators keep their registers in each.
    for (int i = 0; i < tiles;) {
      for (; i < tiles && full(i); ++i) {
        advance(i);
        turn(i);
        attn_tile<FMT, D, NQ, false, LS>(w, ring + slot * T::BYTES, false, a, lds.lut, lds.q, first + i * ROUND, lane);
        done();
      }
      for (; i < tiles && !full(i); ++i) {
        advance(i);
        turn(i);
        const bool off = ((bad >> (2 * slot + (lane >> 5))) & 1u) != 0;
        attn_tile<FMT, D, NQ, true, LS>(w, ring + slot * T::BYTES, off, a, lds.lut, lds.q, first + i * ROUND, lane);
        done();
      }
    }

    // ---- join the waves
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      w.l[n] = sum_xor16_32(w.l[n]);
      if (g == 0) {
        lds.sm[wave][n * 16 + c] = w.m[n];
        lds.sl[wave][n * 16 + c] = w.l[n];
      }
    }
    __syncthreads();                                         // all tiles are read: their slots become red
    // a problem that goes on from the workgroup before lies in this one's first
    // slot of the partial results, one that goes on in the next in its second
    const int64_t part = 2 * (int64_t)blockIdx.x + (q0 == 0 ? 1 : 0);
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = n * 16 + c;
      float top = lds.sm[0][r];
#pragma unroll
      for (int v = 1; v < NW; ++v) top = fmaxf(top, lds.sm[v][r]);
      const float f = __builtin_amdgcn_exp2f(w.m[n] - (top == kNegInf ? 0.0f : top));
      float *mine = lds.red + (wave * 16 + c) * (D + 4);
      // four values of the row at a time: MXFP4 row index 4g + i of every tile d
      // is value (4g + i) D/16 + d, NF4 value 64 (d / 4) + 4 (4g + i) + d % 4
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int d = 0; d < ND; d += 4)
          *reinterpret_cast<float4 *>(mine + (MX ? (g * 4 + i) * (D / 16) + d : d * 16 + (g * 4 + i) * 4)) =
              make_float4(w.o[n][d][i] * f, w.o[n][d + 1][i] * f, w.o[n][d + 2][i] * f, w.o[n][d + 3][i] * f);
      __syncthreads();
      for (int k4 = tid; k4 < 16 * (D / 4); k4 += NT) {
        const int rr = k4 / (D / 4), d4 = (k4 - rr * (D / 4)) * 4;
        const int kr = n * 16 + rr, row = row0 + kr;
        if (row < x.rows) {
          float4 s = make_float4(0, 0, 0, 0);
          float mr = lds.sm[0][kr], l = 0.0f;
#pragma unroll
          for (int v = 0; v < NW; ++v) {
            const float4 o = *reinterpret_cast<const float4 *>(lds.red + (v * 16 + rr) * (D + 4) + d4);
            s.x += o.x;
            s.y += o.y;
            s.z += o.z;
            s.w += o.w;
            mr = fmaxf(mr, lds.sm[v][kr]);
          }
          const float mrs = mr == kNegInf ? 0.0f : mr;
#pragma unroll
          for (int v = 0; v < NW; ++v) l += lds.sl[v][kr] * __builtin_amdgcn_exp2f(lds.sm[v][kr] - mrs);
          if (whole) {
            const int tok = row / a.G, hq = h * a.G + row - tok * a.G;
            const AttnScale z = attn_finish(mr, l, a.sinks, hq);
            *reinterpret_cast<uint2 *>(a.out + (int64_t)(x.r0 + tok) * a.out_stride + (int64_t)hq * D + d4) =
                make_uint2(pk_bf16(s.x * z.mul, s.y * z.mul), pk_bf16(s.z * z.mul, s.w * z.mul));
            if (a.lse && d4 == 0) a.lse[(int64_t)(x.r0 + tok) * Hq + hq] = z.lse;
          } else {
            const int64_t pr = part * M + kr;
            *reinterpret_cast<float4 *>(a.part + pr * D + d4) = s;
            if (d4 == 0) *reinterpret_cast<float2 *>(a.part + 2LL * kAttnGroups * M * D + pr * 2) = make_float2(mr, l);
          }
        }
      }
      __syncthreads();
    }
    if (!a.shared) return;
  }
}

// Puts together the problems that lie in several shares: a workgroup per problem,
// a thread per four values of a row.
constexpr int kJoinThreads = 512;

template <int D>
__global__ __launch_bounds__(kJoinThreads) void kv_attn_join_kernel(KvAttnArgs a, int M) {
  const KvView &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63;
  int idx = (int)blockIdx.x;
  const int h = idx % kv.H;
  idx /= kv.H;
  int mt = idx % a.n_mt;
  const int b = idx / a.n_mt;
  const AttnSeq x = attn_seq(a, attn_raw(kv, b), M);
  int first = 0, total = 0;
  for (int i = 0; i < kv.B; i += 64) {
    const int sum = attn_chunk(a, i, M, lane).sum;
    if (b >= i && b < i + 64) first = total + __builtin_amdgcn_readlane(sum, b - i) - attn_units(a, x);
    total += __builtin_amdgcn_readlane(sum, 63);
  }
  if (mt >= x.mts) return;
  const int share = attn_share(total);
  first += (mt * kv.H + h) * x.units;
  const int w0 = first / share, w1 = (first + x.units - 1) / share;
  if (w0 == w1) return;                                      // written by its only workgroup
  const int n = w1 - w0 + 1;
  mt = (mt & 1) ? x.mts - 1 - (mt >> 1) : mt >> 1;           // the order of the shares
  const float2 *ml = reinterpret_cast<const float2 *>(a.part + 2LL * kAttnGroups * M * D);
  for (int u = tid; u < M * (D / 4); u += kJoinThreads) {
    const int r = u / (D / 4), d4 = (u - r * (D / 4)) * 4, row = mt * M + r;
    if (row >= x.rows) break;
    // the first workgroup's second slot, the first slots of the others
    auto at = [&](int s) { return (int64_t)(2 * (w0 + s) + (s == 0 ? 1 : 0)) * M + r; };
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

// Waves and slots of a workgroup that has a compute unit to itself: eight waves
// of up to 256 registers, four where a wave of 256 values has two tiles or the
// slots would not fit beside the NF4 table (64 of 160 KB); the third slot where
// there is room (for NF4 it takes a smaller table, which costs more than the
// slot gains: 39 us became 42 in the 32 sequences above).
template <int FMT, int D, int NQ>
struct AttnCfg {
  static constexpr bool MX = FMT == GNF4_MXFP4;
  static constexpr int NW = D == 256 && (!MX || NQ == 2) ? 4 : 8;
  static constexpr int S = NW == 8 && MX && D <= 128 ? 3 : 2;
};

// The most 16-row tiles of a wave whose results the registers hold: a step
// decodes K and V once for all of them.
constexpr int attn_most_tiles(int format, int D) {
  return D == 256 ? 2 : D == 64 ? 4 : format == GNF4_MXFP4 ? 3 : 2;
}

constexpr int kAttnShort = 1024;

// Rows per tile from the most new tokens of a sequence. Short contexts take a
// workgroup per problem and one launch; where these are at least as many as
// compute units, of four waves, so that several fit on one.
bool kv_attention_plan(int32_t format, int32_t D, int32_t H, int32_t G, int32_t B, int64_t n_tokens, int32_t max_new,
                       int64_t max_len, int64_t capacity, int32_t window, KvAttnPlan *p) {
  const int64_t rows = (int64_t)max_new * G;
  p->nq = rows <= 16 ? 1 : rows <= 32 ? 2 : attn_most_tiles(format, D);
  // a short context is a small problem also with many rows
  const int64_t seen = window > 0 ? std::min<int64_t>(max_len, (int64_t)window + 64) : max_len;
  if (seen <= kAttnShort && p->nq > 2) p->nq = 2;
  // Two tiles of 256 values take four waves a compute unit. NF4 has no more with
  // one (2 x 1024 rows of 4 heads over 4000: 401 us, 565 with one); MXFP4 has
  // eight, so that two pay only over many positions (226 us, 262; 8 x 40 rows
  // over 4097: 39 us, 34).
  if (D == 256 && format == GNF4_MXFP4 && p->nq == 2 &&
      (seen <= kAttnShort || (int64_t)B * H * ((rows + 31) / 32) * seen < 1 << 19))
    p->nq = 1;
  const int M = 16 * p->nq;
  const int64_t n_mt = (rows + M - 1) / M;
  p->items = (int64_t)B * n_mt * H;
  int64_t len = std::max<int64_t>(max_len, 1);
  p->tile_tokens = (int32_t)std::min<int64_t>((M - 1 + G - 1) / G + 1, max_new);
  if (window > 0) len = std::min<int64_t>(len, (int64_t)window + p->tile_tokens - 1 + 31);
  if (p->items >= 1 << 23) return false;                     // a launch has fewer than 2^32 threads
  p->n_mt = (int32_t)n_mt;
  p->shared = len > kAttnShort;
  p->small = !p->shared && p->items >= kAttnGroups;
  // the runs are counted in 32 bits
  if (p->shared && p->items * ((capacity + kAttnUnit - 1) / kAttnUnit) > 0x7fff0000LL) p->shared = 0;
  p->bytes = p->shared ? (size_t)(2 * kAttnGroups * M) * (D + 2) * 4 : 0;
  return true;
}

template <int FMT, int D, int NQ, int NW, int S>
static hipError_t attn_go(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  hipLaunchKernelGGL((kv_attn_kernel<FMT, D, NQ, NW, S>), dim3(p.shared ? kAttnGroups : (unsigned)p.items), dim3(64 * NW),
                     0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.shared) return e;
  hipLaunchKernelGGL((kv_attn_join_kernel<D>), dim3((unsigned)p.items), dim3(kJoinThreads), 0, s, a, 16 * NQ);
  return hipGetLastError();
}

template <int FMT, int D>
static hipError_t attn_nq(const KvAttnArgs &a, const KvAttnPlan &p, hipStream_t s) {
  if constexpr (D <= 128) {
    if (p.small && p.nq == 2) return attn_go<FMT, D, 2, 4, 2>(a, p, s);
    constexpr int most = attn_most_tiles(FMT, D);
    if (p.nq == most && most > 2) return attn_go<FMT, D, most, AttnCfg<FMT, D, most>::NW, AttnCfg<FMT, D, most>::S>(a, p, s);
    if (p.nq == 2) return attn_go<FMT, D, 2, AttnCfg<FMT, D, 2>::NW, AttnCfg<FMT, D, 2>::S>(a, p, s);
  }
  if constexpr (D == 256) {
    if (p.nq == 2) return attn_go<FMT, D, 2, AttnCfg<FMT, D, 2>::NW, AttnCfg<FMT, D, 2>::S>(a, p, s);
  }
  if (p.small) return attn_go<FMT, D, 1, 4, 2>(a, p, s);
  return attn_go<FMT, D, 1, AttnCfg<FMT, D, 1>::NW, AttnCfg<FMT, D, 1>::S>(a, p, s);
}

hipError_t launch_kv_attention(const KvAttnArgs &args, const KvAttnPlan &p, int32_t format, hipStream_t s) {
  KvAttnArgs a = args;
  a.n_mt = p.n_mt;
  a.shared = p.shared;
  a.tile_tokens = p.tile_tokens;
  // The running maximum is taken before the scale, which therefore must not be
  // negative (the queries change sign instead) nor 0 (0 times the -inf of a
  // masked place; 2^-100 leaves the weights equal) nor infinite (0 times that).
  a.q_sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
  a.scale_log2 = std::min(std::max(std::fabs(a.scale_log2), 0x1p-100f), 0x1p127f);
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
