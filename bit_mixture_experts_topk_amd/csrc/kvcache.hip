// The paged 4-bit cache of keys and values: quantize new rows into it, and
// read rows back.
//
// The formats are those of the packed weights, along a head's D values: NF4
// with one float32 absmax per 64, MXFP4 with one e8m0 scale per 32 (the pages
// list paged decode attention over a quantized cache among the package's
// tasks: "MoE Training on Consumer GPUs -- Loggetta & Cerin Amroth", Task
// guides table; the 4-bit cache is this library's form of it). Both kernels
// are bound by the bytes they move (4 bytes in, about 0.55 out per pair of
// values for the write, the reverse for the read), so a thread takes 8
// consecutive values: one 16-byte access on the bf16 side and one dword of
// codes, neighbouring threads neighbouring chunks. A block's largest value is
// found across the 4 (MXFP4) or 8 (NF4) lanes that hold it.
#include "kvcache.h"

namespace gnf4 {

constexpr int kKvThreads = 256;

// max over the lane's aligned group of 4 (quad_perm swaps) or 8 lanes
// (row_half_mirror joins the two quads).
template <int GROUP>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));   // quad_perm 1,0,3,2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));   // quad_perm 2,3,0,1
  if (GROUP == 8)
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));  // row_half_mirror
  return v;
}

// floor(log2) of a positive bf16 value given by its 15 magnitude bits.
__device__ __forceinline__ int bf16_floor_log2(uint32_t mag) {
  return mag >= 0x80u ? (int)(mag >> 7) - 127 : (31 - __builtin_clz(mag)) - 133;
}

// The midpoint m_i of codebook entries i and i+1 is half the sum of two
// float32 values: a float32 hi and, where that sum needs one more bit, a
// remainder lo (both exact). base counts the midpoints below the cell.
struct Nf4Cell {
  float hi, lo;
  int base;
};
constexpr int kNf4Cells = 65;

// Cell c covers x in [c/32 - 1, (c+1)/32 - 1): at most one midpoint lies in it
// (the closest two are 0.08 apart), so the code of x is base + (x > that
// midpoint), for x in the cell and up to the midpoints on either side.
__device__ __forceinline__ void fill_nf4_cells(Nf4Cell *cells, int tid) {
  if (tid < kNf4Cells) {
    const double left = (double)tid / 32.0 - 1.0;
    int base = 0;
    double mid = 2.0;                            // past every x / absmax
#pragma unroll
    for (int i = 0; i < 15; ++i) {
      const double m = 0.5 * ((double)__builtin_bit_cast(float, kNF4Bits[i]) +
                              (double)__builtin_bit_cast(float, kNF4Bits[i + 1]));
      if (m < left) base = i + 1;
    }
#pragma unroll
    for (int i = 14; i >= 0; --i) {
      const double m = 0.5 * ((double)__builtin_bit_cast(float, kNF4Bits[i]) +
                              (double)__builtin_bit_cast(float, kNF4Bits[i + 1]));
      if (i == base) mid = m;
    }
    cells[tid].hi = (float)mid;
    cells[tid].lo = (float)(mid - (double)(float)mid);
    cells[tid].base = base;
  }
}

// NF4 code of w against its block's a, both scaled so that a is in [1, 2): w
// > mid * a exactly. w and a hold 8 significant bits and mid 25, so hi * a - w
// is exact where it is small (the fma rounds once and keeps the sign
// otherwise), and it is compared with the exact lo * a. inv = 1 / a picks the
// cell only.
__device__ __forceinline__ uint32_t nf4_code(const Nf4Cell *cells, float w, float a, float inv) {
  const float t = fminf(fmaxf(w * inv, -1.0f), 1.0f);
  const Nf4Cell c = cells[(int)((t + 1.0f) * 32.0f)];
  return (uint32_t)c.base + (fmaf(-c.hi, a, w) > c.lo * a ? 1u : 0u);
}

// One thread per 8 values: the H*D/8 chunks of a token's keys, then those of
// its values. H*D/4 is a multiple of 16, so a block's lanes are together.
template <int FMT>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(KvRowsArgs a) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  __shared__ Nf4Cell cells[MX ? 1 : kNf4Cells];
  const KvView &kv = a.kv;
  const int lane = threadIdx.x & 63;
  const int side = kv.H * (kv.D >> 3), per = 2 * side;       // chunks per token
  const int64_t idx = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
  const int t = (int)(idx / per);
  const int rem = (int)(idx - (int64_t)t * per);
  const bool live = t < kv.n_tokens;
  const bool is_v = rem >= side;
  const int hc = is_v ? rem - side : rem;                    // chunk within the token's heads
  const int h = hc / (kv.D >> 3), c = hc - h * (kv.D >> 3);
  uint4 x = make_uint4(0, 0, 0, 0);
  if (live) {
    const uint16_t *src = is_v ? a.v + (int64_t)t * a.v_stride : a.k + (int64_t)t * a.k_stride;
    x = *reinterpret_cast<const uint4 *>(src + (int64_t)hc * 8);
  }
  if (!MX) {
    fill_nf4_cells(cells, threadIdx.x);
    __syncthreads();
  }
  // the row of every token of this wave (at most four)
  int64_t row = -1;
  uint64_t todo = __ballot(live);
  while (todo) {
    const int first = __builtin_ctzll(todo);
    const int r = __builtin_amdgcn_readlane(t, first);
    const int b = find_seq(kv.offsets, kv.B, r, lane);
    int64_t got = -1;
    if (b >= 0) got = kv_row0(kv, b, kv.lens[b] - kv.offsets[b + 1] + r);
    if (t == r) row = got;
    todo &= ~__ballot(t == r);
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) mag = max(mag, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  mag = group_max_u32<MX ? 4 : 8>(mag);
  uint32_t codes = 0;
  const bool finite = mag < 0x7f80u;                         // else: the block reads back as NaN
  if constexpr (MX) {
    int s = 255;
    if (finite) {
      s = mag ? min(max(bf16_floor_log2(mag) - 2 + 127, 0), 254) : 0;
      // The conversion divides by the scale. A scale below 2^-63 is brought up
      // with its values by 2^64 (exact: such values are below 2^-60).
      const bool tiny = s < 64;
      const float up = tiny ? 0x1p64f : 1.0f;
      const float sc = __builtin_bit_cast(float, (uint32_t)(tiny ? s + 64 : s) << 23);
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __builtin_bit_cast(float, w[i] << 16) * up;
        f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u) * up;
      }
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[0], f[1], sc, 0);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[2], f[3], sc, 1);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[4], f[5], sc, 2);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[6], f[7], sc, 3);
    }
    if (row < 0) return;
    row += (int64_t)h << kv.page_shift;
    uint8_t *dst = is_v ? kv.v_codes : kv.k_codes;
    reinterpret_cast<uint32_t *>(dst + row * (kv.D >> 1))[c] = codes;
    if ((c & 3) == 0)
      static_cast<uint8_t *>(is_v ? kv.v_scales : kv.k_scales)[row * (kv.D >> 5) + (c >> 2)] = (uint8_t)s;
  } else {
    float absmax = __builtin_bit_cast(float, finite ? mag << 16 : 0x7fc00000u);
    codes = 0x77777777u;                                     // code 7 is the exact zero
    if (finite && mag) {
      const int e = -bf16_floor_log2(mag);
      const float an = ldexpf(absmax, e), inv = 1.0f / an;
      codes = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f0 = ldexpf(__builtin_bit_cast(float, w[i] << 16), e);
        const float f1 = ldexpf(__builtin_bit_cast(float, w[i] & 0xffff0000u), e);
        codes |= ((nf4_code(cells, f0, an, inv) << 4) | nf4_code(cells, f1, an, inv)) << (8 * i);
      }
    }
    if (row < 0) return;
    row += (int64_t)h << kv.page_shift;
    uint8_t *dst = is_v ? kv.v_codes : kv.k_codes;
    reinterpret_cast<uint32_t *>(dst + row * (kv.D >> 1))[c] = codes;
    if ((c & 7) == 0)
      static_cast<float *>(is_v ? kv.v_scales : kv.k_scales)[row * (kv.D >> 6) + (c >> 3)] = absmax;
  }
}

// The reverse: one thread per 8 values of the step's rows. The 16 code values
// sit in lanes 0..15 of a register and reach each lane through ds_bpermute.
template <int FMT, bool F32>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvRowsArgs a) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  const KvView &kv = a.kv;
  const int lane = threadIdx.x & 63;
  const int side = kv.H * (kv.D >> 3), per = 2 * side;
  const int64_t idx = (int64_t)blockIdx.x * kKvThreads + threadIdx.x;
  const int t = (int)(idx / per);
  const int rem = (int)(idx - (int64_t)t * per);
  const bool live = t < kv.n_tokens;
  const bool is_v = rem >= side;
  const int hc = is_v ? rem - side : rem;
  const int h = hc / (kv.D >> 3), c = hc - h * (kv.D >> 3);
  int64_t row = -1;
  uint64_t todo = __ballot(live);
  while (todo) {
    const int first = __builtin_ctzll(todo);
    const int r = __builtin_amdgcn_readlane(t, first);
    const int b = find_seq(kv.offsets, kv.B, r, lane);
    int64_t got = -1;
    if (b >= 0) got = kv_row0(kv, b, kv.lens[b] - kv.offsets[b + 1] + r);
    if (t == r) row = got;
    todo &= ~__ballot(t == r);
  }
  uint32_t q = 0;
  float sc = 0.0f;
  if (row >= 0) {
    row += (int64_t)h << kv.page_shift;
    q = reinterpret_cast<const uint32_t *>((is_v ? kv.v_codes : kv.k_codes) + row * (kv.D >> 1))[c];
    const void *scales = is_v ? kv.v_scales : kv.k_scales;
    if (MX) sc = e8m0_to_f32(static_cast<const uint8_t *>(scales)[row * (kv.D >> 5) + (c >> 2)]);
    else sc = static_cast<const float *>(scales)[row * (kv.D >> 6) + (c >> 3)];
  }
  const float m = kE2M1[lane & 7];
  const float table = MX ? ((lane & 8) ? -m : m) : __builtin_bit_cast(float, kNF4Bits[lane & 15]);
  const int tbits = __builtin_bit_cast(int, table);
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = MX ? i : i ^ 1;                            // NF4: element 2i in the high nibble
    const int code = (int)((q >> (4 * n)) & 15u);
    f[i] = __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(code << 2, tbits)) * sc;
  }
  if (row < 0) return;
  const int64_t at = (int64_t)t * side * 8 + (int64_t)hc * 8;
  if constexpr (F32) {
    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(is_v ? a.v_out : a.k_out) + at);
    dst[0] = make_float4(f[0], f[1], f[2], f[3]);
    dst[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u0 = __builtin_bit_cast(uint32_t, f[2 * i]), u1 = __builtin_bit_cast(uint32_t, f[2 * i + 1]);
      const uint32_t r0 = f[2 * i] != f[2 * i] ? 0x7fc0u : bf16_rne(u0);
      const uint32_t r1 = f[2 * i + 1] != f[2 * i + 1] ? 0x7fc0u : bf16_rne(u1);
      o[i] = r0 | (r1 << 16);
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_v ? a.v_out : a.k_out) + at) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

static unsigned kv_blocks(const KvView &kv) {
  const int64_t threads = (int64_t)kv.n_tokens * 2 * kv.H * (kv.D / 8);
  return (unsigned)((threads + kKvThreads - 1) / kKvThreads);
}

hipError_t launch_kv_write(const KvRowsArgs &a, int32_t format, hipStream_t s) {
  const dim3 grid(kv_blocks(a.kv)), block(kKvThreads);
  if (format == GNF4_MXFP4) hipLaunchKernelGGL(kv_write_kernel<GNF4_MXFP4>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(kv_write_kernel<GNF4_NF4>, grid, block, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvRowsArgs &a, int32_t format, int32_t out_f32, hipStream_t s) {
  const dim3 grid(kv_blocks(a.kv)), block(kKvThreads);
  if (format == GNF4_MXFP4) {
    if (out_f32) hipLaunchKernelGGL((kv_read_kernel<GNF4_MXFP4, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((kv_read_kernel<GNF4_MXFP4, false>), grid, block, 0, s, a);
  } else {
    if (out_f32) hipLaunchKernelGGL((kv_read_kernel<GNF4_NF4, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((kv_read_kernel<GNF4_NF4, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace gnf4
