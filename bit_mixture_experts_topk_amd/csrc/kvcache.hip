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
// found across the 4 (MXFP4) or 8 (NF4) lanes that hold it. 5 prompts, 12500
// tokens of 8 heads of 128, NF4 (61 MB each way): write 19.1 to 21 us, read 13.7
// to 15, 3 to 4.3 TB/s; below that lie the search for a row's place and the
// codes' arithmetic, which the loads of other workgroups cover in part.
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

// NF4 codes of x = w / absmax by one look-up and one comparison. Cell c covers
// [c/32 - 1, (c+1)/32 - 1): at most one midpoint of neighbouring codebook values
// lies in it (the closest two are 0.08 apart), so the code of x, in the cell
// or beside it, is base + (x > that midpoint), base the midpoints below the
// cell. A word holds both: the midpoint's float32 with base in its low four
// bits, within 8 units in the last place of it.
// That float32 decides as exact arithmetic does: w and absmax are bf16, and
// of all quotients of two 8-bit significands the one nearest to a midpoint is
// 5.4e-7 off (enumerated), while x = w * (1/absmax) is off by 0.7e-7 at most
// there and the word by 2.4e-7.
constexpr int kNf4Cells = 65;

struct Nf4CellTable {
  uint32_t w[kNf4Cells];
};

constexpr Nf4CellTable nf4_cells() {
  Nf4CellTable t{};
  for (int c = 0; c < kNf4Cells; ++c) {
    const double left = c / 32.0 - 1.0;
    uint32_t base = 0;
    double mid = 2.0;                                        // past every x
    for (int i = 14; i >= 0; --i) {
      const double m = 0.5 * ((double)__builtin_bit_cast(float, kNF4Bits[i]) +
                              (double)__builtin_bit_cast(float, kNF4Bits[i + 1]));
      if (m >= left) mid = m;
      else if (base == 0) base = (uint32_t)i + 1;
    }
    t.w[c] = ((__builtin_bit_cast(uint32_t, (float)mid) - base + 8u) & ~15u) | base;
  }
  return t;
}

__constant__ const Nf4CellTable kCells = nf4_cells();

__device__ __forceinline__ uint32_t nf4_code(const uint32_t *cells, float x) {
  const uint32_t w = cells[(int)fmaf(x, 32.0f, 32.0f)];
  return (w & 15u) + (x > __builtin_bit_cast(float, w) ? 1u : 0u);
}

// How a workgroup of 256 goes through the chunks of 8 values of its tokens: a
// token has 2 H D/8 of them, its keys' then its values'. Tokens of few chunks
// are taken side by side, long ones in several steps; a thread's chunk then
// stays the same from token to token. H*D/4 is a multiple of 16, so the lanes of
// a block are together.
struct KvWalk {
  int per, side, abreast;                                    // chunks per token and side, tokens side by side
  int i, rem;                                                // the thread's first token and chunk
};

__device__ __forceinline__ KvWalk kv_walk(const KvView &kv, int tid) {
  KvWalk x;
  x.side = kv.H * (kv.D >> 3);
  x.per = 2 * x.side;
  x.abreast = x.per >= kKvThreads ? 1 : kKvThreads / x.per;
  x.i = x.per >= kKvThreads ? 0 : tid / x.per;
  x.rem = tid - x.i * x.per;
  if (x.i >= x.abreast) x.rem = x.per;                       // the threads that are left over
  return x;
}

// Where the tokens' rows lie is found once per workgroup, by every wave for
// itself (its lane i holds token t0 + i's).
template <int FMT>
__global__ __launch_bounds__(kKvThreads) void kv_write_kernel(KvRowsArgs a, int tokens) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  __shared__ uint32_t cells[MX ? 1 : kNf4Cells];
  const KvView &kv = a.kv;
  const int lane = threadIdx.x & 63, tid = threadIdx.x;
  const int t0 = (int)blockIdx.x * tokens, n = min(tokens, kv.n_tokens - t0);
  const KvWalk z = kv_walk(kv, tid);
  const int dshift = __builtin_ctz(kv.D) - 3;                // chunks per head
  if (!MX) {
    if (tid < kNf4Cells) cells[tid] = kCells.w[tid];
    __syncthreads();
  }
  const int64_t rows = kv_rows(kv, t0, n, lane);
  for (int rem = z.rem; rem - z.rem < z.per; rem += kKvThreads) {
    const bool mine = rem < z.per, is_v = rem >= z.side;
    const int hc = is_v ? rem - z.side : rem, h = hc >> dshift, c = hc & ((1 << dshift) - 1);
    const uint16_t *src = (is_v ? a.v : a.k) + (int64_t)hc * 8;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    uint8_t *codes_at = (is_v ? kv.v_codes : kv.k_codes) + 4 * c;
    uint8_t *scales_at = static_cast<uint8_t *>(is_v ? kv.v_scales : kv.k_scales);
    auto chunk = [&](int i) {
      return mine && i < n ? *reinterpret_cast<const uint4 *>(src + (t0 + i) * stride) : make_uint4(0, 0, 0, 0);
    };
    uint4 x = chunk(z.i), xn = chunk(z.i + z.abreast);
    for (int i0 = 0; i0 < n; i0 += z.abreast) {              // whole waves: lanes share their blocks
      const int i = i0 + z.i;
      const uint4 xf = chunk(i + 2 * z.abreast);
      int64_t row = __shfl(rows, i & 63, 64);
      if (!mine || i >= n) row = -1;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      x = xn;
      xn = xf;
      uint32_t mag = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) mag = max(mag, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
      mag = group_max_u32<MX ? 4 : 8>(mag);
      uint32_t codes = 0;
      const bool finite = mag < 0x7f80u;                     // else: the block reads back as NaN
      if constexpr (MX) {
        int s = 255;
        if (finite) {
          s = mag ? min(max(bf16_floor_log2(mag) - 2 + 127, 0), 254) : 0;
          // The conversion divides by the scale. A scale below 2^-63 is brought
          // up with its values by 2^64 (exact: such values are below 2^-60).
          const bool tiny = s < 64;
          const float up = tiny ? 0x1p64f : 1.0f;
          const float sc = __builtin_bit_cast(float, (uint32_t)(tiny ? s + 64 : s) << 23);
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[2 * j] = __builtin_bit_cast(float, w[j] << 16) * up;
            f[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xffff0000u) * up;
          }
          codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[0], f[1], sc, 0);
          codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[2], f[3], sc, 1);
          codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[4], f[5], sc, 2);
          codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, f[6], f[7], sc, 3);
        }
        if (row < 0) continue;
        row += (int64_t)h << kv.page_shift;
        *reinterpret_cast<uint32_t *>(codes_at + row * (kv.D >> 1)) = codes;
        if ((c & 3) == 0) scales_at[row * (kv.D >> 5) + (c >> 2)] = (uint8_t)s;
      } else {
        const float absmax = __builtin_bit_cast(float, finite ? mag << 16 : 0x7fc00000u);
        codes = 0x77777777u;                                 // code 7 is the exact zero
        if (finite && mag) {
          // absmax brought into [1, 2), its reciprocal is then within an ulp
          const int e = -bf16_floor_log2(mag);
          const float inv = __builtin_amdgcn_rcpf(ldexpf(absmax, e));
          codes = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t q0 = nf4_code(cells, ldexpf(__builtin_bit_cast(float, w[j] << 16), e) * inv);
            const uint32_t q1 = nf4_code(cells, ldexpf(__builtin_bit_cast(float, w[j] & 0xffff0000u), e) * inv);
            codes |= ((q0 << 4) | q1) << (8 * j);
          }
        }
        if (row < 0) continue;
        row += (int64_t)h << kv.page_shift;
        *reinterpret_cast<uint32_t *>(codes_at + row * (kv.D >> 1)) = codes;
        if ((c & 7) == 0) reinterpret_cast<float *>(scales_at)[row * (kv.D >> 6) + (c >> 3)] = absmax;
      }
    }
  }
}

// The reverse. NF4 values come two at a time from an LDS table of the 256
// bytes, MXFP4 values from the hardware conversion.
template <int FMT, bool F32>
__global__ __launch_bounds__(kKvThreads) void kv_read_kernel(KvRowsArgs a, int tokens) {
  constexpr bool MX = FMT == GNF4_MXFP4;
  __shared__ float2 pairs[MX ? 1 : 256];
  const KvView &kv = a.kv;
  const int lane = threadIdx.x & 63, tid = threadIdx.x;
  const int t0 = (int)blockIdx.x * tokens, n = min(tokens, kv.n_tokens - t0);
  const KvWalk z = kv_walk(kv, tid);
  const int dshift = __builtin_ctz(kv.D) - 3;
  if (!MX) {                                                 // element 2j in the high nibble
    pairs[tid] = make_float2(__builtin_bit_cast(float, kNF4Bits[tid >> 4]), __builtin_bit_cast(float, kNF4Bits[tid & 15]));
    __syncthreads();
  }
  const int64_t rows = kv_rows(kv, t0, n, lane);
  constexpr int U = 4;                                       // tokens whose loads are in flight together
  for (int rem = z.rem; rem - z.rem < z.per; rem += kKvThreads) {
    const bool mine = rem < z.per, is_v = rem >= z.side;
    const int hc = is_v ? rem - z.side : rem, h = hc >> dshift, c = hc & ((1 << dshift) - 1);
    const uint8_t *codes = (is_v ? kv.v_codes : kv.k_codes) + 4 * c;
    const uint8_t *scales = static_cast<const uint8_t *>(is_v ? kv.v_scales : kv.k_scales);
    for (int i0 = z.i; i0 - z.i < n; i0 += U * z.abreast) {
      uint32_t q[U], s[U];
      bool live[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * z.abreast;
        int64_t row = __shfl(rows, i & 63, 64);
        live[u] = mine && i < n && row >= 0;
        row = live[u] ? row + ((int64_t)h << kv.page_shift) : 0;
        q[u] = *reinterpret_cast<const uint32_t *>(codes + row * (kv.D >> 1));
        if (MX) s[u] = scales[row * (kv.D >> 5) + (c >> 2)];
        else s[u] = reinterpret_cast<const uint32_t *>(scales)[row * (kv.D >> 6) + (c >> 3)];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!live[u]) continue;
        const int64_t at = (int64_t)(t0 + i0 + u * z.abreast) * z.side * 8 + (int64_t)hc * 8;
        void *dst = is_v ? a.v_out : a.k_out;
        if constexpr (MX && !F32) {
          // exact in bf16: the conversion's result is the value (255 gives NaN)
          const float sc = __builtin_bit_cast(float, s[u] << 23);
          uint4 o = make_uint4(fp4_pair<0>(q[u], sc), fp4_pair<1>(q[u], sc), fp4_pair<2>(q[u], sc), fp4_pair<3>(q[u], sc));
          if (s[u] == 255u) o = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
          *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + at) = o;
        } else {
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (MX) {
              const float sc = e8m0_to_f32(s[u]);
              const uint32_t b = (q[u] >> (8 * j)) & 0xffu;
              const float m0 = kE2M1[b & 7u], m1 = kE2M1[(b >> 4) & 7u];
              f[2 * j] = ((b & 8u) ? -m0 : m0) * sc;
              f[2 * j + 1] = ((b & 0x80u) ? -m1 : m1) * sc;
            } else {
              const float sc = __builtin_bit_cast(float, s[u]);
              const float2 p = pairs[(q[u] >> (8 * j)) & 0xffu];
              f[2 * j] = p.x * sc;
              f[2 * j + 1] = p.y * sc;
            }
          }
          if constexpr (F32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(dst) + at);
            o[0] = make_float4(f[0], f[1], f[2], f[3]);
            o[1] = make_float4(f[4], f[5], f[6], f[7]);
          } else {
            typedef float f32x2_t __attribute__((ext_vector_type(2)));
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x2_t v = {f[2 * j], f[2 * j + 1]};
              o[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
              if (f[2 * j] != f[2 * j]) o[j] = (o[j] & 0xffff0000u) | 0x7fc0u;
              if (f[2 * j + 1] != f[2 * j + 1]) o[j] = (o[j] & 0xffffu) | 0x7fc00000u;
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + at) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    }
  }
}

// Tokens per workgroup: up to 16, over which the search for their rows is
// spread, as long as eight workgroups per compute unit remain (12500 tokens of
// 8 heads, NF4: 19.9 us to write with 4, 22.7 with 2, 21.3 with 16).
static int kv_tokens(const KvView &kv) {
  int n = 1;
  while (n < 16 && kv.n_tokens / (2 * n) >= 2048) n *= 2;
  return n;
}

hipError_t launch_kv_write(const KvRowsArgs &a, int32_t format, hipStream_t s) {
  const int n = kv_tokens(a.kv);
  const dim3 grid((unsigned)((a.kv.n_tokens + n - 1) / n)), block(kKvThreads);
  if (format == GNF4_MXFP4) hipLaunchKernelGGL(kv_write_kernel<GNF4_MXFP4>, grid, block, 0, s, a, n);
  else hipLaunchKernelGGL(kv_write_kernel<GNF4_NF4>, grid, block, 0, s, a, n);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvRowsArgs &a, int32_t format, int32_t out_f32, hipStream_t s) {
  const int n = kv_tokens(a.kv);
  const dim3 grid((unsigned)((a.kv.n_tokens + n - 1) / n)), block(kKvThreads);
  if (format == GNF4_MXFP4) {
    if (out_f32) hipLaunchKernelGGL((kv_read_kernel<GNF4_MXFP4, true>), grid, block, 0, s, a, n);
    else hipLaunchKernelGGL((kv_read_kernel<GNF4_MXFP4, false>), grid, block, 0, s, a, n);
  } else {
    if (out_f32) hipLaunchKernelGGL((kv_read_kernel<GNF4_NF4, true>), grid, block, 0, s, a, n);
    else hipLaunchKernelGGL((kv_read_kernel<GNF4_NF4, false>), grid, block, 0, s, a, n);
  }
  return hipGetLastError();
}

}  // namespace gnf4
