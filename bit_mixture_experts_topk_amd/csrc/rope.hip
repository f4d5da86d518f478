// Norm of every query and key head and the rotation by position, in one pass,
// and its backward pass.
//
//   n = w * x / sqrt(mean(x^2) + eps)                 (w NULL: n = x)
//   pairs (a, b) of the first rot_dim values of n, with angle t = pos * f_i:
//   y = mscale * (a cos t - b sin t, b cos t + a sin t), the rest of n as it is
//
// The pages run the packed experts behind a real attention (Jordan Anderson,
// jordananderson-pages.pages.dev, section "grouped-nf4-gemm & experts-4bit",
// demonstration paragraph of the first bullet) without describing it; the
// form is that of the public models the workloads are shaped after.
//
// Bound by memory: 4 bytes per value forward, 6 backward, and a handful of
// float32 operations. A head row lies in 8, 16 or 32 lanes (8 values each, one
// 16-byte access), its sums in DPP steps; a workgroup takes one token at a
// time, so that the angles, formed in float64 (pos * f of far positions has
// no fraction left in float32), are computed once for all its heads. 8192
// tokens of 64 + 4 heads of 128: 57 us, 5.0 TB/s (a 1 GiB copy: 5.2); backward,
// 4096 tokens of 32 + 4 heads: 32.5 us, 3.5 TB/s, and 4 for the weights' sums.
// The backward has three streams and two chained row sums per row, and its
// workgroups keep the weights' sums in registers over all their tokens.
#include <algorithm>

#include "rope.h"

namespace gnf4 {

constexpr int kRopeThreads = 256;

// Sum over the lane's aligned group of LPR lanes, in every lane.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xf, 0xf, true));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xf, 0xf, true));
  if (LPR >= 16)
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xf, 0xf, true));
  if (LPR >= 32) {
    auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v), __builtin_bit_cast(unsigned, v),
                                              false, false);
    v = __builtin_bit_cast(float, (unsigned)r[0]) + __builtin_bit_cast(float, (unsigned)r[1]);
  }
  return v;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __builtin_bit_cast(float, w[i] << 16);
    f[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2_t v = {f[2 * i], f[2 * i + 1]};
    w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// cos and sin of the token's rot_dim/2 angles into LDS, times mscale. The
// angle in turns, pos * f / 2 pi, is formed in float64 and only its fraction
// goes on in float32.
__device__ __forceinline__ void fill_angles(float *cs, float *sn, const RopeArgs &a, int pos, int tid) {
  if (tid < a.rot / 2) {
    const double turns = (double)pos * ((double)a.inv_freq[tid] * 0.15915494309189533577);
    const float f = (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * f, &s, &c);
    cs[tid] = c * a.mscale;
    sn[tid] = s * a.mscale;
  }
}

// Rotation of the lane's 8 values f (chunk c of a row of LPR lanes). Neighbouring
// pairs sit in the lane; with the half layout the partners of chunk c are those
// of chunk c +- rot/16, fetched across lanes. SIGN -1: the transposed rotation.
template <bool IL, int SIGN>
__device__ __forceinline__ void rotate8(float (&f)[8], const float *cs, const float *sn, int c, int rot, int lane) {
  if constexpr (IL) {
    if (8 * c < rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float co = cs[4 * c + i], si = SIGN * sn[4 * c + i];
        const float x = f[2 * i], y = f[2 * i + 1];
        f[2 * i] = x * co - y * si;
        f[2 * i + 1] = y * co + x * si;
      }
    }
  } else {
    const int half = rot >> 4;                               // chunks of each half
    const bool first = c < half, in = c < 2 * half;
    const int other = in ? (first ? lane + half : lane - half) : lane;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p[i] = __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(other << 2, __builtin_bit_cast(int, f[i])));
    if (in) {
      const int k = first ? 8 * c : 8 * (c - half);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float co = cs[k + i], si = SIGN * sn[k + i];
        f[i] = first ? f[i] * co - p[i] * si : f[i] * co + p[i] * si;
      }
    }
  }
}

// Row rr of a token: a query head, then a key head.
__device__ __forceinline__ uint4 load_row(const uint16_t *q, int64_t qs, const uint16_t *k, int64_t ks, int t, int rr,
                                          int Hq, int D, int d) {
  const uint16_t *p = rr < Hq ? q + (int64_t)t * qs + (int64_t)rr * D : k + (int64_t)t * ks + (int64_t)(rr - Hq) * D;
  return *reinterpret_cast<const uint4 *>(p + d);
}

template <int LPR, bool IL>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_kernel(RopeArgs a, int rows_per_block) {
  __shared__ __attribute__((aligned(16))) float cs[128], sn[128];
  constexpr int RPI = kRopeThreads / LPR;                    // head rows at a time
  const int tid = threadIdx.x, lane = tid & 63, c = tid % LPR, sub = tid / LPR, d = 8 * c;
  const int t = blockIdx.x, rows = a.Hq + a.Hk;
  const int first = (int)blockIdx.y * rows_per_block, last = min(first + rows_per_block, rows);
  const bool in = d < a.D;
  int rr = first + sub;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (in && rr < last) x = load_row(a.q, a.q_stride, a.k, a.k_stride, t, rr, a.Hq, a.D, d);
  float wq[8] = {}, wk[8] = {};
  if (a.wq && in) unpack8(*reinterpret_cast<const uint4 *>(a.wq + d), wq);
  if (a.wk && in) unpack8(*reinterpret_cast<const uint4 *>(a.wk + d), wk);
  if (a.rot) {
    fill_angles(cs, sn, a, a.positions[t], tid);
    __syncthreads();
  }
  for (; first + (rr - first - sub) < last; rr += RPI) {     // the same number of rounds in every wave
    const bool live = in && rr < last;
    const int nx = rr + RPI;
    uint4 xn = make_uint4(0, 0, 0, 0);
    if (in && nx < last) xn = load_row(a.q, a.q_stride, a.k, a.k_stride, t, nx, a.Hq, a.D, d);
    float f[8];
    unpack8(x, f);
    const bool isq = rr < a.Hq;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(f[i], f[i], sq);
    sq = row_sum<LPR>(sq);
    if (isq ? a.wq != nullptr : a.wk != nullptr) {
      const float r = 1.0f / sqrtf(sq / (float)a.D + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * (isq ? wq[i] : wk[i]);
    }
    if (a.rot) rotate8<IL, 1>(f, cs, sn, c, a.rot, lane);
    if (live) {
      uint16_t *o = isq ? a.q_out + (int64_t)t * a.q_out_stride + (int64_t)rr * a.D
                        : a.k_out + (int64_t)t * a.k_out_stride + (int64_t)(rr - a.Hq) * a.D;
      *reinterpret_cast<uint4 *>(o + d) = pack8(f);
    }
    x = xn;
  }
}

// Backward. With g the gradient of y: g_n = R^T g (mscale within), dw = sum
// over rows of g_n * x r, and with h = g_n * w, z = x r: dx = r (h - z mean(h z)).
// A workgroup takes tokens blockIdx.x, + gridDim.x, ... and keeps its part of
// both weight gradients in registers; the parts are summed in a fixed order by
// norm_rope_dw_kernel, so the result does not depend on scheduling.
template <int LPR, bool IL>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_dx_kernel(RopeArgs a) {
  __shared__ __attribute__((aligned(16))) float cs[2][128], sn[2][128];   // of this token and the next
  __shared__ float red[kRopeThreads * 8];
  constexpr int RPI = kRopeThreads / LPR;
  const int tid = threadIdx.x, lane = tid & 63, c = tid % LPR, sub = tid / LPR, d = 8 * c;
  const int rows = a.Hq + a.Hk;
  const bool in = d < a.D;
  float wq[8], wk[8], dwq[8], dwk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wq[i] = wk[i] = dwq[i] = dwk[i] = 0.0f;
  if (a.wq && in) unpack8(*reinterpret_cast<const uint4 *>(a.wq + d), wq);
  if (a.wk && in) unpack8(*reinterpret_cast<const uint4 *>(a.wk + d), wk);
  // gradient and input of row rr of token t
  auto load = [&](int t, int rr, uint4 &g, uint4 &x) {
    g = x = make_uint4(0, 0, 0, 0);
    if (!in || rr >= rows || t >= a.T) return;
    g = load_row(a.dq, a.dq_stride, a.dk, a.dk_stride, t, rr, a.Hq, a.D, d);
    if (rr < a.Hq ? a.wq != nullptr : a.wk != nullptr)
      x = load_row(a.q, a.q_stride, a.k, a.k_stride, t, rr, a.Hq, a.D, d);
  };
  int t = blockIdx.x, r0 = 0, buf = 0;
  uint4 gv, xv;
  load(t, sub, gv, xv);
  if (a.rot) {
    fill_angles(cs[0], sn[0], a, a.positions[t], tid);
    __syncthreads();
  }
  const float inv_d = 1.0f / (float)a.D;
  while (t < a.T) {
    if (r0 == 0 && a.rot && t + (int)gridDim.x < a.T)
      fill_angles(cs[buf ^ 1], sn[buf ^ 1], a, a.positions[t + gridDim.x], tid);
    // the next rows are under way while these are worked on
    const int rn = r0 + RPI < rows ? r0 + RPI : 0, tn = rn ? t : t + (int)gridDim.x;
    uint4 gn, xn;
    load(tn, rn + sub, gn, xn);
    const int rr = r0 + sub;
    const bool live = in && rr < rows, isq = rr < a.Hq, norm = isq ? a.wq != nullptr : a.wk != nullptr;
    float g[8], x[8];
    unpack8(gv, g);
    unpack8(xv, x);
    if (a.rot) rotate8<IL, -1>(g, cs[buf], sn[buf], c, a.rot, lane);
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(x[i], x[i], sq);
    sq = row_sum<LPR>(sq);
    const float r = 1.0f / sqrtf(sq * inv_d + a.eps);
    float dot = 0.0f, h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] *= r;
      h[i] = g[i] * (isq ? wq[i] : wk[i]);
      dot = fmaf(h[i], x[i], dot);
    }
    dot = row_sum<LPR>(dot) * inv_d;
    if (norm) {
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (isq) dwq[i] = fmaf(g[i], x[i], dwq[i]);
          else dwk[i] = fmaf(g[i], x[i], dwk[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = r * (h[i] - x[i] * dot);
    }
    if (live) {
      uint16_t *o = isq ? a.q_out + (int64_t)t * a.q_out_stride + (int64_t)rr * a.D
                        : a.k_out + (int64_t)t * a.k_out_stride + (int64_t)(rr - a.Hq) * a.D;
      *reinterpret_cast<uint4 *>(o + d) = pack8(g);
    }
    if (rn == 0 && a.rot) {
      __syncthreads();                                       // the next token's angles are there
      buf ^= 1;
    }
    gv = gn;
    xv = xn;
    r0 = rn;
    t = tn;
  }
  if (!a.part) return;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[sub * (LPR * 8) + d + i] = side ? dwk[i] : dwq[i];
    __syncthreads();
    for (int j = tid; j < a.D; j += kRopeThreads) {
      float s = 0.0f;
      for (int u = 0; u < RPI; ++u) s += red[u * (LPR * 8) + j];
      a.part[((int64_t)blockIdx.x * 2 + side) * a.D + j] = s;
    }
  }
}

// Sums the workgroups' parts: 16 columns of the 2 D per workgroup, 64 slices of
// the parts each, joined in LDS.
constexpr int kDwSlices = 64;

__global__ __launch_bounds__(16 * kDwSlices) void norm_rope_dw_kernel(const float *__restrict__ part, int n, int D,
                                                                      float *__restrict__ dwq,
                                                                      float *__restrict__ dwk) {
  __shared__ float red[kDwSlices][17];
  const int col = threadIdx.x & 15, slice = threadIdx.x >> 4, j = (int)blockIdx.x * 16 + col;
  float s = 0.0f;
  if (j < 2 * D) {
#pragma unroll 8
    for (int i = slice; i < n; i += kDwSlices) s += part[(int64_t)i * 2 * D + j];
  }
  red[slice][col] = s;
  __syncthreads();
  if (threadIdx.x < 64) {                                    // four lanes per column
    const int q = threadIdx.x >> 4;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kDwSlices / 4; ++i) v += red[q * (kDwSlices / 4) + i][col];
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    if (q == 0 && j < 2 * D) {
      float *o = j < D ? dwq : dwk;
      if (o) o[j < D ? j : j - D] = v;
    }
  }
}

int32_t rope_dx_blocks(int32_t T) { return std::min<int32_t>(T, 1024); }

// A launch has fewer than 2^32 threads: more tokens than this in several.
constexpr int kRopeTokens = 1 << 23;

hipError_t launch_norm_rope(const RopeArgs &args, hipStream_t s) {
  if (args.T > kRopeTokens) {
    RopeArgs a = args;
    for (int64_t t = 0; t < args.T; t += kRopeTokens) {
      a.T = (int32_t)std::min<int64_t>(args.T - t, kRopeTokens);
      if (args.Hq) a.q = args.q + t * args.q_stride, a.q_out = args.q_out + t * args.q_out_stride;
      if (args.Hk) a.k = args.k + t * args.k_stride, a.k_out = args.k_out + t * args.k_out_stride;
      if (args.positions) a.positions = args.positions + t;
      const hipError_t e = launch_norm_rope(a, s);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const RopeArgs &a = args;
  const int rows = a.Hq + a.Hk;
  const int lpr = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32, rpi = kRopeThreads / lpr;
  // few tokens: one round of head rows per workgroup; many: all of a token's
  const int rpb = a.T >= 2048 ? rows : rpi;
  const dim3 grid((unsigned)a.T, (unsigned)((rows + rpb - 1) / rpb)), block(kRopeThreads);
  if (lpr == 8) {
    if (a.interleaved) hipLaunchKernelGGL((norm_rope_kernel<8, true>), grid, block, 0, s, a, rpb);
    else hipLaunchKernelGGL((norm_rope_kernel<8, false>), grid, block, 0, s, a, rpb);
  } else if (lpr == 16) {
    if (a.interleaved) hipLaunchKernelGGL((norm_rope_kernel<16, true>), grid, block, 0, s, a, rpb);
    else hipLaunchKernelGGL((norm_rope_kernel<16, false>), grid, block, 0, s, a, rpb);
  } else {
    if (a.interleaved) hipLaunchKernelGGL((norm_rope_kernel<32, true>), grid, block, 0, s, a, rpb);
    else hipLaunchKernelGGL((norm_rope_kernel<32, false>), grid, block, 0, s, a, rpb);
  }
  return hipGetLastError();
}

hipError_t launch_norm_rope_dx(const RopeArgs &a, hipStream_t s) {
  const int lpr = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  const int n = rope_dx_blocks(a.T);
  const dim3 grid((unsigned)n), block(kRopeThreads);
  if (n > 0) {
    if (lpr == 8) {
      if (a.interleaved) hipLaunchKernelGGL((norm_rope_dx_kernel<8, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((norm_rope_dx_kernel<8, false>), grid, block, 0, s, a);
    } else if (lpr == 16) {
      if (a.interleaved) hipLaunchKernelGGL((norm_rope_dx_kernel<16, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((norm_rope_dx_kernel<16, false>), grid, block, 0, s, a);
    } else {
      if (a.interleaved) hipLaunchKernelGGL((norm_rope_dx_kernel<32, true>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((norm_rope_dx_kernel<32, false>), grid, block, 0, s, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dwq && !a.dwk) return hipSuccess;
  hipLaunchKernelGGL(norm_rope_dw_kernel, dim3((2 * a.D + 15) / 16), dim3(16 * kDwSlices), 0, s, a.part, n, a.D, a.dwq, a.dwk);
  return hipGetLastError();
}

}  // namespace gnf4
