// Shared by the cache's write and read kernels and the attention over it: the
// kernel-side view of a paged 4-bit cache and of a step's rows.
#pragma once

#include "common.h"

namespace gnf4 {

// Cache and step as the kernels see them. Page p of head h starts at row
// (p * H + h) << page_shift of each array; a row is D/2 code bytes.
struct KvView {
  uint8_t *k_codes, *v_codes;
  void *k_scales, *v_scales;
  int32_t n_pages, page_shift, H, D;
  const int32_t *offsets, *lens, *pages;
  int32_t B, n_tokens, max_pages;
};

struct KvRowsArgs {
  KvView kv;
  const uint16_t *k, *v;          // write: bf16 rows, token strides in elements
  int64_t k_stride, v_stride;
  void *k_out, *v_out;            // read: [n_tokens][H][D]
};

struct KvAttnArgs {
  KvView kv;
  const uint16_t *q;
  int64_t q_stride;
  uint16_t *out;
  int64_t out_stride;
  float *lse;                     // [n_tokens][Hq] or NULL
  const float *sinks;             // [Hq] or NULL
  int32_t G;                      // query heads per cache head
  int32_t window;                 // 0: none
  float scale_log2;               // scale * log2(e): the softmax runs in base 2
  uint32_t q_sign;                // flips the queries' signs (a negative scale)
  int32_t n_mt;                   // most row tiles of one sequence
  int32_t tile_tokens;            // most tokens that the rows of one tile belong to
  int32_t shared;                 // 1: equal shares of all work per workgroup; 0: a workgroup per tile
  float *part;                    // [slots][M][D] then [slots][M][2], two slots per workgroup
};

// How one call is cut (attention.hip).
struct KvAttnPlan {
  int32_t nq, n_mt, shared, small, tile_tokens;
  int64_t items;                  // sequences * n_mt * H
  size_t bytes;
};
bool kv_attention_plan(int32_t format, int32_t D, int32_t H, int32_t G, int32_t B, int64_t n_tokens,
                       int32_t max_new, int64_t max_len, int64_t capacity, int32_t window, KvAttnPlan *p);

hipError_t launch_kv_write(const KvRowsArgs &a, int32_t format, hipStream_t s);
hipError_t launch_kv_read(const KvRowsArgs &a, int32_t format, int32_t out_f32, hipStream_t s);
hipError_t launch_kv_attention(const KvAttnArgs &a, const KvAttnPlan &p, int32_t format, hipStream_t s);

// The last b with offsets[b] <= r, b in [0, B], or -1. Called by whole waves with
// a uniform r. Each round the wave's lanes probe 64 evenly spaced entries at
// once, so B < 64 takes one load and B < 4096 two, where a bisection takes 6 and
// 12 in a row.
__device__ __forceinline__ int find_seq(const int32_t *__restrict__ offsets, int B, int r, int lane) {
  int lo = 0, n = B + 1;
  for (;;) {
    const int step = (n + 63) >> 6;
    const int i = lane * step;
    const bool below = i < n && offsets[lo + min(i, n - 1)] <= r;
    const int c = __popcll(__ballot(below));
    if (c == 0) return lo - 1;
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
    if (n == 1) return lo;
  }
}

// Where the row of position pos of sequence b lies: the row index in the code
// arrays for head 0 of its page, or -1 when the position does not exist or its
// page id is outside the cache.
__device__ __forceinline__ int64_t kv_row0(const KvView &kv, int b, int pos) {
  if (pos < 0 || (pos >> kv.page_shift) >= kv.max_pages) return -1;
  const int pid = kv.pages[(int64_t)b * kv.max_pages + (pos >> kv.page_shift)];
  if ((uint32_t)pid >= (uint32_t)kv.n_pages) return -1;
  return ((int64_t)pid * kv.H << kv.page_shift) + (pos & ((1 << kv.page_shift) - 1));
}

// kv_row0 of rows t0 .. t0 + n - 1 of the step (n <= 64), lane i's that of row
// t0 + i; -1 for rows of no sequence. Called by whole waves. The sequence of t0
// is searched for, those of the rows behind it follow from the next 64 offsets.
__device__ __forceinline__ int64_t kv_rows(const KvView &kv, int t0, int n, int lane) {
  const int b0 = find_seq(kv.offsets, kv.B, t0, lane);
  const int k = b0 + 1 + lane;
  const int next = k <= kv.B ? kv.offsets[k] : 0x7fffffff;
  int b = b0;
  for (int i = 1; i < n; ++i) {
    const int c = __popcll(__ballot(next <= t0 + i));
    // 64 offsets passed at once (empty sequences): the window does not reach
    const int at = c < 64 ? b0 + c : find_seq(kv.offsets, kv.B, t0 + i, lane);
    if (lane == i) b = at;
  }
  if (lane >= n || b < 0 || b >= kv.B) return -1;
  const int t = t0 + lane, end = kv.offsets[b + 1];
  return t < end && t < kv.n_tokens ? kv_row0(kv, b, kv.lens[b] - end + t) : -1;
}

}  // namespace gnf4
