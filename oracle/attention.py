"""The attention in front of the experts on a 4-bit cache (oracle): norm of
query and key heads with the rotation by position and its backward pass, the
paged cache's write and read, and the attention over it.

TEST INFRASTRUCTURE (see the package docstring): never imported by the GPU path.

The pages run the packed experts behind a real attention (Jordan Anderson,
jordananderson-pages.pages.dev, section "grouped-nf4-gemm & experts-4bit", the
demonstration paragraph of the first bullet) and list FP8 paged decode attention
with sliding window, sinks and a custom scale among the package's tasks ("MoE
Training on Consumer GPUs -- Loggetta & Cerin Amroth", Task guides table), with
no formula. Readings taken, those of the public models the workloads are shaped
after, everything in float64:

* ``norm_rope``: n = w x / sqrt(mean(x^2) + eps); the first 2 len(inv_freq)
  values of n are rotated in pairs by position * inv_freq (neighbours, or the
  two halves) and multiplied by mscale.
* ``norm_rope_dx``: its gradients, from the chain rule.
* ``Cache``: the packed rows of ``nf4`` and ``mxfp4`` on pages; a block with a
  NaN or an infinity decodes to NaN.
* ``attend``: softmax attention over the decoded rows that a query sees, an
  optional sink logit in the softmax's sum; a row that sees nothing is 0.

Parity: norm_rope pinned (norm of ones, lengths of pairs kept, angles adding up,
both layouts related by a permutation), norm_rope_dx by differences, Cache by
round trips against ``nf4`` / ``mxfp4`` and hand-placed rows, attend by uniform
weights, one-hot scores, and joining two parts by their lse.
"""

import math

import numpy as np

from . import mxfp4, nf4


def bf16_to_f64(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# ------------------------------------------------------- norm and rotation

def angles(positions, inv_freq):
    return np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float32).astype(np.float64)


def rotate(x, ang, interleaved, sign=1.0):
    """x [T, H, D] with pair i of the first 2 n values turned by ang [T, n]."""
    y = np.array(x, dtype=np.float64)
    n = ang.shape[1]
    c, s = np.cos(ang)[:, None], sign * np.sin(ang)[:, None]
    if interleaved:
        ia, ib = 2 * np.arange(n), 2 * np.arange(n) + 1
    else:
        ia, ib = np.arange(n), n + np.arange(n)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def _scale_rotated(y, n, mscale):
    y = np.array(y)
    y[..., :2 * n] *= float(np.float32(mscale))
    return y


def norm_rope(x, w, eps, positions, inv_freq, interleaved, mscale=1.0):
    """x [T, H, D] float64; w [D] float64 or None; inv_freq None: no rotation."""
    y = np.asarray(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps))) * w
    if inv_freq is None:
        return y
    return _scale_rotated(rotate(y, angles(positions, inv_freq), interleaved), len(inv_freq), mscale)


def norm_rope_dx(g, x, w, eps, positions, inv_freq, interleaved, mscale=1.0):
    """(dx [T, H, D], dw [D] or None) from the gradient g of norm_rope's result."""
    g = np.asarray(g, dtype=np.float64)
    if inv_freq is not None:
        g = rotate(_scale_rotated(g, len(inv_freq), mscale), angles(positions, inv_freq), interleaved, -1.0)
    if w is None:
        return g, None
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
    z = x * r
    h = g * w
    return r * (h - z * (h * z).mean(-1, keepdims=True)), (g * z).sum((0, 1))


def rope_frequencies(rot_dim, base, scaling="plain", factor=1.0, original_len=0.0, beta_fast=32.0, beta_slow=1.0):
    """(inv_freq float32, mscale float32) of the header's definition."""
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            turns = original_len * f / (2.0 * math.pi)
            keep = min(max((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0)
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    m = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return np.array(out, dtype=np.float64).astype(np.float32), np.float32(m)


# ------------------------------------------------------------------- cache

class Batch:
    """Rows of one step (see the header): plain lists."""

    def __init__(self, offsets, lens, pages, n_tokens):
        self.offsets, self.lens, self.n_tokens = list(offsets), list(lens), n_tokens
        self.pages = np.asarray(pages, dtype=np.int64)

    def rows(self):
        """(row, sequence, position) of every row that belongs to a sequence."""
        for b, length in enumerate(self.lens):
            lo, hi = self.offsets[b], self.offsets[b + 1]
            for r in range(max(lo, 0), min(hi, self.n_tokens)):
                yield r, b, length - hi + r


class Cache:
    """Packed rows in numpy, [n_pages, H, page, ...]."""

    def __init__(self, fmt, n_pages, page, H, D):
        self.fmt, self.n_pages, self.page, self.H, self.D = fmt, n_pages, page, H, D
        mx = fmt == "mxfp4"
        self.codes = [np.zeros((n_pages, H, page, D // 2), dtype=np.uint8) for _ in range(2)]
        self.scales = [np.zeros((n_pages, H, page, D // (32 if mx else 64)), dtype=np.uint8 if mx else np.float32)
                       for _ in range(2)]

    def place(self, batch, b, pos):
        """(page, place) of a position, or None where it does not exist."""
        if pos < 0 or pos // self.page >= batch.pages.shape[1]:
            return None
        pid = int(batch.pages[b, pos // self.page])
        return (pid, pos % self.page) if 0 <= pid < self.n_pages else None

    def quantize(self, x):
        """(codes, scales) of float rows x [..., D]; blocks that are not finite
        get the NaN scale (and the codes of zeros)."""
        x = np.asarray(x, dtype=np.float32)
        size = 32 if self.fmt == "mxfp4" else 64
        bad = ~np.isfinite(x.reshape(-1, size)).all(1)
        clean = np.where(np.repeat(bad, size).reshape(x.shape), np.float32(0), x)
        codes, scales = (mxfp4 if self.fmt == "mxfp4" else nf4).quantize(clean)
        scales.reshape(-1)[bad] = 255 if self.fmt == "mxfp4" else np.nan
        return codes, scales

    def write(self, batch, k, v):
        """k, v [n_tokens, H, D] float rows."""
        for side, x in enumerate((k, v)):
            codes, scales = self.quantize(x)
            for r, b, pos in batch.rows():
                at = self.place(batch, b, pos)
                if at is not None:
                    self.codes[side][at[0], :, at[1]] = codes[r]
                    self.scales[side][at[0], :, at[1]] = scales[r]

    def values(self, side):
        """Every place's float32 value, [n_pages, H, page, D]."""
        with np.errstate(invalid="ignore"):
            return (mxfp4 if self.fmt == "mxfp4" else nf4).dequantize(self.codes[side], self.scales[side], self.D)

    def read(self, batch, k, v):
        """Fills k, v [n_tokens, H, D] (float32) with the rows' values."""
        vals = [self.values(0), self.values(1)]
        for r, b, pos in batch.rows():
            at = self.place(batch, b, pos)
            if at is not None:
                k[r], v[r] = vals[0][at[0], :, at[1]], vals[1][at[0], :, at[1]]
        return k, v


def attend(q, cache, batch, scale, window=0, sinks=None):
    """(out, lse, spread, reach) for q [n_tokens, Hq, D] float64; rows that
    belong to no sequence are NaN. spread = sum of w |v| [n_tokens, Hq, D] and
    reach = the largest of scale * sum |q_i k_i| over the seen positions
    [n_tokens, Hq] scale the rounding errors of an implementation."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    G = Hq // cache.H
    kv = [cache.values(0).astype(np.float64), cache.values(1).astype(np.float64)]
    out, spread = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    lse, reach = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for r, b, own in batch.rows():
        first = max(0, own - window + 1) if window > 0 else 0
        at = [cache.place(batch, b, p) for p in range(first, own + 1)]
        at = [a for a in at if a is not None]
        pid, off = [a[0] for a in at], [a[1] for a in at]
        for h in range(cache.H):
            k, v = kv[0][pid, h, off].reshape(-1, D), kv[1][pid, h, off].reshape(-1, D)
            for g in range(G):
                hq = h * G + g
                x = scale * (k @ q[r, hq])
                sink = -np.inf if sinks is None else float(sinks[hq])
                top = max(x.max(), sink) if x.size else sink
                if np.isnan(x).any():
                    top = np.nan
                if top == -np.inf:
                    out[r, hq], lse[r, hq] = 0.0, -np.inf
                    continue
                e = np.exp(x - top)
                total = e.sum() + np.exp(sink - top)
                w = e / total
                out[r, hq] = w @ v if x.size else 0.0
                spread[r, hq] = w @ np.abs(v) if x.size else 0.0
                reach[r, hq] = (abs(scale) * (np.abs(k) @ np.abs(q[r, hq]))).max() if x.size else 0.0
                lse[r, hq] = top + math.log(total)
    return out, lse, spread, reach
