"""Helpers of the attention tests: ragged steps on shuffled pages, device
copies, and error bars.

Bars, from the arithmetic of the kernels (eps8 = 2^-8 is half a bf16 step
relative to the value, the most one rounding to bf16 is off):

* head norm + rotation: float32 throughout and one rounding. The terms of a
  rotated value are sums of two products; each passes about eight float32
  operations (2^-24 each) plus an angle known to 2^-23 and a sine / cosine
  within a few ulps: 2e-6 of |a| + |b|, and eps8 of the result.
* its input gradient: the same with about twice the operations: 4e-6 of
  r (|h| + |z| mean |h z|), and eps8 of the result.
* weight gradients: a float32 sum whose longest chain stays below 160 terms
  (160 * 2^-24 = 1e-5) of sum |g z|.
* attention: eps8 |out| for the result. MXFP4: the probabilities are each
  rounded to bf16, eps8 * spread (spread = sum w |v|). NF4: operands in fp16
  (eps11 = 2^-11): eps11 * spread each for the probabilities times absmax and
  for the codebook; for the keys' codebook every score moves by at most
  d = eps11 * reach (reach = scale * sum |q k|), which changes each weight by
  a factor within exp(+-2 d); what lies below fp16's normal range is 2^-32 of
  a row's largest term each. float32 sums, exp2 and the score itself:
  1e-5 * (1 + reach) * spread.
* lse: d (NF4) + 1e-5 * (1 + reach).
"""

import numpy as np
import torch

from oracle import attention as oa

EPS8 = 2.0 ** -8
EPS11 = 2.0 ** -11


def to_bf16(x):
    """float64 / float32 array -> (bf16 bits uint16, their float64 values)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    bits = t.view(torch.int16).numpy().view(np.uint16)
    return bits, oa.bf16_to_f64(bits)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def values(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Step:
    """A ragged step on shuffled pages: the oracle's batch and the device's."""

    def __init__(self, lens, new, page, seed=0, spare=2, slack=0, max_len=None):
        g = np.random.default_rng([77, seed, page, len(lens)])
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        ids = list(g.permutation(self.n_pages))
        width = max(max(need), 1) + slack
        pages = g.choice([-1, -7, 1 << 30, self.n_pages], size=(len(lens), width)).astype(np.int64)
        for b, n in enumerate(need):
            pages[b, :n] = [ids.pop() for _ in range(n)]
        self.page, self.lens, self.new = page, list(lens), list(new)
        self.offsets = [0] + [int(x) for x in np.cumsum(new)]
        self.pages, self.T = pages, self.offsets[-1]
        self.max_len = max(max(lens), 1) if max_len is None else max_len

    def oracle(self):
        return oa.Batch(self.offsets, self.lens, self.pages, self.T)

    def whole(self):
        """The step that holds every position of every sequence."""
        s = Step.__new__(Step)
        s.__dict__.update(self.__dict__)
        s.new, s.offsets = self.lens, [0] + [int(x) for x in np.cumsum(self.lens)]
        s.T = s.offsets[-1]
        return s

    def device(self, g):
        i32 = lambda x: dev(np.asarray(x, dtype=np.int32))  # noqa: E731
        return g.KVBatch(i32(self.offsets), i32(self.lens), i32(self.pages), self.T, max(max(self.new), 1),
                         self.max_len)


def device_cache(g, c):
    """The oracle's cache on the device."""
    return g.KVCache(g.FORMATS[c.fmt], c.n_pages, c.page, c.H, c.D, dev(c.codes[0]), dev(c.scales[0]),
                     dev(c.codes[1]), dev(c.scales[1]))


def attention_bars(fmt, out, spread, reach):
    """(bar of out, bar of lse) elementwise."""
    small = 1e-5 * (1.0 + reach)
    d = EPS11 * reach if fmt == "nf4" else np.zeros_like(reach)
    w = small + (2 * EPS11 + np.expm1(2 * d) * (1 + EPS8) if fmt == "nf4" else EPS8)
    return EPS8 * np.abs(out) + w[..., None] * spread * (1 + EPS8) + 1e-30, d + small


def check_attention(fmt, got, got_lse, ref, rows=None):
    out, lse, spread, reach = ref
    rows = np.arange(out.shape[0]) if rows is None else rows
    out, lse, spread, reach = out[rows], lse[rows], spread[rows], reach[rows]
    bar, lbar = attention_bars(fmt, out, spread, reach)
    got = got[rows]
    assert np.array_equal(np.isnan(got), np.isnan(out)), "NaN in other places"
    f = ~np.isnan(out)
    assert out.size, "comparing nothing proves nothing"
    worst = (np.abs(got - out)[f] / bar[f]).max(initial=0.0)     # every row may be NaN
    assert worst <= 1.0, "error %.3g of its bar" % worst
    if got_lse is not None:
        got_lse = got_lse[rows]
        fin = np.isfinite(lse)
        assert np.array_equal(got_lse[~fin], lse[~fin], equal_nan=True)
        assert np.all(np.abs(got_lse - lse)[fin] <= lbar[fin])
    return worst
