"""Pins of the attention oracle that do not re-run its formulas (CPU)."""

import math

import numpy as np
import pytest

from oracle import attention as oa
from oracle import mxfp4, nf4


def rng(*seed):
    return np.random.default_rng(list(seed))


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_keeps_pair_lengths_and_adds_angles(interleaved):
    x = rng(1).standard_normal((5, 3, 64))
    f = (10.0 ** -np.arange(16)).astype(np.float32)
    pos = np.array([0, 1, 7, 100000, -3])
    y = oa.norm_rope(x, None, 0.0, pos, f, interleaved)
    assert np.array_equal(y[0], x[0])                        # position 0: no turn
    assert np.array_equal(y[..., 32:], x[..., 32:])          # the rest of the head
    pair = (lambda z: (z[..., 0:32:2], z[..., 1:32:2])) if interleaved else (lambda z: (z[..., :16], z[..., 16:32]))
    (a, b), (u, v) = pair(x), pair(y)
    assert np.allclose(a * a + b * b, u * u + v * v, rtol=1e-12)
    turn = np.angle((u + 1j * v) / (a + 1j * b))
    want = np.remainder(pos[:, None].astype(float) * f.astype(float) + math.pi, 2 * math.pi) - math.pi
    diff = np.remainder(turn - want[:, None] + math.pi, 2 * math.pi) - math.pi
    assert np.abs(diff).max() < 1e-9
    back = oa.norm_rope(y, None, 0.0, -pos, f, interleaved)
    assert np.allclose(back, x, atol=1e-9)


def test_layouts_differ_by_a_permutation():
    x = rng(2).standard_normal((4, 2, 32))
    f = (3.0 ** -np.arange(16)).astype(np.float32)
    order = np.concatenate((np.arange(0, 32, 2), np.arange(1, 32, 2)))
    a = oa.norm_rope(x, None, 0.0, [1, 2, 3, 4], f, True)[..., order]
    b = oa.norm_rope(x[..., order], None, 0.0, [1, 2, 3, 4], f, False)
    assert np.allclose(a, b, atol=1e-15)


def test_norm_of_constant_rows():
    x = np.full((1, 1, 16), -2.0)
    w = np.arange(16.0)
    assert np.allclose(oa.norm_rope(x, w, 0.0, [0], None, False)[0, 0], -w, rtol=1e-15)
    assert np.allclose(oa.norm_rope(x, w, 12.0, [0], None, False)[0, 0], -w / 2, rtol=1e-6)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_dx_by_differences(interleaved, norm):
    g = rng(3, interleaved)
    x, grad = g.standard_normal((2, 2, 32)), g.standard_normal((2, 2, 32))
    w = g.standard_normal(32) if norm else None
    f = (5.0 ** -np.arange(8)).astype(np.float32)
    args = (1e-3, [3, 11], f, interleaved, 1.25)
    dx, dw = oa.norm_rope_dx(grad, x, w, *args)
    loss = lambda x, w: float((oa.norm_rope(x, w, *args) * grad).sum())  # noqa: E731
    for at in [(0, 0, 0), (0, 1, 9), (1, 0, 17), (1, 1, 31)]:
        e = np.zeros_like(x)
        e[at] = 1e-6
        assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-6 - dx[at]) < 1e-7
    if norm:
        for i in (0, 8, 31):
            e = np.zeros(32)
            e[i] = 1e-6
            assert abs((loss(x, w + e) - loss(x, w - e)) / 2e-6 - dw[i]) < 1e-7
    else:
        assert dw is None


def test_rope_frequencies():
    f, m = oa.rope_frequencies(8, 10000.0)
    assert np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-7) and m == 1.0
    g, _ = oa.rope_frequencies(8, 10000.0, "linear", 4.0)
    assert np.allclose(g * 4, f, rtol=1e-7)
    y, m = oa.rope_frequencies(64, 10000.0, "yarn", 8.0, 4096.0)
    p, _ = oa.rope_frequencies(64, 10000.0)
    turns = 4096 * p.astype(float) / (2 * math.pi)
    assert np.array_equal(y[turns > 32], p[turns > 32])      # fast pairs as trained
    assert np.allclose(y[turns < 1], p[turns < 1] / 8, rtol=1e-6)   # slow ones interpolated
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((y[mid] < p[mid]) & (y[mid] > p[mid] / 8))
    assert abs(m - (0.1 * math.log(8) + 1)) < 1e-6


def batch_of(lens, new, page, extra=0):
    """Sequences on pages handed out from the back."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + extra
    ids = iter(range(total - 1, -1, -1))
    pages = -np.ones((len(lens), max(max(need), 1)), dtype=np.int64)
    for b, n in enumerate(need):
        pages[b, :n] = [next(ids) for _ in range(n)]
    off = np.concatenate(([0], np.cumsum(new)))
    return oa.Batch(off, lens, pages, int(off[-1])), total


@pytest.mark.parametrize("fmt", ["nf4", "mxfp4"])
def test_cache_round_trip(fmt):
    batch, n_pages = batch_of([5, 0, 33], [5, 0, 33], 16)
    k, v = rng(5).standard_normal((2, 38, 2, 64)).astype(np.float32)
    c = oa.Cache(fmt, n_pages, 16, 2, 64)
    c.write(batch, k, v)
    kb, vb = c.read(batch, np.zeros_like(k), np.zeros_like(v))
    mod = nf4 if fmt == "nf4" else mxfp4
    for x, y in ((k, kb), (v, vb)):
        assert np.array_equal(y, mod.dequantize(*mod.quantize(x), 64))
    # sequence 2's position 17 is the second place of its second page
    assert np.array_equal(c.codes[0][batch.pages[2, 1], 1, 1], mod.quantize(k[5 + 17, 1])[0])


def test_cache_drops_what_does_not_exist_and_marks_nan():
    c = oa.Cache("mxfp4", 2, 16, 1, 64)
    batch = oa.Batch([1, 3, 5], [1, 40], [[0, 9], [1, 5]], 6)
    x = rng(6).standard_normal((6, 1, 64)).astype(np.float32)
    x[2, 0, 40] = np.inf
    c.write(batch, x, x)
    # row 1 is position -1, rows 3 and 4 lie past their pages; row 2 is position 0
    assert c.codes[0][0, 0, 0].any() and not c.codes[0][0, 0, 1:].any() and not c.codes[0][1].any()
    k = np.full((6, 1, 64), 7.0, dtype=np.float32)
    c.read(batch, k, k.copy())
    assert np.all(k[[0, 1, 3, 4, 5]] == 7.0)
    assert np.isnan(k[2, 0, 32:]).all() and np.isfinite(k[2, 0, :32]).all()


def test_attend_uniform_and_one_hot():
    batch, n = batch_of([20], [2], 16)
    whole, _ = batch_of([20], [20], 16)
    g = rng(7)
    k, v = g.standard_normal((2, 20, 1, 64))
    c = oa.Cache("mxfp4", n, 16, 1, 64)
    c.write(whole, k, v)
    vals = c.read(whole, np.zeros((20, 1, 64), np.float32), np.zeros((20, 1, 64), np.float32))
    q = np.zeros((2, 3, 64))
    out, lse, _, _ = oa.attend(q, c, batch, 0.3)
    for r, seen in ((0, 19), (1, 20)):
        assert np.allclose(out[r], vals[1][:seen, 0].astype(float).mean(0), atol=1e-12)
        assert np.allclose(lse[r], math.log(seen))
    out, _, _, _ = oa.attend(q, c, batch, 0.3, window=4, sinks=[math.log(4.0)] * 3)
    assert np.allclose(out[1], vals[1][16:, 0].astype(float).sum(0) / 8, atol=1e-12)
    q = np.tile(1000.0 * vals[0][6, 0].astype(float), (2, 3, 1))
    best = int(np.argmax(vals[0][:19, 0].astype(float) @ vals[0][6, 0].astype(float)))
    out, _, _, _ = oa.attend(q, c, batch, 1.0)
    assert np.allclose(out[0], vals[1][best, 0], atol=1e-9)


def test_attend_joins_by_lse_and_empty_rows():
    batch, n = batch_of([40], [1], 16)
    whole, _ = batch_of([40], [40], 16)
    k, v = rng(8).standard_normal((2, 40, 2, 64))
    c = oa.Cache("nf4", n, 16, 2, 64)
    c.write(whole, k, v)
    q = rng(9).standard_normal((1, 4, 64))
    out, lse, _, _ = oa.attend(q, c, batch, 0.125)
    near, l1, _, _ = oa.attend(q, c, batch, 0.125, window=10)
    far, l2, _, _ = oa.attend(q, c, oa.Batch([0, 1], [30], batch.pages, 1), 0.125)
    w1, w2 = np.exp(l1 - lse)[..., None], np.exp(l2 - lse)[..., None]
    assert np.allclose(w1 * near + w2 * far, out, atol=1e-12) and np.allclose(w1 + w2, 1.0)
    nothing = oa.Batch([0, 1], [0], batch.pages, 1)
    out, lse, _, _ = oa.attend(q, c, nothing, 0.125)
    assert not out.any() and np.all(lse == -np.inf)
    out, lse, _, _ = oa.attend(q, c, nothing, 0.125, sinks=[1.0, 2.0, 3.0, 4.0])
    assert not out.any() and np.allclose(lse, [[1, 2, 3, 4]])
