"""GPU parity of the paged 4-bit cache: written bytes and values read back
equal the oracle's exactly."""

import numpy as np
import pytest
import torch

from oracle import attention as oa

from .attention_util import Step, dev, dev_bf16, device_cache, to_bf16
from .gpu_util import gnf4, say

pytestmark = pytest.mark.gpu

FMTS = ["nf4", "mxfp4"]


def same_bytes(c, gc):
    """Every code and scale of the oracle's cache, except the codes of NaN blocks."""
    for side, (codes, scales) in enumerate(((gc.k_codes, gc.k_scales), (gc.v_codes, gc.v_scales))):
        s = c.scales[side]
        gs = scales.cpu().numpy()
        nan = s == 255 if c.fmt == "mxfp4" else np.isnan(s)
        assert np.array_equal(nan, gs == 255 if c.fmt == "mxfp4" else np.isnan(gs))
        assert np.array_equal(s[~nan], gs[~nan])
        ok = np.repeat(~nan, (32 if c.fmt == "mxfp4" else 64) // 2, axis=-1)
        assert np.array_equal(c.codes[side][ok], codes.cpu().numpy()[ok])


def run_write(fmt, step, H, D, k, v, kd, vd, seed=0):
    """The oracle's cache and the device's after writing the step over random bytes."""
    g = gnf4()
    c = oa.Cache(fmt, step.n_pages, step.page, H, D)
    r = np.random.default_rng([seed, H, D])
    for side in range(2):
        c.codes[side][:] = r.integers(0, 256, c.codes[side].shape)
        c.scales[side][:] = r.integers(1, 255, c.scales[side].shape)
    gc = device_cache(g, c)
    c.write(step.oracle(), k, v)
    g.kv_cache_write(gc, kd, vd, step.device(g))
    torch.cuda.synchronize()
    same_bytes(c, gc)
    return c, gc


def rows_of(T, H, D, seed, spread=3.0):
    """k and v as parts of wider rows: (k, kd, v, vd)."""
    r = np.random.default_rng([T, H, D, seed])
    x = r.standard_normal((T, 3 * H * D)) * np.exp(spread * r.standard_normal((T, 1)))
    bits, x = to_bf16(x)
    xd = dev_bf16(bits)
    cut = lambda a, i: a[:, i * H * D:(i + 1) * H * D].reshape(T, H, D) if isinstance(a, np.ndarray) else (  # noqa: E731
        a[:, i * H * D:(i + 1) * H * D].view(T, H, D))
    return cut(x, 1), cut(xd, 1), cut(x, 2), cut(xd, 2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,new,page,H,D", [
    ([1], [1], 16, 1, 64), ([17, 40, 3], [1, 1, 1], 16, 4, 128), ([33, 100, 64], [33, 7, 64], 32, 2, 128),
    ([5, 0, 130, 9], [5, 0, 1, 0], 64, 3, 64), ([300], [257], 128, 1, 256), ([2] * 70, [1] * 70, 16, 8, 128),
    ([3] * 300, [1] * 300, 16, 1, 64), ([31], [31], 256, 5, 64)])
def test_write_then_read(fmt, lens, new, page, H, D):
    g = gnf4()
    say("kv write/read", fmt, len(lens), "seqs", sum(new), "rows page", page, "H", H, "D", D)
    step = Step(lens, new, page)
    k, kd, v, vd = rows_of(step.T, H, D, 1)
    c, gc = run_write(fmt, step, H, D, k, v, kd, vd)
    whole = step.whole()
    z = [np.zeros((whole.T, H, D), np.float32) for _ in range(2)]
    kr, vr = c.read(whole.oracle(), *z)
    b = whole.device(g)
    for dtype in (torch.float32, torch.bfloat16):
        kg, vg = g.kv_cache_read(gc, b, dtype)
        for want, got in ((kr, kg), (vr, vg)):
            assert got.dtype == dtype
            assert torch.equal(torch.from_numpy(want).to(dtype), got.cpu())


@pytest.mark.parametrize("fmt", FMTS)
def test_every_magnitude(fmt):
    """All finite bf16 values, each block a binade of scales: subnormals, the
    largest, zeros of both signs, exact midpoints."""
    g = gnf4()
    say("kv write, every bf16", fmt)
    bits = np.arange(65536, dtype=np.uint16)
    bits = bits[(bits & 0x7f80) != 0x7f80]
    x = np.concatenate((bits, bits[::-1], np.random.default_rng(0).permutation(bits), np.zeros(64, np.uint16),
                        np.full(64, 0x8000, np.uint16)))
    # mixed with much smaller and larger neighbours too
    x = np.concatenate((x, np.random.default_rng(1).permutation(x)))
    T = -(-x.size // 256)
    x = np.resize(x, (T, 4, 64))
    step = Step([T], [T], 16)
    f = oa.bf16_to_f64(x)
    run_write(fmt, step, 4, 64, f, f[::-1], dev_bf16(x), dev_bf16(x[::-1]))


@pytest.mark.parametrize("fmt", FMTS)
def test_midpoints_and_neighbours(fmt):
    """Values on, just above and just below every border between two codes, at several scales."""
    say("kv write, borders", fmt)
    if fmt == "mxfp4":
        mids, size, top = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), 32, [4.0, 6.0, 7.9]
    else:
        from oracle import nf4
        cb = nf4.codebook().astype(np.float64)
        mids, size, top = np.abs((cb[1:] + cb[:-1]) / 2), 64, [1.0, 1.5, 1.9921875]
    rows = []
    for e in (-100, -20, -3, 0, 9, 100):
        for t in top:
            m = np.concatenate((mids * (1.0 if fmt == "mxfp4" else t), [t]))
            b = to_bf16(np.resize(m, size - 1) * 2.0 ** e)[0].astype(np.int32)
            for d in (-1, 0, 1):
                sign = np.where(np.arange(size - 1) % 2 == 0, 0, 0x8000)
                blk = np.concatenate(((b + d) | sign, to_bf16([t * 2.0 ** e])[0]))
                rows.append(np.resize(blk, 64))
    x = np.array(rows, dtype=np.uint16)[:, None]
    T = len(rows)
    f = oa.bf16_to_f64(x)
    run_write(fmt, Step([T], [T], 32), 1, 64, f, -f, dev_bf16(x), dev_bf16(x ^ 0x8000))


@pytest.mark.parametrize("fmt", FMTS)
def test_every_quotient_of_two_significands(fmt):
    """A block's largest value with each of the 128 bf16 significands, against
    every significand at ten binades, of both signs."""
    say("kv write, all quotients", fmt)
    top = 0x3f80 + np.arange(128)                            # [1, 2)
    rows = []
    for e in range(10):
        w = 0x3f80 + np.arange(128) - 128 * e
        for a in top:
            for part in w.reshape(2, 64):
                ok = np.where(part <= a, part, a)            # not above the largest
                rows.append(np.concatenate((ok[:63], [a])))
                rows.append(np.concatenate(([a], ok[1:] | 0x8000)))
    x = np.array(rows, dtype=np.uint16).reshape(-1, 4, 64)
    T = x.shape[0]
    f = oa.bf16_to_f64(x)
    run_write(fmt, Step([T], [T], 64), 4, 64, f, -f, dev_bf16(x), dev_bf16(x ^ 0x8000))


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_and_infinity_mark_their_block(fmt):
    g = gnf4()
    say("kv write NaN / inf", fmt)
    k, _, v, _ = rows_of(20, 2, 128, 3, 0.0)
    k[3, 1, 70], k[4, 0, 0], v[5, 1, 127], v[6, 0, 33] = np.inf, -np.inf, np.nan, np.nan
    (kb, k), (vb, v) = to_bf16(k), to_bf16(v)
    step = Step([20], [20], 16)
    c, gc = run_write(fmt, step, 2, 128, k, v, dev_bf16(kb), dev_bf16(vb))
    kr, vr = c.read(step.oracle(), *(np.zeros((20, 2, 128), np.float32) for _ in range(2)))
    for dtype in (torch.float32, torch.bfloat16):
        kg, vg = g.kv_cache_read(gc, step.device(g), dtype)
        for want, got in ((kr, kg), (vr, vg)):
            want, got = torch.from_numpy(want).to(dtype), got.cpu()
            assert torch.isnan(want).any() and torch.equal(torch.isnan(want), torch.isnan(got))
            assert torch.equal(torch.nan_to_num(want), torch.nan_to_num(got))


@pytest.mark.parametrize("fmt", FMTS)
def test_every_code_and_scale_reads_back(fmt):
    """All code bytes under every scale (MXFP4) or assorted absmax (NF4)."""
    g = gnf4()
    say("kv read, every byte", fmt)
    c = oa.Cache(fmt, 1, 4096, 1, 64)
    c.codes[0][0, 0] = np.resize(np.arange(256), (4096, 32))
    c.codes[1][0, 0] = np.resize(np.arange(256)[::-1], (4096, 32))
    if fmt == "mxfp4":
        s = np.resize(np.arange(256).repeat(16), (4096, 2))
    else:
        s = np.resize(np.array([0.0, 1.0, 2.0 ** -149, 2.0 ** -126, 1e-30, 0.3, 3.4028235e38, np.inf, np.nan], np.float32), (4096, 1))
    for side in range(2):
        c.scales[side][0, 0] = s
    step = Step([4096], [4096], 4096, spare=0)
    step.pages[:] = 0
    gc = device_cache(g, c)
    kr, vr = c.read(step.oracle(), *(np.zeros((4096, 1, 64), np.float32) for _ in range(2)))
    for dtype in (torch.float32, torch.bfloat16):
        kg, vg = g.kv_cache_read(gc, step.device(g), dtype)
        for want, got in ((kr, kg), (vr, vg)):
            want, got = torch.from_numpy(want).to(dtype), got.cpu()
            assert torch.equal(torch.isnan(want), torch.isnan(got))
            assert torch.equal(torch.nan_to_num(want, nan=0.0), torch.nan_to_num(got, nan=0.0))


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_and_positions_that_do_not_exist(fmt):
    """Bad page ids, negative positions, positions past the table, rows outside
    the offsets: nothing is written or read there."""
    g = gnf4()
    say("kv bad pages", fmt)
    H, D = 2, 64
    step = Step([40, 50, 3], [10, 4, 6], 16, slack=0)
    step.pages[0, 2] = -1                                    # positions 32..39 of sequence 0
    step.pages[1, 3] = step.n_pages                          # 48, 49 of sequence 1
    step.offsets = [2, 12, 16, 22]                           # two rows before, three behind
    step.T = 25
    k, kd, v, vd = rows_of(25, H, D, 5)
    c, gc = run_write(fmt, step, H, D, k, v, kd, vd)
    want = c.read(step.oracle(), *(np.full((25, H, D), 7.0, np.float32) for _ in range(2)))
    kg, vg = (torch.full((25, H, D), 7.0, device="cuda") for _ in range(2))
    g.kv_cache_read(gc, step.device(g), torch.float32, kg, vg)
    # rows 4..11 of sequence 0 and 14, 15 of sequence 1 are on bad pages, row 16..18 at negative positions
    for w, got in zip(want, (kg, vg)):
        assert np.array_equal(w, got.cpu().numpy())
        left = {0, 1, *range(4, 12), 14, 15, 16, 17, 18, 22, 23, 24}
        assert {r for r in range(25) if (w[r] == 7.0).all()} == left


def test_positions_behind_four_gib():
    """A cache whose code array is longer than 2^32 bytes."""
    g = gnf4()
    page, H, D = 65536, 4, 256
    n = (1 << 32) // (page * H * D // 2) + 2
    say("kv large cache", n, "pages")
    gc = g.empty_kv_cache("mxfp4", n, page, H, D)
    step = Step([3], [3], 64)
    step.page, step.n_pages, step.pages = page, n, np.array([[n - 1]])
    k, kd, v, vd = rows_of(3, H, D, 8, 0.0)
    g.kv_cache_write(gc, kd, vd, step.device(g))
    kg, vg = g.kv_cache_read(gc, step.device(g), torch.float32)
    small = oa.Cache("mxfp4", 1, 16, H, D)
    near = Step([3], [3], 16, spare=0)
    near.pages[:] = 0
    small.write(near.oracle(), k, v)
    kr, vr = small.read(near.oracle(), *(np.zeros((3, H, D), np.float32) for _ in range(2)))
    assert np.array_equal(kr, kg.cpu().numpy()) and np.array_equal(vr, vg.cpu().numpy())
    assert np.array_equal(gc.k_codes[n - 1, :, :3].cpu().numpy(), small.codes[0][0, :, :3])


def test_binding_refusals():
    g = gnf4()
    gc = g.empty_kv_cache("nf4", 4, 16, 2, 64)
    step = Step([5], [5], 16)
    b = step.device(g)
    x = torch.zeros((5, 2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        g.kv_cache_write(gc, x[:4], x, b)
    with pytest.raises(ValueError):
        g.kv_cache_write(gc, x.float(), x, b)
    with pytest.raises(ValueError):
        g.kv_cache_read(gc, b, torch.float16)
    with pytest.raises(ValueError):
        g.KVCache(g.MXFP4, 4, 16, 2, 64, gc.k_codes, gc.k_scales, gc.v_codes, gc.v_scales).packed(0)
    with pytest.raises(ValueError):
        g.KVCache(g.NF4, 5, 16, 2, 64, gc.k_codes, gc.k_scales, gc.v_codes, gc.v_scales).packed(0)
    with pytest.raises(ValueError):
        g.kv_cache_write(gc, x, x, g.KVBatch(b.offsets[:1], b.lens, b.pages, 5, 5, 5))
    with pytest.raises(g.Gnf4Error) as e:
        g.kv_cache_write(gc, x, x, g.KVBatch(b.offsets, b.lens, b.pages, 5, 0, 5))
    assert e.value.status == 1


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B", [63, 65, 200])
def test_many_sequences(fmt, B):
    """More sequences than lanes, and more without new tokens in a row."""
    r = np.random.default_rng(B)
    lens = r.integers(0, 40, B)
    new = np.where(r.random(B) < 0.5, lens, np.minimum(lens, 1))
    new[3:3 + B // 2] = 0
    new[-1] = lens[-1] = 33
    step = Step([int(x) for x in lens], [int(x) for x in new], 16, seed=B)
    k, kd, v, vd = rows_of(step.T, 2, 64, 4)
    c, gc = run_write(fmt, step, 2, 64, k, v, kd, vd)
    g = gnf4()
    want = c.read(step.oracle(), *(np.full((step.T, 2, 64), 7.0, np.float32) for _ in range(2)))
    for w, got in zip(want, g.kv_cache_read(gc, step.device(g), torch.float32)):
        assert np.array_equal(w, got.cpu().numpy())
