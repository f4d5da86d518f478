"""GPU parity of attention over the paged 4-bit cache with the float64 oracle,
and the whole path norm + rotation -> cache write -> attention."""

import numpy as np
import pytest
import torch

from oracle import attention as oa

from .attention_util import (EPS8, Step, attention_bars, check_attention, dev, dev_bf16, device_cache, to_bf16, values)
from .gpu_util import gnf4, say

pytestmark = pytest.mark.gpu

FMTS = ["nf4", "mxfp4"]


def filled(fmt, step, H, D, seed, sharp=1.0):
    """An oracle cache holding every position of the step's sequences; what lies
    elsewhere is NaN scales and random codes."""
    r = np.random.default_rng([seed, H, D, step.page])
    c = oa.Cache(fmt, step.n_pages, step.page, H, D)
    for side in range(2):
        c.codes[side][:] = r.integers(0, 256, c.codes[side].shape)
        c.scales[side][:] = 255 if fmt == "mxfp4" else np.nan
    whole = step.whole()
    k, v = r.standard_normal((2, whole.T, H, D))
    k[..., ::19] *= 2.0
    c.write(whole.oracle(), sharp * k, v)
    return c


def queries(T, Hq, D, seed):
    return to_bf16(np.random.default_rng([T, Hq, D, seed]).standard_normal((T, Hq, D)))


def run(fmt, step, H, G, D, window=0, sinks=False, scale=None, seed=0, sharp=1.0, cache=None, q=None):
    g = gnf4()
    say("kv_attention", fmt, "lens", step.lens[:6], "new", step.new[:6], "page", step.page, "H", H, "G", G, "D", D,
        "window", window, "sinks", sinks)
    c = filled(fmt, step, H, D, seed, sharp) if cache is None else cache
    bits, qv = queries(step.T, H * G, D, seed) if q is None else q
    sk = np.random.default_rng(seed).standard_normal(H * G).astype(np.float32) if sinks else None
    sc = D ** -0.5 if scale is None else scale
    lse = torch.full((step.T, H * G), 5.0, device="cuda")
    out = torch.full((step.T, H * G, D), 7.0, dtype=torch.bfloat16, device="cuda")
    g.kv_attention(dev_bf16(bits), device_cache(g, c), step.device(g), scale, window, None if sk is None else dev(sk),
                   out, lse)
    torch.cuda.synchronize()
    ref = oa.attend(qv, c, step.oracle(), float(np.float32(sc)), window, sk)
    rows = sorted(r for r, _, _ in step.oracle().rows())
    worst = check_attention(fmt, values(out), lse.cpu().numpy().astype(np.float64), ref, rows)
    left = sorted(set(range(step.T)) - set(rows))
    assert torch.all(out[left] == 7.0) and torch.all(lse[left] == 5.0)
    return worst, out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_decode_lengths(fmt, D, G):
    """One new token at lengths around every border of a tile, a round and a page."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]
    run(fmt, Step(lens, [1] * len(lens), 16), 2, G, D)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G,new", [(1, 1), (3, 5), (16, 1), (16, 2), (5, 7), (8, 17), (7, 1), (1, 64), (1, 65), (64, 1), (40, 3)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_row_tiles(fmt, G, new, D):
    """Every count of 16-row tiles, rows that do not fill one, several tiles, causal among the new tokens."""
    run(fmt, Step([new + 40, new, new + 3], [new, new, max(new - 1, 0)], 32), 1 if G > 8 else 2, G, D)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_pages(fmt, page):
    run(fmt, Step([page * 2 + 5, page, 3, page - 1], [2, 1, 3, 1], page, slack=3), 2, 4, 128)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window", [1, 2, 31, 128, 200, 100000, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [False, True])
def test_window_and_sinks(fmt, window, sinks):
    run(fmt, Step([400, 5, 131, 260], [1, 5, 4, 70], 16), 1, 4, 64, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_split_over_workgroups(fmt, D):
    """Few rows over a long context: ranges of it in separate workgroups, joined."""
    g = gnf4()
    step = Step([3000, 900], [1, 1], 64)
    c = filled(fmt, step, 1, D, 3)
    assert g.kv_attention_workspace_bytes(device_cache(g, c), step.device(g), 8) > 0
    run(fmt, step, 1, 8, D, cache=c, sinks=True)
    run(fmt, Step([1500], [19], 32), 1, 3, D)


@pytest.mark.parametrize("fmt", FMTS)
def test_lengths_beyond_the_bound(fmt):
    """max_len only decides the split: sequences longer than it are computed whole."""
    run(fmt, Step([700, 90, 260], [1, 1, 1], 16, max_len=100), 1, 4, 128)
    run(fmt, Step([1700, 90], [1, 1], 16, max_len=600), 1, 4, 128)
    run(fmt, Step([300, 90], [1, 1], 16, max_len=1 << 30), 1, 4, 128)


@pytest.mark.parametrize("fmt", FMTS)
def test_empty_sequences_and_rows_that_see_nothing(fmt):
    """Sequences without new tokens; lengths below the new tokens (rows at
    negative positions); rows before and behind the sequences are left alone."""
    for sinks in (False, True):
        step = Step([30, 0, 12, 7], [2, 0, 0, 7], 16)
        step.lens[3] = 4                                     # rows at -3 .. 3
        step.offsets = [1, 3, 3, 3, 10]
        step.T = 12
        c = filled(fmt, Step([30, 0, 12, 7], [2, 0, 0, 7], 16), 2, 64, 4)
        run(fmt, step, 2, 2, 64, sinks=sinks, cache=c)


@pytest.mark.parametrize("fmt", FMTS)
def test_bad_pages_are_not_attended(fmt):
    step = Step([200, 70], [3, 1], 16)
    c = filled(fmt, step, 2, 128, 5)
    for p in (2, 7):
        step.pages[0, p] = -1
    step.pages[0, 11] = step.n_pages
    step.pages[1, :] = 1 << 30                               # sequence 1 sees nothing
    _, out = run(fmt, step, 2, 4, 128, cache=c)
    assert not out[3].any()
    assert out[:3].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("side", [0, 1])
def test_nan_reaches_only_rows_that_see_it(fmt, D, side):
    """A NaN block at a position that some rows of a tile see and others do not,
    and one inside a full tile."""
    step = Step([300], [40], 16)
    c = filled(fmt, step, 1, D, 6)
    for pos in (280, 289):
        at = c.place(step.oracle(), 0, pos)
        c.scales[side][at[0], 0, at[1], -1] = 255 if fmt == "mxfp4" else np.nan
    _, out = run(fmt, step, 1, 2, D, cache=c)
    bad = torch.isnan(out).any(-1).any(-1).cpu().numpy()
    assert list(bad) == [260 + i >= 280 for i in range(40)]
    c = filled(fmt, step, 1, D, 6)
    at = c.place(step.oracle(), 0, 20)
    c.scales[side][at[0], 0, at[1], 0] = 255 if fmt == "mxfp4" else np.nan
    _, out = run(fmt, step, 1, 2, D, cache=c)
    assert torch.isnan(out).any(-1).all()
    # the window has left position 20 behind for every row
    _, out = run(fmt, step, 1, 2, D, cache=c, window=100)
    assert not torch.isnan(out).any()


@pytest.mark.parametrize("fmt", FMTS)
def test_special_queries(fmt):
    """Infinite and NaN queries give NaN in their own row only; zero queries the mean."""
    step = Step([50, 60], [3, 2], 16)
    c = filled(fmt, step, 1, 64, 7)
    bits, q = queries(5, 2, 64, 7)
    q = q.copy()
    q[0, 0, 3], q[1, 1, 9], q[2] = np.nan, np.inf, 0.0
    bits, q = to_bf16(q)
    g = gnf4()
    say("kv_attention special queries", fmt)
    out = g.kv_attention(dev_bf16(bits), device_cache(g, c), step.device(g))
    assert torch.isnan(out).any(-1).nonzero().tolist() == [[0, 0], [1, 1]]
    with np.errstate(invalid="ignore"):
        ref = oa.attend(q, c, step.oracle(), 0.125)
    bar, _ = attention_bars(fmt, *(ref[i] for i in (0, 2, 3)))
    got = values(out)
    for r, h in ((2, 0), (2, 1), (3, 0), (4, 1), (0, 1), (1, 0)):
        assert np.all(np.abs(got[r, h] - ref[0][r, h]) <= bar[r, h])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales_and_peaked_rows(fmt, scale):
    run(fmt, Step([150, 33], [2, 1], 16), 2, 4, 64, scale=scale)
    run(fmt, Step([150, 33], [2, 1], 16), 2, 4, 64, sharp=4.0)


def test_equal_heads_and_shuffled_pages_give_equal_bits():
    """The result depends on what the pages hold, not on where they lie."""
    g = gnf4()
    say("kv_attention page order")
    a, b = Step([500, 77], [1, 3], 32, seed=1), Step([500, 77], [1, 3], 32, seed=2, spare=9)
    q = dev_bf16(queries(4, 16, 128, 1)[0])
    outs = []
    for s in (a, b):
        c = oa.Cache("nf4", s.n_pages, 32, 2, 128)
        r = np.random.default_rng(5)
        c.write(s.whole().oracle(), *r.standard_normal((2, 577, 2, 128)))
        outs.append(g.kv_attention(q, device_cache(g, c), s.device(g)))
    assert torch.equal(*outs) and torch.equal(outs[0], g.kv_attention(q, device_cache(g, c), b.device(g)))


def test_strides_and_int16_bits():
    g = gnf4()
    say("kv_attention strides")
    step = Step([100, 260], [1, 4], 16)
    c = filled("mxfp4", step, 2, 128, 9)
    gc, b = device_cache(g, c), step.device(g)
    bits, _ = queries(5, 8, 128, 9)
    q = dev_bf16(bits)
    want = g.kv_attention(q, gc, b)
    wide = torch.zeros((5, 3000), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 1024] = q.view(5, 1024)
    out = torch.full((5, 2000), 7.0, dtype=torch.bfloat16, device="cuda")
    g.kv_attention(wide[:, 8:8 + 1024].view(5, 8, 128), gc, b, out=out[:, 16:16 + 1024].view(5, 8, 128))
    assert torch.equal(out[:, 16:16 + 1024].view(5, 8, 128), want)
    assert torch.all(out[:, :16] == 7) and torch.all(out[:, 16 + 1024:] == 7)
    assert torch.equal(g.kv_attention(q.view(torch.int16), gc, b).view(torch.bfloat16), want)


def test_decode_loop_through_a_graph_and_another_stream():
    """Norm + rotation, write and attention of a decode step, captured once and
    replayed while the sequences grow (new lengths and pages come in through
    the same arrays), against eager steps on a second cache and stream."""
    g = gnf4()
    say("decode loop")
    H, Hq, D, page, B, steps = 2, 8, 128, 16, 3, 5
    r = np.random.default_rng(11)
    start = np.array([14, 30, 3])
    width = 4
    pages = r.permutation(B * width).reshape(B, width).astype(np.int32)
    off = dev(np.arange(B + 1, dtype=np.int32))
    lens = dev((start + 1).astype(np.int32))
    pos = dev(start.astype(np.int32))
    batch = g.KVBatch(off, lens, dev(pages), B, 1, 64)
    rope = g.rope_frequencies(D, 10000.0)
    w = dev_bf16(to_bf16(1 + 0.1 * r.standard_normal(D))[0])
    caches = [g.empty_kv_cache("nf4", B * width, page, H, D) for _ in range(2)]
    whole = g.KVBatch(dev(np.concatenate(([0], np.cumsum(start))).astype(np.int32)), dev(start.astype(np.int32)),
                      dev(pages), int(start.sum()), int(start.max()), 64)
    k0, v0 = (dev_bf16(to_bf16(r.standard_normal((int(start.sum()), H, D)))[0]) for _ in range(2))
    for c in caches:
        g.kv_cache_write(c, k0, v0, whole)
    x = torch.zeros((B, (Hq + 2 * H) * D), dtype=torch.bfloat16, device="cuda")
    q, k, v = (x[:, a * D:b * D].view(B, b - a, D) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))

    def step(cache):
        qr, kr = g.qk_norm_rope(q, k, pos, rope, w, w)
        g.kv_cache_write(cache, kr, v, batch)
        return g.kv_attention(qr, cache, batch, sinks=None)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(caches[0])                                      # warm up; rewritten by the first replay
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(caches[0])
    for i in range(steps):
        x.copy_(dev_bf16(to_bf16(r.standard_normal(x.shape))[0]))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = step(caches[1])
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.isfinite(got).all(), i
        lens += 1
        pos += 1
    n = int(lens.sum().item()) - B
    end = g.KVBatch(dev(np.concatenate(([0], np.cumsum(start + steps))).astype(np.int32)), dev((start + steps).astype(np.int32)),
                    dev(pages), n, 64, 64)
    for a, b in zip(g.kv_cache_read(caches[0], end), g.kv_cache_read(caches[1], end)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_path_norm_write_attend_against_the_oracle(fmt):
    """The three calls of a step chained on the device against the oracle's chain on the device's own rounded rows."""
    g = gnf4()
    say("path", fmt)
    H, Hq, D = 2, 8, 64
    step = Step([40, 9, 70], [40, 9, 70], 16)
    r = np.random.default_rng(13)
    pos = np.concatenate([np.arange(n) for n in step.lens]).astype(np.int32)
    rope = g.rope_frequencies(D, 500.0, "linear", 2.0)
    w = dev_bf16(to_bf16(1 + 0.1 * r.standard_normal(D))[0])
    q, k, v = (to_bf16(r.standard_normal((step.T, h, D))) for h in (Hq, H, H))
    qr, kr = g.qk_norm_rope(dev_bf16(q[0]), dev_bf16(k[0]), dev(pos), rope, w, w)
    gc = g.empty_kv_cache(fmt, step.n_pages, 16, H, D)
    b = step.device(g)
    g.kv_cache_write(gc, kr, dev_bf16(v[0]), b)
    out = g.kv_attention(qr, gc, b)
    c = oa.Cache(fmt, step.n_pages, 16, H, D)
    c.write(step.oracle(), values(kr), v[1])
    ref = oa.attend(values(qr), c, step.oracle(), D ** -0.5)
    check_attention(fmt, values(out), None, ref)
    # and the rotated rows are those of the oracle within a bf16 step
    f = rope.inv_freq.cpu().numpy()
    want = oa.norm_rope(k[1], values(w), 1e-6, pos, f, False)
    assert np.all(np.abs(values(kr) - want) <= EPS8 * np.abs(want) + 1e-5)


def test_workspace_and_binding_refusals():
    g = gnf4()
    step = Step([3000], [1], 64)
    c = filled("mxfp4", step, 1, 64, 1)
    gc, b = device_cache(g, c), step.device(g)
    q = dev_bf16(queries(1, 4, 64, 1)[0])
    need = g.kv_attention_workspace_bytes(gc, b, 4)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")      # NaN everywhere: contents do not matter
    assert torch.equal(g.kv_attention(q, gc, b, workspace=ws), g.kv_attention(q, gc, b))
    with pytest.raises(g.Gnf4Error) as e:
        g.kv_attention(q, gc, b, workspace=ws[:need - 16])
    assert e.value.status == 3
    with pytest.raises(ValueError):
        g.kv_attention(q[:, :, :32], gc, b)
    with pytest.raises(ValueError):
        g.kv_attention(q, gc, b, sinks=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        g.kv_attention(q, gc, b, lse=torch.zeros(4, dtype=torch.float64, device="cuda"))


def many(B, seed, longest=60):
    """Lengths and new tokens of B sequences, long runs of which have no new token."""
    r = np.random.default_rng([B, seed])
    lens = r.integers(0, longest, B)
    new = np.where(r.random(B) < 0.4, np.minimum(lens, r.integers(1, 4, B)), 0)
    new[5:5 + B // 2] = 0                                    # more than 64 in a row
    new[-1], lens[-1] = 2, longest
    return [int(x) for x in lens], [int(x) for x in new]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("max_len", [None, 5000])
@pytest.mark.parametrize("B", [63, 64, 65, 200])
def test_many_sequences(fmt, max_len, B):
    """More sequences than lanes, and more empty ones in a row; a workgroup per
    problem (None) and shares of the positions (5000)."""
    lens, new = many(B, 1)
    run(fmt, Step(lens, new, 16, seed=B, max_len=max_len), 2, 2, 64, sinks=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new", [(4, 1), (16, 1), (8, 4), (10, 4)])
def test_many_short_problems(fmt, D, G, new):
    """So many problems that they get small workgroups, each with every row count."""
    lens = [1 + (37 * i) % 90 for i in range(90)]
    run(fmt, Step(lens, [min(n, new) for n in lens], 32, max_len=90), 3, G, D, window=50)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 256])
def test_a_wave_with_more_tiles_than_page_ids(fmt, D):
    """One workgroup over a context of more than 64 of each wave's tiles (the
    ids of a wave's next 64 pages are held in its lanes)."""
    n = 64 * 256 + 300
    run(fmt, Step([n, 40], [2, 1], 16, max_len=1000), 1, 1, D)
    run(fmt, Step([n], [1], 64, max_len=1000), 1, 1, D, window=n - 150)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[700], [3000, 40]])
def test_values_of_very_different_size(fmt, D, lens):
    """Values 2^-20 to 2^20 apart between positions, blocks 2^-6 to 2^6, and positions that are zero."""
    step = Step(lens, [2] * len(lens), 16)
    r = np.random.default_rng([D, len(lens)])
    c = oa.Cache(fmt, step.n_pages, 16, 2, D)
    whole = step.whole()
    k, v = r.standard_normal((2, whole.T, 2, D))
    e = r.integers(-20, 21, (whole.T, 2, 1)) + np.repeat(r.integers(-6, 7, (whole.T, 2, D // 64)), 64, -1)
    v = v * np.exp2(e) * (r.random((whole.T, 2, 1)) < 0.8)
    c.write(whole.oracle(), 2.0 * k, v)
    run(fmt, step, 2, 4, D, cache=c)
    c.write(whole.oracle(), k, v * 2.0 ** -30)
    run(fmt, step, 2, 4, D, cache=c, sinks=True)
    c.write(whole.oracle(), k, np.zeros_like(v))
    _, out = run(fmt, step, 2, 4, D, cache=c)
    assert not out.any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [-100, -30, 30, 60])
def test_queries_of_every_size(fmt, size):
    """Query rows far from 1, undone by the scale or by the keys' size."""
    step = Step([200, 60], [3, 1], 16)
    c = filled(fmt, step, 2, 64, 2)
    _, q = queries(step.T, 8, 64, 3)
    q = q * 2.0 ** (size + np.arange(8) % 3)[:, None]
    run(fmt, step, 2, 4, 64, cache=c, q=to_bf16(q), scale=0.125 * 2.0 ** -size)


def test_positions_behind_four_gib():
    """A sequence whose pages are the first and the last of a cache longer than 2^32 bytes."""
    g = gnf4()
    page, H, D = 65536, 4, 256
    n = (1 << 32) // (page * H * D // 2) + 2
    say("kv_attention large cache", n, "pages")
    gc = g.empty_kv_cache("mxfp4", n, page, H, D)
    r = np.random.default_rng(3)
    near = Step([70], [70], 16, spare=0)
    k, v = r.standard_normal((2, 70, H, D))
    small = oa.Cache("mxfp4", near.n_pages, 16, H, D)
    small.write(near.oracle(), k, v)
    far = Step([70], [2], 64)
    far.page, far.n_pages, far.pages = page, n, np.array([[n - 1]])
    b = far.device(g)
    rows = g.KVBatch(dev(np.array([0, 70], dtype=np.int32)), b.lens, b.pages, 70, 70, 70)
    g.kv_cache_write(gc, dev(k.astype(np.float32)).bfloat16(), dev(v.astype(np.float32)).bfloat16(), rows)
    small.write(near.oracle(), *(to_bf16(x)[1] for x in (k, v)))
    near.new, near.offsets, near.T = [2], [0, 2], 2
    bits, q = queries(2, 8, D, 4)
    out = g.kv_attention(dev_bf16(bits), gc, b)
    check_attention("mxfp4", values(out), None, oa.attend(q, small, near.oracle(), D ** -0.5))


def test_two_streams_and_graphs_with_their_own_workspaces():
    """Two captured calls and two eager ones at once, a workspace each."""
    g = gnf4()
    say("kv_attention two graphs")
    steps = [Step([3000, 1200], [1, 1], 64, seed=1), Step([2500], [3], 32, seed=2)]
    gcs = [device_cache(g, filled("nf4", s, 2, 128, 3)) for s in steps]
    bs = [s.device(g) for s in steps]
    qs = [dev_bf16(queries(s.T, 8, 128, 5)[0]) for s in steps]
    want = [g.kv_attention(*a) for a in zip(qs, gcs, bs)]
    outs = [torch.zeros_like(w) for w in want]
    graphs = []
    for q, c, b, o in zip(qs, gcs, bs, outs):
        ws = torch.empty(g.kv_attention_workspace_bytes(c, b, 8), dtype=torch.uint8, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            g.kv_attention(q, c, b, out=o, workspace=ws)
        graphs.append((gr, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    for i in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, (gr, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        eager = [g.kv_attention(*a) for a in zip(qs, gcs, bs)]
        torch.cuda.synchronize()
        for w, o, e in zip(want, outs, eager):
            assert torch.equal(w, o) and torch.equal(w, e), i


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window", [3, 2 ** 31 - 1])
def test_windows_of_rows_below_position_zero(fmt, window):
    """A tile whose first rows stand below position 0: the widest window takes nothing from its other rows."""
    step = Step([9, 40], [9, 3], 16)
    c = filled(fmt, step, 1, 64, 8)
    step.lens[0] = 4                                         # rows at -5 .. 3
    _, out = run(fmt, step, 1, 2, 64, window=window, cache=c)
    assert not out[:5].any() and out[5:].any(-1).any(-1).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_wide_heads_in_pairs_of_tiles(fmt):
    """D = 256 with more than 16 rows over many positions: two tiles per wave, of
    which the last is part empty."""
    run(fmt, Step([2100, 1300], [50, 33], 32), 2, 8, 256, window=0, sinks=True)
    run(fmt, Step([1500] * 2, [20, 1], 64), 1, 1, 256, window=1100)
    run(fmt, Step([2000] * 24, [5] * 24, 64), 2, 4, 256)


@pytest.mark.parametrize("D", [128, 256])
def test_blocks_of_a_head_far_apart(D):
    """One block of V 2^-18 of the others: the products of its probabilities reach
    below fp16's normal range, 2^-25 of absolute error beside terms around 2^-13,
    which is 2^-12 of their sum and stays inside the bar's two 2^-11."""
    step = Step([400, 60], [2, 1], 16)
    r = np.random.default_rng(D)
    c = oa.Cache("nf4", step.n_pages, 16, 2, D)
    whole = step.whole()
    k, v = r.standard_normal((2, whole.T, 2, D))
    v[..., 64:128] *= 2.0 ** -18
    c.write(whole.oracle(), k, v)
    _, out = run("nf4", step, 2, 4, D, cache=c)
    assert (out[..., 64:128] != 0).float().mean() > 0.99
