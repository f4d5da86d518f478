"""GPU parity of the head norm + rotation and its backward pass with the
float64 oracle."""

import numpy as np
import pytest
import torch

from oracle import attention as oa

from .attention_util import EPS8, dev, dev_bf16, to_bf16, values
from .gpu_util import gnf4, say

pytestmark = pytest.mark.gpu


def case(T, Hq, Hk, D, rot, interleaved, norm, seed=0, fused=True, far=5000, mscale=1.0):
    """Inputs on the host (float64) and the device; q, k as parts of one projection's rows."""
    r = np.random.default_rng([T, Hq, Hk, D, rot, seed])
    bits, x = to_bf16(r.standard_normal((T, (Hq + 2 * Hk) * D)) * np.exp(r.standard_normal((T, 1))))
    q = x[:, :Hq * D].reshape(T, Hq, D)
    k = x[:, Hq * D:(Hq + Hk) * D].reshape(T, Hk, D)
    xd = dev_bf16(bits)
    qd, kd = xd[:, :Hq * D].view(T, Hq, D), xd[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    if not fused:
        qd, kd = qd.contiguous(), kd.contiguous()
    pos = r.integers(-3, far, size=T).astype(np.int32)
    f = (10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32) if rot else None
    w = [to_bf16(1.0 + 0.3 * r.standard_normal(D)) if norm else (None, None) for _ in range(2)]
    return dict(q=q, k=k, qd=qd, kd=kd, pos=pos, posd=dev(pos), f=f, w=[w[0][1], w[1][1]],
                wd=[None if b is None else dev_bf16(b) for b, _ in w], interleaved=interleaved, mscale=mscale)


def rope_of(g, c):
    return None if c["f"] is None else g.Rope(dev(c["f"]), c["interleaved"], c["mscale"])


def check_forward(c, y, i, eps):
    x, w, got = c["qk"[i]], c["w"][i], values(y)
    ref = oa.norm_rope(x, w, eps, c["pos"], c["f"], c["interleaved"], c["mscale"])
    n = oa.norm_rope(x, w, eps, c["pos"], None, False)
    size = np.abs(n)
    if c["f"] is not None:                                   # |a| + |b| of each pair, by the oracle's own pairing
        h = len(c["f"])
        for a, b in ([(2 * j, 2 * j + 1) for j in range(h)] if c["interleaved"] else [(j, j + h) for j in range(h)]):
            size[..., a] = size[..., b] = (size[..., a] + size[..., b]) * c["mscale"]
    worst = (np.abs(got - ref) / (EPS8 * np.abs(ref) + 2e-6 * size + 1e-30)).max()
    assert worst <= 1.0


SHAPES = [(1, 1, 1, 64, 64), (1, 32, 4, 128, 128), (3, 5, 5, 128, 64), (7, 4, 1, 256, 256), (2, 3, 2, 80, 32),
          (5, 2, 1, 16, 16), (33, 16, 16, 96, 96), (4, 8, 2, 256, 64), (2, 1, 0, 128, 128), (2, 0, 3, 64, 16),
          (70, 9, 3, 192, 192), (2049, 2, 1, 64, 64)]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", SHAPES)
def test_forward(T, Hq, Hk, D, rot, interleaved, norm):
    g = gnf4()
    say("norm_rope", T, Hq, Hk, D, rot, interleaved, norm)
    c = case(T, Hq, Hk, D, rot, interleaved, norm, mscale=1.25)
    yq, yk = g.qk_norm_rope(c["qd"], c["kd"], c["posd"], rope_of(g, c), *c["wd"], eps=1e-5)
    torch.cuda.synchronize()
    for i, y in enumerate((yq, yk)):
        if y.numel():
            check_forward(c, y, i, 1e-5)


def test_forward_without_rotation_and_with_one_norm():
    g = gnf4()
    say("norm_rope: no rotation; one weight only")
    c = case(9, 3, 2, 128, 0, False, True)
    c["wd"][1], c["w"][1] = None, None
    yq, yk = g.qk_norm_rope(c["qd"], c["kd"], None, None, *c["wd"], eps=1e-6)
    check_forward(c, yq, 0, 1e-6)
    assert torch.equal(yk, c["kd"])


def test_far_positions():
    """Angles of positions in the millions keep their fraction."""
    g = gnf4()
    say("norm_rope far")
    c = case(64, 2, 1, 128, 128, False, False, far=2 ** 31 - 1)
    yq, yk = g.qk_norm_rope(c["qd"], c["kd"], c["posd"], rope_of(g, c))
    check_forward(c, yq, 0, 0.0)
    check_forward(c, yk, 1, 0.0)


def test_in_place_and_strided_results():
    g = gnf4()
    say("norm_rope in place")
    c = case(21, 6, 2, 128, 64, False, True)
    rope = rope_of(g, c)
    yq, yk = g.qk_norm_rope(c["qd"], c["kd"], c["posd"], rope, *c["wd"])
    wide = torch.full((21, 8, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q2, k2 = wide.view(21, -1)[:, :6 * 128].view(21, 6, 128), wide.view(21, -1)[:, 8 * 128:10 * 128].view(21, 2, 128)
    g.qk_norm_rope(c["qd"], c["kd"], c["posd"], rope, *c["wd"], q_out=q2, k_out=k2)
    assert torch.equal(q2, yq) and torch.equal(k2, yk)
    assert torch.all(wide.view(21, -1)[:, 6 * 128:8 * 128] == 7) and torch.all(wide.view(21, -1)[:, 10 * 128:] == 7)
    g.qk_norm_rope(c["qd"], c["kd"], c["posd"], rope, *c["wd"], q_out=c["qd"], k_out=c["kd"])
    assert torch.equal(c["qd"], yq) and torch.equal(c["kd"], yk)


def test_special_values_stay_in_their_row():
    g = gnf4()
    say("norm_rope NaN / inf / zero rows")
    c = case(6, 2, 1, 128, 128, False, True)
    q = c["qd"].contiguous()
    q[1, 0, 5], q[2, 1, 77], q[3] = float("nan"), float("inf"), 0.0
    y, _ = g.qk_norm_rope(q, c["kd"], c["posd"], rope_of(g, c), *c["wd"])
    nan = torch.isnan(y).any(-1).cpu()
    assert nan.nonzero().tolist() == [[1, 0], [2, 1]] and torch.isnan(y[1, 0]).all()
    assert not y[3].any()


def check_backward(c, dq, dk, out, eps):
    for i, (x, gr, w) in enumerate(((c["q"], dq, c["w"][0]), (c["k"], dk, c["w"][1]))):
        if x.shape[1] == 0:
            continue
        dx, dw = oa.norm_rope_dx(gr, x, w, eps, c["pos"], c["f"], c["interleaved"], c["mscale"])
        gn = oa.norm_rope_dx(gr, x, None, eps, c["pos"], c["f"], c["interleaved"], c["mscale"])[0]
        pair = np.abs(gr)
        if c["f"] is not None:                               # |a| + |b| before the rotation
            h = len(c["f"])
            for a, b in ([(2 * j, 2 * j + 1) for j in range(h)] if c["interleaved"] else [(j, j + h) for j in range(h)]):
                pair[..., a] = pair[..., b] = (pair[..., a] + pair[..., b]) * c["mscale"]
        if w is None:
            size = pair
        else:
            r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
            h, z = pair * np.abs(w), np.abs(x * r)
            size = r * (h + z * (h * z).mean(-1, keepdims=True))
            got = values(out[2 + i])
            bar = 1e-5 * (np.abs(pair) * z).sum((0, 1))
            worst = (np.abs(got - dw) / bar).max()
            assert worst <= 1.0
        got = values(out[i])
        worst = (np.abs(got - dx) / (EPS8 * np.abs(dx) + 4e-6 * size + 1e-30)).max()
        assert worst <= 1.0
        assert gn.shape == dx.shape


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", SHAPES)
def test_backward(T, Hq, Hk, D, rot, interleaved, norm):
    g = gnf4()
    say("norm_rope_dx", T, Hq, Hk, D, rot, interleaved, norm)
    c = case(T, Hq, Hk, D, rot, interleaved, norm, seed=1, mscale=0.75)
    r = np.random.default_rng([T, D, 9])
    (bq, dq), (bk, dk) = to_bf16(r.standard_normal((T, Hq, D))), to_bf16(r.standard_normal((T, Hk, D)))
    out = g.qk_norm_rope_dx(dev_bf16(bq), dev_bf16(bk), c["qd"], c["kd"], c["posd"], rope_of(g, c), *c["wd"], eps=1e-5)
    torch.cuda.synchronize()
    check_backward(c, dq, dk, out, 1e-5)
    again = g.qk_norm_rope_dx(dev_bf16(bq), dev_bf16(bk), c["qd"], c["kd"], c["posd"], rope_of(g, c), *c["wd"], eps=1e-5)
    for a, b in zip(out, again):
        assert (a is None and b is None) or torch.equal(a, b), "two calls differ"


def test_backward_in_place_one_weight_and_no_tokens():
    g = gnf4()
    say("norm_rope_dx in place, one weight, T = 0")
    c = case(13, 4, 2, 128, 128, True, True, seed=2)
    c["wd"][0], c["w"][0] = None, None
    r = np.random.default_rng(3)
    (bq, dq), (bk, dk) = to_bf16(r.standard_normal((13, 4, 128))), to_bf16(r.standard_normal((13, 2, 128)))
    a, b = dev_bf16(bq), dev_bf16(bk)
    out = g.qk_norm_rope_dx(a, b, c["qd"], c["kd"], c["posd"], rope_of(g, c), *c["wd"], gq=a, gk=b)
    assert out[0] is a and out[1] is b and out[2] is None
    check_backward(c, dq, dk, out, 1e-6)
    e = case(0, 4, 2, 128, 128, True, True)
    w = dev_bf16(to_bf16(np.ones(128))[0])
    z = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    out = g.qk_norm_rope_dx(z, z[:, :2], z, z[:, :2], e["posd"], rope_of(g, e), w, w)
    assert not out[2].any() and not out[3].any()


def test_replayed_from_a_graph():
    """Forward and backward captured once and replayed on new inputs."""
    g = gnf4()
    say("norm_rope graph")
    c = case(40, 8, 2, 128, 128, False, True)
    rope = rope_of(g, c)
    r = np.random.default_rng(4)
    d = [dev_bf16(to_bf16(r.standard_normal((40, h, 128)))[0]) for h in (8, 2)]
    q, k = c["qd"].contiguous(), c["kd"].contiguous()
    step = lambda: (*g.qk_norm_rope(q, k, c["posd"], rope, *c["wd"]),  # noqa: E731
                    *g.qk_norm_rope_dx(*d, q, k, c["posd"], rope, *c["wd"]))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        q.copy_(torch.roll(q, 1, 0))
        c["posd"].add_(i)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_binding_refusals():
    g = gnf4()
    c = case(4, 2, 1, 128, 128, False, True)
    rope = rope_of(g, c)
    with pytest.raises(ValueError):
        g.qk_norm_rope(c["qd"].half(), c["kd"], c["posd"], rope)
    with pytest.raises(ValueError):
        g.qk_norm_rope(c["qd"].transpose(0, 1), c["kd"], c["posd"], rope)
    with pytest.raises(ValueError):
        g.qk_norm_rope(c["qd"], c["kd"], c["posd"].long(), rope)
    with pytest.raises(ValueError):
        g.qk_norm_rope(c["qd"], c["kd"], c["posd"][:3], rope)
    with pytest.raises(ValueError):
        g.qk_norm_rope(c["qd"], c["kd"], c["posd"], rope, wq=c["wd"][0][:64])
    with pytest.raises(ValueError):
        g.qk_norm_rope(c["qd"].cpu(), c["kd"], c["posd"], rope)


def test_more_tokens_than_a_launch_has_threads_for():
    """2^24 tokens and some: every one as in a call of its own part."""
    g = gnf4()
    T = (1 << 24) + 5
    say("norm_rope", T, "tokens")
    q = torch.randn((T, 1, 16), dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    w = torch.ones(16, dtype=torch.bfloat16, device="cuda")
    rope = g.rope_frequencies(16, 10000.0)
    k = torch.empty((T, 0, 16), dtype=torch.bfloat16, device="cuda")
    out = g.qk_norm_rope(q, k, pos, rope, w, None)[0]
    for lo, hi in ((0, 9), ((1 << 23) - 4, (1 << 23) + 4), ((1 << 24) - 4, T)):
        part = g.qk_norm_rope(q[lo:hi].contiguous(), k[lo:hi], pos[lo:hi].contiguous(), rope, w, None)[0]
        assert torch.equal(out[lo:hi], part)
