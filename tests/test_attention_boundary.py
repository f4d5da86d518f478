"""Refusals of the attention calls and the host-side frequency table: every
check runs before any HIP call (no GPU needed)."""

import ctypes
import os

import numpy as np
import pytest

from oracle import attention as oa

gnf4 = pytest.importorskip("bit_mixture_experts_topk_amd.gnf4")

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x10000                                   # an aligned address that is never touched


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gnf4.LIB_PATH):
        pytest.fail("libgnf4.so is not built (run python -m bit_mixture_experts_topk_amd.build)")
    return gnf4.lib()


def refused(st, want, text):
    assert st == want and text in gnf4.last_error(), (st, gnf4.last_error())


@pytest.mark.parametrize("args", [(64, 10000.0, "plain", 1.0, 0.0, 32.0, 1.0), (128, 5e5, "linear", 4.0, 0.0, 32.0, 1.0),
                                  (64, 150000.0, "yarn", 32.0, 4096.0, 32.0, 1.0), (2, 1.5, "yarn", 1.0, 10.0, 4.0, 0.0),
                                  (256, 1e6, "plain", 1.0, 0.0, 32.0, 1.0)])
def test_rope_frequencies_match_the_oracle(L, args):
    rot, base, kind, factor, length, fast, slow = args
    f, m = (ctypes.c_float * (rot // 2))(), ctypes.c_float()
    assert L.gnf4_rope_frequencies(rot, base, gnf4.ROPE_SCALINGS[kind], factor, length, fast, slow, f, ctypes.byref(m)) == OK
    want, wm = oa.rope_frequencies(*args)
    # float64 formulas of a few operations each, rounded once: at most a float32 step apart
    assert np.allclose(np.array(list(f), dtype=np.float32), want, rtol=2.0 ** -23, atol=0)
    assert abs(m.value - wm) <= 2.0 ** -23 * wm


@pytest.mark.parametrize("kw,text", [
    (dict(rot=0), "rot_dim"), (dict(rot=63), "rot_dim"), (dict(rot=258), "rot_dim"), (dict(base=1.0), "base"),
    (dict(base=float("nan")), "base"), (dict(kind=3), "scaling"), (dict(kind=1, factor=0.5), "factor"),
    (dict(kind=2, factor=2.0, length=0.0), "YARN"), (dict(kind=2, factor=2.0, fast=1.0), "YARN"),
    (dict(out=False), "NULL")])
def test_rope_frequencies_refusals(L, kw, text):
    d = dict(rot=64, base=1e4, kind=0, factor=1.0, length=1e3, fast=32.0, slow=1.0, out=True)
    d.update(kw)
    f = (ctypes.c_float * 128)()
    st = L.gnf4_rope_frequencies(d["rot"], d["base"], d["kind"], d["factor"], d["length"], d["fast"], d["slow"],
                                 f if d["out"] else None, None)
    refused(st, INVALID, text)


NORM = dict(q=A, qs=512, k=A, ks=256, T=2, Hq=4, Hk=2, D=128, wq=A, wk=A, eps=1e-6, rot=128, il=0, f=A, rope=True,
            pos=A, qo=A, qos=512, ko=A, kos=256)


def norm_call(L, **kw):
    d = dict(NORM)
    d.update(kw)
    r = gnf4.CRope(d["rot"], d["il"], d["f"], 1.0)
    return L.gnf4_qk_norm_rope(d["q"], d["qs"], d["k"], d["ks"], d["T"], d["Hq"], d["Hk"], d["D"], d["wq"], d["wk"],
                               d["eps"], ctypes.byref(r) if d["rope"] else None, d["pos"], d["qo"], d["qos"], d["ko"],
                               d["kos"], None)


def dx_call(L, dwq=A, dwk=A, ws=A, wsb=1 << 30, **kw):
    d = dict(NORM)
    d.update(kw)
    r = gnf4.CRope(d["rot"], d["il"], d["f"], 1.0)
    return L.gnf4_qk_norm_rope_dx(d.get("dq", A), d.get("dqs", 512), A, 256, d["q"], d["qs"], d["k"], d["ks"], d["T"],
                                  d["Hq"], d["Hk"], d["D"], d["wq"], d["wk"], d["eps"],
                                  ctypes.byref(r) if d["rope"] else None, d["pos"], d["qo"], d["qos"], d["ko"],
                                  d["kos"], dwq, dwk, ws, wsb, None)


BAD_NORM = [
    (dict(T=-1), "T = -1"), (dict(Hq=-1), "heads"), (dict(Hq=0, Hk=0), "heads"), (dict(Hq=65535), "heads"),
    (dict(D=8), "D = 8"), (dict(D=264), "D = 264"), (dict(D=100), "D = 100"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(wq=A + 2), "wq"),
    (dict(rot=0), "rot_dim"), (dict(rot=24), "rot_dim"), (dict(rot=144), "rot_dim"), (dict(il=2), "interleaved"),
    (dict(f=None), "inv_freq"), (dict(f=A + 1), "inv_freq"), (dict(pos=None), "positions"), (dict(q=None), "q is NULL"),
    (dict(q=A + 8), "16-byte"), (dict(qs=504), "stride"), (dict(qs=516), "stride"), (dict(ks=0), "stride"),
    (dict(qo=None), "NULL"), (dict(ko=A + 4), "16-byte"), (dict(kos=248), "stride")]


@pytest.mark.parametrize("kw,text", BAD_NORM)
def test_norm_rope_refusals(L, kw, text):
    refused(norm_call(L, **kw), INVALID, text)
    refused(dx_call(L, **kw), INVALID, text)


def test_norm_rope_dx_refusals(L):
    refused(dx_call(L, wq=None), INVALID, "without a weight")
    refused(dx_call(L, dwk=A + 2), INVALID, "4-byte")
    refused(dx_call(L, dq=None), INVALID, "dq is NULL")
    refused(dx_call(L, dqs=256), INVALID, "stride")
    need = L.gnf4_qk_norm_rope_dx_workspace_bytes(2, 128)
    assert need > 0 and L.gnf4_qk_norm_rope_dx_workspace_bytes(2, 100) == 0
    assert L.gnf4_qk_norm_rope_dx_workspace_bytes(-1, 128) == 0
    refused(dx_call(L, wsb=need - 1), WORKSPACE, "needed")
    refused(dx_call(L, ws=None), INVALID, "workspace")
    refused(dx_call(L, ws=A + 4), INVALID, "workspace")


def test_norm_rope_of_nothing_is_ok(L):
    assert norm_call(L, T=0, q=None, k=None, qo=None, ko=None, pos=None) == OK
    assert dx_call(L, T=0, wq=None, wk=None, dwq=None, dwk=None, ws=None, wsb=0) == OK


CACHE = dict(fmt=2, n_pages=4, page=16, H=2, D=128, kc=A, ks=A, vc=A, vs=A)
BATCH = dict(B=2, n=3, max_new=2, max_len=40, off=A, lens=A, pages=A, max_pages=3)


def structs(kw):
    c, b = dict(CACHE), dict(BATCH)
    for k, v in kw.items():
        (c if k in c else b)[k] = v
    return (gnf4.CKVCache(c["fmt"], c["n_pages"], c["page"], c["H"], c["D"], c["kc"], c["ks"], c["vc"], c["vs"]),
            gnf4.CKVBatch(b["B"], b["n"], b["max_new"], b["max_len"], b["off"], b["lens"], b["pages"], b["max_pages"]))


def calls(L, kw):
    c, b = structs(kw)
    c, b = ctypes.byref(c), ctypes.byref(b)
    return [L.gnf4_kv_cache_write(c, b, A, 256, A, 256, None), L.gnf4_kv_cache_read(c, b, 0, A, A, None),
            L.gnf4_kv_attention(A, 1024, c, b, 8, 0.1, 0, None, A, 1024, None, A, 1 << 40, None)]


@pytest.mark.parametrize("kw,want,text", [
    (dict(fmt=1), UNSUPPORTED, "NF4_DQ"), (dict(fmt=5), INVALID, "format"), (dict(n_pages=0), INVALID, "n_pages"),
    (dict(page=8), INVALID, "page_size"), (dict(page=48), INVALID, "page_size"), (dict(page=1 << 17), INVALID, "page_size"),
    (dict(H=0), INVALID, "H = 0"), (dict(H=1025), INVALID, "H = 1025"), (dict(D=96), UNSUPPORTED, "D = 96"),
    (dict(kc=None), INVALID, "NULL"), (dict(vs=None), INVALID, "NULL"), (dict(vc=A + 8), INVALID, "16-byte"),
    (dict(ks=A + 4), INVALID, "16-byte"), (dict(B=-1), INVALID, "B = -1"), (dict(B=(1 << 20) + 1), INVALID, "B ="),
    (dict(n=-1), INVALID, "n_tokens"), (dict(max_new=0), INVALID, "max_new"), (dict(max_pages=0), INVALID, "max_pages"),
    (dict(max_pages=1 << 27), INVALID, "max_pages"), (dict(off=None), INVALID, "NULL"), (dict(lens=None), INVALID, "NULL"),
    (dict(pages=A + 2), INVALID, "4-byte"), (dict(n=(1 << 31) - 1, H=1024), UNSUPPORTED, "too many rows")])
def test_cache_and_batch_refusals(L, kw, want, text):
    c, b = structs(kw)
    c, b = ctypes.byref(c), ctypes.byref(b)
    refused(L.gnf4_kv_cache_write(c, b, A, 1 << 20, A, 1 << 20, None), want, text)
    refused(L.gnf4_kv_cache_read(c, b, 0, A, A, None), want, text)
    refused(L.gnf4_kv_attention(A, 1 << 20, c, b, 8, 0.1, 0, None, A, 1 << 20, None, A, 1 << 40, None), want, text)


def test_null_descriptors_are_refused(L):
    c, b = structs({})
    refused(L.gnf4_kv_cache_write(None, ctypes.byref(b), A, 256, A, 256, None), INVALID, "descriptor")
    refused(L.gnf4_kv_attention(A, 1024, ctypes.byref(c), None, 8, 0.1, 0, None, A, 1024, None, A, 1 << 40, None),
            INVALID, "descriptor")
    assert L.gnf4_kv_attention_workspace_bytes(None, None, 8, 0) == 0


def test_row_arguments_refusals(L):
    c, b = (ctypes.byref(x) for x in structs({}))
    refused(L.gnf4_kv_cache_write(c, b, None, 256, A, 256, None), INVALID, "k is NULL")
    refused(L.gnf4_kv_cache_write(c, b, A, 248, A, 256, None), INVALID, "stride")
    refused(L.gnf4_kv_cache_write(c, b, A, 256, A + 2, 256, None), INVALID, "16-byte")
    refused(L.gnf4_kv_cache_read(c, b, 2, A, A, None), INVALID, "out_f32")
    refused(L.gnf4_kv_cache_read(c, b, 1, None, A, None), INVALID, "NULL")
    refused(L.gnf4_kv_cache_read(c, b, 1, A, A + 8, None), INVALID, "16-byte")


@pytest.mark.parametrize("kw,want,text", [
    (dict(Hq=7), INVALID, "Hq = 7"), (dict(Hq=0), INVALID, "Hq = 0"), (dict(Hq=131072), INVALID, "Hq ="),
    (dict(scale=float("nan")), INVALID, "scale"), (dict(scale=float("inf")), INVALID, "scale"),
    (dict(window=-1), INVALID, "window"), (dict(q=None), INVALID, "q is NULL"), (dict(qs=1016), INVALID, "stride"),
    (dict(out=A + 2), INVALID, "16-byte"), (dict(os=1000), INVALID, "stride"), (dict(sinks=A + 1), INVALID, "4-byte"),
    (dict(lse=A + 2), INVALID, "4-byte"), (dict(wsb=-1), WORKSPACE, "needed"), (dict(ws=None), INVALID, "workspace"),
    (dict(ws=A + 8), INVALID, "workspace")])
def test_attention_refusals(L, kw, want, text):
    c, b = (ctypes.byref(x) for x in structs(dict(max_len=4096, max_pages=400)))
    need = L.gnf4_kv_attention_workspace_bytes(c, b, 8, 0)
    assert need > 0
    d = dict(q=A, qs=1024, Hq=8, scale=0.1, window=0, sinks=None, out=A, os=1024, lse=None, ws=A, wsb=0)
    d.update(kw)
    refused(L.gnf4_kv_attention(d["q"], d["qs"], c, b, d["Hq"], d["scale"], d["window"], d["sinks"], d["out"], d["os"],
                                d["lse"], d["ws"], need + d["wsb"], None), want, text)


def test_a_step_without_rows_is_ok(L):
    for kw in (dict(n=0, off=None, lens=None, pages=None), dict(B=0, off=None, lens=None, pages=None)):
        assert calls(L, kw) == [OK, OK, OK]
    c, b = (ctypes.byref(x) for x in structs(dict(n=0)))
    assert L.gnf4_kv_attention_workspace_bytes(c, b, 8, 0) == 0
    refused(L.gnf4_kv_attention(A, 1024, c, b, 7, 0.1, 0, None, A, 1024, None, None, 0, None), INVALID, "Hq = 7")


def test_workspace_does_not_grow_with_the_bounds(L):
    """A short context needs none; wide bounds do not make it large."""
    for D in (64, 128, 256):
        for max_len in (1, 128, 1 << 15, 1 << 30):
            for n, new in ((1, 1), (64, 1), (64, 64), (1000, 1 << 30)):
                c, b = (ctypes.byref(x) for x in structs(dict(D=D, B=4, n=n, max_new=new, max_len=max_len,
                                                              max_pages=1 << 26)))
                need = L.gnf4_kv_attention_workspace_bytes(c, b, 16, 0)
                assert need <= 256 << 20, (D, max_len, n, new, need)
                if max_len <= 128:
                    assert need == 0


def test_launches_stay_below_their_thread_limit(L):
    """Problems and tokens whose launch would have 2^32 threads are refused."""
    ok = dict(B=1 << 19, H=8, n=1 << 19, max_new=1, max_len=100)
    for kw, bad in ((ok, False), (dict(ok, B=1 << 20, n=1 << 20), True), (dict(ok, max_new=1 << 19), True)):
        c, b = (ctypes.byref(x) for x in structs(kw))
        st = L.gnf4_kv_attention(None, 1024, c, b, 8, 0.1, 0, None, A, 1024, None, None, 0, None)
        refused(st, UNSUPPORTED if bad else INVALID, "too many rows" if bad else "q")
    c, b = (ctypes.byref(x) for x in structs(dict(n=(1 << 27) + 1)))
    refused(L.gnf4_kv_cache_write(c, b, A, 256, A, 256, None), UNSUPPORTED, "too many rows")
