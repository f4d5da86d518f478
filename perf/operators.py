"""The attention side of a mixture-of-experts layer on 4-bit storage, as cases to measure.

Four operators, in the order in which a model step meets them:

* ``norm_rope``  root-mean-square norm of every query and key head with a learned
  weight, and the rotation by position, in one pass
* ``norm_rope_grad``  its backward pass: gradients of queries, keys and both weights
* ``cache``  new keys and values quantized into a paged 4-bit cache (NF4 or MXFP4)
  as they are written, and read back
* ``attend``  attention of the new tokens' queries over that cache: grouped heads,
  ragged lengths, causal among the new tokens, sliding window, sink logits

``prepare`` makes the inputs of a case from a seed, ``run`` is one pass (plain torch
where ``own`` is false, the library's calls where it is true), ``exact`` the same
result in float64.
"""

import math

import torch

own = False

BF, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
DEV = "cuda"

# The 16 NormalFloat-4 values (float32) and the 8 e2m1 magnitudes.
NF4 = torch.tensor([0xbf800000, 0xbf3239b1, 0xbf066b2e, 0xbeca329e, 0xbe91a24b, 0xbe3d353d,
                    0xbdba7869, 0x00000000, 0x3da2fb01, 0x3e24cadf, 0x3e7c04da, 0x3ead0336,
                    0x3ee1a4b5, 0x3f1007a9, 0x3f3913b0, 0x3f800000],
                   dtype=torch.int64).to(torch.uint32).view(F32)
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F32)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one step of a serving batch: 64 sequences, one token each
        dict(name="norm+rope step", op="norm_rope", T=64, Hq=32, Hk=4, D=128, rot=128,
             interleaved=False, norm=True, far=40000),
        # a long prompt in a context stretched to far positions
        dict(name="norm+rope prompt", op="norm_rope", T=8192, Hq=64, Hk=4, D=128, rot=128,
             interleaved=False, norm=True, far=131072),
        # fine-tuning on one packed batch
        dict(name="norm+rope grad", op="norm_rope_grad", T=4096, Hq=32, Hk=4, D=128, rot=128,
             interleaved=False, norm=True, far=4096),
        # a short odd batch, neighbouring pairs, half of the head rotated
        dict(name="norm+rope grad odd", op="norm_rope_grad", T=257, Hq=16, Hk=16, D=128, rot=64,
             interleaved=True, norm=True, far=2000),
        # what every layer of a decode step stores
        dict(name="cache step", op="cache", fmt="mxfp4", B=64, new=1, even=True, len=2048,
             ragged=0.9, Hk=4, D=128, page=16),
        # prompts of several users stored at once, ragged
        dict(name="cache prompts", op="cache", fmt="nf4", B=5, new=4096, even=False, len=6000,
             ragged=0.3, Hk=8, D=128, page=64),
        # one user, a short context: latency
        dict(name="attend one short", op="attend", fmt="mxfp4", B=1, new=1, even=True, len=777,
             ragged=0.0, Hq=32, Hk=4, D=128, page=16, window=0, sinks=False),
        # an ordinary serving batch
        dict(name="attend batch nf4", op="attend", fmt="nf4", B=32, new=1, even=True, len=8192,
             ragged=0.9, Hq=64, Hk=4, D=128, page=32, window=0, sinks=False),
        # a layer with a sliding window and sinks, 64-wide heads
        dict(name="attend window sinks", op="attend", fmt="mxfp4", B=64, new=1, even=True,
             len=4096, ragged=0.9, Hq=64, Hk=8, D=64, page=16, window=128, sinks=True),
        # long contexts
        dict(name="attend long", op="attend", fmt="mxfp4", B=16, new=1, even=True, len=32768,
             ragged=0.5, Hq=32, Hk=8, D=128, page=64, window=0, sinks=False),
        # a few drafted tokens checked at once
        dict(name="attend draft", op="attend", fmt="nf4", B=8, new=5, even=False, len=4097,
             ragged=0.5, Hq=32, Hk=4, D=128, page=16, window=0, sinks=False),
        # the next chunk of a long prompt
        dict(name="attend chunk", op="attend", fmt="mxfp4", B=2, new=1024, even=False, len=8192,
             ragged=0.4, Hq=32, Hk=4, D=128, page=64, window=0, sinks=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "cache", "cache", "attend", "attend", "attend"])
    if op.startswith("norm"):
        D = rng.choice([64, 128, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 5, 8])
        T = _log(rng, 1, max(1, 8192 * 68 * 128 // ((Hq + Hk) * D * (1 if op == "norm_rope" else 2))))
        T = min(T, 16000)
        return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, rot=rng.choice([D, D, D // 2, D // 4]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8, far=_log(rng, 100, 200000))
    fmt = rng.choice(["mxfp4", "nf4"])
    D = rng.choice([64, 128, 128, 256])
    Hk = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    ragged = round(rng.uniform(0.0, 1.0), 3)
    even = rng.random() < 0.5
    B = _log(rng, 1, 64)
    if op == "cache":
        new = _log(rng, 1, max(1, min(4096, 20000 * 1024 // (B * Hk * D))))
        return dict(op=op, fmt=fmt, B=B, new=new, even=even, len=new + rng.randrange(0, 3000), ragged=ragged,
                    Hk=Hk, D=D, page=page)
    Hq = Hk * rng.choice([1, 2, 4, 7, 8, 16])
    length = _log(rng, 2, max(2, min(32768, 16 * 32768 * 1024 // (B * Hk * D))))
    new = rng.choice([1, 1, 1, _log(rng, 1, 16), _log(rng, 1, 1024)])
    # the products of a drawn case stay below those of the chunk of a long prompt
    new = max(1, min(new, length, 2 * 1024 * 8192 * 32 * 128 // (B * length * Hq * D)))
    return dict(op=op, fmt=fmt, B=B, new=new, even=even, len=length, ragged=ragged, Hq=Hq, Hk=Hk, D=D,
                page=page, window=rng.choice([0, 0, 1, 128, 1000]), sinks=rng.random() < 0.4)


def _lengths(case):
    """(new tokens, lengths) of the sequences: the first has the most of both, the others are spread
    evenly below it. Lengths include the new tokens."""
    new, lens = [], []
    for b in range(case["B"]):
        f, g = (b * 0.6180339887) % 1.0, (b * 0.4142135623) % 1.0
        n = case["new"] if case["even"] else 1 + int((case["new"] - 1) * (1.0 - g))
        new.append(n)
        lens.append(max(n, int(math.ceil(case["len"] * (1.0 - case["ragged"] * f)))))
    return new, lens


def work(case):
    """Each input read once, each output written once."""
    D = case["D"]
    if case["op"].startswith("norm"):
        heads = case["T"] * (case["Hq"] + case["Hk"])
        if case["op"] == "norm_rope":
            return {"bytes": heads * D * 2 * 2 + case["T"] * 4, "flops": heads * D * 7}
        return {"bytes": heads * D * 2 * 3 + case["T"] * 4 + 12 * D, "flops": heads * D * 16}
    row = D // 2 + (D // 32 if case["fmt"] == "mxfp4" else D // 16)
    new, lens = _lengths(case)
    H = case["Hk"]
    if case["op"] == "cache":
        # rows in, codes and scales out, and the same back
        return {"bytes": sum(new) * H * 2 * (2 * D * 2 + 2 * row), "flops": sum(new) * H * 2 * D * 4}
    w, toks, pairs = case["window"], 0, 0
    for n, l in zip(new, lens):
        first = l - n
        toks += l - (max(0, first - w + 1) if w else 0)
        if w:
            pairs += sum(min(w, p + 1) for p in range(first, l))
        else:
            pairs += n * (first + 1) + n * (n - 1) // 2
    return {"bytes": toks * H * 2 * row + sum(new) * case["Hq"] * D * 2 * 2,
            "flops": 4.0 * D * pairs * case["Hq"]}


# ----------------------------------------------------------------- inputs

def _normal(gen, *shape, dtype=BF):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=F32).to(dtype)


def _batch(case, gen):
    """Which rows are new, how long each sequence is, and where its pages lie."""
    new, lens = _lengths(case)
    order = torch.randperm(case["B"], generator=gen, device=DEV).tolist()
    new, lens = [new[i] for i in order], [lens[i] for i in order]
    page = case["page"]
    need = [-(-l // page) for l in lens]
    n_pages = sum(need) + 3
    ids = torch.randperm(n_pages, generator=gen, device=DEV).to(I32)
    table = torch.full((case["B"], max(need)), -1, dtype=I32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    offsets = [0]
    for n in new:
        offsets.append(offsets[-1] + n)
    return dict(offsets=torch.tensor(offsets, dtype=I32, device=DEV),
                lens=torch.tensor(lens, dtype=I32, device=DEV), pages=table, n_tokens=offsets[-1],
                max_new=max(new), max_len=max(lens), page=page, n_pages=n_pages, B=case["B"])


def _stored(case, gen, n_pages, like_keys):
    """Codes and scales of a cache filled with quantized rows, [n_pages][Hk][page][..]. Keys have a few
    channels that are larger than the others, as a model's have."""
    H, P, D = case["Hk"], case["page"], case["D"]
    codes = torch.empty((n_pages, H, P, D // 2), dtype=torch.uint8, device=DEV)
    mx = case["fmt"] == "mxfp4"
    scales = torch.empty((n_pages, H, P, D // (32 if mx else 64)), dtype=torch.uint8 if mx else F32, device=DEV)
    step = max(1, (1 << 26) // (H * P * D))
    for s in range(0, n_pages, step):
        n = min(step, n_pages - s)
        x = torch.randn((n, H, P, D), generator=gen, device=DEV)
        if like_keys:
            x[..., ::37] *= 3.0
        b = x.view(-1, 32 if mx else 64)
        top = b.abs().amax(-1, keepdim=True)
        if mx:
            e = torch.frexp(top)[1] - 3
            m = torch.ldexp(b, -e)
            q = torch.bucketize(m.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)) + 8 * (m < 0)
            scales[s:s + n] = (e + 127).view(n, H, P, D // 32).to(torch.uint8)
            q = q.view(n, H, P, D // 2, 2)
            codes[s:s + n] = (q[..., 0] + 16 * q[..., 1]).to(torch.uint8)
        else:
            t = NF4.to(DEV)
            q = torch.bucketize(b / top, (t[1:] + t[:-1]) / 2).view(n, H, P, D // 2, 2)
            scales[s:s + n] = top.view(n, H, P, D // 64)
            codes[s:s + n] = (16 * q[..., 0] + q[..., 1]).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    D, s = case["D"], dict(case)
    if case["op"].startswith("norm"):
        T, Hq, Hk = case["T"], case["Hq"], case["Hk"]
        # queries, keys and values of a token lie in one row of the projection's output
        qkv = _normal(gen, T, (Hq + 2 * Hk) * D)
        s["q"], s["k"] = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["positions"] = torch.randint(0, case["far"], (T,), generator=gen, device=DEV, dtype=I32)
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=F64) / half)).to(F32).to(DEV)
        for n in ("wq", "wk"):
            s[n] = (1.0 + 0.2 * _normal(gen, D, dtype=F32)).to(BF) if case["norm"] else None
        s["eps"], s["mscale"] = 1e-6, 1.0
        if case["op"] == "norm_rope_grad":
            s["dq"], s["dk"] = _normal(gen, T, Hq, D), _normal(gen, T, Hk, D)
        return s
    s["batch"] = _batch(case, gen)
    n_pages = s["batch"]["n_pages"]
    s["k_codes"], s["k_scales"] = _stored(case, gen, n_pages, True)
    s["v_codes"], s["v_scales"] = _stored(case, gen, n_pages, False)
    T, H = s["batch"]["n_tokens"], case["Hk"]
    if case["op"] == "cache":
        qkv = _normal(gen, T, (4 + 2) * H * D)
        s["k"], s["v"] = qkv[:, 4 * H * D:5 * H * D].view(T, H, D), qkv[:, 5 * H * D:].view(T, H, D)
    else:
        s["q"] = (1.5 * _normal(gen, T, case["Hq"], D, dtype=F32)).to(BF)
        s["sink"] = _normal(gen, case["Hq"], dtype=F32) if case["sinks"] else None
    return s


# ------------------------------------------------------------ plain forms

def _sincos(s):
    """Cosine and sine of position * frequency, [T, 1, rot/2]: the angle in float64."""
    a = s["positions"].to(F64)[:, None] * s["inv_freq"].to(F64)
    return (torch.cos(a) * s["mscale"]).to(F32)[:, None], (torch.sin(a) * s["mscale"]).to(F32)[:, None]


def _rotate(x, c, n, rot, interleaved):
    """Rotates the first rot values of each head by the angle with cosine c and sine n."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, v = a * c - b * n, b * c + a * n
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _norm_rope(s, x, w):
    x = x.to(F32)
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.to(F32)
    c, n = _sincos(s)
    return _rotate(x, c, n, s["rot"], s["interleaved"]).to(BF)


def _norm_rope_grad(s, g, x, w):
    c, n = _sincos(s)
    g = _rotate(g.to(F32), c, -n, s["rot"], s["interleaved"])
    if w is None:
        return g.to(BF), None
    x = x.to(F32)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    z = x * r
    gw = (g * z).sum((0, 1))
    h = g * w.to(F32)
    return ((h - z * (h * z).mean(-1, keepdim=True)) * r).to(BF), gw


def _spots(s):
    """Page and place in it of every new token's row."""
    b = s["batch"]
    off, rows = b["offsets"].long(), torch.arange(b["n_tokens"], device=DEV)
    seq = torch.bucketize(rows, off[1:], right=True)
    pos = b["lens"].long()[seq] - off[seq + 1] + rows
    return b["pages"].long()[seq, pos // b["page"]], pos % b["page"]


def _quantize(fmt, x):
    """Codes (two to a byte) and scales of x [..., D], decided in float64."""
    mx = fmt == "mxfp4"
    b = x.to(F64).unflatten(-1, (-1, 32 if mx else 64))
    top = b.abs().amax(-1, keepdim=True)
    if mx:
        e = torch.clamp(torch.frexp(top)[1] - 1 - 2 + 127, 0, 254) * (top > 0)
        m = torch.ldexp(b, 127 - e)
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=F64, device=DEV)
        up, down = torch.bucketize(m.abs(), mids, right=True), torch.bucketize(m.abs(), mids)
        q = torch.where(up % 2 == 0, up, down) + 8 * torch.signbit(m)     # on a border: the even code
        scale = e[..., 0].to(torch.uint8)
    else:
        t = NF4.to(DEV).to(F64)
        q = torch.where(top > 0, torch.bucketize(b / top.clamp_min(1e-300), (t[1:] + t[:-1]) / 2), 7)
        scale = top[..., 0].to(F32)
    q = q.flatten(-2).unflatten(-1, (-1, 2))
    return (q[..., 0] + 16 * q[..., 1] if mx else 16 * q[..., 0] + q[..., 1]).to(torch.uint8), scale


def _values(fmt, codes, scales):
    """The float32 values that codes [..., D/2] and their scales stand for."""
    byte = torch.arange(256, device=DEV)
    if fmt == "mxfp4":
        t = torch.cat((E2M1, -E2M1)).to(DEV)
        pair = torch.stack((t[byte % 16], t[byte // 16]), -1)
        scale = torch.ldexp(torch.ones((), device=DEV), scales.to(I32) - 127)
    else:
        t = NF4.to(DEV)
        pair = torch.stack((t[byte // 16], t[byte % 16]), -1)
        scale = scales
    x = pair.index_select(0, codes.reshape(-1).to(I32)).view(*codes.shape[:-1], scales.shape[-1], -1)
    return (x * scale[..., None]).flatten(-2)


def _store_and_read(s, n, pid, at):
    codes, scales = _quantize(s["fmt"], s[n])
    s[n + "_codes"][pid, :, at], s[n + "_scales"][pid, :, at] = codes, scales
    return _values(s["fmt"], s[n + "_codes"][pid, :, at], s[n + "_scales"][pid, :, at]).to(BF)


def _cache(s):
    pid, at = _spots(s)
    return _store_and_read(s, "k", pid, at), _store_and_read(s, "v", pid, at)


def _attend(s):
    b, D, Hq, Hk = s["batch"], s["D"], s["Hq"], s["Hk"]
    off, lens = b["offsets"].long(), b["lens"].long()
    tok = torch.arange(b["max_len"], device=DEV)
    # the new rows of each sequence, padded to the most of any
    i = torch.arange(b["max_new"], device=DEV)
    live = i < (off[1:] - off[:-1])[:, None]
    rows = (off[:-1, None] + i).clamp_max(b["n_tokens"] - 1)
    pos = lens[:, None] - (off[1:] - off[:-1])[:, None] + i
    q = s["q"][rows].to(F32).view(b["B"], -1, Hk, Hq // Hk, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    pid = b["pages"].long()[:, tok // b["page"]].clamp_min(0)
    at = tok % b["page"]
    k = _values(s["fmt"], s["k_codes"][pid, :, at], s["k_scales"][pid, :, at])     # [B, L, Hk, D]
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (D ** -0.5)                       # [B, Hk, G*new, L]
    del k
    see = tok <= pos[..., None]
    if s["window"]:
        see &= tok > pos[..., None] - s["window"]
    see &= live[..., None]
    x = x.unflatten(2, (Hq // Hk, -1)).masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    sink = s["sink"].view(1, Hk, -1, 1, 1) if s["sink"] is not None else None
    top = torch.maximum(top, sink) if sink is not None else top
    x = x.sub_(top.clamp_min(-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    total = total + torch.exp(sink - top) if sink is not None else total
    v = _values(s["fmt"], s["v_codes"][pid, :, at], s["v_scales"][pid, :, at])
    y = torch.matmul(x.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (Hq // Hk, -1)) / total
    return y.permute(0, 3, 1, 2, 4)[live].reshape(b["n_tokens"], Hq, D).to(BF)


# -------------------------------------------------------------------- run

def run(state):
    s = state
    if own:
        from bit_mixture_experts_topk_amd import gnf4
        if s["op"].startswith("norm"):
            rope = gnf4.Rope(s["inv_freq"], s["interleaved"], s["mscale"])
            if s["op"] == "norm_rope":
                return gnf4.qk_norm_rope(s["q"], s["k"], s["positions"], rope, s["wq"], s["wk"], s["eps"])
            return gnf4.qk_norm_rope_dx(s["dq"], s["dk"], s["q"], s["k"], s["positions"], rope,
                                        s["wq"], s["wk"], s["eps"])
        b = s["batch"]
        cache = gnf4.KVCache(gnf4.FORMATS[s["fmt"]], b["n_pages"], b["page"], s["Hk"], s["D"],
                             s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
        batch = gnf4.KVBatch(b["offsets"], b["lens"], b["pages"], b["n_tokens"], b["max_new"], b["max_len"])
        if s["op"] == "cache":
            gnf4.kv_cache_write(cache, s["k"], s["v"], batch)
            return gnf4.kv_cache_read(cache, batch, BF)
        return gnf4.kv_attention(s["q"], cache, batch, window=s["window"], sinks=s["sink"])
    if s["op"] == "norm_rope":
        return _norm_rope(s, s["q"], s["wq"]), _norm_rope(s, s["k"], s["wk"])
    if s["op"] == "norm_rope_grad":
        gq, gwq = _norm_rope_grad(s, s["dq"], s["q"], s["wq"])
        gk, gwk = _norm_rope_grad(s, s["dk"], s["k"], s["wk"])
        return gq, gk, gwq, gwk
    return _cache(s) if s["op"] == "cache" else _attend(s)


# ------------------------------------------------------------------ exact

def _turn(s):
    """The rotation of every token as a complex number per frequency, float64."""
    a = torch.outer(s["positions"].double(), s["inv_freq"].double())
    return torch.polar(torch.full_like(a, s["mscale"]), a)[:, None]


def _apply(x, z, rot, interleaved):
    pair = x[..., :rot].unflatten(-1, (rot // 2, 2) if interleaved else (2, rot // 2))
    pair = pair if interleaved else pair.transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    y = (y if interleaved else y.transpose(-1, -2)).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _row_values(s, which, b):
    """Keys or values of sequence b, [len, Hk, D] in float64, from the stored bytes."""
    bat, P = s["batch"], s["page"]
    n = int(bat["lens"][b])
    pages = bat["pages"][b, :-(-n // P)].long()
    codes, scales = s[which + "_codes"][pages], s[which + "_scales"][pages]
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    if s["fmt"] == "mxfp4":
        t = torch.tensor([m * g for g in (1, -1) for m in (0, .5, 1, 1.5, 2, 3, 4, 6)], dtype=F64, device=DEV)
        x, size = torch.stack((t[lo], t[hi]), -1), torch.exp2(scales.double() - 127.0)
    else:
        t = NF4.to(DEV).double()
        x, size = torch.stack((t[hi], t[lo]), -1), scales.double()
    x = x.flatten(-2).unflatten(-1, (size.shape[-1], -1)) * size[..., None]
    return x.flatten(-2).transpose(1, 2).reshape(-1, s["Hk"], s["D"])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    D = s["D"]
    if s["op"].startswith("norm"):
        z, rot, il = _turn(s), s["rot"], s["interleaved"]
        ys, gxs, gws = [], [], []
        for n in ("q", "k"):
            x, w = s[n].double(), s["w" + n]
            r = (x.square().sum(-1, keepdim=True) / D + s["eps"]).pow(-0.5) if w is not None else 1.0
            weight = w.double() if w is not None else 1.0
            ys.append(_apply(x * r * weight, z, rot, il))
            if s["op"] == "norm_rope_grad":
                g = _apply(s["d" + n].double(), z.conj(), rot, il)
                if w is None:
                    gxs.append(g)
                    gws.append(None)
                else:
                    gws.append(torch.einsum("thd,thd->d", g, x * r))
                    u = g * weight
                    gxs.append(r * u - x * r ** 3 * (u * x).sum(-1, keepdim=True) / D)
        return tuple(ys) if s["op"] == "norm_rope" else (*gxs, *gws)
    if s["op"] == "cache":
        out = []
        for n in ("k", "v"):
            x = s[n].double()
            if s["fmt"] == "mxfp4":
                t = x.unflatten(-1, (-1, 32))
                size = torch.exp2(torch.floor(torch.log2(t.abs().amax(-1, keepdim=True))) - 2)
                grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=F64, device=DEV)
                a = (t / size).abs().clamp_max(6.0)
                step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(F64)
                a = torch.round(a / step) * step         # to the even multiple of the step
                assert torch.isin(a, grid).all()
                out.append((torch.sign(t) * a * size).flatten(-2))
            else:
                t = x.unflatten(-1, (-1, 64))
                top = t.abs().amax(-1, keepdim=True)
                c = NF4.to(DEV).double()
                y, best = torch.zeros_like(t), torch.full_like(t, math.inf)
                for v in c:
                    d = (t - v * top).abs()
                    y, best = torch.where(d < best, v * top, y), torch.minimum(d, best)
                out.append(y.flatten(-2))
        return tuple(out)
    bat, G = s["batch"], s["Hq"] // s["Hk"]
    off, lens = bat["offsets"].tolist(), bat["lens"].tolist()
    out = torch.empty(bat["n_tokens"], s["Hq"], D, dtype=F64, device=DEV)
    for b in range(bat["B"]):
        n, L = off[b + 1] - off[b], lens[b]
        k, v = _row_values(s, "k", b), _row_values(s, "v", b)
        p = torch.arange(L - n, L, device=DEV)[:, None]
        t = torch.arange(L, device=DEV)
        hide = (t > p) | ((t <= p - s["window"]) if s["window"] else False)
        for h in range(s["Hq"]):
            x = s["q"][off[b]:off[b + 1], h].double() @ k[:, h // G].T / math.sqrt(D)
            x = x.masked_fill(hide, -math.inf)
            if s["sink"] is not None:
                x = torch.cat((x, s["sink"][h].double().expand(n, 1)), 1)
            x = torch.softmax(x, -1)[:, :L]
            out[off[b]:off[b + 1], h] = x @ v[:, h // G]
    return out
