"""Python binding of libgnf4 (ctypes): argument marshalling only.

Every step of the path runs in the HIP library; this module checks tensor
placement, allocates outputs with torch (device memory is torch's), passes raw
device pointers and torch's current HIP stream, and raises on a non-OK status.
There is no fallback: if the library is missing or a call fails, it raises.

Names follow the C ABI in include/gnf4.h: route, grouped_gemm, combine,
dequant, quantize, nf4_codebook, rope_frequencies, qk_norm_rope, kv_cache_write,
kv_cache_read, kv_attention, last_error, build_id.
"""

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgnf4.so")

NF4, NF4_DQ, MXFP4 = 0, 1, 2
FORMATS = {"nf4": NF4, "nf4_dq": NF4_DQ, "mxfp4": MXFP4}
STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE", 4: "DEVICE"}

# Every entry point declared in include/gnf4.h.
EXPORTS = ("gnf4_route", "gnf4_route_workspace_bytes", "gnf4_route_noalloc", "gnf4_route_logits", "gnf4_route_grouped_gemm",
           "gnf4_route_logits_grouped_gemm", "gnf4_grouped_gemm",
           "gnf4_grouped_gemm_swiglu", "gnf4_grouped_gemm_combine",
           "gnf4_grouped_gemm_dx", "gnf4_swiglu", "gnf4_combine",
           "gnf4_dequant", "gnf4_dequant_experts_bf16", "gnf4_quantize", "gnf4_nf4_codebook",
           "gnf4_nf4_codebook_bf16", "gnf4_read_probe",
           "gnf4_expert_cache_state_words", "gnf4_expert_cache_copies_words",
           "gnf4_expert_cache_reset", "gnf4_expert_cache_stage", "gnf4_expert_cache_fill",
           "gnf4_rope_frequencies", "gnf4_qk_norm_rope", "gnf4_qk_norm_rope_dx",
           "gnf4_qk_norm_rope_dx_workspace_bytes", "gnf4_kv_cache_write", "gnf4_kv_cache_read",
           "gnf4_kv_attention", "gnf4_kv_attention_workspace_bytes",
           "gnf4_last_error",
           "gnf4_build_id")


class Gnf4Error(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s failed with %s: %s" % (what, STATUS.get(status, status), last_error()))
        self.status = status


class CWeights(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("E", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("scales2", ctypes.c_void_p)]


class CRope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p), ("mscale", ctypes.c_float)]


class CKVCache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("H", ctypes.c_int32), ("D", ctypes.c_int32), ("k_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class CKVBatch(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("offsets", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("pages", ctypes.c_void_p), ("max_pages", ctypes.c_int32)]


_lib = None


def lib():
    """Load libgnf4.so (built in-tree by bit_mixture_experts_topk_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libgnf4.so is not built; run `python -m bit_mixture_experts_topk_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p
        Z = ctypes.c_size_t
        L.gnf4_route_workspace_bytes.argtypes = [I, I, I]
        L.gnf4_route_workspace_bytes.restype = Z
        L.gnf4_route.argtypes = [P, I, I, I, P, P, P, P, P, P, P, P, Z, S]
        L.gnf4_route_logits.argtypes = [P, I, I, I, P, P, P, P, P, P, P, P, P, P, Z, S]
        L.gnf4_route_noalloc.argtypes = [P, I, I, I, P, P, P, P, P, P, P, S]
        L.gnf4_swiglu.argtypes = [P, I, I, P, S]
        L.gnf4_grouped_gemm.argtypes = [ctypes.POINTER(CWeights), P, I, P, P, P, P, I, I, P, S]
        L.gnf4_grouped_gemm_swiglu.argtypes = [ctypes.POINTER(CWeights), P, I, P, P, P, P, I, I, P, S]
        L.gnf4_route_grouped_gemm.argtypes = [P, I, I, P, P, P, P, P, P, P, P, Z,
                                              ctypes.POINTER(CWeights), P, P, P, S]
        L.gnf4_grouped_gemm_combine.argtypes = [ctypes.POINTER(CWeights), P, P, P, P, P, P, P, I, I,
                                                P, P, S]
        L.gnf4_route_logits_grouped_gemm.argtypes = [P, I, I, P, P, P, P, P, P, P, P, P, P, Z,
                                                     ctypes.POINTER(CWeights), P, P, P, S]
        L.gnf4_grouped_gemm_dx.argtypes = [ctypes.POINTER(CWeights), P, P, I, I, P, S]
        L.gnf4_combine.argtypes = [P, P, P, I, I, I, P, S]
        L.gnf4_dequant.argtypes = [ctypes.POINTER(CWeights), I, P, S]
        L.gnf4_dequant_experts_bf16.argtypes = [ctypes.POINTER(CWeights), P, P, I, P, S]
        L.gnf4_quantize.argtypes = [I, P, I, I, P, P, P, S]
        L.gnf4_expert_cache_state_words.argtypes = [I, I]
        L.gnf4_expert_cache_state_words.restype = ctypes.c_size_t
        L.gnf4_expert_cache_copies_words.argtypes = [I, I, I, I]
        L.gnf4_expert_cache_copies_words.restype = ctypes.c_size_t
        L.gnf4_expert_cache_reset.argtypes = [P, I, I, S]
        L.gnf4_expert_cache_stage.argtypes = [P, I, I, I, I, P, P, P, S]
        L.gnf4_expert_cache_fill.argtypes = [ctypes.POINTER(CWeights), ctypes.POINTER(CWeights), P, I, S]
        F, W = ctypes.c_float, ctypes.c_int64
        # descriptors: a pointer to the structure, or its packed bytes
        D, RP, CP, BP = ctypes.c_double, P, P, P
        L.gnf4_rope_frequencies.argtypes = [I, D, I, D, D, D, D, ctypes.POINTER(F), ctypes.POINTER(F)]
        L.gnf4_qk_norm_rope.argtypes = [P, W, P, W, I, I, I, I, P, P, F, RP, P, P, W, P, W, S]
        L.gnf4_qk_norm_rope_dx.argtypes = [P, W, P, W, P, W, P, W, I, I, I, I, P, P, F, RP, P, P, W, P, W,
                                           P, P, P, Z, S]
        L.gnf4_qk_norm_rope_dx_workspace_bytes.argtypes = [I, I]
        L.gnf4_qk_norm_rope_dx_workspace_bytes.restype = Z
        L.gnf4_kv_cache_write.argtypes = [CP, BP, P, W, P, W, S]
        L.gnf4_kv_cache_read.argtypes = [CP, BP, I, P, P, S]
        L.gnf4_kv_attention.argtypes = [P, W, CP, BP, I, F, I, P, P, W, P, P, Z, S]
        L.gnf4_kv_attention_workspace_bytes.argtypes = [CP, BP, I, I]
        L.gnf4_kv_attention_workspace_bytes.restype = Z
        L.gnf4_nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
        L.gnf4_nf4_codebook.restype = None
        L.gnf4_nf4_codebook_bf16.argtypes = [ctypes.POINTER(ctypes.c_uint16), ctypes.POINTER(ctypes.c_float)]
        L.gnf4_nf4_codebook_bf16.restype = None
        L.gnf4_read_probe.argtypes = [P, ctypes.c_size_t, I, P, S]
        L.gnf4_last_error.restype = ctypes.c_char_p
        L.gnf4_build_id.restype = ctypes.c_char_p
        for name in ("gnf4_route", "gnf4_grouped_gemm", "gnf4_combine", "gnf4_dequant", "gnf4_quantize"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def last_error():
    return lib().gnf4_last_error().decode()


def build_id():
    return lib().gnf4_build_id().decode()


def nf4_codebook():
    buf = (ctypes.c_float * 16)()
    lib().gnf4_nf4_codebook(buf)
    return [buf[i] for i in range(16)]


def nf4_codebook_bf16():
    """(bf16 bits of the 16 NF4 operand values, their scale s): the values
    are bf16(s * c[q]) and the kernels scale partial sums by absmax / s."""
    buf = (ctypes.c_uint16 * 16)()
    sc = ctypes.c_float()
    lib().gnf4_nf4_codebook_bf16(buf, ctypes.byref(sc))
    return [buf[i] for i in range(16)], sc.value


def _check(status, what):
    if status != 0:
        raise Gnf4Error(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dev(t, dtype, name):
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s CUDA tensor" % (name, dtype))
    return t


@dataclass
class PackedWeights:
    """Packed experts of one projection: W [E, N, K] in a 4-bit format."""
    format: int
    E: int
    N: int
    K: int
    codes: torch.Tensor                  # uint8 [E, N, K/2]
    scales: torch.Tensor                 # float32 / int8 / uint8 per format
    scales2: Optional[torch.Tensor] = None

    def cstruct(self):
        return CWeights(self.format, self.E, self.N, self.K, self.codes.data_ptr(),
                        self.scales.data_ptr(),
                        self.scales2.data_ptr() if self.scales2 is not None else None)

    def nbytes(self):
        n = self.codes.numel() + self.scales.numel() * self.scales.element_size()
        if self.scales2 is not None:
            n += self.scales2.numel() * 4
        return n


def empty_packed(fmt, E, N, K, device="cuda", pin_memory=False):
    """Uninitialised packed weights; device="cpu", pin_memory=True gives pinned
    host memory (the host side of the expert streaming cache)."""
    fmt = FORMATS.get(fmt, fmt)
    kw = dict(device=device, pin_memory=pin_memory)
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, **kw)
    scales2 = None
    if fmt == MXFP4:
        scales = torch.empty((E, N, K // 32), dtype=torch.uint8, **kw)
    elif fmt == NF4:
        scales = torch.empty((E, N, K // 64), dtype=torch.float32, **kw)
    else:
        scales = torch.empty((E, N, K // 64), dtype=torch.int8, **kw)
        nb = E * N * (K // 64)
        scales2 = torch.empty(((nb + 255) // 256,), dtype=torch.float32, **kw)
    return PackedWeights(fmt, E, N, K, codes, scales, scales2)


def quantize(fmt, W, out=None):
    """Pack float32 W [E, N, K] (CUDA) with gnf4_quantize."""
    fmt = FORMATS.get(fmt, fmt)
    _dev(W, torch.float32, "W")
    E, N, K = W.shape
    pw = out if out is not None else empty_packed(fmt, E, N, K, W.device)
    _check(lib().gnf4_quantize(fmt, _ptr(W), E * N, K, _ptr(pw.codes), _ptr(pw.scales),
                               _ptr(pw.scales2), _stream()), "gnf4_quantize")
    return pw


def quantize_into(fmt, W, pw, e0):
    """Pack float32 W [n, N, K] into experts [e0, e0 + n) of pw."""
    fmt = FORMATS.get(fmt, fmt)
    _dev(W, torch.float32, "W")
    n, N, K = W.shape
    if fmt == NF4_DQ:
        raise ValueError("NF4_DQ groups span experts; quantize the whole layer at once")
    codes = pw.codes[e0:e0 + n]
    scales = pw.scales[e0:e0 + n]
    _check(lib().gnf4_quantize(fmt, _ptr(W), n * N, K, _ptr(codes), _ptr(scales), None, _stream()),
           "gnf4_quantize")


def route_workspace_bytes(T, k, E):
    return int(lib().gnf4_route_workspace_bytes(T, k, E))


def route_buffers(T, k, E, device="cuda"):
    """Output buffers for route(): counts, offsets, perm, inv, active,
    n_active, bad, and the route's workspace (empty when none is needed)."""
    i32 = dict(dtype=torch.int32, device=device)
    ws = route_workspace_bytes(T, k, E)
    return {"counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
            "perm": torch.empty(max(T * k, 1), **i32), "inv": torch.empty(max(T * k, 1), **i32),
            "active": torch.empty(E, **i32), "n_active": torch.empty(1, **i32),
            "bad": torch.empty(1, **i32),
            "workspace": torch.empty(max(ws, 16), dtype=torch.uint8, device=device)}


def _ws(r):
    """(pointer, bytes) of a route dict's workspace."""
    w = r.get("workspace")
    return (None, 0) if w is None else (_ptr(w), w.numel())


def route(topk_ids, E, out=None):
    """Route int32 topk_ids [T, k] (CUDA) over E experts; returns a dict of tensors."""
    _dev(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    r = dict(out) if out is not None else route_buffers(T, k, E, topk_ids.device)
    _check(lib().gnf4_route(_ptr(topk_ids), T, k, E, _ptr(r["counts"]), _ptr(r["offsets"]),
                            _ptr(r["perm"]), _ptr(r["inv"]), _ptr(r["active"]),
                            _ptr(r["n_active"]), _ptr(r["bad"]), *_ws(r), _stream()), "gnf4_route")
    r["perm"] = r["perm"][:T * k]
    r["inv"] = r["inv"][:T * k]
    return r


def route_noalloc(topk_ids, E, out=None):
    """route() through gnf4_route_noalloc: the library's static workspace,
    no workspace argument (out's "workspace" entry, if any, is not used)."""
    _dev(topk_ids, torch.int32, "topk_ids")
    T, k = topk_ids.shape
    r = dict(out) if out is not None else route_buffers(T, k, E, topk_ids.device)
    _check(lib().gnf4_route_noalloc(_ptr(topk_ids), T, k, E, _ptr(r["counts"]), _ptr(r["offsets"]),
                                    _ptr(r["perm"]), _ptr(r["inv"]), _ptr(r["active"]),
                                    _ptr(r["n_active"]), _ptr(r["bad"]), _stream()),
           "gnf4_route_noalloc")
    r["perm"] = r["perm"][:T * k]
    r["inv"] = r["inv"][:T * k]
    return r


def route_grouped_gemm(topk_ids, w, X, out=None, Y=None, H=None, swiglu=False):
    """route() then grouped_gemm(gather=1) (or grouped_gemm_swiglu when
    swiglu), one launch for a single token; returns (route dict, Y or H)."""
    _dev(topk_ids, torch.int32, "topk_ids")
    if not (X.is_cuda and X.is_contiguous() and X.element_size() == 2):
        raise ValueError("X must be a contiguous bf16 (or 16-bit bit pattern) CUDA tensor")
    T, k = topk_ids.shape
    r = dict(out) if out is not None else route_buffers(T, k, w.E, topk_ids.device)
    if swiglu:
        if H is None:
            H = torch.empty((max(T * k, 1), w.N // 2), dtype=torch.int16, device=X.device)
        res = H
    else:
        if Y is None:
            Y = torch.empty((max(T * k, 1), w.N), dtype=torch.float32, device=X.device)
        res = Y
    cw = w.cstruct()
    _check(lib().gnf4_route_grouped_gemm(_ptr(topk_ids), T, k, _ptr(r["counts"]), _ptr(r["offsets"]),
                                         _ptr(r["perm"]), _ptr(r["inv"]), _ptr(r["active"]),
                                         _ptr(r["n_active"]), _ptr(r["bad"]), *_ws(r), ctypes.byref(cw),
                                         _ptr(X), None if swiglu else _ptr(Y),
                                         _ptr(H) if swiglu else None, _stream()),
           "gnf4_route_grouped_gemm")
    r["perm"] = r["perm"][:T * k]
    r["inv"] = r["inv"][:T * k]
    return r, res


def route_logits_grouped_gemm(logits, k, w, X, out=None, Y=None, H=None, swiglu=False):
    """route_logits() then grouped_gemm(gather=1) (or grouped_gemm_swiglu),
    one launch for a single token; returns (route dict with topk_ids and
    topk_w, Y or H)."""
    _dev(logits, torch.float32, "logits")
    if not (X.is_cuda and X.is_contiguous() and X.element_size() == 2):
        raise ValueError("X must be a contiguous bf16 (or 16-bit bit pattern) CUDA tensor")
    T, E = logits.shape
    r = dict(out) if out is not None else route_buffers(T, k, E, logits.device)
    if "topk_ids" not in r:
        r["topk_ids"] = torch.empty((max(T, 1), k), dtype=torch.int32, device=logits.device)
        r["topk_w"] = torch.empty((max(T, 1), k), dtype=torch.float32, device=logits.device)
    if swiglu:
        if H is None:
            H = torch.empty((max(T * k, 1), w.N // 2), dtype=torch.int16, device=X.device)
        res = H
    else:
        if Y is None:
            Y = torch.empty((max(T * k, 1), w.N), dtype=torch.float32, device=X.device)
        res = Y
    cw = w.cstruct()
    _check(lib().gnf4_route_logits_grouped_gemm(
        _ptr(logits), T, k, _ptr(r["topk_ids"]), _ptr(r["topk_w"]), _ptr(r["counts"]),
        _ptr(r["offsets"]), _ptr(r["perm"]), _ptr(r["inv"]), _ptr(r["active"]), _ptr(r["n_active"]),
        _ptr(r["bad"]), *_ws(r), ctypes.byref(cw), _ptr(X), None if swiglu else _ptr(Y),
        _ptr(H) if swiglu else None, _stream()), "gnf4_route_logits_grouped_gemm")
    r["perm"] = r["perm"][:T * k]
    r["inv"] = r["inv"][:T * k]
    r["topk_ids"] = r["topk_ids"][:T]
    r["topk_w"] = r["topk_w"][:T]
    return r, res


def route_logits(logits, k, out=None):
    """Top-k of float32 router logits [T, E] (CUDA) with softmax weights, then
    route; returns the route dict plus "topk_ids" [T, k] and "topk_w" [T, k]."""
    _dev(logits, torch.float32, "logits")
    T, E = logits.shape
    r = dict(out) if out is not None else route_buffers(T, k, E, logits.device)
    if "topk_ids" not in r:
        r["topk_ids"] = torch.empty((max(T, 1), k), dtype=torch.int32, device=logits.device)
        r["topk_w"] = torch.empty((max(T, 1), k), dtype=torch.float32, device=logits.device)
    _check(lib().gnf4_route_logits(_ptr(logits), T, k, E, _ptr(r["topk_ids"]), _ptr(r["topk_w"]),
                                   _ptr(r["counts"]), _ptr(r["offsets"]), _ptr(r["perm"]),
                                   _ptr(r["inv"]), _ptr(r["active"]), _ptr(r["n_active"]),
                                   _ptr(r["bad"]), *_ws(r), _stream()), "gnf4_route_logits")
    r["perm"] = r["perm"][:T * k]
    r["inv"] = r["inv"][:T * k]
    r["topk_ids"] = r["topk_ids"][:T]
    r["topk_w"] = r["topk_w"][:T]
    return r


def swiglu(Y, I, H=None):
    """H [rows, I] bf16 bits (int16) = bf16(silu(Y[:, :I]) * Y[:, I:2I])."""
    _dev(Y, torch.float32, "Y")
    rows = Y.shape[0]
    if Y.shape[1] != 2 * I:
        raise ValueError("Y must have 2*I columns")
    if H is None:
        H = torch.empty((max(rows, 1), I), dtype=torch.int16, device=Y.device)
    _check(lib().gnf4_swiglu(_ptr(Y), rows, I, _ptr(H), _stream()), "gnf4_swiglu")
    return H


def grouped_gemm(w, X, gather, r, T, k, Y=None):
    """Y [T*k, N] float32 = grouped GEMM of bf16 X over the routed rows."""
    if not (X.is_cuda and X.is_contiguous() and X.element_size() == 2):
        raise ValueError("X must be a contiguous bf16 (or 16-bit bit pattern) CUDA tensor")
    if Y is None:
        Y = torch.empty((max(T * k, 1), w.N), dtype=torch.float32, device=X.device)
    cw = w.cstruct()
    _check(lib().gnf4_grouped_gemm(ctypes.byref(cw), _ptr(X), gather, _ptr(r["offsets"]),
                                   _ptr(r["perm"]), _ptr(r["active"]), _ptr(r["n_active"]),
                                   T, k, _ptr(Y), _stream()), "gnf4_grouped_gemm")
    return Y


def grouped_gemm_swiglu(w, X, gather, r, T, k, H=None):
    """H [T*k, N/2] bf16 bits (int16) = SwiGLU of the grouped GEMM, fused."""
    if not (X.is_cuda and X.is_contiguous() and X.element_size() == 2):
        raise ValueError("X must be a contiguous bf16 (or 16-bit bit pattern) CUDA tensor")
    if H is None:
        H = torch.empty((max(T * k, 1), w.N // 2), dtype=torch.int16, device=X.device)
    cw = w.cstruct()
    _check(lib().gnf4_grouped_gemm_swiglu(ctypes.byref(cw), _ptr(X), gather, _ptr(r["offsets"]),
                                          _ptr(r["perm"]), _ptr(r["active"]), _ptr(r["n_active"]),
                                          T, k, _ptr(H), _stream()), "gnf4_grouped_gemm_swiglu")
    return H


def grouped_gemm_combine(w, X, r, topk_w, T, k, out=None, Y=None):
    """grouped_gemm(gather=0) then combine: out [T, N] float32; one launch for
    a single token. Y is the [T*k, N] intermediate of the two-launch path
    (allocated here when needed)."""
    if not (X.is_cuda and X.is_contiguous() and X.element_size() == 2):
        raise ValueError("X must be a contiguous bf16 (or 16-bit bit pattern) CUDA tensor")
    _dev(topk_w, torch.float32, "topk_w")
    if out is None:
        out = torch.empty((max(T, 1), w.N), dtype=torch.float32, device=X.device)
    if Y is None and not (T == 1 and w.K <= 8192):
        Y = torch.empty((max(T * k, 1), w.N), dtype=torch.float32, device=X.device)
    cw = w.cstruct()
    _check(lib().gnf4_grouped_gemm_combine(ctypes.byref(cw), _ptr(X), _ptr(r["offsets"]), _ptr(r["perm"]),
                                           _ptr(r["inv"]), _ptr(r["active"]), _ptr(r["n_active"]),
                                           _ptr(topk_w), T, k, _ptr(Y), _ptr(out), _stream()),
           "gnf4_grouped_gemm_combine")
    return out


def grouped_gemm_dx(w, dY, r, T, k, dA=None):
    """dA [T*k, K] float32 = dY [T*k, N] (bf16 bits, routed order) times the
    dequantized weights of each row's expert: the input gradient of
    grouped_gemm with frozen weights. Rows past the routed ones are left as
    they are (uninitialised when dA is allocated here)."""
    if not (dY.is_cuda and dY.is_contiguous() and dY.element_size() == 2):
        raise ValueError("dY must be a contiguous bf16 (or 16-bit bit pattern) CUDA tensor")
    if dA is None:
        dA = torch.empty((max(T * k, 1), w.K), dtype=torch.float32, device=dY.device)
    cw = w.cstruct()
    _check(lib().gnf4_grouped_gemm_dx(ctypes.byref(cw), _ptr(dY), _ptr(r["offsets"]), T, k,
                                      _ptr(dA), _stream()), "gnf4_grouped_gemm_dx")
    return dA


def token_grad(dA, r, T, k, out=None):
    """dX [T, K] float32: the sum of each token's k routed copies of dA (the
    gradient through the gather of a first projection), via gnf4_combine
    with unit weights."""
    ones = torch.ones((max(T, 1), k), dtype=torch.float32, device=dA.device)
    return combine(dA, r["inv"], ones, T, k, out=out)


def combine(Y, inv, topk_w, T, k, out=None):
    _dev(Y, torch.float32, "Y")
    _dev(topk_w, torch.float32, "topk_w")
    N = Y.shape[1]
    if out is None:
        out = torch.empty((max(T, 1), N), dtype=torch.float32, device=Y.device)
    _check(lib().gnf4_combine(_ptr(Y), _ptr(inv), _ptr(topk_w), T, k, N, _ptr(out), _stream()),
           "gnf4_combine")
    return out


def dequant_experts_bf16(w, experts, count, max_experts, out=None):
    """bf16 bits (int16) [max_experts, N, K] of the listed experts (device
    int32 experts[], count[1]); slots past *count are left untouched."""
    _dev(experts, torch.int32, "experts")
    _dev(count, torch.int32, "count")
    if out is None:
        out = torch.zeros((max(max_experts, 1), w.N, w.K), dtype=torch.int16, device=w.codes.device)
    cw = w.cstruct()
    _check(lib().gnf4_dequant_experts_bf16(ctypes.byref(cw), _ptr(experts), _ptr(count), max_experts,
                                           _ptr(out), _stream()), "gnf4_dequant_experts_bf16")
    return out


def read_probe(buf, nbytes=None, workgroups=0, sink=None):
    """Read nbytes (default: all) of the CUDA tensor buf once (the achievable
    HBM read rate; over more than 256 MB it also evicts the Infinity Cache)."""
    if not (buf.is_cuda and buf.is_contiguous()):
        raise ValueError("buf must be a contiguous CUDA tensor")
    n = buf.numel() * buf.element_size() if nbytes is None else nbytes
    if sink is None:
        sink = torch.empty(1, dtype=torch.int32, device=buf.device)
    _check(lib().gnf4_read_probe(_ptr(buf), n, workgroups, _ptr(sink), _stream()), "gnf4_read_probe")
    return sink


def dequant(w, e):
    out = torch.empty((w.N, w.K), dtype=torch.float32, device=w.codes.device)
    cw = w.cstruct()
    _check(lib().gnf4_dequant(ctypes.byref(cw), e, _ptr(out), _stream()), "gnf4_dequant")
    return out


# ------------------------------------------------ expert streaming cache

def expert_cache_state(E, S):
    """A reset residency state for S slots over E experts (device int32)."""
    n = lib().gnf4_expert_cache_state_words(E, S)
    if n == 0:
        raise ValueError("invalid cache shape E=%d S=%d" % (E, S))
    state = torch.empty((n,), dtype=torch.int32, device="cuda")
    expert_cache_reset(state, E, S)
    return state


def expert_cache_reset(state, E, S):
    _dev(state, torch.int32, "state")
    _check(lib().gnf4_expert_cache_reset(_ptr(state), E, S, _stream()), "gnf4_expert_cache_reset")


def expert_cache_copies_words(T, k, E, S):
    return int(lib().gnf4_expert_cache_copies_words(T, k, E, S))


def expert_cache_stage(topk_ids, E, S, state, slot_ids=None, copies=None):
    """Residency decision for int32 topk_ids [T, k]: (slot_ids [T, k], copies)."""
    _dev(topk_ids, torch.int32, "topk_ids")
    _dev(state, torch.int32, "state")
    T, k = topk_ids.shape
    if slot_ids is None:
        slot_ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    if copies is None:
        copies = torch.empty((max(expert_cache_copies_words(T, k, E, S), 1),), dtype=torch.int32,
                             device="cuda")
    _check(lib().gnf4_expert_cache_stage(_ptr(topk_ids), T, k, E, S, _ptr(state), _ptr(slot_ids),
                                         _ptr(copies), _stream()), "gnf4_expert_cache_stage")
    return slot_ids, copies


def expert_cache_fill(host_w, cache_w, copies, max_copies):
    """Copy the listed experts of host_w (pinned host memory) into cache_w."""
    _dev(copies, torch.int32, "copies")
    hw, cw = host_w.cstruct(), cache_w.cstruct()
    _check(lib().gnf4_expert_cache_fill(ctypes.byref(hw), ctypes.byref(cw), _ptr(copies), max_copies,
                                        _stream()), "gnf4_expert_cache_fill")


# ------------------------------------------------ attention

ROPE_SCALINGS = {"plain": 0, "linear": 1, "yarn": 2}

# A decode step makes several of these calls per layer and each runs for a few
# microseconds, so the binding's own time is kept down: descriptors are packed
# as bytes (CRope, CKVCache, CKVBatch above give the fields) and every tensor
# is looked at once.
_BITS16 = frozenset((torch.bfloat16, torch.int16))
_pack_rope = struct.Struct("@2iPf4x").pack
_pack_cache = struct.Struct("@5i4x4P").pack
_pack_batch = struct.Struct("@4i3Pi4x").pack
_device = torch.cuda.current_device


def _here(t, dtype, name, dev):
    """Address of t, a contiguous tensor of that type on the current device."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        if t.is_cuda and t.get_device() != dev:
            raise ValueError("%s lies on %s, which is not the current device" % (name, t.device))
        raise ValueError("%s must be a contiguous %s CUDA tensor" % (name, dtype))
    return t.data_ptr()


def _heads(t, T, H, D, name, dev):
    """Token stride of t, bf16 (or 16-bit pattern) [T, H, D] on the current
    device with each token's heads contiguous."""
    if t.dtype not in _BITS16 or t.get_device() != dev or t.shape != (T, H, D):
        if t.is_cuda and t.get_device() != dev:
            raise ValueError("%s lies on %s, which is not the current device" % (name, t.device))
        raise ValueError("%s must be a bf16 (or 16-bit bit pattern) CUDA tensor [%d, %d, %d]" % (name, T, H, D))
    s0, s1, s2 = t.stride()
    if (s2 != 1 or (s1 != D and H > 1)) and T * H:
        raise ValueError("the heads of %s must be contiguous within a token" % name)
    return s0 if T > 1 else H * D                            # a single token: its own size


def _weight(w, D, name, dev):
    if w is None:
        return None
    if w.dtype not in _BITS16 or w.numel() != D:
        raise ValueError("%s must hold D = %d bf16 values" % (name, D))
    return _here(w, w.dtype, name, dev)


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


@dataclass
class Rope:
    """Rotation by position: pair i of a head's first 2 * len(inv_freq) values
    turns by position * inv_freq[i] (float32, CUDA); pairs are neighbours when
    interleaved, else the two halves; both are multiplied by mscale."""
    inv_freq: torch.Tensor
    interleaved: bool = False
    mscale: float = 1.0

    def packed(self, dev):
        f = self.inv_freq
        return _pack_rope(2 * f.numel(), bool(self.interleaved), _here(f, torch.float32, "inv_freq", dev), self.mscale)


@dataclass
class KVCache:
    """A paged 4-bit cache of keys and values: codes uint8 [n_pages, H,
    page_size, D/2], scales float32 [.., D/64] (NF4) or uint8 [.., D/32] (MXFP4)."""
    format: int
    n_pages: int
    page_size: int
    H: int
    D: int
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor

    def packed(self, dev):
        mx = self.format == MXFP4
        kc, ks, vc, vs = self.k_codes, self.k_scales, self.v_codes, self.v_scales
        rows, kind = self.n_pages * self.H * self.page_size, torch.uint8 if mx else torch.float32
        nc, ns = rows * (self.D // 2), rows * (self.D // (32 if mx else 64))
        if kc.numel() != nc or vc.numel() != nc or ks.numel() != ns or vs.numel() != ns:
            raise ValueError("the cache arrays do not hold n_pages * H * page_size rows of D values")
        return _pack_cache(self.format, self.n_pages, self.page_size, self.H, self.D,
                           _here(kc, torch.uint8, "k_codes", dev), _here(ks, kind, "k_scales", dev),
                           _here(vc, torch.uint8, "v_codes", dev), _here(vs, kind, "v_scales", dev))

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales))


@dataclass
class KVBatch:
    """The rows of a step: sequence b's new tokens are rows [offsets[b],
    offsets[b+1]), lens[b] its length with them, pages[b] its page ids (all
    int32, CUDA). max_new bounds the new tokens of one sequence, max_len is
    the longest length expected."""
    offsets: torch.Tensor
    lens: torch.Tensor
    pages: torch.Tensor
    n_tokens: int
    max_new: int
    max_len: int

    def packed(self, dev):
        B, shape = self.lens.numel(), self.pages.shape
        if self.offsets.numel() != B + 1 or len(shape) != 2 or shape[0] != B:
            raise ValueError("offsets must hold B + 1, lens B and pages B rows of ids")
        return _pack_batch(B, self.n_tokens, self.max_new, min(self.max_len, 0x7fffffff),
                           _here(self.offsets, torch.int32, "offsets", dev), _here(self.lens, torch.int32, "lens", dev),
                           _here(self.pages, torch.int32, "pages", dev), shape[1])


def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, beta_fast=32.0,
                     beta_slow=1.0, interleaved=False, device="cuda"):
    """A Rope with the frequencies of gnf4_rope_frequencies on the device."""
    f, m = (ctypes.c_float * max(rot_dim // 2, 1))(), ctypes.c_float()
    _check(lib().gnf4_rope_frequencies(rot_dim, base, ROPE_SCALINGS.get(scaling, scaling), factor, original_len,
                                       beta_fast, beta_slow, f, ctypes.byref(m)), "gnf4_rope_frequencies")
    return Rope(torch.tensor(list(f), dtype=torch.float32, device=device), interleaved, m.value)


def _positions(positions, rope, T, dev):
    """(packed rotation, address of the positions), or nothing."""
    if rope is None:
        return None, None
    if positions.numel() != T:
        raise ValueError("positions must hold T = %d values" % T)
    return rope.packed(dev), _here(positions, torch.int32, "positions", dev)


def _result(out, like, T, H, D, name, dev):
    """(tensor, token stride) of a result [T, H, D]: the given one, or a new one like `like`."""
    if out is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format), H * D
    return out, _heads(out, T, H, D, name, dev)


def qk_norm_rope(q, k, positions, rope=None, wq=None, wk=None, eps=1e-6, q_out=None, k_out=None):
    """Norm (bf16 weights wq, wk [D]; None: no norm) and rotation (None: none)
    of q [T, Hq, D] and k [T, Hk, D] (bf16, any token stride) at int32
    positions [T]; returns (q_out, k_out), which may be q and k themselves."""
    dev = _device()
    T, Hq, D = q.shape
    Hk = k.shape[1]
    qs, ks = _heads(q, T, Hq, D, "q", dev), _heads(k, T, Hk, D, "k", dev)
    r, pos = _positions(positions, rope, T, dev)
    q_out, qos = _result(q_out, q, T, Hq, D, "q_out", dev)
    k_out, kos = _result(k_out, k, T, Hk, D, "k_out", dev)
    _check(lib().gnf4_qk_norm_rope(q.data_ptr(), qs, k.data_ptr(), ks, T, Hq, Hk, D, _weight(wq, D, "wq", dev),
                                   _weight(wk, D, "wk", dev), eps, r, pos, q_out.data_ptr(), qos, k_out.data_ptr(), kos,
                                   _raw_stream(dev)), "gnf4_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_dx(dq, dk, q, k, positions, rope=None, wq=None, wk=None, eps=1e-6, gq=None, gk=None,
                    workspace=None):
    """Backward pass of qk_norm_rope: (gq, gk, dwq, dwk) from the gradients dq,
    dk of its results and its inputs; dwq / dwk float32 [D], None without a
    weight. gq and gk may be dq and dk."""
    dev = _device()
    T, Hq, D = dq.shape
    Hk = dk.shape[1]
    dqs, dks = _heads(dq, T, Hq, D, "dq", dev), _heads(dk, T, Hk, D, "dk", dev)
    qs, ks = _heads(q, T, Hq, D, "q", dev), _heads(k, T, Hk, D, "k", dev)
    r, pos = _positions(positions, rope, T, dev)
    pq, pk = _weight(wq, D, "wq", dev), _weight(wk, D, "wk", dev)
    gq, gqs = _result(gq, dq, T, Hq, D, "gq", dev)
    gk, gks = _result(gk, dk, T, Hk, D, "gk", dev)
    dwq = dwk = None
    L, wsp, wsn = lib(), None, 0
    if pq is not None or pk is not None:
        dw = torch.empty((2, D), dtype=torch.float32, device=dq.device)
        dwq, dwk = dw[0] if pq is not None else None, dw[1] if pk is not None else None
        if workspace is None:
            workspace = torch.empty(L.gnf4_qk_norm_rope_dx_workspace_bytes(T, D), dtype=torch.uint8, device=dq.device)
        wsp, wsn = _here(workspace, workspace.dtype, "workspace", dev), workspace.numel() * workspace.element_size()
    _check(L.gnf4_qk_norm_rope_dx(dq.data_ptr(), dqs, dk.data_ptr(), dks, q.data_ptr(), qs, k.data_ptr(), ks, T, Hq, Hk,
                                  D, pq, pk, eps, r, pos, gq.data_ptr(), gqs, gk.data_ptr(), gks,
                                  dwq.data_ptr() if dwq is not None else None, dwk.data_ptr() if dwk is not None else None,
                                  wsp, wsn, _raw_stream(dev)), "gnf4_qk_norm_rope_dx")
    return gq, gk, dwq, dwk


def empty_kv_cache(fmt, n_pages, page_size, H, D, device="cuda"):
    """An uninitialised cache of n_pages pages of page_size positions."""
    fmt = FORMATS.get(fmt, fmt)
    codes = [torch.empty((n_pages, H, page_size, D // 2), dtype=torch.uint8, device=device) for _ in range(2)]
    mx = fmt == MXFP4
    scales = [torch.empty((n_pages, H, page_size, D // (32 if mx else 64)),
                          dtype=torch.uint8 if mx else torch.float32, device=device) for _ in range(2)]
    return KVCache(fmt, n_pages, page_size, H, D, codes[0], scales[0], codes[1], scales[1])


def kv_cache_write(cache, k, v, batch):
    """Quantize the step's k and v [n_tokens, H, D] (bf16, any token stride)
    into the cache."""
    dev = _device()
    T, H, D = batch.n_tokens, cache.H, cache.D
    ks, vs = _heads(k, T, H, D, "k", dev), _heads(v, T, H, D, "v", dev)
    _check(lib().gnf4_kv_cache_write(cache.packed(dev), batch.packed(dev), k.data_ptr(), ks, v.data_ptr(), vs,
                                     _raw_stream(dev)), "gnf4_kv_cache_write")


def kv_cache_read(cache, batch, dtype=torch.bfloat16, k=None, v=None):
    """The values of the step's rows, (k, v) [n_tokens, H, D] in bf16 or
    float32. Rows that are not in the cache are left as they are (uninitialised
    when k and v are allocated here)."""
    dev = _device()
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be bfloat16 or float32")
    cc, cb = cache.packed(dev), batch.packed(dev)
    shape = (batch.n_tokens, cache.H, cache.D)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache.k_codes.device)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=cache.k_codes.device)
    if k.shape != shape or v.shape != shape:
        raise ValueError("k and v must be [n_tokens, H, D]")
    _check(lib().gnf4_kv_cache_read(cc, cb, dtype is torch.float32, _here(k, dtype, "k", dev), _here(v, dtype, "v", dev),
                                    _raw_stream(dev)), "gnf4_kv_cache_read")
    return k, v


def kv_attention_workspace_bytes(cache, batch, Hq, window=0):
    dev = _device()
    return int(lib().gnf4_kv_attention_workspace_bytes(cache.packed(dev), batch.packed(dev), Hq, window))


def kv_attention(q, cache, batch, scale=None, window=0, sinks=None, out=None, lse=None, workspace=None):
    """Attention of q [n_tokens, Hq, D] (bf16, any token stride) over the cache:
    out [n_tokens, Hq, D] bf16. scale None: 1/sqrt(D); window 0: all earlier
    positions; sinks float32 [Hq]; lse float32 [n_tokens, Hq] is filled when
    given. Rows that belong to no sequence are left as they are (uninitialised
    when out is allocated here)."""
    dev = _device()
    T, Hq, D = batch.n_tokens, q.shape[1], cache.D
    qs = _heads(q, T, Hq, D, "q", dev)
    out, outs = _result(out, q, T, Hq, D, "out", dev)
    if sinks is not None:
        if sinks.numel() != Hq:
            raise ValueError("sinks must hold Hq = %d values" % Hq)
        sinks = _here(sinks, torch.float32, "sinks", dev)
    if lse is not None:
        if lse.numel() != T * Hq:
            raise ValueError("lse must be [n_tokens, Hq]")
        lse = _here(lse, torch.float32, "lse", dev)
    cc, cb, L, wsp, wsn = cache.packed(dev), batch.packed(dev), lib(), None, 0
    if workspace is None:
        need = L.gnf4_kv_attention_workspace_bytes(cc, cb, Hq, window)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    if workspace is not None:
        wsp, wsn = _here(workspace, workspace.dtype, "workspace", dev), workspace.numel() * workspace.element_size()
    _check(L.gnf4_kv_attention(q.data_ptr(), qs, cc, cb, Hq, D ** -0.5 if scale is None else scale, window, sinks,
                               out.data_ptr(), outs, lse, wsp, wsn, _raw_stream(dev)), "gnf4_kv_attention")
    return out
