"""ctypes binding of the layer operators of liblora_mlp.so (include/lora_layer.h): attention over
packed documents and to the states of another length, the residual add with the norms before and after a block, log probabilities
of given tokens, norms of query and key heads with the rotation by position, and distillation from a
teacher's top logits, forward and backward.

Argument marshalling only, as in lib.py: types and layouts are checked here, sizes and pointers by
the C entry point of the same name, and every non-zero status raises ``LmError``.  Every operator
takes ``stream`` (a torch stream or a raw handle; None: the current one): its results and workspace
are allocated on the stream that its kernels run on.
"""
from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass
from typing import Optional

import torch

from . import lib as L
from .lib import LmError, workspace  # noqa: F401  (re-exported)

HEADER = os.path.join(os.path.dirname(L.PKG), "include", "lora_layer.h")
LM_BF16, LM_F32 = 0, 1
LM_I32, LM_I64 = 0, 1
_DTYPES = {torch.bfloat16: LM_BF16, torch.float32: LM_F32}
_INDEX = {torch.int32: LM_I32, torch.int64: LM_I64}

_P, _I64, _I32, _SZ, _SZP, _F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                                 ctypes.POINTER(ctypes.c_size_t), ctypes.c_float)


class lm_heads(ctypes.Structure):
    _fields_ = [("p", _P), ("token_stride", _I64), ("head_stride", _I64)]


class lm_attn(ctypes.Structure):
    _fields_ = [("scale", _F), ("cap", _F), ("slopes", _P), ("causal", _I32), ("window", _I32), ("cu_docs", _P),
                ("prefix", _P), ("n_docs", _I32), ("reserved", _I32)]


class lm_cross(ctypes.Structure):
    _fields_ = [("scale", _F), ("cap", _F), ("cu_q", _P), ("cu_k", _P), ("k_len", _P), ("n_docs", _I32), ("reserved", _I32)]


class lm_addnorm(ctypes.Structure):
    _fields_ = [("w_in", _P), ("w_post", _P), ("gate", _P), ("alpha", _F), ("eps", _F), ("w_offset", _F),
                ("h_dtype", _I32), ("w_dtype", _I32), ("reserved", _I32)]


class lm_qkrope(ctypes.Structure):
    _fields_ = [("inv_freq", _P), ("pos", _P), ("axis", _P), ("w_q", _P), ("w_k", _P), ("factor", _F), ("eps", _F),
                ("w_offset", _F), ("rot", _I32), ("axes", _I32), ("interleaved", _I32), ("norm", _I32), ("pos_index", _I32),
                ("w_dtype", _I32), ("reserved", _I32)]


class lm_teacher(ctypes.Structure):
    _fields_ = [("ids", _P), ("values", _P), ("K", _I32), ("index", _I32), ("dtype", _I32), ("rest", _I32)]


_HP = ctypes.POINTER(lm_heads)
_AP = ctypes.POINTER(lm_attn)
_CP = ctypes.POINTER(lm_cross)
_NP = ctypes.POINTER(lm_addnorm)
_RP = ctypes.POINTER(lm_qkrope)
_TP = ctypes.POINTER(lm_teacher)

_SIGS = {
    "attn_workspace_size": ([_I64, _I32, _I32, _I32, _SZP], _I32),
    "attn_debug_inject": ([_I32, ctypes.c_uint64], _I32),
    "attn_fwd": ([_I64, _I32, _I32, _I32, _HP, _HP, _HP, _AP, _P, _P, _P, _P, _SZ, _P], _I32),
    "attn_bwd": ([_I64, _I32, _I32, _I32, _HP, _HP, _HP, _HP, _P, _P, _P, _AP, _P, _P, _P, _P, _SZ, _P], _I32),
    "cross_workspace_size": ([_I64, _I64, _I32, _I32, _I32, _SZP], _I32),
    "cross_fwd": ([_I64, _I64, _I32, _I32, _I32, _HP, _HP, _HP, _CP, _P, _P, _P, _P, _SZ, _P], _I32),
    "cross_bwd": ([_I64, _I64, _I32, _I32, _I32, _HP, _HP, _HP, _HP, _P, _P, _P, _CP, _P, _P, _P, _P, _SZ, _P], _I32),
    "addnorm_workspace_size": ([_I64, _I64, _SZP], _I32),
    "addnorm_fwd": ([_I64, _I64, _P, _P, _NP, _P, _P, _P, _P, _P], _I32),
    "addnorm_bwd": ([_I64, _I64, _P, _P, _P, _P, _P, _P, _NP, _P, _P, _P, _P, _P, _P, _SZ, _P], _I32),
    "logprob_fwd": ([_I64, _I64, _I64, _P, _I32, _P, _I32, _F, _I32, _P, _P, _P, _P, _P, _P], _I32),
    "logprob_bwd": ([_I64, _I64, _I64, _P, _I32, _P, _I32, _F, _P, _P, _P, _P, _P, _I64, _P], _I32),
    "qkrope_workspace_size": ([_I64, _I32, _I32, _I32, _SZP], _I32),
    "qkrope_fwd": ([_I64, _I32, _I32, _I32, _HP, _HP, _RP, _HP, _HP, _P], _I32),
    "qkrope_bwd": ([_I64, _I32, _I32, _I32, _HP, _HP, _HP, _HP, _RP, _HP, _HP, _P, _P, _P, _SZ, _P], _I32),
    "distill_fwd": ([_I64, _I64, _I64, _P, _I32, _TP, _P, _I32, _F, _P, _P, _P, _P, _P], _I32),
    "distill_bwd": ([_I64, _I64, _I64, _P, _I32, _TP, _P, _I32, _F, _P, _P, _P, _P, _I64, _P], _I32),
}

_fns = {}


def header_symbols() -> list:
    """Names of the entry points declared in include/lora_layer.h."""
    with open(HEADER) as f:
        return re.findall(r"LM_API\s+[\w\s\*]+?\b(\w+)\s*\(", f.read())


def _fn(name: str):
    fn = _fns.get(name)
    if fn is None:
        fn = getattr(L.load(), name)
        fn.argtypes, fn.restype = _SIGS[name]
        _fns[name] = fn
    return fn


def call_status(name: str, *args) -> int:
    """Call an entry point and return its raw status (for tests of the error paths)."""
    return _fn(name)(*args)


def _call(name: str, *args) -> None:
    st = _fn(name)(*args)
    if st != L.LM_OK:
        raise LmError(st, name, L.last_error())


def _size(name: str, *args) -> int:
    out = ctypes.c_size_t(0)
    _call(name, *args, ctypes.byref(out))
    return out.value


def _refuse(t, shape, dtype, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be contiguous" % name)


def _shaped(t: Optional[torch.Tensor], shape, dtype, name: str) -> int:
    """Device address of a contiguous tensor of this shape and type (None: a null pointer)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _refuse(t, shape, dtype, name)
    return t.data_ptr() or L._empty_ptr(t.device)


_raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream() -> int:
    """The current raw stream, without building a Stream object (3 us of a call's 20)."""
    return _raw_stream(_device())


def _on(stream):
    """The stream made the current one, so that what a call allocates and zeroes is ordered before its kernels."""
    if not isinstance(stream, torch.cuda.Stream):
        raw = L._stream(stream)
        stream = torch.cuda.ExternalStream(raw) if raw else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _new(shape, dtype, dev):
    """A contiguous tensor of the call's own and its address (no checks: a small call takes as long as its checks; with
    its strides given, torch makes one in 60 % of the time)."""
    n = len(shape)
    strides = (1,) if n == 1 else (shape[1], 1) if n == 2 else (shape[1] * shape[2], shape[2], 1)
    t = torch.empty_strided(shape, strides, dtype=dtype, device=dev)
    return t, t.data_ptr() or L._empty_ptr(dev)


def _out(t, shape, dtype, dev, name):
    """The caller's tensor, or a new one, and its address."""
    return _new(shape, dtype, dev) if t is None else (t, _shaped(t, shape, dtype, name))


# ---------------------------------------------------------------------------------------------
# attention


@dataclass
class Attn:
    """What one attention call computes (lm_attn): scores scale * q.k, capped by cap * tanh(. / cap)
    when cap > 0 (2^-14 to 2^12), less slopes[head] * |i - j| when slopes is given; token i sees the tokens j <= i of
    its document (all of it when not causal, and always the document's first prefix tokens) nearer
    than window (0: no limit).  cu_docs: int32 document offsets (n + 1; None: one document), prefix:
    int32 (n), slopes: float32 (query heads)."""
    scale: float
    cap: float = 0.0
    causal: bool = True
    window: int = 0
    cu_docs: Optional[torch.Tensor] = None
    prefix: Optional[torch.Tensor] = None
    slopes: Optional[torch.Tensor] = None

    def c_struct(self, hq: int) -> lm_attn:
        n = 0 if self.cu_docs is None else self.cu_docs.numel() - 1
        return lm_attn(self.scale, self.cap, _shaped(self.slopes, (hq,), torch.float32, "slopes"), bool(self.causal),
                       self.window, _shaped(self.cu_docs, (n + 1,), torch.int32, "cu_docs"),
                       _shaped(self.prefix, (n,), torch.int32, "prefix"), n, 0)


def _heads(t: torch.Tensor, T: int, h: int, d: int, name: str) -> lm_heads:
    """A (T, heads, d) bf16 tensor whose tokens and heads may be strided."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != torch.bfloat16:
        raise TypeError("%s must be %s, got %s" % (name, torch.bfloat16, t.dtype))
    if t.shape != (T, h, d):
        raise ValueError("%s must have shape %s, got %s" % (name, (T, h, d), tuple(t.shape)))
    ts, hs, one = t.stride()
    if one != 1 and d > 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    if h == 1:  # the stride of a dimension of size one is not used, and torch may report any value
        hs = d
    if T <= 1:
        ts = h * max(hs, d)
    return lm_heads(t.data_ptr() if T else L._empty_ptr(t.device), ts, hs)


def _d16(d: int) -> int:
    return (d + 15) // 16 * 16


def attn_workspace_size(T: int, hq: int, hk: int, d: int) -> int:
    return _size("attn_workspace_size", T, hq, hk, d)


def attn_fwd(q, k, v, a: Attn, train: bool = True, O=None, lse=None, O_lo=None, ws=None, stream=None) -> dict:
    """q (T, hq, d), k and v (T, hk, d) -> O (T, hq, d), lse (hq, T) and, with ``train``, O_lo (int8: more
    bits of O, for the backward)."""
    if stream is not None:
        with _on(stream):
            return attn_fwd(q, k, v, a, train, O, lse, O_lo, ws)
    (T, hq, d), hk = q.shape, k.shape[1]
    dev = q.device
    hs = _heads(q, T, hq, d, "q"), _heads(k, T, hk, d, "k"), _heads(v, T, hk, d, "v")
    O, pO = _out(O, (T, hq, d), torch.bfloat16, dev, "O")
    lse, pl = _out(lse, (hq, T), torch.float32, dev, "lse")
    plo = 0
    if train or O_lo is not None:
        O_lo, plo = _out(O_lo, (T, hq, _d16(d)), torch.int8, dev, "O_lo")
    ws = workspace(attn_workspace_size(T, hq, hk, d), dev) if ws is None else ws
    _call("attn_fwd", T, hq, hk, d, *hs, a.c_struct(hq), pO, plo, pl, L._ptr(ws, torch.uint8, "ws"), ws.numel(), _stream())
    return {"O": O, "lse": lse, "O_lo": O_lo, "ws": ws}


def attn_bwd(q, k, v, dO, fwd: dict, a: Attn, dQ=None, dK=None, dV=None, ws=None, stream=None) -> dict:
    """The gradients of q, k and v from dO (T, hq, d) and the forward's result."""
    if stream is not None:
        with _on(stream):
            return attn_bwd(q, k, v, dO, fwd, a, dQ, dK, dV, ws)
    (T, hq, d), hk = q.shape, k.shape[1]
    dev, bf = q.device, torch.bfloat16
    hs = _heads(q, T, hq, d, "q"), _heads(k, T, hk, d, "k"), _heads(v, T, hk, d, "v"), _heads(dO, T, hq, d, "dO")
    dQ, pq = _out(dQ, (T, hq, d), bf, dev, "dQ")
    dK, pk = _out(dK, (T, hk, d), bf, dev, "dK")
    dV, pv = _out(dV, (T, hk, d), bf, dev, "dV")
    ws = fwd["ws"] if ws is None else ws
    _call("attn_bwd", T, hq, hk, d, *hs, _shaped(fwd["O"], (T, hq, d), bf, "O"),
          _shaped(fwd["O_lo"], (T, hq, _d16(d)), torch.int8, "O_lo"), _shaped(fwd["lse"], (hq, T), torch.float32, "lse"),
          a.c_struct(hq), pq, pk, pv, L._ptr(ws, torch.uint8, "ws"), ws.numel(), _stream())
    return {"dQ": dQ, "dK": dK, "dV": dV}


# ---------------------------------------------------------------------------------------------
# residual add and norms


@dataclass
class AddNorm:
    """h_out = h + alpha * gate * N(y; w_post), x = N(h_out; w_in), N the root-mean-square norm with
    weight w + w_offset.  Each vector (d values, all bf16 or all float32) may be None: no norm after
    the block, no gate, no norm before the next block."""
    w_in: Optional[torch.Tensor] = None
    w_post: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    alpha: float = 1.0
    eps: float = 1e-5
    w_offset: float = 0.0

    def c_struct(self, d: int, h_dtype) -> lm_addnorm:
        w = self.w_in if self.w_in is not None else self.w_post if self.w_post is not None else self.gate
        wt = torch.bfloat16 if w is None else w.dtype
        hc, wc = _DTYPES.get(h_dtype), _DTYPES.get(wt)
        if hc is None or wc is None:
            raise TypeError("h and the norm's vectors must be bfloat16 or float32, got %s and %s" % (h_dtype, wt))
        shape = (d,)
        return lm_addnorm(_shaped(self.w_in, shape, wt, "w_in"), _shaped(self.w_post, shape, wt, "w_post"),
                          _shaped(self.gate, shape, wt, "gate"), self.alpha, self.eps, self.w_offset, hc, wc, 0)


def addnorm_workspace_size(T: int, d: int) -> int:
    return _size("addnorm_workspace_size", T, d)


def addnorm_fwd(h, y, n: AddNorm, h_out=None, x=None, stream=None) -> dict:
    """h (T, d) bf16 or float32, y (T, d) bf16 or None -> h (the sum; h itself without y), x (None
    without w_in), rstd_y, rstd_h."""
    if stream is not None:
        with _on(stream):
            return addnorm_fwd(h, y, n, h_out, x)
    T, d = h.shape
    dev, ht, f32, bf = h.device, h.dtype, torch.float32, torch.bfloat16
    td = (T, d)
    ph, py, c = _shaped(h, td, ht, "h"), _shaped(y, td, bf, "y"), n.c_struct(d, ht)
    rstd_y = rstd_h = None
    po = px = pry = prh = 0
    if y is not None or h_out is not None:
        h_out, po = _out(h_out, td, ht, dev, "h_out")
    if n.w_in is not None:
        rstd_h, prh = _new((T,), f32, dev)
    if n.w_in is not None or x is not None:
        x, px = _out(x, td, bf, dev, "x")
    if n.w_post is not None:
        rstd_y, pry = _new((T,), f32, dev)
    _call("addnorm_fwd", T, d, ph, py, c, po, px, pry, prh, _stream())
    # (a buffer given for a result that is not there is checked, not written and not returned)
    return {"h": h if y is None else h_out, "x": x if n.w_in is not None else None, "rstd_y": rstd_y, "rstd_h": rstd_h}


def addnorm_bwd(h, y, dh_out, dx, fwd: dict, n: AddNorm, weights: bool = True, dh=None, dy=None, ws=None,
                stream=None) -> dict:
    """Gradients from those of the sum (dh_out, None: zero) and of x (dx), with the forward's inputs h and
    y: dh, dy, and with ``weights`` the float32 gradients of the vectors that are there."""
    if stream is not None:
        with _on(stream):
            return addnorm_bwd(h, y, dh_out, dx, fwd, n, weights, dh, dy, ws)
    T, d = h.shape
    dev, ht, f32, bf = h.device, h.dtype, torch.float32, torch.bfloat16
    td = (T, d)
    ins = (_shaped(h, td, ht, "h"), _shaped(y, td, bf, "y"), _shaped(dh_out, td, ht, "dh_out"), _shaped(dx, td, bf, "dx"),
           _shaped(fwd["rstd_y"], (T,), f32, "rstd_y"), _shaped(fwd["rstd_h"], (T,), f32, "rstd_h"), n.c_struct(d, ht))
    dh, ph = _out(dh, td, ht, dev, "dh")
    py = 0
    if y is not None or dy is not None:
        dy, py = _out(dy, td, bf, dev, "dy")

    def grad(w):
        return _new((d,), f32, dev) if weights and w is not None else (None, 0)

    (dw_in, pi), (dw_post, pp), (dgate, pg) = grad(n.w_in), grad(n.w_post), grad(n.gate)
    ws = workspace(addnorm_workspace_size(T, d), dev) if ws is None else ws
    _call("addnorm_bwd", T, d, *ins, ph, py, pi, pp, pg, L._ptr(ws, torch.uint8, "ws"), ws.numel(), _stream())
    return {"dh": dh, "dy": dy if y is not None else None, "dw_in": dw_in, "dw_post": dw_post, "dgate": dgate, "ws": ws}


# ---------------------------------------------------------------------------------------------
# log probabilities


def _rows2d(t: torch.Tensor, name: str):
    """(address, row stride, type) of a (T, V) tensor with contiguous rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TypeError("%s must be a 2D torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in _DTYPES:
        raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))
    T, V = t.shape
    if V > 1 and t.stride(1) != 1:
        raise ValueError("%s must have contiguous rows" % name)
    return t.data_ptr() if t.numel() else L._empty_ptr(t.device), t.stride(0) if T > 1 else V, _DTYPES[t.dtype]


def _targets(t: torch.Tensor, T: int):
    if not isinstance(t, torch.Tensor) or t.dtype not in _INDEX:
        raise TypeError("targets must be an int32 or int64 tensor")
    return _shaped(t, (T,), t.dtype, "targets"), _INDEX[t.dtype]


def logprob_fwd(logits, targets, k: int = 0, scale: float = 1.0, stream=None) -> dict:
    """logits (T, V) bf16 or float32 (rows may be strided), targets (T) -> logp, entropy, lse (T) float32 and,
    for k > 0, top_ids (T, k) int32 and top_logp (T, k) float32."""
    if stream is not None:
        with _on(stream):
            return logprob_fwd(logits, targets, k, scale)
    p, ld, dt = _rows2d(logits, "logits")
    T, V = logits.shape
    tp, ti = _targets(targets, T)
    dev, f32 = logits.device, torch.float32
    logp, pl = _new((T,), f32, dev)
    entropy, pe = _new((T,), f32, dev)
    lse, ps = _new((T,), f32, dev)
    ids = top = None
    pi = pt = 0
    if k > 0:
        ids, pi = _new((T, k), torch.int32, dev)
        top, pt = _new((T, k), f32, dev)
    _call("logprob_fwd", T, V, ld, p, dt, tp, ti, scale, k, pl, pe, ps, pi, pt, _stream())
    return {"logp": logp, "entropy": entropy, "lse": lse, "top_ids": ids, "top_logp": top}


def logprob_bwd(logits, targets, fwd: dict, dlogp=None, dentropy=None, scale: float = 1.0, dlogits=None,
                stream=None) -> dict:
    """dlogits (T, V), in the logits' type, from the gradients of logp and entropy (T float32; None: zero).
    ``dlogits`` may be ``logits`` itself; for logits whose rows have gaps that is where it is written fastest, or in a
    buffer with the same gaps (without them about seven times slower)."""
    if stream is not None:
        with _on(stream):
            return logprob_bwd(logits, targets, fwd, dlogp, dentropy, scale, dlogits)
    p, ld, dt = _rows2d(logits, "logits")
    T, V = logits.shape
    tp, ti = _targets(targets, T)
    f32 = torch.float32
    if dlogits is None:
        dlogits = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
    po, ldo, dto = _rows2d(dlogits, "dlogits")
    if dlogits.shape != (T, V) or dto != dt:
        raise ValueError("dlogits must have the logits' shape and type")
    _call("logprob_bwd", T, V, ld, p, dt, tp, ti, scale, _shaped(fwd["lse"], (T,), f32, "lse"),
          _shaped(fwd["entropy"], (T,), f32, "entropy"), _shaped(dlogp, (T,), f32, "dlogp"),
          _shaped(dentropy, (T,), f32, "dentropy"), po, ldo, _stream())
    return {"dlogits": dlogits}


# ---------------------------------------------------------------------------------------------
# norms of query and key heads, rotation by position


def _here(*tensors) -> None:
    """Every tensor on the current device, whose stream a call is made on."""
    at = _device()
    for t in tensors:
        if t is not None and t.get_device() != at:
            raise ValueError("a call's tensors must lie on the current device (cuda:%d), got one on %s" % (at, t.device))


# The usual tensor of a call in as few questions as say that it is one (get_device is -1 on the host); others take the
# long way, which says what is wrong with them.
def _flat(t, shape, dtype, dev: int, name: str) -> int:
    """Device address of a contiguous tensor on the current device (None: a null pointer)."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor):
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr() or L._empty_ptr(t.device)
        _here(t)
    return _shaped(t, shape, dtype, name)


def _heads_at(t, T: int, h: int, d: int, dev: int, name: str) -> lm_heads:
    if isinstance(t, torch.Tensor):
        if T > 1 and h > 1 and t.dtype is torch.bfloat16 and t.get_device() == dev and t.shape == (T, h, d):
            ts, hs, one = t.stride()
            if one == 1:
                return lm_heads(t.data_ptr(), ts, hs)
        _here(t)
    return _heads(t, T, h, d, name)


@dataclass
class QkRope:
    """Norm of each query and key head (``norm``; root mean square, weights w_q and w_k + w_offset of d values, all
    bf16 or all float32, None: 1), then the rotation of its first 2 len(inv_freq) dims by position (inv_freq
    None: no rotation): pair p turns by pos[axis[p]][token] * inv_freq[p], and the rotated dims are multiplied
    by ``factor``.  Pairs are dims (p, p + len) or, ``interleaved``, (2p, 2p + 1).  inv_freq: float32; pos: int32 or
    int64, (T), or (axes, T) with axis (int32, an axis for each pair; numbers outside are clamped); None: the
    token's index.  eps: at least 2^-126."""
    inv_freq: Optional[torch.Tensor] = None
    pos: Optional[torch.Tensor] = None
    axis: Optional[torch.Tensor] = None
    interleaved: bool = False
    factor: float = 1.0
    norm: bool = False
    w_q: Optional[torch.Tensor] = None
    w_k: Optional[torch.Tensor] = None
    eps: float = 1e-6
    w_offset: float = 0.0

    def c_struct(self, T: int, d: int) -> lm_qkrope:
        f, pos, axis, wq, wk = self.inv_freq, self.pos, self.axis, self.w_q, self.w_k
        half, pairs, pp, axes, pi = (), 0, 0, 1, LM_I32
        if f is not None:
            pairs = f.numel()
            half = (pairs,)
        elif pos is not None or axis is not None:
            raise ValueError("pos and axis need inv_freq")
        dev = _device()
        if pos is not None:
            dt, shape = pos.dtype, (T,)
            if dt not in _INDEX:
                raise TypeError("pos must be int32 or int64, got %s" % dt)
            pi = _INDEX[dt]
            if pos.dim() == 2:
                axes = pos.shape[0]
                shape = (axes, T)
            pp = _flat(pos, shape, dt, dev, "pos")
        wt = wq.dtype if wq is not None else wk.dtype if wk is not None else torch.bfloat16
        wc = _DTYPES.get(wt)
        if wc is None:
            raise TypeError("w_q and w_k must be bfloat16 or float32, got %s" % wt)
        one = (d,)
        return lm_qkrope(_flat(f, half, torch.float32, dev, "inv_freq"), pp, _flat(axis, half, torch.int32, dev, "axis"),
                         _flat(wq, one, wt, dev, "w_q"), _flat(wk, one, wt, dev, "w_k"), self.factor, self.eps, self.w_offset,
                         2 * pairs, axes, bool(self.interleaved), bool(self.norm), pi, wc, 0)


def _heads_out(t, T, h, d, dev, at: int, name):
    """The caller's strided tensor, or a new contiguous one."""
    if t is None:
        t, p = _new((T, h, d), torch.bfloat16, dev)
        return t, lm_heads(p, h * d, d)
    return t, _heads_at(t, T, h, d, at, name)


def qkrope_workspace_size(T: int, hq: int, hk: int, d: int) -> int:
    return _size("qkrope_workspace_size", T, hq, hk, d)


def qkrope_fwd(q, k, r: QkRope, q_out=None, k_out=None, stream=None) -> dict:
    """q (T, hq, d) and k (T, hk, d; or None) bf16, strided like attn_fwd's -> q and k, normed and rotated.  q_out and
    k_out may be q and k themselves, or other slices of one buffer."""
    if stream is not None:
        with _on(stream):
            return qkrope_fwd(q, k, r, q_out, k_out)
    (T, hq, d), dev, at = q.shape, q.device, _device()
    hk = 0 if k is None else k.shape[1]
    sq, c = _heads_at(q, T, hq, d, at, "q"), r.c_struct(T, d)
    q_out, oq = _heads_out(q_out, T, hq, d, dev, at, "q_out")
    sk = ok = None
    if hk:
        sk = _heads_at(k, T, hk, d, at, "k")
        k_out, ok = _heads_out(k_out, T, hk, d, dev, at, "k_out")
    _call("qkrope_fwd", T, hq, hk, d, sq, sk, c, oq, ok, _raw_stream(at))
    return {"q": q_out, "k": k_out if hk else None}


def qkrope_bwd(q, k, dq, dk, r: QkRope, weights: bool = True, dq_in=None, dk_in=None, ws=None, stream=None) -> dict:
    """The gradients of the forward's inputs q and k from those of its results, and with ``weights`` the float32
    gradients dw_q and dw_k of the weights that are there.  Without a norm q and k are not read and may be None.
    dq_in may be dq, dk_in may be dk."""
    if stream is not None:
        with _on(stream):
            return qkrope_bwd(q, k, dq, dk, r, weights, dq_in, dk_in, ws)
    (T, hq, d), dev, at = dq.shape, dq.device, _device()
    hk = 0 if dk is None else dk.shape[1]
    gq, c = _heads_at(dq, T, hq, d, at, "dq"), r.c_struct(T, d)
    dq_in, oq = _heads_out(dq_in, T, hq, d, dev, at, "dq_in")
    sq = sk = gk = ok = dw_q = dw_k = None
    pq = pk = pw = n = 0
    if hk:
        gk = _heads_at(dk, T, hk, d, at, "dk")
        dk_in, ok = _heads_out(dk_in, T, hk, d, dev, at, "dk_in")
    if r.norm:
        sq, sk = _heads_at(q, T, hq, d, at, "q"), _heads_at(k, T, hk, d, at, "k") if hk else None
        if weights and r.w_q is not None:
            dw_q, pq = _new((d,), torch.float32, dev)
        if weights and r.w_k is not None:
            dw_k, pk = _new((d,), torch.float32, dev)
        if ws is None:
            ws = torch.empty(qkrope_workspace_size(T, hq, hk, d), dtype=torch.uint8, device=dev)
        n = ws.numel()
        pw = _flat(ws, (n,), torch.uint8, at, "ws")
    _call("qkrope_bwd", T, hq, hk, d, sq, sk, gq, gk, c, oq, ok, pq, pk, pw, n, _raw_stream(at))
    return {"dq": dq_in, "dk": dk_in if hk else None, "dw_q": dw_q, "dw_k": dw_k, "ws": ws}


# ---------------------------------------------------------------------------------------------
# distillation from a teacher's top logits


@dataclass
class Teacher:
    """What a teacher says of each row: ``ids`` (T, K; int32 or int64, outside [0, V): no entry) and ``values``
    (T, K; bfloat16 or float32), K at most 128.  ``rest`` False: logits, a softmax of scale * values over the
    row's entries is the teacher; True: log probabilities, and what they leave is one more outcome."""
    ids: torch.Tensor
    values: torch.Tensor
    rest: bool = False

    def c_struct(self, T: int) -> lm_teacher:
        ids, values = self.ids, self.values
        if not isinstance(ids, torch.Tensor) or ids.dtype not in _INDEX or ids.dim() != 2:
            raise TypeError("ids must be a 2D int32 or int64 tensor")
        if not isinstance(values, torch.Tensor) or values.dtype not in _DTYPES:
            raise TypeError("values must be a bfloat16 or float32 tensor")
        it, vt, K, dev = ids.dtype, values.dtype, ids.shape[1], _device()
        return lm_teacher(_flat(ids, (T, K), it, dev, "ids"), _flat(values, (T, K), vt, dev, "values"), K, _INDEX[it], _DTYPES[vt],
                          bool(self.rest))


def _alike(t):
    """A new tensor whose rows lie as t's do, modulo 16 bytes (t: 2D with contiguous rows)."""
    T, V = t.shape
    ld, es = t.stride(0) if T > 1 else V, t.element_size()
    off = t.data_ptr() % 16 // es
    if ld > 2 * V + 16 // es:  # (not the gaps of a much wider buffer: the nearest stride that lies alike)
        ld = V + (ld - V) % (16 // es)
    buf = torch.empty(off + T * ld, dtype=t.dtype, device=t.device)
    return buf.as_strided((T, V), (ld, 1), off)


def distill_fwd(logits, teacher: Teacher, targets=None, scale: float = 1.0, stream=None) -> dict:
    """logits (T, V) bf16 or float32 (rows may be strided) -> kl (T), the divergence from the teacher at scale * logits,
    lse (T) and, with targets (T; int32 or int64), logp (T), their log probabilities at scale 1, all float32;
    ``saved`` is for the backward."""
    if stream is not None:
        with _on(stream):
            return distill_fwd(logits, teacher, targets, scale)
    p, ld, dt = _rows2d(logits, "logits")
    T, V = logits.shape
    _here(logits, targets)
    tp, ti = (0, LM_I32) if targets is None else _targets(targets, T)
    dev, f32 = logits.device, torch.float32
    kl, pk = _new((T,), f32, dev)
    lse, pl = _new((T,), f32, dev)
    saved, ps = _new((T, 8), f32, dev)
    logp, pp = (None, 0) if targets is None else _new((T,), f32, dev)
    _call("distill_fwd", T, V, ld, p, dt, teacher.c_struct(T), tp, ti, scale, pk, pp, pl, ps, _stream())
    return {"kl": kl, "logp": logp, "lse": lse, "saved": saved}


def distill_bwd(logits, teacher: Teacher, fwd: dict, dkl=None, targets=None, dlogp=None, scale: float = 1.0, dlogits=None,
                stream=None) -> dict:
    """dlogits (T, V), in the logits' type, from the gradients of kl and logp (T float32; None: zero), with the
    forward's arguments.  ``dlogits`` may be ``logits`` itself; a new one has rows that lie as the logits' do."""
    if stream is not None:
        with _on(stream):
            return distill_bwd(logits, teacher, fwd, dkl, targets, dlogp, scale, dlogits)
    if dlogp is not None and fwd["logp"] is None:
        raise ValueError("dlogp needs a forward with targets")
    p, ld, dt = _rows2d(logits, "logits")
    T, V = logits.shape
    _here(logits, targets, dlogits)
    tp, ti = (0, LM_I32) if targets is None else _targets(targets, T)
    f32, at, t1 = torch.float32, _device(), (T,)
    if dlogits is None:
        dlogits = _alike(logits)
    po, ldo, dto = _rows2d(dlogits, "dlogits")
    if dlogits.shape != (T, V) or dto != dt:
        raise ValueError("dlogits must have the logits' shape and type")
    _call("distill_bwd", T, V, ld, p, dt, teacher.c_struct(T), tp, ti, scale, _flat(fwd["saved"], (T, 8), f32, at, "saved"),
          _flat(dkl, t1, f32, at, "dkl"), _flat(dlogp, t1, f32, at, "dlogp"), po, ldo, _raw_stream(at))
    return {"dlogits": dlogits}


# ---------------------------------------------------------------------------------------------
# attention to the states of another length


@dataclass
class Cross:
    """What one cross-attention call computes (lm_cross): scores scale * q.k, capped by cap * tanh(. / cap) when cap > 0.
    Without cu_q every query sees every key; with it document m's queries [cu_q[m], cu_q[m + 1]) see the first
    k_len[m] (None: all) of its keys [cu_k[m], cu_k[m + 1]) (int32: n + 1 offsets each, n lengths)."""
    scale: float
    cap: float = 0.0
    cu_q: Optional[torch.Tensor] = None
    cu_k: Optional[torch.Tensor] = None
    k_len: Optional[torch.Tensor] = None

    def c_struct(self) -> lm_cross:
        if self.cu_q is None and self.cu_k is None and self.k_len is None:
            return lm_cross(self.scale, self.cap, 0, 0, 0, 0, 0)
        if self.cu_q is None or self.cu_k is None:
            raise ValueError("cu_q and cu_k belong together, and k_len to them")
        _here(self.cu_q, self.cu_k, self.k_len)
        n = self.cu_q.numel() - 1
        return lm_cross(self.scale, self.cap, _shaped(self.cu_q, (n + 1,), torch.int32, "cu_q"),
                        _shaped(self.cu_k, (n + 1,), torch.int32, "cu_k"), _shaped(self.k_len, (n,), torch.int32, "k_len"), n, 0)


def cross_workspace_size(Tq: int, Tk: int, hq: int, hk: int, d: int) -> int:
    return _size("cross_workspace_size", Tq, Tk, hq, hk, d)


def cross_fwd(q, k, v, a: Cross, train: bool = True, O=None, lse=None, O_lo=None, ws=None, stream=None) -> dict:
    """q (Tq, hq, d), k and v (Tk, hk, d) -> O (Tq, hq, d), lse (hq, Tq) and, with ``train``, O_lo (as attn_fwd's)."""
    if stream is not None:
        with _on(stream):
            return cross_fwd(q, k, v, a, train, O, lse, O_lo, ws)
    (Tq, hq, d), (Tk, hk, _) = q.shape, k.shape
    dev, at = q.device, _device()
    hs = _heads_at(q, Tq, hq, d, at, "q"), _heads_at(k, Tk, hk, d, at, "k"), _heads_at(v, Tk, hk, d, at, "v")
    O, pO = _new((Tq, hq, d), torch.bfloat16, dev) if O is None else (O, _flat(O, (Tq, hq, d), torch.bfloat16, at, "O"))
    lse, pl = _new((hq, Tq), torch.float32, dev) if lse is None else (lse, _flat(lse, (hq, Tq), torch.float32, at, "lse"))
    plo = 0
    if train or O_lo is not None:
        shape = (Tq, hq, _d16(d))
        O_lo, plo = _new(shape, torch.int8, dev) if O_lo is None else (O_lo, _flat(O_lo, shape, torch.int8, at, "O_lo"))
    if ws is None:
        ws = torch.empty(cross_workspace_size(Tq, Tk, hq, hk, d), dtype=torch.uint8, device=dev)
        ws[:256].zero_()  # (the error word; the parts' sums may be megabytes)
    n = ws.numel()
    _call("cross_fwd", Tq, Tk, hq, hk, d, *hs, a.c_struct(), pO, plo, pl, _flat(ws, (n,), torch.uint8, at, "ws"), n,
          _raw_stream(at))
    return {"O": O, "lse": lse, "O_lo": O_lo, "ws": ws}


def cross_bwd(q, k, v, dO, fwd: dict, a: Cross, dQ=None, dK=None, dV=None, ws=None, stream=None) -> dict:
    """The gradients of q, k and v from dO (Tq, hq, d) and the forward's result."""
    if stream is not None:
        with _on(stream):
            return cross_bwd(q, k, v, dO, fwd, a, dQ, dK, dV, ws)
    (Tq, hq, d), (Tk, hk, _) = q.shape, k.shape
    dev, at, bf = q.device, _device(), torch.bfloat16
    sq, sk = (Tq, hq, d), (Tk, hk, d)
    ws = fwd["ws"] if ws is None else ws
    hs = (_heads_at(q, Tq, hq, d, at, "q"), _heads_at(k, Tk, hk, d, at, "k"), _heads_at(v, Tk, hk, d, at, "v"),
          _heads_at(dO, Tq, hq, d, at, "dO"))
    dQ, pq = _new(sq, bf, dev) if dQ is None else (dQ, _flat(dQ, sq, bf, at, "dQ"))
    dK, pk = _new(sk, bf, dev) if dK is None else (dK, _flat(dK, sk, bf, at, "dK"))
    dV, pv = _new(sk, bf, dev) if dV is None else (dV, _flat(dV, sk, bf, at, "dV"))
    n = ws.numel()
    _call("cross_bwd", Tq, Tk, hq, hk, d, *hs, _flat(fwd["O"], sq, bf, at, "O"),
          _flat(fwd["O_lo"], (Tq, hq, _d16(d)), torch.int8, at, "O_lo"), _flat(fwd["lse"], (hq, Tq), torch.float32, at, "lse"),
          a.c_struct(), pq, pk, pv, _flat(ws, (n,), torch.uint8, at, "ws"), n, _raw_stream(at))
    return {"dQ": dQ, "dK": dK, "dV": dV}
