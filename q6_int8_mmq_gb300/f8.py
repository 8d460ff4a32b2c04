"""The 8-bit steps around the projections: the norm with the residual's addition
and the gated activation that end in quantised activations, and products of
e4m3 blocks (8-bit floating point, a scale for each 128).

Argument marshalling over the C ABI, as in the package's other calls. Sums are
f32; nothing is kept between calls.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import NamedTuple

from . import (PATH_NAMES, Q6_EINVAL, Activations, Q6Error, _c_ints, _check, _same_device,
               act_plane_bytes, alloc_activations, load)
from .moe import _empty, _made, _on, _rows, _rows2d, _stream, _type, _types, _whole


@functools.lru_cache(maxsize=None)
def _f8():
    import torch
    return torch.float8_e4m3fn


@functools.lru_cache(maxsize=256)
def f8_act_bytes(N: int, K: int):
    """(xq_bytes, sx_bytes, ldsx) of N x K e4m3 activations."""
    _c_ints(N=N, K=K)
    a, b, ld = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int()
    _check(load().q6_f8_act_bytes(N, K, ctypes.byref(a), ctypes.byref(b), ctypes.byref(ld)))
    return a.value, b.value, ld.value


@functools.lru_cache(maxsize=256)
def f8_weight_bytes(M: int, K: int):
    """(wq_bytes, sw_bytes) of an M x K e4m3 weight."""
    _c_ints(M=M, K=K)
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().q6_f8_weight_bytes(M, K, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def _blocks(n):
    return -(-n // 128)


@dataclasses.dataclass(frozen=True)
class F8Activations:
    """e4m3 activations on the device: xq [N, K] float8_e4m3fn, sx [ceil(K / 128), ldsx] f32, the
    scale of each token's 128 values (ldsx: N rounded up to 4; the columns past N are not
    looked at). Checked once, when made; read-only."""
    N: int
    K: int
    xq: object
    sx: object

    def __post_init__(self):
        import torch
        _same_device((self.xq, "xq", _f8(), (self.N, self.K)),
                     (self.sx, "sx", torch.float32,
                      (_blocks(self.K), f8_act_bytes(self.N, self.K)[2])))

    @property
    def device(self):
        return self.sx.device


@dataclasses.dataclass(frozen=True)
class F8Weights:
    """An e4m3 weight on the device, as checkpoints hold it: wq [M, K] float8_e4m3fn, sw
    [ceil(M / 128), ceil(K / 128)] f32, the scale of each block of 128 x 128. Checked once, when
    made; read-only."""
    M: int
    K: int
    wq: object
    sw: object

    def __post_init__(self):
        import torch
        f8_weight_bytes(self.M, self.K)      # the sizes the kernels take
        _same_device((self.wq, "wq", _f8(), (self.M, self.K)),
                     (self.sw, "sw", torch.float32, (_blocks(self.M), _blocks(self.K))))

    @property
    def device(self):
        return self.wq.device


def _cuda(device):
    import torch
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        raise Q6Error(Q6_EINVAL, f"buffers have to be on a CUDA device, not {dev}")
    return dev


def alloc_f8_activations(N: int, K: int, device=None) -> F8Activations:
    """Buffers for N x K e4m3 activations (K a multiple of 16)."""
    import torch
    dev, ldsx = _cuda(device), f8_act_bytes(N, K)[2]
    return _made(F8Activations, N=N, K=K, xq=torch.empty((N, K), dtype=_f8(), device=dev),
                 sx=torch.empty((_blocks(K), ldsx), dtype=torch.float32, device=dev))


def alloc_f8_weights(M: int, K: int, device=None) -> F8Weights:
    """Buffers for an M x K e4m3 weight (K a multiple of 16)."""
    import torch
    dev = _cuda(device)
    f8_weight_bytes(M, K)
    return _made(F8Weights, M=M, K=K, wq=torch.empty((M, K), dtype=_f8(), device=dev),
                 sw=torch.empty((_blocks(M), _blocks(K)), dtype=torch.float32, device=dev))


def _input(X, name):
    """(type code, shape, device, row stride) of a 2-D view of rows."""
    try:
        code, shape, dev = _types().get(X.dtype), X.shape, X.device
        if code is not None and len(shape) == 2 and X.is_contiguous() and dev.type == "cuda":
            return code, shape, dev, shape[1] or 1
    except AttributeError:
        pass
    code = _type(X, name)
    _rows2d(X, name)
    return code, X.shape, X.device, _rows(X, name, X.dtype, X.shape, X.device)


def _fits(out, cls, N, K, dev):
    """Whether the rows a call writes go to `out`; raises if they do not fit."""
    if out.__class__ is cls and out.N == N and out.K == K and out.device == dev:
        return
    if not isinstance(out, cls):
        raise Q6Error(Q6_EINVAL, f"out must be {cls.__name__}, not {type(out).__name__}")
    if out.N != N or out.K != K or out.device != dev:
        raise Q6Error(Q6_EINVAL, f"out holds {out.N} x {out.K} activations on {out.device}, not "
                                 f"{N} x {K} on {dev}")


def _q8_out(out, N, K, dev, want_xh, want_xq, want_us, stream):
    """int8 activations of N x K: `out`, which has to fit, or new ones."""
    if out is not None:
        _fits(out, Activations, N, K, dev)
        return out
    act_plane_bytes(N, K)
    if not (want_xh or want_xq):
        raise Q6Error(Q6_EINVAL, "one of want_xh and want_xq is needed")
    with _on(stream):
        return alloc_activations(N, K, dev, want_xh, want_xq, want_us)


def _q8_pointers(act):
    xq, xh, us = act.xq, act.xh, act.us
    return (None if xq is None else xq.data_ptr(), act.da.data_ptr(),
            None if xh is None else xh.data_ptr(), None if us is None else us.data_ptr())


def _f8_out(out, N, K, dev, stream):
    if out is not None:
        _fits(out, F8Activations, N, K, dev)
        return out
    with _on(stream):
        return alloc_f8_activations(N, K, dev)


def f8_quantize_act(X, out: F8Activations | None = None, stream=None) -> F8Activations:
    """Quantises activations X [N, K] (f32, bf16 or f16 rows, 16-byte aligned; K a multiple of
    16) to e4m3 with a scale for each 128 of a row: largest magnitude / 448."""
    code, (N, K), dev, ldx = _input(X, "X")
    out = _f8_out(out, N, K, dev, stream)
    _check(load().q6_f8_quantize_act(X.data_ptr(), code, N, K, ldx, out.xq.data_ptr(),
                                     out.sx.data_ptr(), _stream(stream, dev)))
    return out


def f8_quantize_weights(W, out: F8Weights | None = None, stream=None) -> F8Weights:
    """Quantises a weight W [M, K] (f32, bf16 or f16 rows, 16-byte aligned; K a multiple of 16)
    to e4m3 with a scale for each block of 128 x 128: largest magnitude / 448."""
    code, (M, K), dev, ldw = _input(W, "W")
    if out is None:
        with _on(stream):
            out = alloc_f8_weights(M, K, dev)
    elif not isinstance(out, F8Weights) or (out.M, out.K, out.device) != (M, K, dev):
        raise Q6Error(Q6_EINVAL, f"out must be F8Weights of {M} x {K} on {dev}")
    _check(load().q6_f8_quantize_weights(W.data_ptr(), code, M, K, ldw, out.wq.data_ptr(),
                                         out.sw.data_ptr(), _stream(stream, dev)))
    return out


def _eps(eps):
    try:
        return float(eps)
    except (TypeError, ValueError):
        raise Q6Error(Q6_EINVAL, f"eps must be a number, not {eps!r}") from None


def _norm_args(X, weight, residual, h):
    """What both norms pass on of their inputs: (shape, device, h, arguments up to the weight's
    type, h's pointer and row stride)."""
    code, shape, dev, ldx = _input(X, "X")
    types = _types()
    wtype = types.get(getattr(weight, "dtype", None))
    if (wtype is None or weight.device != dev or weight.dim() != 1 or weight.shape[0] != shape[1]
            or not weight.is_contiguous()):
        wtype = _type(weight, "weight")
        _whole(weight, "weight", weight.dtype, (shape[1],), dev)
    if residual is None:
        if h is not None:
            raise Q6Error(Q6_EINVAL, "h without a residual")
        return shape, dev, X, (X.data_ptr(), code, ldx, None, 0, 0, weight.data_ptr(), wtype), None, 0
    rtype = types.get(getattr(residual, "dtype", None))
    if rtype is None:
        rtype = _type(residual, "residual")
    dtype, width = residual.dtype, shape[1] or 1
    ldr = ldh = (width if residual.shape == shape and residual.device == dev and residual.is_contiguous()
                 else _rows(residual, "residual", dtype, shape, dev))
    r = p = residual.data_ptr()
    if h is None:
        h = residual
    else:
        try:
            plain = h.dtype is dtype and h.shape == shape and h.device == dev and h.is_contiguous()
        except AttributeError:
            plain = False
        ldh, p = width if plain else _rows(h, "h", dtype, shape, dev), h.data_ptr()
    return shape, dev, h, (X.data_ptr(), code, ldx, r, rtype, ldr, weight.data_ptr(), wtype), p, ldh


def rms_norm_q8(X, weight, eps: float, residual=None, h=None, out: Activations | None = None,
                want_xh: bool = True, want_xq: bool = True, want_us: bool = False, stream=None):
    """h = X + residual, and the root-mean-square norm h / sqrt(mean(h^2) + eps) * weight as int8
    activations for mmq() and q4k_mmq() (want_us): X, residual [N, K] of f32, bf16 or f16 each
    (rows 16-byte aligned, K a multiple of 256), weight [K]. h gets the sum, rounded to
    residual's type; without h it goes into residual. Without a residual it is the norm of X.
    Codes are those of h * weight, the norm is in the scales. Returns (Activations, h)."""
    (N, K), dev, h, args, p, ldh = _norm_args(X, weight, residual, h)
    out = _q8_out(out, N, K, dev, want_xh, want_xq, want_us, stream)
    _check(load().q6_rms_norm_q8(*args, _eps(eps), N, K, p, ldh, *_q8_pointers(out), _stream(stream, dev)))
    return out, h


def rms_norm_f8(X, weight, eps: float, residual=None, h=None, out: F8Activations | None = None,
                stream=None):
    """The same norm as e4m3 activations for f8_mmq() (K a multiple of 16). Returns
    (F8Activations, h)."""
    (N, K), dev, h, args, p, ldh = _norm_args(X, weight, residual, h)
    out = _f8_out(out, N, K, dev, stream)
    _check(load().q6_rms_norm_f8(*args, _eps(eps), N, K, p, ldh, out.xq.data_ptr(), out.sx.data_ptr(),
                                 _stream(stream, dev)))
    return out, h


def _gate_up(X):
    code, (N, width), dev, ldx = _input(X, "X")
    if width % 2:
        raise Q6Error(Q6_EINVAL, f"X has {width} columns, not gate and up halves")
    return code, N, width // 2, dev, ldx


def silu_mul_q8(X, out: Activations | None = None, want_xh: bool = True, want_xq: bool = True,
                want_us: bool = False, stream=None) -> Activations:
    """silu(gate) * up of X [N, 2 K] (f32, bf16 or f16 rows, 16-byte aligned: K gate, then K up
    values) as int8 activations for mmq() and q4k_mmq() (want_us); K a multiple of 256."""
    code, N, K, dev, ldx = _gate_up(X)
    out = _q8_out(out, N, K, dev, want_xh, want_xq, want_us, stream)
    _check(load().q6_silu_mul_q8(X.data_ptr(), code, N, K, ldx, *_q8_pointers(out),
                                 _stream(stream, dev)))
    return out


def silu_mul_f8(X, out: F8Activations | None = None, stream=None) -> F8Activations:
    """The same as e4m3 activations for f8_mmq(); K a multiple of 16."""
    code, N, K, dev, ldx = _gate_up(X)
    out = _f8_out(out, N, K, dev, stream)
    _check(load().q6_silu_mul_f8(X.data_ptr(), code, N, K, ldx, out.xq.data_ptr(),
                                 out.sx.data_ptr(), _stream(stream, dev)))
    return out


def f8_mmq(w: F8Weights, act: F8Activations, out=None, dtype=None, stream=None):
    """Y [N, M] = the product of e4m3 activations and an e4m3 weight, each block of 128 of K times
    its two scales, summed in f32 and rounded once to dtype (f32, bf16 or f16; bf16 without dtype
    or out). Returns (Y, path name)."""
    M, K, N, dev = w.M, w.K, act.N, w.wq.device
    if act.K != K or act.device != dev:
        raise Q6Error(Q6_EINVAL, f"activations of K = {act.K} on {act.device} for weights of "
                                 f"K = {K} on {dev}")
    if out is None:
        if dtype is None:
            import torch
            dtype = torch.bfloat16
        if dtype not in _types():
            raise Q6Error(Q6_EINVAL, f"dtype must be float32, bfloat16 or float16, not {dtype}")
        out = _empty((N, M), dtype, dev, stream)
    elif dtype is not None and getattr(out, "dtype", None) is not dtype:
        raise Q6Error(Q6_EINVAL, f"out is not of dtype {dtype}")
    code, ldy = _types().get(getattr(out, "dtype", None)), M
    if code is None or out.shape != (N, M) or out.device != dev or not out.is_contiguous():
        code = _type(out, "out")
        ldy = _rows(out, "out", out.dtype, (N, M), dev)
    path = ctypes.c_int(-1)
    _check(load().q6_f8_mmq(w.wq.data_ptr(), w.sw.data_ptr(), M, K, act.xq.data_ptr(),
                            act.sx.data_ptr(), N, out.data_ptr(), code, ldy, ctypes.byref(path),
                            _stream(stream, dev)))
    return out, PATH_NAMES.get(path.value, str(path.value))


class F8Form(NamedTuple):
    """How a product of e4m3 blocks runs: the path's name, the tokens and weight rows of a tile,
    the parts of K that the CTAs (on the path "f8_tc" pairs of CTAs) of a cluster take, and how
    many such clusters the device runs at a time (0 where it could not say)."""
    path: str
    tokens: int
    rows: int
    parts: int
    room: int


def f8_mmq_form(M: int, K: int, N: int) -> F8Form:
    """How f8_mmq() runs N tokens on an M x K weight on the current device."""
    _c_ints(M=M, K=K, N=N)
    form = [ctypes.c_int() for _ in range(5)]
    _check(load().q6_f8_mmq_form(M, K, N, *map(ctypes.byref, form)))
    path, *rest = (v.value for v in form)
    return F8Form(PATH_NAMES.get(path, str(path)), *rest)
