"""Projections whose weights each token chooses: expert routing and grouping,
grouped products of K-quant experts, their combination, and low-rank adapters
of many requests beside a shared projection.

Argument marshalling over the C ABI, as in the package's other calls. 16-bit
activations are taken as they are; sums are f32 and rounded once. Group sizes
stay on the device: no call waits for them. Scratch memory comes from PyTorch's
allocator on the stream the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import functools

from . import (PATH_NAMES, Q6_EINVAL, Q6Error, _check, _ptr, _row_stride, _same_device, _tensor,
               load)

FORMATS = {"q4_K": 4, "q6_K": 6}
BLOCK_BYTES = {"q4_K": 144, "q6_K": 210}
MAX_GROUPS = 1024
MAX_TOPK = 32
LORA_MAX_RANK = 256


@functools.lru_cache(maxsize=None)
def _types():
    import torch
    return {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _type(t, name, half=False):
    code = _types().get(getattr(t, "dtype", None))
    if code is None or (half and code == 0):
        import torch
        if not isinstance(t, torch.Tensor):
            raise Q6Error(Q6_EINVAL, f"{name} must be a torch tensor")
        raise Q6Error(Q6_EINVAL, f"{name} must be {'' if half else 'float32, '}bfloat16 or "
                                 f"float16, not {t.dtype}")
    return code


def _rows2d(t, name, width=None):
    """The number of rows of a 2-D tensor of this width."""
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise Q6Error(Q6_EINVAL, f"{name} must have shape [rows, {width or 'columns'}], not "
                                 f"{tuple(t.shape)}")
    return t.shape[0]


def _stream(stream, device):
    """The raw handle of the stream a call runs on: `stream`, or the current
    one of the tensors' device, which has to be the current device."""
    current_device, current_stream = _current()
    index = device.index
    if current_device() != index:
        raise Q6Error(Q6_EINVAL, f"the tensors are on {device}, the current device is "
                                 f"cuda:{current_device()}")
    return current_stream(index) if stream is None else stream.cuda_stream


@functools.lru_cache(maxsize=None)
def _current():
    """() -> the current device's index, and device index -> the current
    stream's raw handle (the direct calls, where this PyTorch has them; a call
    has a CUDA tensor, so CUDA is initialised)."""
    import torch
    return (getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device,
            getattr(torch._C, "_cuda_getCurrentRawStream", None)
            or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _rows(t, name, dtype, shape, device):
    """Checks a 2-D view of rows as _tensor() does and returns its row stride.
    A contiguous tensor of this dtype and shape on this device, what callers
    mostly have, is recognised quickly."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device
                and device.type == "cuda"):
            return max(shape[1], 1)
    except AttributeError:
        pass
    return _row_stride(_tensor(t, name, dtype, shape, device, rows=True))


def _whole(t, name, dtype, shape, device):
    """The same for a tensor that has to be contiguous."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
            return
    except AttributeError:
        pass
    _tensor(t, name, dtype, shape, device)


def _on(stream):
    """Scratch and outputs are allocated on the stream the call runs on."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


@functools.lru_cache(maxsize=None)
def _alloc():
    import torch
    return torch.empty, torch.uint8, torch.cuda.stream


def _empty(shape, dtype, device, stream):
    empty, _, on = _alloc()
    if stream is None:
        return empty(shape, dtype=dtype, device=device)
    with on(stream):
        return empty(shape, dtype=dtype, device=device)


def _scratch(nbytes, device, stream):
    return _empty(nbytes, _alloc()[1], device, stream)


@functools.lru_cache(maxsize=None)
def _f32_i32():
    import torch
    return torch.float32, torch.int32


def _made(cls, **fields):
    """An object of a frozen class from buffers allocated here, which need no checks."""
    made = object.__new__(cls)
    made.__dict__.update(fields)
    return made


# ---------------------------------------------------------------- grouping ---

@functools.lru_cache(maxsize=256)
def group_workspace_bytes(N: int, per_row: int, groups: int) -> int:
    b = ctypes.c_size_t()
    _check(load().q6_group_workspace_bytes(N, per_row, groups, ctypes.byref(b)))
    return b.value


@dataclasses.dataclass(frozen=True)
class Groups:
    """N * per_row items sorted by group, in item order within one (device,
    int32): offsets [n_groups + 2] (the last section holds the items of no
    group), rows [N * per_row] (each sorted item's token), pos [N, per_row]
    (each item's place, -1 without a group). Checked once, when made."""
    N: int
    per_row: int
    n_groups: int
    offsets: object
    rows: object
    pos: object
    workspace: object = None

    def __post_init__(self):
        import torch
        n, need = self.N * self.per_row, group_workspace_bytes(self.N, self.per_row, self.n_groups)
        _same_device((self.offsets, "offsets", torch.int32, (self.n_groups + 2,)),
                     (self.rows, "rows", torch.int32, (n,)),
                     (self.pos, "pos", torch.int32, (self.N, self.per_row)),
                     (self.workspace, "workspace", torch.uint8, (need,)))
        if need and self.workspace is None:
            raise Q6Error(Q6_EINVAL, f"this grouping needs a workspace of {need} bytes")

        object.__setattr__(self, "items", n)
        object.__setattr__(self, "device", self.offsets.device)


def alloc_groups(N: int, per_row: int, n_groups: int, device=None) -> Groups:
    """Buffers for a grouping."""
    import torch
    need = group_workspace_bytes(N, per_row, n_groups)
    dev = device or torch.device("cuda")

    def i32(*shape):
        return torch.empty(shape, dtype=torch.int32, device=dev)

    offsets = i32(n_groups + 2)
    return _made(Groups, N=N, per_row=per_row, n_groups=n_groups, offsets=offsets,
                 rows=i32(N * per_row), pos=i32(N, per_row), items=N * per_row,
                 device=offsets.device,
                 workspace=torch.empty(need, dtype=torch.uint8, device=dev) if need else None)


def group_rows(ids, n_groups: int, out: Groups | None = None, stream=None) -> Groups:
    """Groups tokens by ids, int32 [N] or [N, per_row] (contiguous CUDA
    tensor); an id outside 0 .. n_groups - 1 belongs to no group."""
    import torch
    if not isinstance(ids, torch.Tensor) or ids.dim() not in (1, 2):
        raise Q6Error(Q6_EINVAL, "ids must be a torch tensor [N] or [N, per_row]")
    _tensor(ids, "ids", torch.int32, ids.shape)
    N, per_row = ids.shape[0], ids.shape[1] if ids.dim() == 2 else 1
    if out is None:
        with _on(stream):
            out = alloc_groups(N, per_row, n_groups, ids.device)
    elif (out.N, out.per_row, out.n_groups, out.device) != (N, per_row, n_groups, ids.device):
        raise Q6Error(Q6_EINVAL, "out holds another grouping than ids and n_groups ask for")
    ws = out.workspace
    _check(load().q6_group_rows(ids.data_ptr(), N, per_row, n_groups, out.offsets.data_ptr(),
                                out.rows.data_ptr(), out.pos.data_ptr(),
                                None if ws is None else ws.data_ptr(),
                                0 if ws is None else ws.numel(), _stream(stream, ids.device)))
    return out


@dataclasses.dataclass(frozen=True)
class Route:
    """A router's choice: ids [N, topk] int32 (-1: no expert), weights
    [N, topk] f32, and the items grouped by expert."""
    ids: object
    weights: object
    groups: Groups

    def __post_init__(self):
        import torch
        g = self.groups
        _same_device((self.ids, "ids", torch.int32, (g.N, g.per_row)),
                     (self.weights, "weights", torch.float32, (g.N, g.per_row)),
                     (g.offsets, "offsets", torch.int32, (g.n_groups + 2,)))


def alloc_route(N: int, E: int, topk: int, device=None) -> Route:
    """Buffers for the routing of N tokens to topk of E experts."""
    import torch
    dev = device or torch.device("cuda")
    return _made(Route, groups=alloc_groups(N, topk, E, dev),
                 ids=torch.empty((N, topk), dtype=torch.int32, device=dev),
                 weights=torch.empty((N, topk), dtype=torch.float32, device=dev))


def moe_route(logits, topk: int, renormalize: bool = True, out: Route | None = None,
              stream=None) -> Route:
    """Routes each token to the experts of its topk largest logits [N, E]
    (f32, bf16 or f16, CUDA; ties to the lowest index) and groups the tokens
    by expert. A logit of -inf or NaN is never chosen: slots left over get id
    -1 and weight 0. weights: softmax over the chosen experts (renormalize) or
    over all of them; a NaN logit makes its token's weights NaN."""
    code = _type(logits, "logits")
    N = _rows2d(logits, "logits")
    E = logits.shape[1]
    dev = logits.device
    ldl = _rows(logits, "logits", logits.dtype, (N, E), dev)
    if out is None:
        with _on(stream):
            out = alloc_route(N, E, topk, dev)
    g = out.groups
    if g.N != N or g.per_row != topk or g.n_groups != E or g.device != dev:
        raise Q6Error(Q6_EINVAL, f"out holds {g.N} x {g.per_row} of {g.n_groups} experts on "
                                 f"{g.device}, not {N} x {topk} of {E} on {dev}")
    ws = g.workspace
    _check(load().q6_moe_route(logits.data_ptr(), code, N, E, ldl, topk,
                               1 if renormalize else 0, out.ids.data_ptr(),
                               out.weights.data_ptr(), g.offsets.data_ptr(), g.rows.data_ptr(),
                               g.pos.data_ptr(), None if ws is None else ws.data_ptr(),
                               0 if ws is None else ws.numel(), _stream(stream, dev)))
    return out


# ----------------------------------------------------------------- experts ---

@functools.lru_cache(maxsize=256)
def expert_plane_bytes(fmt: str, E: int, M: int, K: int, swiglu: bool = False) -> int:
    if fmt not in FORMATS:
        raise Q6Error(Q6_EINVAL, f"fmt must be one of {sorted(FORMATS)}, not {fmt}")
    b = ctypes.c_size_t()
    _check(load().q6_expert_plane_bytes(FORMATS[fmt], E, M, K, int(swiglu), ctypes.byref(b)))
    return b.value


@dataclasses.dataclass(frozen=True)
class ExpertWeights:
    """E packed K-quant experts of M x K on the device; with swiglu the first
    M / 2 rows are gate rows, the others up rows. Checked once, when made."""
    fmt: str
    E: int
    M: int
    K: int
    swiglu: bool
    plane: object

    def __post_init__(self):
        import torch
        need = expert_plane_bytes(self.fmt, self.E, self.M, self.K, self.swiglu)
        _same_device((self.plane, "plane", torch.uint8, (need,)))

    @property
    def device(self):
        return self.plane.device

    @property
    def out_features(self):
        return self.M // 2 if self.swiglu else self.M


def pack_experts(raw, fmt: str, E: int, M: int, K: int, swiglu: bool = False, stream=None,
                 device=None) -> ExpertWeights:
    """Packs E raw GGUF matrices of M x K ("q4_K" or "q6_K" bytes, one expert
    after another): a contiguous uint8 tensor on a CUDA device or in host
    memory, as pack_weights(). swiglu: the rows are M / 2 gate rows, then
    M / 2 up rows, and the product returns silu(gate) * up."""
    import torch
    swiglu = bool(swiglu)
    need = expert_plane_bytes(fmt, E, M, K, swiglu)
    if (not isinstance(raw, torch.Tensor) or raw.numel() != E * M * (K // 256) * BLOCK_BYTES[fmt]
            or raw.dtype != torch.uint8 or not raw.is_contiguous()):
        raise Q6Error(Q6_EINVAL, f"raw must be a contiguous uint8 tensor of "
                                 f"E*M*K/256*{BLOCK_BYTES[fmt]} bytes")
    on_host = not raw.is_cuda
    if on_host:
        dev = torch.device(device) if device is not None else torch.device(
            "cuda", torch.cuda.current_device())
        if not raw.is_pinned():
            raw = raw.pin_memory()
    else:
        dev = raw.device
    with torch.cuda.device(dev), _on(stream):
        plane = torch.empty(need, dtype=torch.uint8, device=dev)
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        _check(load().q6_pack_experts(FORMATS[fmt], _ptr(raw), E, M, K, int(swiglu), _ptr(plane),
                                      s.cuda_stream))
        if on_host:
            s.synchronize()      # the kernel has read the host bytes
    return ExpertWeights(fmt, E, M, K, swiglu, plane)


@functools.lru_cache(maxsize=256)
def experts_workspace_bytes(E: int, K: int, type: int, items: int, gather: bool) -> int:
    b = ctypes.c_size_t()
    _check(load().q6_experts_workspace_bytes(E, K, type, items, int(gather), ctypes.byref(b)))
    return b.value


def experts_mmq(w: ExpertWeights, X, groups: Groups, gather: bool = True, out=None, stream=None):
    """The grouped product: row i of the result is W[e] x for the sorted item
    i of `groups` (one group per expert), x the item's token's row of X
    [N, K] (gather) or row i of X [items, K]; silu(gate) * up for swiglu
    weights. X is bf16 or f16 (rows 16-byte aligned), the result the same.
    Items of no expert get zeros. Returns (Y [items, out_features], path
    name)."""
    code = _type(X, "X", half=True)
    K = w.K
    nx = _rows2d(X, "X", K)
    dev, items, dtype = w.plane.device, groups.items, X.dtype
    ldx = _rows(X, "X", dtype, (nx, K), dev)
    if groups.n_groups != w.E or groups.device != dev:
        raise Q6Error(Q6_EINVAL, f"a grouping of {groups.n_groups} groups on {groups.device} for "
                                 f"{w.E} experts on {dev}")
    if nx != (groups.N if gather else items):
        raise Q6Error(Q6_EINVAL, f"X has {nx} rows, the grouping {groups.N} tokens and {items} "
                                 "items")
    shape = (items, w.out_features)
    if out is None:
        out = _empty(shape, dtype, dev, stream)
    ldy = _rows(out, "out", dtype, shape, dev)
    need, ws = experts_workspace_bytes(w.E, K, code, items, bool(gather)), None
    if need:
        ws = _scratch(need, dev, stream)
    path = ctypes.c_int(-1)
    _check(load().q6_experts_mmq(FORMATS[w.fmt], w.plane.data_ptr(), w.E, w.M, K,
                                 1 if w.swiglu else 0, X.data_ptr(), code, nx, ldx, 1 if gather else 0,
                                 groups.offsets.data_ptr(), groups.rows.data_ptr(), items,
                                 out.data_ptr(), ldy, None if ws is None else ws.data_ptr(), need,
                                 ctypes.byref(path), _stream(stream, dev)))
    return out, PATH_NAMES.get(path.value, str(path.value))


def moe_combine(Y, pos, weights, shared=None, out=None, stream=None):
    """out [N, M] = shared + the weighted sum of each token's rows of Y
    [items, M] (bf16 or f16): pos [N, topk] int32 are their places (-1 adds
    nothing; others are below items, which is not checked), weights [N, topk]
    f32, shared f32 [N, M] or None."""
    f32, i32 = _f32_i32()
    code = _type(Y, "Y", half=True)
    items = _rows2d(Y, "Y")
    dev, dtype, M = Y.device, Y.dtype, Y.shape[1]
    ldy = _rows(Y, "Y", dtype, (items, M), dev)
    if getattr(pos, "dtype", None) is not i32 or pos.dim() != 2:
        raise Q6Error(Q6_EINVAL, "pos must be a 2-D int32 torch tensor [N, topk]")
    slots = N, topk = pos.shape
    _whole(pos, "pos", i32, slots, dev)
    _whole(weights, "weights", f32, slots, dev)
    lds = 0 if shared is None else _rows(shared, "shared", f32, (N, M), dev)
    if out is None:
        out = _empty((N, M), dtype, dev, stream)
    ldo = _rows(out, "out", dtype, (N, M), dev)
    _check(load().q6_moe_combine(Y.data_ptr(), code, ldy, pos.data_ptr(), weights.data_ptr(), N,
                                 topk, M, None if shared is None else shared.data_ptr(), lds,
                                 out.data_ptr(), ldo, _stream(stream, dev)))
    return out


# ---------------------------------------------------------------- adapters ---

@functools.lru_cache(maxsize=256)
def lora_workspace_bytes(items: int, L: int, r: int, K: int) -> int:
    b = ctypes.c_size_t()
    _check(load().q6_lora_workspace_bytes(items, L, r, K, ctypes.byref(b)))
    return b.value


@dataclasses.dataclass(frozen=True)
class LoraAdapters:
    """L low-rank adapters of one projection on the device: A [L, r, K], B
    [L, M, r] (bf16 or f16, contiguous), scale f32 [L]. r is a multiple of 8
    (pad with zeros). Checked once, when made."""
    A: object
    B: object
    scale: object

    def __post_init__(self):
        import torch
        _type(self.A, "A", half=True)
        if not isinstance(self.B, torch.Tensor) or self.A.dim() != 3 or self.B.dim() != 3:
            raise Q6Error(Q6_EINVAL, "A and B must be tensors [L, r, K] and [L, M, r]")
        L, r, K = self.A.shape
        _same_device((self.A, "A", self.A.dtype, (L, r, K)),
                     (self.B, "B", self.A.dtype, (L, self.B.shape[1], r)),
                     (self.scale, "scale", torch.float32, (L,)))
        lora_workspace_bytes(1, L, r, K)     # the sizes the kernels take

    @property
    def device(self):
        return self.A.device


def lora_add(adapters: LoraAdapters, X, groups: Groups, Y, out=None, stream=None):
    """out [N, M] = Y + scale[a] * B[a] (A[a] x) for each token, a its adapter
    (groups: the tokens grouped by adapter, one id a token); tokens of no
    adapter keep Y. X [N, K] is f32, bf16 or f16 (rows 16-byte aligned), Y and
    out are f32; without out the result goes into Y. Returns out."""
    A, B, f32 = adapters.A, adapters.B, _f32_i32()[0]
    L, r, K = A.shape
    M, dev, N = B.shape[1], A.device, groups.items
    code = _type(X, "X")
    ldx = _rows(X, "X", X.dtype, (N, K), dev)
    if groups.n_groups != L or groups.per_row != 1 or groups.device != dev:
        raise Q6Error(Q6_EINVAL, f"adapters need one id a token in {L} groups on {dev}")
    ldy = ldo = _rows(Y, "Y", f32, (N, M), dev)
    if out is None:
        out = Y
    else:
        ldo = _rows(out, "out", f32, (N, M), dev)
    need, ws = lora_workspace_bytes(N, L, r, K), None
    if need:
        ws = _scratch(need, dev, stream)
    _check(load().q6_lora_add(A.data_ptr(), B.data_ptr(), adapters.scale.data_ptr(),
                              _types()[A.dtype], L, r, M, K, X.data_ptr(), code, ldx,
                              groups.offsets.data_ptr(), groups.rows.data_ptr(), N, Y.data_ptr(),
                              ldy, out.data_ptr(), ldo, None if ws is None else ws.data_ptr(),
                              need, _stream(stream, dev)))
    return out
