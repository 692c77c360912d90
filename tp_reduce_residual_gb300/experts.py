"""Python binding of the operators around the experts of a mixture-of-experts layer.

``route`` chooses each token's experts and weights from the router's logits
(``route_backward`` is its gradient), ``plan`` groups the token slots by expert,
``quantize_fp4`` / ``dequantize_fp4`` take rows to 4-bit microscaled floating
point and back, and ``expert_product`` multiplies grouped rows with each
expert's weights.  ``plan(...).perm``, ``route(...)``'s weights and the product
are what ``beamnorm.finalize_reduce_norm`` takes.

As in ``beamnorm``, a function checks its arguments, then calls the C entry
point with raw device pointers and the current CUDA stream; the arithmetic runs
in the library's kernels and there is no fallback.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass
from typing import NamedTuple, Optional

import torch

from . import beamnorm as _bn

SCORES = {"softmax": 0, "sigmoid": 1}
FORMATS = {"nvfp4": 0, "mxfp4": 1}
#: values along a row that share a scale
BLOCK = {"nvfp4": 16, "mxfp4": 32}
_CHUNK = {"nvfp4": 64, "mxfp4": 128}   # values along a row in one scale tile
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

_FLOAT32, _INT32, _UINT8 = torch.float32, torch.int32, torch.uint8


class Plan(NamedTuple):
    """Where token slots go when they are grouped by expert: perm [R,T,k] the
    place of each slot, offsets [E+1] the groups' first places, rows [T*k] the
    token at each place (all int32)."""
    perm: torch.Tensor
    offsets: torch.Tensor
    rows: torch.Tensor


@dataclass
class FP4:
    """Quantised rows: ``data`` uint8 [..., K/2] (element 2i in the low half of
    byte i) and ``scales`` uint8 [tiles, chunks, 512] in the layout that
    ``include/beamnorm.h`` describes at bn_fp4_scale_bytes.  ``offsets`` are the
    ragged groups' first rows (int32 [groups+1]; of a longer list a part, then the
    rows before its first are in no group) or None: one group per leading index of
    a 3-D ``data``, one group for a 2-D one."""
    data: torch.Tensor
    scales: torch.Tensor
    format: str
    offsets: Optional[torch.Tensor] = None
    tensor_scale: float = 1.0

    @property
    def shape(self):
        return (*self.data.shape[:-1], 2 * self.data.shape[-1])


@dataclass
class Int8:
    """Rows in 8-bit integers: ``data`` int8 [..., K] and a scale for each row, ``scales``
    FP32 [...].  ``offsets`` as in FP4."""
    data: torch.Tensor
    scales: torch.Tensor
    offsets: Optional[torch.Tensor] = None

    @property
    def shape(self):
        return tuple(self.data.shape)


# A decoded token's operators take a few microseconds on the GPU, so the checks
# below are written for the host's time: an argument that is as it should be passes
# in one expression, and only one that is not goes through beamnorm's checks for
# the message.


def _call(name, args, index, stream):
    """One C call with device ``index`` current, on ``stream`` or the current one."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    else:
        stream = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    fn = getattr(_bn._lib or _bn.load(), name)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status:
        _bn._check(status)


def _ptr(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this type, shape and device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev and t.is_cuda \
            and t.is_contiguous():
        return t.data_ptr()
    return _bn._need(t, name, dtype, tuple(shape), dev)


def _out(t, name, dtype, shape, dev, stream):
    """An output and its address: the caller's, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev) if stream is None else _bn._empty(shape, dtype, dev, stream)
        return t, t.data_ptr()
    return t, _ptr(t, name, dtype, shape, dev)


def _name(table, value, what):
    if value not in table:
        raise ValueError(f"{what} must be one of {', '.join(table)} (got {value!r})")
    return table[value]


def _dtype(t, name, fp32=True):
    d = _DTYPES.get(t.dtype)
    if d is None or (d == 2 and not fp32):
        raise TypeError(f"{name} must be torch.bfloat16, torch.float16{' or torch.float32' if fp32 else ''} (got {t.dtype})")
    return d


def _rows2d(t, name):
    """A 2-D CUDA tensor whose rows are contiguous; returns its row stride."""
    if isinstance(t, torch.Tensor) and t.is_cuda:
        shape = t.shape
        if len(shape) == 2:
            if t.is_contiguous():
                return shape[1]
            ld, inner = t.stride()
            if inner == 1 or shape[1] <= 1:
                if shape[0] <= 1:
                    return shape[1]
                if ld >= shape[1]:
                    return ld
                raise ValueError(f"{name} must have rows that do not overlap (row stride {ld} below {shape[1]})")
            raise ValueError(f"{name} must have contiguous rows")
        raise ValueError(f"{name} must have 2 dimensions (got {len(shape)})")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")


def route(logits, k: int, bias=None, score: str = "softmax", groups: int = 1, top_groups: int = 1,
          group_top: int = 1, renormalize: bool = True, scale: float = 1.0, shards: int = 1,
          ids=None, w=None, stream=None):
    """Each token's k experts and their weights: ``(ids [T,k] int32, w [shards,T,k] FP32)``.

    ``logits`` [T,E] BF16, FP16 or FP32 (any row stride).  Experts rank by
    score + ``bias`` [E] (FP32, for the choice only), equal ones by index;
    weights are the scores (``renormalize``: over their sum) times ``scale``.
    With ``groups`` > 1 only the ``top_groups`` groups of consecutive experts
    with the largest sum of their ``group_top`` (1 or 2) best are left.  Logits
    of -inf take experts out; slots without an expert get id -1, weight 0."""
    ld = _rows2d(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    dtype = _dtype(logits, "logits")
    bp = None if bias is None else _ptr(bias, "bias", _FLOAT32, (E,), dev)
    ids, ip = _out(ids, "ids", _INT32, (T, k), dev, stream)
    w, wp = _out(w, "w", _FLOAT32, (shards, T, k), dev, stream)
    _call("bn_route", (logits.data_ptr(), dtype, ld, T, E, k, bp, _name(SCORES, score, "score"), groups, top_groups,
                       group_top, 1 if renormalize else 0, scale, shards, ip, wp), dev.index, stream)
    return ids, w


def route_backward(logits, ids, dw, score: str = "softmax", renormalize: bool = True,
                   scale: float = 1.0, dlogits=None, stream=None) -> torch.Tensor:
    """Gradient of ``route``'s weights: dlogits [T,E] in the logits' dtype from
    ``dw`` [shards,T,k] FP32 (summed over the shards) and the chosen ``ids``."""
    ld = _rows2d(logits, "logits")
    T, E = logits.shape
    dev = logits.device
    dtype = _dtype(logits, "logits")
    if not isinstance(dw, torch.Tensor) or dw.dim() != 3:
        raise ValueError("dw must be a tensor of 3 dimensions [shards, T, k]")
    R, _, k = dw.shape
    ip = _ptr(ids, "ids", _INT32, (T, k), dev)
    dp = _ptr(dw, "dw", _FLOAT32, (R, T, k), dev)
    dlogits, op = _out(dlogits, "dlogits", logits.dtype, (T, E), dev, stream)
    _call("bn_route_backward", (logits.data_ptr(), dtype, ld, T, E, k, ip, dp, R, _name(SCORES, score, "score"),
                                1 if renormalize else 0, scale, op), dev.index, stream)
    return dlogits


def plan(ids, experts: int, shards: int = 1, perm=None, offsets=None, rows=None, stream=None) -> Plan:
    """Group the slots of ``ids`` [T,k] by expert, in slot order within each;
    slots with id -1 come last.  ``perm`` is repeated for ``shards`` shards."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a tensor of 2 dimensions [T, k]")
    T, k = ids.shape
    dev = ids.device
    ip = _ptr(ids, "ids", _INT32, (T, k), dev)
    perm, pp = _out(perm, "perm", _INT32, (shards, T, k), dev, stream)
    offsets, op = _out(offsets, "offsets", _INT32, (experts + 1,), dev, stream)
    rows, rp = _out(rows, "rows", _INT32, (T * k,), dev, stream)
    _call("bn_expert_plan", (ip, T, k, experts, shards, pp, op, rp), dev.index, stream)
    return Plan(perm, offsets, rows)


def fp4_scales_shape(M: int, K: int, format: str, groups: int = 1, ragged: bool = False):
    """Shape of the scales of M rows of K values: [tiles, chunks, 512]."""
    tiles = M // 128 + groups + 1 if ragged else groups * (-(-(M // groups) // 128))
    return tiles, -(-K // _CHUNK[format]), 512


def _layout(q: FP4, name: str):
    """(M, K, groups, and the pointers of offsets, data and scales) of quantised rows, after checks."""
    if not isinstance(q, FP4):
        raise TypeError(f"{name} must be an FP4")
    _name(FORMATS, q.format, "format")
    data = q.data
    shape, dev = data.shape, data.device
    n = len(shape)
    if n not in (2, 3) or (n == 3 and q.offsets is not None):
        raise ValueError(f"{name}.data must be [M, K/2], or [groups, rows, K/2] without offsets")
    dp = _ptr(data, f"{name}.data", _UINT8, shape, dev)
    K = 2 * shape[-1]
    groups = shape[0] if n == 3 else 1
    M = groups * shape[1] if n == 3 else shape[0]
    op = None
    if q.offsets is not None:
        groups = q.offsets.numel() - 1
        op = _ptr(q.offsets, f"{name}.offsets", _INT32, (groups + 1,), dev)
    sp = _ptr(q.scales, f"{name}.scales", _UINT8, fp4_scales_shape(M, K, q.format, max(groups, 1), op is not None), dev)
    return M, K, groups, op, dp, sp


@functools.lru_cache(maxsize=256)
def quantize_workspace_bytes(n: int, M: int, K: int, format: str) -> int:
    """Workspace bytes with which ``quantize_fp4`` quantises n rows once for M
    places, or 0 where that does not pay."""
    return (_bn._lib or _bn.load()).bn_quantize_fp4_workspace_bytes(n, M, K, _name(FORMATS, format, "format"))


def quantize_fp4(x, format: str, rows=None, offsets=None, tensor_scale: float = 1.0,
                 data=None, scales=None, workspace=None, stream=None) -> FP4:
    """Rows of ``x`` ([n,K], or [groups,n,K] such as weights; BF16 or FP16) in
    4-bit floating point.  ``rows`` (int32 [M]) picks the rows, ``offsets``
    (int32 [groups+1]) are the ragged groups of the result, as ``plan`` gives
    them; ``tensor_scale`` is a power of two.  Where many places take the same
    row, rows are quantised once into a ``workspace`` (a 1-D uint8 tensor of
    ``quantize_workspace_bytes``; by default one is allocated for the call when
    it runs on the current stream) and copied from there: the same result."""
    fmt = _name(FORMATS, format, "format")
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    lead = None
    if x.dim() == 3:
        if rows is not None or offsets is not None:
            raise ValueError("a 3-D x has equal groups: it takes neither rows nor offsets")
        if not x.is_contiguous():
            raise ValueError("a 3-D x must be contiguous")
        lead = x.shape[:2]
        x = x.view(-1, x.shape[2])
    ld = _rows2d(x, "x")
    n, K = x.shape
    if n <= 1:
        ld = -(-K // 8) * 8
    dtype = _dtype(x, "x", fp32=False)
    M, rp = n, None
    if rows is not None:
        M = rows.numel()
        rp = _ptr(rows, "rows", _INT32, (M,), dev)
    groups, op = 1, None
    if offsets is not None:
        groups = offsets.numel() - 1
        op = _ptr(offsets, "offsets", _INT32, (groups + 1,), dev)
    elif lead is not None:
        groups = lead[0]
    if K % 32 or K == 0:
        raise ValueError(f"x has rows of {K} values, not a positive multiple of 32")
    if M and groups < 1:
        raise ValueError("offsets must have 2 entries or more")
    dshape = (*lead, K // 2) if lead is not None else (M, K // 2)
    groups = max(groups, 1)
    data, dp = _out(data, "data", _UINT8, dshape, dev, stream)
    scales, sp = _out(scales, "scales", _UINT8, fp4_scales_shape(M, K, format, groups, op is not None), dev, stream)
    wp, wn = None, 0
    if workspace is not None:
        wp, wn = _bn._workspace(workspace, dev)
    elif rp is not None and stream is None:
        wn = quantize_workspace_bytes(n, M, K, format)
        if wn:
            workspace = torch.empty(wn, dtype=_UINT8, device=dev)
            wp = workspace.data_ptr()
    _call("bn_quantize_fp4", (x.data_ptr(), dtype, ld, n, rp, M, K, op, groups, fmt, tensor_scale, dp, sp, wp, wn), dev.index,
          stream)
    return FP4(data, scales, format, offsets, tensor_scale)


def dequantize_fp4(q: FP4, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """The values of quantised rows ([..., K]) in BF16, FP16 or FP32."""
    M, K, groups, op, dp, sp = _layout(q, "q")
    dev = q.data.device
    out, yp = _out(out, "out", dtype if out is None else out.dtype, q.shape, dev, stream)
    _call("bn_dequantize_fp4", (dp, sp, M, K, op, max(groups, 1), FORMATS[q.format], q.tensor_scale, yp, _dtype(out, "out")),
          dev.index, stream)
    return out


def expert_product(a, w, scale: float = 1.0, out=None, stream=None, workspace=None) -> torch.Tensor:
    """out [M,N] BF16: each row of ``a`` ([M,K], grouped by ``a.offsets``) times
    its group's weights of ``w`` ([E,N,K]; [N,K] is one expert), times ``scale``
    and the operands' scales.  Both are FP4 or both Int8, whose sums are exact.  Rows
    before the first group and past the last are zeros.  Int8 rows of large groups go
    through a ``workspace`` (a 1-D uint8 tensor of ``product_int8_workspace_bytes``; by
    default one is allocated for the call); FP4 ones take none."""
    if isinstance(a, Int8):
        return _expert_product_int8(a, w, scale, out, workspace, stream)
    if workspace is not None:
        raise ValueError("FP4 rows take no workspace")
    M, K, groups, op, ap, sp = _layout(a, "a")
    _, wK, E, wo, wp, wsp = _layout(w, "w")
    if wo is not None:
        raise ValueError("w must have equal groups (no offsets)")
    if a.data.dim() != 2:
        raise ValueError("a.data must be [M, K/2]")
    if wK != K or a.format != w.format:
        raise ValueError(f"a has rows of {K} {a.format} values, w of {wK} {w.format} values")
    if groups != E:
        raise ValueError(f"a has {groups} groups, w has {E} experts")
    dev = a.data.device
    if w.data.device != dev:
        raise ValueError(f"w is on {w.data.device}, expected {dev}")
    N = w.data.shape[-2]
    out, yp = _out(out, "out", torch.bfloat16, (M, N), dev, stream)
    _call("bn_expert_product", (ap, sp, M, wp, wsp, E, N, K, op, FORMATS[a.format], scale * a.tensor_scale * w.tensor_scale, yp),
          dev.index, stream)
    return out


def _groups(offsets, E, dev):
    """The address of the groups' offsets of E experts, or None where one expert has every row."""
    if offsets is None:
        if E != 1:
            raise ValueError(f"offsets are required with {E} experts")
        return None
    return _ptr(offsets, "offsets", _INT32, (E + 1,), dev)


def _weights(w, dtype, dev):
    """(E, N, K) and the address of the experts' weights [E,N,K], or [N,K]: one expert."""
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w must be a tensor [experts, N, K] or [N, K]")
    shape = w.shape
    E, N, K = shape if len(shape) == 3 else (1, *shape)
    return E, N, K, _ptr(w, "w", dtype, shape, dev)


def _places(x, rows):
    """M and the address of ``rows``: the rows of x, or one for every entry of ``rows``."""
    if rows is None:
        return x.shape[0], None
    return rows.numel(), _ptr(rows, "rows", _INT32, (rows.numel(),), x.device)


def _stride(t, name):
    """The row stride of a 2-D tensor for the kernels that copy rows in 16-byte pieces."""
    ld = _rows2d(t, name)
    return ld if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def linear_workspace_bytes(M: int, K: int) -> int:
    """Workspace bytes with which ``expert_linear`` and ``expert_linear_dw`` bring rows of
    K values to M places by index, or 0 where they need none."""
    return (_bn._lib or _bn.load()).bn_expert_linear_workspace_bytes(M, K)


def _call_workspace(workspace, n, dev, stream):
    """The caller's workspace, or one of n bytes for the call from its stream's pool: address, bytes, and the
    tensor to keep."""
    if workspace is not None:
        return (*_bn._workspace(workspace, dev), workspace)
    if n == 0:
        return None, 0, None
    workspace = torch.empty(n, dtype=_UINT8, device=dev) if stream is None else _bn._empty((n,), _UINT8, dev, stream)
    return workspace.data_ptr(), n, workspace


def expert_linear(x, w, offsets=None, rows=None, out=None, workspace=None, stream=None) -> torch.Tensor:
    """The experts' linear layer in 16 bits: out [M,N], each row of ``x`` ([n,K] BF16 or
    FP16, any row stride that is a multiple of 8) times its group's weights of ``w``
    ([E,N,K]; [N,K] is one expert), summed in FP32.  ``offsets`` (int32 [E+1]) are the
    groups, ``rows`` (int32 [M]) the row of x at each place, as ``plan`` gives them;
    without ``rows`` x is grouped already.  Rows of no group are zeros, whatever ``rows``
    holds there.  More than a few
    rows by index go through a ``workspace`` (a 1-D uint8 tensor of
    ``linear_workspace_bytes``; by default one is allocated for the call).  One
    workspace serves one call at a time."""
    ld = _stride(x, "x")
    dev = x.device
    dtype = _dtype(x, "x", fp32=False)
    M, rp = _places(x, rows)
    E, N, K, wp = _weights(w, x.dtype, dev)
    if x.shape[1] != K:
        raise ValueError(f"x has rows of {x.shape[1]} values, w of {K}")
    op = _groups(offsets, E, dev)
    out, yp = _out(out, "out", x.dtype, (M, N), dev, stream)
    sp, n, workspace = _call_workspace(workspace, linear_workspace_bytes(M, K) if rp is not None else 0, dev, stream)
    _call("bn_expert_linear", (x.data_ptr(), dtype, ld, x.shape[0], rp, M, wp, E, N, K, op, yp, sp, n), dev.index, stream)
    return out


def expert_linear_dx(dy, w, offsets=None, dx=None, stream=None) -> torch.Tensor:
    """Gradient of ``expert_linear`` with respect to the grouped rows: dx [M,K] from ``dy``
    [M,N].  Where ``rows`` took a row several times, its gradient is the sum over its
    places: ``beamnorm.finalize_reduce_only`` with the plan's perm and weights of 1 (FP32,
    each shard's sum rounded to BF16 once).  It takes BF16 rows, as every finalize does:
    rows in FP16, dx or the layer's output, are for the caller to add up."""
    ld = _stride(dy, "dy")
    dev = dy.device
    dtype = _dtype(dy, "dy", fp32=False)
    M = dy.shape[0]
    E, N, K, wp = _weights(w, dy.dtype, dev)
    if dy.shape[1] != N:
        raise ValueError(f"dy has rows of {dy.shape[1]} values, w has {N} rows")
    op = _groups(offsets, E, dev)
    dx, xp = _out(dx, "dx", dy.dtype, (M, K), dev, stream)
    _call("bn_expert_linear_dx", (dy.data_ptr(), dtype, ld, M, wp, E, N, K, op, xp), dev.index, stream)
    return dx


def expert_linear_dw(dy, x, offsets=None, rows=None, dtype=None, dw=None, accumulate: bool = False, workspace=None,
                     stream=None) -> torch.Tensor:
    """Gradient of ``expert_linear`` with respect to the weights: dw [E,N,K] from ``dy``
    [M,N] and the layer's ``x`` and ``rows``, in x's dtype or FP32 (``dtype``, or that of
    ``dw``).  ``accumulate`` adds to what an FP32 ``dw`` holds.  Without ``offsets`` there
    is one expert and dw is [N,K].  ``workspace`` as in ``expert_linear``."""
    ld_dy = _stride(dy, "dy")
    ld = _stride(x, "x")
    dev = dy.device
    d = _dtype(dy, "dy", fp32=False)
    if x.device != dev or x.dtype is not dy.dtype:
        raise ValueError(f"x ({x.dtype} on {x.device}) must be as dy ({dy.dtype} on {dev})")
    M, rp = _places(x, rows)
    if dy.shape[0] != M:
        raise ValueError(f"dy has {dy.shape[0]} rows, expected {M}")
    E = 1 if offsets is None else offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets must have 2 entries or more")
    op = _groups(offsets, E, dev)
    N, K = dy.shape[1], x.shape[1]
    if accumulate and dw is None:
        raise ValueError("accumulate adds to a dw that is given")
    want = dw.dtype if isinstance(dw, torch.Tensor) else x.dtype if dtype is None else dtype
    if want not in (x.dtype, _FLOAT32) or (dtype is not None and dtype is not want):
        raise TypeError(f"dw must be {x.dtype} or torch.float32 (got {dtype or want})")
    dw, wp = _out(dw, "dw", want, (N, K) if offsets is None else (E, N, K), dev, stream)
    sp, n, workspace = _call_workspace(workspace, linear_workspace_bytes(M, K) if rp is not None else 0, dev, stream)
    _call("bn_expert_linear_dw", (dy.data_ptr(), d, ld_dy, M, x.data_ptr(), ld, x.shape[0], rp, E, N, K, op, wp, _DTYPES[want],
                                  1 if accumulate else 0, sp, n), dev.index, stream)
    return dw


def swiglu(x, out=None, stream=None) -> torch.Tensor:
    """The gated activation between an expert's two layers: [M,F], gate / (1 + exp(-gate)) * up
    of ``x`` [M,2F] (gate and up side by side; BF16, FP16 or FP32, any row stride)."""
    ld = _rows2d(x, "x")
    M, n = x.shape
    if n == 0 or n % 2:
        raise ValueError(f"x must have rows of gate and up side by side (got {n} values)")
    dev = x.device
    dtype = _dtype(x, "x")
    out, yp = _out(out, "out", x.dtype, (M, n // 2), dev, stream)
    _call("bn_swiglu", (x.data_ptr(), dtype, ld, M, n // 2, yp), dev.index, stream)
    return out


def swiglu_backward(x, dy, dx=None, stream=None) -> torch.Tensor:
    """Gradient of ``swiglu``: dx [M,2F] from its ``x`` and ``dy`` [M,F] (any row strides)."""
    ld, ld_dy = _rows2d(x, "x"), _rows2d(dy, "dy")
    M, n = x.shape
    if n == 0 or n % 2:
        raise ValueError(f"x must have rows of gate and up side by side (got {n} values)")
    dev = x.device
    dtype = _dtype(x, "x")
    if dy.shape != (M, n // 2) or dy.dtype is not x.dtype or dy.device != dev:
        raise ValueError(f"dy must be {x.dtype} of shape {(M, n // 2)} on {dev} (got {dy.dtype}, {tuple(dy.shape)}, {dy.device})")
    dx, xp = _out(dx, "dx", x.dtype, (M, n), dev, stream)
    _call("bn_swiglu_backward", (x.data_ptr(), dtype, ld, M, n // 2, dy.data_ptr(), ld_dy, xp), dev.index, stream)
    return dx


@functools.lru_cache(maxsize=256)
def quantize_int8_workspace_bytes(n: int, M: int, K: int) -> int:
    """Workspace bytes with which ``quantize_int8`` quantises n rows once for M places, or
    0 where that does not pay."""
    return (_bn._lib or _bn.load()).bn_quantize_int8_workspace_bytes(n, M, K)


def quantize_int8(x, rows=None, offsets=None, data=None, scales=None, workspace=None, stream=None) -> Int8:
    """Rows of ``x`` ([n,K], or [groups,n,K] such as weights, whose rows are the output
    channels; BF16, FP16 or FP32) in 8-bit integers with a scale a row.  ``rows`` (int32
    [M]) picks the rows; ``offsets`` are kept with the result.  Where many places take
    the same row, rows are quantised once into a ``workspace`` (a 1-D uint8 tensor of
    ``quantize_int8_workspace_bytes``; by default one is allocated for the call) and copied
    from there: the same result."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    lead = None
    if x.dim() == 3:
        if rows is not None or offsets is not None:
            raise ValueError("a 3-D x has equal groups: it takes neither rows nor offsets")
        if not x.is_contiguous():
            raise ValueError("a 3-D x must be contiguous")
        lead = x.shape[:2]
        x = x.view(-1, x.shape[2])
    ld = _rows2d(x, "x")
    n, K = x.shape
    dev = x.device
    dtype = _dtype(x, "x")
    if n <= 1:
        ld = -(-K // 8) * 8
    if offsets is not None:
        _ptr(offsets, "offsets", _INT32, (offsets.numel(),), dev)
    M, rp = _places(x, rows)
    shape = lead if lead is not None else (M,)
    data, dp = _out(data, "data", torch.int8, (*shape, K), dev, stream)
    scales, sp = _out(scales, "scales", _FLOAT32, tuple(shape), dev, stream)
    need = quantize_int8_workspace_bytes(n, M, K) if workspace is None and rp is not None else 0
    wp, wn, workspace = _call_workspace(workspace, need, dev, stream)
    _call("bn_quantize_int8", (x.data_ptr(), dtype, ld, n, rp, M, K, dp, sp, wp, wn), dev.index, stream)
    return Int8(data, scales, offsets)


def _layout_int8(q: Int8, name: str):
    """(rows, K, and the addresses of data and scales) of 8-bit rows, after checks."""
    if not isinstance(q, Int8):
        raise TypeError(f"{name} must be an Int8")
    data = q.data
    shape = data.shape
    if len(shape) not in (2, 3) or (len(shape) == 3 and q.offsets is not None):
        raise ValueError(f"{name}.data must be [M, K], or [groups, rows, K] without offsets")
    dp = _ptr(data, f"{name}.data", torch.int8, shape, data.device)
    sp = _ptr(q.scales, f"{name}.scales", _FLOAT32, shape[:-1], data.device)
    return q.scales.numel(), shape[-1], dp, sp


def dequantize_int8(q: Int8, dtype=torch.bfloat16, out=None, stream=None) -> torch.Tensor:
    """The values of 8-bit rows ([..., K]) in BF16, FP16 or FP32."""
    M, K, dp, sp = _layout_int8(q, "q")
    dev = q.data.device
    out, yp = _out(out, "out", dtype if out is None else out.dtype, q.shape, dev, stream)
    _call("bn_dequantize_int8", (dp, sp, M, K, yp, _dtype(out, "out")), dev.index, stream)
    return out


def product_int8_workspace_bytes(M: int, E: int, N: int, K: int) -> int:
    """Workspace bytes with which ``expert_product`` widens M Int8 rows of K values once
    for E experts of N rows, or 0 where it needs none."""
    return (_bn._lib or _bn.load()).bn_expert_product_int8_workspace_bytes(M, E, N, K)


def _expert_product_int8(a: Int8, w: Int8, scale, out, workspace, stream) -> torch.Tensor:
    M, K, ap, sp = _layout_int8(a, "a")
    _, wK, wp, wsp = _layout_int8(w, "w")
    dev = a.data.device
    if a.data.dim() != 2:
        raise ValueError("a.data must be [M, K]")
    if w.offsets is not None:
        raise ValueError("w must have equal groups (no offsets)")
    if w.data.device != dev:
        raise ValueError(f"w is on {w.data.device}, expected {dev}")
    if wK != K:
        raise ValueError(f"a has rows of {K} values, w of {wK}")
    shape = w.data.shape
    E, N = shape[:2] if len(shape) == 3 else (1, shape[0])
    op = _groups(a.offsets, E, dev)
    out, yp = _out(out, "out", torch.bfloat16, (M, N), dev, stream)
    xp, n, workspace = _call_workspace(workspace, 0 if workspace is not None else product_int8_workspace_bytes(M, E, N, K), dev, stream)
    _call("bn_expert_product_int8", (ap, sp, M, wp, wsp, E, N, K, op, scale, yp, xp, n), dev.index, stream)
    return out
