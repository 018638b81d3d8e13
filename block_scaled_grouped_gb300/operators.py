"""The operators around the grouped GEMM of an expert layer, on torch tensors.

``route`` (softmax top-k) -> ``sort_tokens`` (tokens by expert, rows padded to
128) -> ``dispatch`` (rows quantized into A and SFA) -> the grouped GEMMs ->
``combine`` (rows back to tokens), the dense layers beside the experts
(``linear``), and their gradients.  As in the rest of the binding nothing is
computed here: shapes and types are checked, outputs allocated (on the stream the
call runs on), and the C ABI's entry points called.  ``include/bsgg.h`` states
each operator's formula, layouts and errors.

Tensors of values are torch tensors of bfloat16, float16 or float32 whose last
dimension is contiguous; a row pitch is taken from their strides.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

from . import BsggError, IN_FORMATS, OUT_FORMATS, _check, _ptr, _stream, lib, sf_bytes

ROW_FORMATS = {**IN_FORMATS, "f16": 6}
ACTIVATIONS = {"none": 0, "relu": 1, "srelu": 2, "silu": 3, "gelu": 4}


class RouteDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("ld", ctypes.c_int64), ("num_experts", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("logit_format", ctypes.c_int32), ("normalize", ctypes.c_int32)]


class TokensDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("hidden", ctypes.c_int64), ("m_pad", ctypes.c_int64),
                ("ld_token", ctypes.c_int64), ("ld_residual", ctypes.c_int64), ("topk", ctypes.c_int32),
                ("token_format", ctypes.c_int32), ("row_format", ctypes.c_int32), ("d_format", ctypes.c_int32)]


class LinearDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("m", "n", "k", "ldx", "ldw", "ld_residual", "ldy", "ldz")] + \
               [(n, ctypes.c_int32) for n in ("in_format", "out_format", "bias_format", "activation")]


class LinearBwdDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("m", "n", "k", "ld_dy", "ldz", "ld_dz", "ldx", "ldw", "ld_dx", "ld_dw")] + \
               [(n, ctypes.c_int32) for n in ("in_format", "dx_format", "dw_format", "activation", "accumulate_dw")]


class TokenMap(NamedTuple):
    """bsgg_sort_tokens' outputs: padded_offsets (num_experts), row_of_slot
    (tokens, topk), slot_of_row (m_pad), prob (m_pad) and rows_used (1)."""
    padded_offsets: "object"
    row_of_slot: "object"
    slot_of_row: "object"
    prob: "object"
    rows_used: "object"


def bind(L) -> None:
    """ctypes signatures of the operators' entry points."""
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    L.bsgg_route.argtypes = [ctypes.POINTER(RouteDesc)] + [vp] * 4
    L.bsgg_route_backward.argtypes = [ctypes.POINTER(RouteDesc)] + [vp] * 5 + [i64, vp, vp]
    L.bsgg_sort_rows.restype, L.bsgg_sort_rows.argtypes = i64, [i64, i32]
    L.bsgg_sort_workspace_bytes.restype, L.bsgg_sort_workspace_bytes.argtypes = ctypes.c_uint64, [i64, i32]
    L.bsgg_sort_tokens.argtypes = [i64, i32, i64] + [vp] * 10
    L.bsgg_dispatch.argtypes = [ctypes.POINTER(TokensDesc)] + [vp] * 6
    L.bsgg_combine.argtypes = [ctypes.POINTER(TokensDesc)] + [vp] * 6
    L.bsgg_combine_backward.argtypes = [ctypes.POINTER(TokensDesc)] + [vp] * 9
    L.bsgg_linear.argtypes = [ctypes.POINTER(LinearDesc)] + [vp] * 8
    L.bsgg_linear_backward.argtypes = [ctypes.POINTER(LinearBwdDesc)] + [vp] * 10
    L.bsgg_query_status_word.argtypes = [vp, vp]
    for name in ("bsgg_route", "bsgg_route_backward", "bsgg_sort_tokens", "bsgg_dispatch", "bsgg_combine",
                 "bsgg_combine_backward", "bsgg_linear", "bsgg_linear_backward", "bsgg_query_status_word"):
        getattr(L, name).restype = ctypes.c_int


# ---------------------------------------------------------------- arguments
_formats = None


def _format(t, what: str) -> int:
    """The ABI's code of a tensor's type."""
    global _formats
    if _formats is None:
        import torch
        _formats = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
    code = _formats.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: bfloat16, float16 or float32 expected, got {t.dtype}")
    return code


def _dtype(name: str):
    import torch
    d = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}.get(name)
    if d is None:
        raise ValueError(f"format: bf16, f16 or f32 expected, got {name!r}")
    return d


def _matrix(t, what: str, rows=None, cols=None, dtype=None):
    """A CUDA matrix with contiguous rows of the given shape; its row pitch."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{what}: a CUDA matrix expected, got {tuple(t.shape)} on {t.device}")
    if (rows is not None and t.shape[0] != rows) or (cols is not None and t.shape[1] != cols):
        raise ValueError(f"{what}: ({rows}, {cols}) expected, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: rows must be contiguous (strides {t.stride()})")
    if t.shape[0] <= 1:
        return -(-t.shape[1] // 8) * 8       # no second row: any pitch will do
    if t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}: rows must not overlap (strides {t.stride()})")
    return t.stride(0)


def _flat(t, what: str, numel: int, dtype_name: str):
    """A contiguous CUDA tensor of int32 or float32 values (None passes)."""
    import torch
    if t is None:
        return None
    if not t.is_cuda or t.dtype != getattr(torch, dtype_name) or t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{what}: {numel} contiguous {dtype_name} values on the GPU expected, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t


def _on(stream):
    """Allocations of the body belong to `stream` (None: torch's current one)."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


_status_words = {}


def _status(device):
    """The device's status word that calls without one of their own share."""
    import torch
    w = _status_words.get(device)
    if w is None:
        w = _status_words[device] = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.synchronize(device)
    return w


def operators_status(stream=None, status=None) -> int:
    """Synchronize and read/clear the status word of sort_tokens, linear and
    linear_backward on the current device (0 = ok)."""
    import torch
    w = status if status is not None else _status(torch.device("cuda", torch.cuda.current_device()))
    return int(lib().bsgg_query_status_word(_ptr(w), _stream(stream)))


# ---------------------------------------------------------------- routing
def _route_desc(logits, topk: int, normalize: bool):
    ld = _matrix(logits, "logits")
    return RouteDesc(logits.shape[0], ld, logits.shape[1], int(topk), _format(logits, "logits"), int(bool(normalize)))


def route(logits, topk: int, normalize: bool = True, ids=None, weights=None, stream=None):
    """Softmax top-k of (tokens, experts) logits: (ids int32, weights float32),
    each (tokens, topk)."""
    import torch
    desc = _route_desc(logits, topk, normalize)
    n = logits.shape[0] * int(topk)
    with _on(stream):
        if ids is None:
            ids = torch.empty(logits.shape[0], int(topk), dtype=torch.int32, device=logits.device)
        if weights is None:
            weights = torch.empty(logits.shape[0], int(topk), dtype=torch.float32, device=logits.device)
    _flat(ids, "ids", n, "int32"), _flat(weights, "weights", n, "float32")
    _check(lib().bsgg_route(ctypes.byref(desc), _ptr(logits), _ptr(ids), _ptr(weights), _stream(stream)), "bsgg_route")
    return ids, weights


def route_backward(logits, ids, weights, dweights, normalize: bool = True, row_of_slot=None, dlogits=None, stream=None):
    """Gradient of route with respect to the logits, in their type.  dweights is
    (tokens, topk), or with row_of_slot a per-row gradient (the backward GEMM's
    dprob)."""
    import torch
    if ids.dim() != 2 or ids.shape[0] != logits.shape[0]:
        raise ValueError(f"ids: (tokens, topk) expected, got {tuple(ids.shape)}")
    desc = _route_desc(logits, ids.shape[1], normalize)
    n = ids.numel()
    _flat(ids, "ids", n, "int32"), _flat(weights, "weights", n, "float32")
    _flat(row_of_slot, "row_of_slot", n, "int32")
    _flat(dweights, "dweights", dweights.numel() if row_of_slot is not None else n, "float32")
    with _on(stream):
        if dlogits is None:
            # the logits' pitch, so that one desc serves both
            dlogits = torch.empty(logits.shape[0], desc.ld, dtype=logits.dtype, device=logits.device)[:, :logits.shape[1]]
    if _matrix(dlogits, "dlogits", *logits.shape, dtype=logits.dtype) != desc.ld:
        raise ValueError("dlogits: the logits' row pitch expected")
    _check(lib().bsgg_route_backward(ctypes.byref(desc), _ptr(logits), _ptr(ids), _ptr(weights), _ptr(dweights),
                                     _ptr(row_of_slot), dweights.numel() if row_of_slot is not None else 0, _ptr(dlogits),
                                     _stream(stream)), "bsgg_route_backward")
    return dlogits


# ---------------------------------------------------------------- tokens <-> rows
def sort_rows(slots: int, num_experts: int) -> int:
    """An m_pad that holds `slots` routed choices however they fall."""
    m = int(lib().bsgg_sort_rows(slots, num_experts))
    if m < 0:
        raise BsggError(1, "bsgg_sort_rows")
    return m


def sort_tokens(ids, num_experts: int, m_pad: Optional[int] = None, weights=None, status=None, stream=None) -> TokenMap:
    """Tokens by expert: ids (tokens, topk) int32 -> TokenMap.  m_pad: rows to lay
    out, by default sort_rows(ids.numel(), num_experts); pass the value of
    rows_used read back to the host for the least."""
    import torch
    n = ids.numel()
    if ids.dim() != 2:
        raise ValueError(f"ids: (tokens, topk) expected, got {tuple(ids.shape)}")
    _flat(ids, "ids", n, "int32"), _flat(weights, "weights", n, "float32")
    if m_pad is None:
        m_pad = sort_rows(n, num_experts)
    L = lib()
    nws = int(L.bsgg_sort_workspace_bytes(n, num_experts))
    with _on(stream):
        i32 = dict(dtype=torch.int32, device=ids.device)
        # one allocation: offsets, rows_used, slots, rows, workspace
        buf = torch.empty(num_experts + 1 + n + max(m_pad, 0) + nws // 4, **i32)
        prob = torch.empty(max(m_pad, 0), dtype=torch.float32, device=ids.device)
    offsets, used, row_of_slot, slot_of_row, ws = buf.split([num_experts, 1, n, max(m_pad, 0), nws // 4])
    status = _status(ids.device) if status is None else status
    _check(L.bsgg_sort_tokens(n, num_experts, m_pad, _ptr(ids), _ptr(weights), _ptr(offsets), _ptr(row_of_slot),
                              _ptr(slot_of_row), _ptr(prob), _ptr(used), _ptr(ws) if nws else None, _ptr(status),
                              _stream(stream)), "bsgg_sort_tokens")
    return TokenMap(offsets, row_of_slot.view(ids.shape), slot_of_row, prob, used)


def _row_buffers(m_pad: int, hidden: int, row_format: str, device):
    """Buffers of rows and scale factors: uint8 codes, or 16-bit values."""
    import torch
    if row_format in ("bf16", "f16"):
        return torch.empty(m_pad, hidden, dtype=_dtype(row_format), device=device), None
    fp4 = row_format in ("nvfp4", "fp4_ue8m0_16", "mxfp4")
    v = 16 if row_format in ("nvfp4", "fp4_ue8m0_16") else 32
    a = torch.empty(m_pad, hidden // 2 if fp4 else hidden, dtype=torch.uint8, device=device)
    return a, torch.empty(sf_bytes(m_pad, hidden, v), dtype=torch.uint8, device=device)


def _row_format(name: str) -> int:
    if name not in ROW_FORMATS:
        raise ValueError(f"row format: one of {sorted(ROW_FORMATS)} expected, got {name!r}")
    return ROW_FORMATS[name]


def _maps(row_of_slot, slot_of_row, tokens: int):
    if row_of_slot.dim() != 2 or row_of_slot.shape[0] != tokens:
        raise ValueError(f"row_of_slot: ({tokens}, topk) expected, got {tuple(row_of_slot.shape)}")
    _flat(row_of_slot, "row_of_slot", row_of_slot.numel(), "int32")
    if slot_of_row is not None:
        _flat(slot_of_row, "slot_of_row", slot_of_row.numel(), "int32")


def dispatch(x, row_of_slot, slot_of_row, in_format: str = "mxfp8_e4m3", stream=None):
    """Tokens x (tokens, hidden) into the grouped GEMM's A and SFA: (a, sfa);
    a is uint8 codes ((m_pad, hidden), FP4 packed) with the swizzled scale codes
    sfa, or bfloat16 / float16 values with sfa None."""
    ld = _matrix(x, "x")
    T, H = x.shape
    _maps(row_of_slot, slot_of_row, T)
    m_pad = slot_of_row.numel()
    desc = TokensDesc(T, H, m_pad, ld, 0, row_of_slot.shape[1], _format(x, "x"), _row_format(in_format), 0)
    with _on(stream):
        a, sfa = _row_buffers(m_pad, H, in_format, x.device)
    _check(lib().bsgg_dispatch(ctypes.byref(desc), _ptr(x), _ptr(row_of_slot), _ptr(slot_of_row), _ptr(a), _ptr(sfa),
                               _stream(stream)), "bsgg_dispatch")
    return a, sfa


def combine(d, row_of_slot, weights=None, residual=None, out_format: Optional[str] = None, out=None, stream=None):
    """Rows d (m_pad, hidden) back to tokens: residual + sum_j weights[t, j] *
    d[row_of_slot[t, j]], (tokens, hidden) in out_format (by default the
    residual's type, or d's)."""
    import torch
    _matrix(d, "d")
    if not d.is_contiguous():
        raise ValueError("d: a contiguous matrix expected")
    m_pad, H = d.shape
    T = row_of_slot.shape[0]
    _maps(row_of_slot, None, T)
    _flat(weights, "weights", row_of_slot.numel(), "float32")
    dt = _dtype(out_format) if out_format is not None else residual.dtype if residual is not None else d.dtype
    ldr = _matrix(residual, "residual", T, H, dt) if residual is not None else 0
    with _on(stream):
        y = out if out is not None else torch.empty(T, H, dtype=dt, device=d.device)
    ldy = _matrix(y, "out", T, H, dt)
    desc = TokensDesc(T, H, m_pad, ldy, ldr, row_of_slot.shape[1], _format(y, "out"), 0, _format(d, "d"))
    _check(lib().bsgg_combine(ctypes.byref(desc), _ptr(d), _ptr(row_of_slot), _ptr(weights), _ptr(residual), _ptr(y),
                              _stream(stream)), "bsgg_combine")
    return y


def combine_backward(dy, d, row_of_slot, slot_of_row, weights=None, out_format: str = "bf16", want_dweights: bool = True,
                     stream=None):
    """Gradient of combine: (dd, sfd, dweights); dd (m_pad, hidden) in the row
    format out_format with its scale factors sfd (None for bf16 and f16)."""
    import torch
    ld = _matrix(dy, "dy")
    T, H = dy.shape
    _maps(row_of_slot, slot_of_row, T)
    m_pad = slot_of_row.numel()
    _flat(weights, "weights", row_of_slot.numel(), "float32")
    if want_dweights:
        _matrix(d, "d", m_pad, H)
        if not d.is_contiguous():
            raise ValueError("d: a contiguous matrix expected")
    desc = TokensDesc(T, H, m_pad, ld, 0, row_of_slot.shape[1], _format(dy, "dy"), _row_format(out_format),
                      _format(d, "d") if want_dweights else 0)
    with _on(stream):
        dd, sfd = _row_buffers(m_pad, H, out_format, dy.device)
        dw = torch.empty(row_of_slot.shape, dtype=torch.float32, device=dy.device) if want_dweights else None
    _check(lib().bsgg_combine_backward(ctypes.byref(desc), _ptr(dy), _ptr(d) if want_dweights else None, _ptr(row_of_slot),
                                       _ptr(slot_of_row), _ptr(weights), _ptr(dd), _ptr(sfd), _ptr(dw), _stream(stream)),
           "bsgg_combine_backward")
    return dd, sfd, dw


# ---------------------------------------------------------------- dense layer
def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation: one of {sorted(ACTIVATIONS)} expected, got {name!r}")
    return ACTIVATIONS[name]


def _rows_of(cols: int, rows: int, dtype, device):
    """An empty matrix whose row pitch is a multiple of 8 elements."""
    import torch
    ld = -(-cols // 8) * 8
    return torch.empty(rows, ld, dtype=dtype, device=device)[:, :cols]


def linear(x, w, bias=None, activation: str = "none", residual=None, want_z: bool = False,
           out_format: Optional[str] = None, out=None, status=None, stream=None):
    """act(x w^T + bias) + residual: x (m, k), w (n, k) bfloat16 or float16,
    bias (n), residual (m, n) in x's type -> (y, z); z, the pre-activation in
    x's type, is None unless want_z."""
    import torch
    ldx = _matrix(x, "x")
    m, k = x.shape
    ldw = _matrix(w, "w", None, k, x.dtype)
    n = w.shape[0]
    dt = _dtype(out_format) if out_format is not None else x.dtype
    if bias is not None and (bias.dim() != 1 or bias.numel() != n or not bias.is_contiguous() or not bias.is_cuda):
        raise ValueError(f"bias: {n} contiguous values on the GPU expected, got {tuple(bias.shape)}")
    ldr = _matrix(residual, "residual", m, n, x.dtype) if residual is not None else 0
    with _on(stream):
        y = out if out is not None else torch.empty(m, n, dtype=dt, device=x.device)
        z = _rows_of(n, m, x.dtype, x.device) if want_z else None
    ldy = _matrix(y, "out", m, n, dt)
    desc = LinearDesc(m, n, k, ldx, ldw, ldr, ldy, _matrix(z, "z") if want_z else 0, _format(x, "x"), _format(y, "out"),
                      _format(bias, "bias") if bias is not None else 0, _activation(activation))
    status = _status(x.device) if status is None else status
    _check(lib().bsgg_linear(ctypes.byref(desc), _ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y), _ptr(z),
                             _ptr(status), _stream(stream)), "bsgg_linear")
    return y, z


def linear_backward(dy, x, w, z=None, activation: str = "none", want_dx: bool = True, want_dw: bool = True,
                    want_dbias: bool = False, dx_format: Optional[str] = None, dw_format: Optional[str] = None, dw=None,
                    status=None, stream=None):
    """Gradient of linear: (dx, dw, dbias), each None where not wanted.  z is the
    pre-activation linear kept (None without an activation).  A given dw is
    added to."""
    import torch
    ld_dy = _matrix(dy, "dy")
    m, n = dy.shape
    ldx = _matrix(x, "x", m, None, dy.dtype)
    k = x.shape[1]
    ldw = _matrix(w, "w", n, k, dy.dtype)
    act = _activation(activation)
    accumulate = dw is not None
    with _on(stream):
        dz = _rows_of(n, m, dy.dtype, dy.device) if act else None
        dx = torch.empty(m, k, dtype=_dtype(dx_format) if dx_format else dy.dtype, device=dy.device) if want_dx else None
        if want_dw and dw is None:
            dw = torch.empty(n, k, dtype=_dtype(dw_format) if dw_format else dy.dtype, device=dy.device)
        dbias = torch.empty(n, dtype=torch.float32, device=dy.device) if want_dbias else None
    if not want_dw:
        dw = None
    if act and z is None:
        raise ValueError("z: the pre-activation is needed for an activation's gradient")
    desc = LinearBwdDesc(m, n, k, ld_dy, _matrix(z, "z", m, n, dy.dtype) if act else 0, _matrix(dz, "dz") if act else 0,
                         ldx, ldw, _matrix(dx, "dx") if want_dx else 0,
                         _matrix(dw, "dw", n, k) if dw is not None else 0, _format(dy, "dy"),
                         _format(dx, "dx") if want_dx else 0, _format(dw, "dw") if dw is not None else 0, act,
                         int(accumulate and want_dw))
    status = _status(dy.device) if status is None else status
    _check(lib().bsgg_linear_backward(ctypes.byref(desc), _ptr(dy), _ptr(x), _ptr(w), _ptr(z) if act else None, _ptr(dz),
                                      _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(status), _stream(stream)),
           "bsgg_linear_backward")
    return dx, dw, dbias
