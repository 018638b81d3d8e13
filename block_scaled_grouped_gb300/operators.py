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

import ctypes
import threading
from ctypes import byref
from typing import NamedTuple, Optional

import torch

from . import BsggError, IN_FORMATS, _check, _stream, lib

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
# A decode step's kernels take a few microseconds, so the host's share of a call
# counts: types and shapes are looked at once, through the cheapest calls torch has.
_FORMATS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8


def _format(t, what: str) -> int:
    """The ABI's code of a tensor's type."""
    code = _FORMATS.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: bfloat16, float16 or float32 expected, got {t.dtype}")
    return code


def _dtype(name: str):
    d = _DTYPES.get(name)
    if d is None:
        raise ValueError(f"format: bf16, f16 or f32 expected, got {name!r}")
    return d


def _matrix(t, what: str, rows=None, cols=None, dtype=None):
    """A CUDA matrix with contiguous rows of the given shape; its row pitch."""
    shape = t.shape
    if len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{what}: a CUDA matrix expected, got {tuple(shape)} on {t.device}")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{what}: ({rows}, {cols}) expected, got {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    pitch, step = t.stride()
    if c > 1 and step != 1:
        raise ValueError(f"{what}: rows must be contiguous (strides {t.stride()})")
    if r <= 1:
        return (c + 7) // 8 * 8              # no second row: any pitch will do
    if pitch < c:
        raise ValueError(f"{what}: rows must not overlap (strides {t.stride()})")
    return pitch


def _flat(t, what: str, numel: int, dtype):
    """The address of a contiguous CUDA tensor of `numel` int32 or float32
    values (None passes)."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != numel or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: {numel} contiguous {dtype} values on the GPU expected, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


_empty = torch.empty


def _empty_on(stream):
    """torch.empty whose memory belongs to `stream` (None: torch's current one)."""
    if stream is None:
        return _empty
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)

    def empty(*shape, **kw):
        with torch.cuda.stream(stream):
            return _empty(*shape, **kw)
    return empty


def _handle(stream, t, *others):
    """The stream's handle; the tensors (None: absent) have to be on the current device."""
    dev = t.get_device()
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError(f"tensors on {t.device} and {o.device}: one device expected")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{dev}, but cuda:{torch._C._cuda_getDevice()} is the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


_status_words = {}
_status_lock = threading.Lock()


def _status_of(t, status):
    """The address of the given status word, or of the one that calls without one
    share on t's device."""
    if status is not None:
        return _flat(status, "status", 1, _I32)
    dev = t.get_device()
    w = _status_words.get(dev)
    if w is None:
        # one word per device for good: kernels hold its address
        with _status_lock:
            w = _status_words.get(dev)
            if w is None:
                word = torch.zeros(1, dtype=_I32, device=t.device)
                torch.cuda.synchronize(t.device)
                w = _status_words[dev] = (word, word.data_ptr())
    return w[1]


def operators_status(stream=None, status=None) -> int:
    """Synchronize and read/clear the status word of sort_tokens, linear and
    linear_backward on the current device (0 = ok).  The word that calls without one
    share is read after all the device's work; a given `status` after `stream`'s."""
    if status is None:
        w = _status_words.get(torch.cuda.current_device())
        if w is None:                        # nothing has run here
            return 0
        torch.cuda.synchronize()             # any stream's kernels may report to it
        status = w[0]
    return int(lib().bsgg_query_status_word(status.data_ptr(), _stream(stream)))


# ---------------------------------------------------------------- routing
def route(logits, topk: int, normalize: bool = True, ids=None, weights=None, stream=None):
    """Softmax top-k of (tokens, experts) logits: (ids int32, weights float32),
    each (tokens, topk)."""
    ld = _matrix(logits, "logits")
    T, L = logits.shape
    k = int(topk)
    desc = RouteDesc(T, ld, L, k, _format(logits, "logits"), 1 if normalize else 0)
    handle = _handle(stream, logits, ids, weights)
    if ids is None or weights is None:
        empty, dev = _empty_on(stream), logits.device
        if ids is None:
            ids = empty((T, max(k, 0)), dtype=_I32, device=dev)
        if weights is None:
            weights = empty((T, max(k, 0)), dtype=_F32, device=dev)
    _check(lib().bsgg_route(byref(desc), logits.data_ptr(), _flat(ids, "ids", T * k, _I32),
                            _flat(weights, "weights", T * k, _F32), handle), "bsgg_route")
    return ids, weights


def route_backward(logits, ids, weights, dweights, normalize: bool = True, row_of_slot=None, dlogits=None, stream=None):
    """Gradient of route with respect to the logits, in their type.  dweights is
    (tokens, topk), or with row_of_slot a per-row gradient (the backward GEMM's
    dprob)."""
    ld = _matrix(logits, "logits")
    T, L = logits.shape
    if ids.dim() != 2 or ids.shape[0] != T:
        raise ValueError(f"ids: ({T}, topk) expected, got {tuple(ids.shape)}")
    n = ids.numel()
    rows = 0 if row_of_slot is None else dweights.numel()
    desc = RouteDesc(T, ld, L, ids.shape[1], _format(logits, "logits"), 1 if normalize else 0)
    handle = _handle(stream, logits, ids, weights, dweights, row_of_slot, dlogits)
    if dlogits is None:
        # the logits' pitch, so that one desc serves both
        dlogits = _empty_on(stream)((T, ld), dtype=logits.dtype, device=logits.device)
        if ld != L:
            dlogits = dlogits[:, :L]
    elif _matrix(dlogits, "dlogits", T, L, logits.dtype) != ld:
        raise ValueError("dlogits: the logits' row pitch expected")
    _check(lib().bsgg_route_backward(byref(desc), logits.data_ptr(), _flat(ids, "ids", n, _I32),
                                     _flat(weights, "weights", n, _F32), _flat(dweights, "dweights", rows or n, _F32),
                                     _flat(row_of_slot, "row_of_slot", n, _I32), rows, dlogits.data_ptr(), handle),
           "bsgg_route_backward")
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
    n = ids.numel()
    if ids.dim() != 2:
        raise ValueError(f"ids: (tokens, topk) expected, got {tuple(ids.shape)}")
    p_ids, p_weights = _flat(ids, "ids", n, _I32), _flat(weights, "weights", n, _F32)
    if m_pad is None:
        m_pad = sort_rows(n, num_experts)
    L = lib()
    nws = L.bsgg_sort_workspace_bytes(n, num_experts) // 4
    handle = _handle(stream, ids, weights, status)
    empty, dev = _empty_on(stream), ids.device
    m, e = max(m_pad, 0), max(num_experts, 0)
    # a tensor each (a view of a larger one costs the host as much as an allocation)
    i32 = {"dtype": _I32, "device": dev}
    offsets, used, row_of_slot, slot_of_row = empty(e, **i32), empty(1, **i32), empty(ids.shape, **i32), empty(m, **i32)
    prob = empty(m, dtype=_F32, device=dev)
    ws = empty(nws, **i32) if nws else None
    _check(L.bsgg_sort_tokens(n, num_experts, m_pad, p_ids, p_weights, offsets.data_ptr(), row_of_slot.data_ptr(),
                              slot_of_row.data_ptr(), prob.data_ptr(), used.data_ptr(),
                              ws.data_ptr() if nws else None, _status_of(ids, status), handle), "bsgg_sort_tokens")
    return TokenMap(offsets, row_of_slot, slot_of_row, prob, used)


def _row_buffers(m_pad: int, hidden: int, row_format: str, device, empty):
    """Buffers of rows and scale factors: uint8 codes, or 16-bit values."""
    if row_format in ("bf16", "f16"):
        return empty((m_pad, hidden), dtype=_DTYPES[row_format], device=device), None
    v = 16 if row_format in ("nvfp4", "fp4_ue8m0_16") else 32
    a = empty((m_pad, hidden // 2 if row_format in _FP4 else hidden), dtype=_U8, device=device)
    # bsgg_sf_bytes(m_pad, hidden, v, 1), without the call
    blocks = (hidden + v - 1) // v
    return a, empty(((m_pad + 127) // 128) * ((blocks + 3) // 4) * 512, dtype=_U8, device=device)


_FP4 = ("nvfp4", "fp4_ue8m0_16", "mxfp4")


def _row_format(name: str) -> int:
    f = ROW_FORMATS.get(name)
    if f is None:
        raise ValueError(f"row format: one of {sorted(ROW_FORMATS)} expected, got {name!r}")
    return f


def _slots_of(row_of_slot, tokens: int):
    """topk and the address of a (tokens, topk) map."""
    shape = row_of_slot.shape
    if len(shape) != 2 or shape[0] != tokens:
        raise ValueError(f"row_of_slot: ({tokens}, topk) expected, got {tuple(shape)}")
    k = shape[1]
    return k, _flat(row_of_slot, "row_of_slot", tokens * k, _I32)


def _rows_matrix(d, rows, cols):
    _matrix(d, "d", rows, cols)
    if not d.is_contiguous():
        raise ValueError("d: a contiguous matrix expected")


def dispatch(x, row_of_slot, slot_of_row, in_format: str = "mxfp8_e4m3", stream=None):
    """Tokens x (tokens, hidden) into the grouped GEMM's A and SFA: (a, sfa);
    a is uint8 codes ((m_pad, hidden), FP4 packed) with the swizzled scale codes
    sfa, or bfloat16 / float16 values with sfa None."""
    ld = _matrix(x, "x")
    T, H = x.shape
    k, p_rows = _slots_of(row_of_slot, T)
    m_pad = slot_of_row.numel()
    p_slots = _flat(slot_of_row, "slot_of_row", m_pad, _I32)
    desc = TokensDesc(T, H, m_pad, ld, 0, k, _format(x, "x"), _row_format(in_format), 0)
    handle = _handle(stream, x, row_of_slot, slot_of_row)
    a, sfa = _row_buffers(m_pad, H, in_format, x.device, _empty_on(stream))
    _check(lib().bsgg_dispatch(byref(desc), x.data_ptr(), p_rows, p_slots, a.data_ptr(),
                               sfa.data_ptr() if sfa is not None else None, handle), "bsgg_dispatch")
    return a, sfa


def combine(d, row_of_slot, weights=None, residual=None, out_format: Optional[str] = None, out=None, stream=None):
    """Rows d (m_pad, hidden) back to tokens: residual + sum_j weights[t, j] *
    d[row_of_slot[t, j]], (tokens, hidden) in out_format (by default the
    residual's type, or d's)."""
    _rows_matrix(d, None, None)
    m_pad, H = d.shape
    T = row_of_slot.shape[0]
    k, p_rows = _slots_of(row_of_slot, T)
    dt = _dtype(out_format) if out_format is not None else residual.dtype if residual is not None else d.dtype
    ldr = _matrix(residual, "residual", T, H, dt) if residual is not None else 0
    handle = _handle(stream, d, row_of_slot, weights, residual, out)
    if out is None:
        y, ldy = _empty_on(stream)((T, H), dtype=dt, device=d.device), H
    else:
        y, ldy = out, _matrix(out, "out", T, H, dt)
    desc = TokensDesc(T, H, m_pad, ldy, ldr, k, _format(y, "out"), 0, _format(d, "d"))
    _check(lib().bsgg_combine(byref(desc), d.data_ptr(), p_rows, _flat(weights, "weights", T * k, _F32),
                              residual.data_ptr() if residual is not None else None, y.data_ptr(), handle), "bsgg_combine")
    return y


def combine_backward(dy, d, row_of_slot, slot_of_row, weights=None, out_format: str = "bf16", want_dweights: bool = True,
                     stream=None, want_dd: bool = True):
    """Gradient of combine: (dd, sfd, dweights); dd (m_pad, hidden) in the row
    format out_format with its scale factors sfd (None for bf16 and f16).  dd and
    dweights are None where not wanted."""
    ld = _matrix(dy, "dy")
    T, H = dy.shape
    k, p_rows = _slots_of(row_of_slot, T)
    m_pad = slot_of_row.numel()
    p_slots, p_weights = _flat(slot_of_row, "slot_of_row", m_pad, _I32), _flat(weights, "weights", T * k, _F32)
    p_d, fd = None, 0
    if want_dweights:
        _rows_matrix(d, m_pad, H)
        p_d, fd = d.data_ptr(), _format(d, "d")
    desc = TokensDesc(T, H, m_pad, ld, 0, k, _format(dy, "dy"), _row_format(out_format), fd)
    handle = _handle(stream, dy, d if want_dweights else None, row_of_slot, slot_of_row, weights)
    empty, dev = _empty_on(stream), dy.device
    dd, sfd = _row_buffers(m_pad, H, out_format, dev, empty) if want_dd else (None, None)
    dw = empty((T, k), dtype=_F32, device=dev) if want_dweights else None
    _check(lib().bsgg_combine_backward(byref(desc), dy.data_ptr(), p_d, p_rows, p_slots, p_weights,
                                       *(v.data_ptr() if v is not None else None for v in (dd, sfd, dw)), handle), "bsgg_combine_backward")
    return dd, sfd, dw


# ---------------------------------------------------------------- dense layer
def _activation(name: str) -> int:
    a = ACTIVATIONS.get(name)
    if a is None:
        raise ValueError(f"activation: one of {sorted(ACTIVATIONS)} expected, got {name!r}")
    return a


def _rows_of(rows: int, cols: int, dtype, device, empty):
    """An empty matrix whose row pitch is a multiple of 8 elements, and that pitch."""
    ld = (cols + 7) // 8 * 8
    t = empty((rows, ld), dtype=dtype, device=device)
    return (t if ld == cols else t[:, :cols]), ld


def linear(x, w, bias=None, activation: str = "none", residual=None, want_z: bool = False,
           out_format: Optional[str] = None, out=None, status=None, stream=None):
    """act(x w^T + bias) + residual: x (m, k), w (n, k) bfloat16 or float16,
    bias (n), residual (m, n) in x's type -> (y, z); z, the pre-activation in
    x's type, is None unless want_z."""
    xt = x.dtype
    ldx = _matrix(x, "x")
    m, k = x.shape
    ldw = _matrix(w, "w", None, k, xt)
    n = w.shape[0]
    p_bias, fb, p_res, ldr, z, p_z, ldz = None, 0, None, 0, None, None, 0
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != n or not bias.is_contiguous() or not bias.is_cuda:
            raise ValueError(f"bias: {n} contiguous values on the GPU expected, got {tuple(bias.shape)}")
        p_bias, fb = bias.data_ptr(), _format(bias, "bias")
    if residual is not None:
        p_res, ldr = residual.data_ptr(), _matrix(residual, "residual", m, n, xt)
    dt = xt if out_format is None else _dtype(out_format)
    handle = _handle(stream, x, w, bias, residual, out, status)
    empty = _empty_on(stream)
    if out is None:
        y, ldy = empty((m, n), dtype=dt, device=x.device), n
    else:
        y, ldy = out, _matrix(out, "out", m, n, dt)
    if want_z:
        z, ldz = _rows_of(m, n, xt, x.device, empty)
        p_z = z.data_ptr()
    desc = LinearDesc(m, n, k, ldx, ldw, ldr, ldy, ldz, _format(x, "x"), _FORMATS[dt], fb, _activation(activation))
    _check(lib().bsgg_linear(byref(desc), x.data_ptr(), w.data_ptr(), p_bias, p_res, y.data_ptr(), p_z,
                             _status_of(x, status), handle), "bsgg_linear")
    return y, z


def linear_backward(dy, x, w, z=None, activation: str = "none", want_dx: bool = True, want_dw: bool = True,
                    want_dbias: bool = False, dx_format: Optional[str] = None, dw_format: Optional[str] = None, dw=None,
                    status=None, stream=None):
    """Gradient of linear: (dx, dw, dbias), each None where not wanted.  z is the
    pre-activation linear kept (None without an activation).  A given dw is
    added to."""
    t = dy.dtype
    ld_dy = _matrix(dy, "dy")
    m, n = dy.shape
    ldx = _matrix(x, "x", m, None, t)
    k = x.shape[1]
    ldw = _matrix(w, "w", n, k, t)
    act = _activation(activation)
    handle = _handle(stream, dy, x, w, z if act else None, dw if want_dw else None, status)
    empty, dev = _empty_on(stream), dy.device
    dz = dx = dbias = p_z = None
    ldz = ld_dz = ld_dx = ld_dw = fx = fw = 0
    if act:
        if z is None:
            raise ValueError("z: the pre-activation is needed for an activation's gradient")
        p_z, ldz = z.data_ptr(), _matrix(z, "z", m, n, t)
        dz, ld_dz = _rows_of(m, n, t, dev, empty)
    if want_dx:
        dx, ld_dx = empty((m, k), dtype=_dtype(dx_format) if dx_format else t, device=dev), k
        fx = _format(dx, "dx")
    accumulate = 0
    if not want_dw:
        dw = None
    else:
        if dw is None:
            dw, ld_dw = empty((n, k), dtype=_dtype(dw_format) if dw_format else t, device=dev), k
        else:
            accumulate, ld_dw = 1, _matrix(dw, "dw", n, k)
        fw = _format(dw, "dw")
    if want_dbias:
        dbias = empty(n, dtype=_F32, device=dev)
    desc = LinearBwdDesc(m, n, k, ld_dy, ldz, ld_dz, ldx, ldw, ld_dx, ld_dw, _format(dy, "dy"), fx, fw, act, accumulate)
    _check(lib().bsgg_linear_backward(byref(desc), dy.data_ptr(), x.data_ptr(), w.data_ptr(), p_z,
                                      *(v.data_ptr() if v is not None else None for v in (dz, dx, dw, dbias)),
                                      _status_of(dy, status), handle), "bsgg_linear_backward")
    return dx, dw, dbias
