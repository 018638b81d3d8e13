"""What the router with scores and groups, the RMS norm and the adapters refuse,
without a GPU, and their references' gradients against differences."""
import ctypes
import math
import os
import re

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
import layer_operator_refs as R
from block_scaled_grouped_gb300 import build as bsgg_build
from block_scaled_grouped_gb300 import operators as ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bsgg.h")
P = ctypes.c_void_p(4096)        # never dereferenced: refused first
Q = ctypes.c_void_p(8192)
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsgg_build.build()
    return bsgg.lib()


@pytest.mark.parametrize("struct,cls", [("bsgg_route_groups_desc", ops.RouteGroupsDesc), ("bsgg_norm_desc", ops.NormDesc),
                                        ("bsgg_norm_bwd_desc", ops.NormBwdDesc), ("bsgg_adapters_desc", ops.AdaptersDesc),
                                        ("bsgg_adapters_bwd_desc", ops.AdaptersBwdDesc)])
def test_binding_structs_match_the_header(struct, cls):
    src = open(HEADER).read()
    end = src.index("} " + struct + ";")
    body = re.sub(r"/\*.*?\*/", "", src[src.rindex("typedef struct {", 0, end) + len("typedef struct {"):end], flags=re.S)
    fields = [(t, n.strip()) for t, names in re.findall(r"(int64_t|int32_t|float)\s+([^;]+);", body) for n in names.split(",")]
    ctype = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float}
    assert [(ctype[t], n) for t, n in fields] == [(t, n) for n, t in cls._fields_]


def desc(cls, base, over):
    d = {**base, **over}
    return ctypes.byref(cls(*[d[n] for n, _ in cls._fields_]))


# ------------------------------------------------------------------ routing
ROUTE = dict(tokens=4, ld=16, num_experts=16, topk=2, groups=4, topk_groups=2, group_top=2, score=1, logit_format=2, normalize=1,
             scale=1.0)


def route(lib, ptrs=(P, P, P, P), **over):
    return lib.bsgg_route_groups(desc(ops.RouteGroupsDesc, ROUTE, over), *ptrs, None)


@pytest.mark.parametrize("over", [dict(tokens=-1), dict(tokens=2 ** 31), dict(num_experts=0), dict(num_experts=1028, ld=2000), dict(topk=0),
                                  dict(topk=9), dict(topk=33, num_experts=128, ld=128), dict(ld=15), dict(logit_format=3), dict(groups=0),
                                  dict(groups=3), dict(groups=33, num_experts=33, ld=33), dict(topk_groups=0), dict(topk_groups=5),
                                  dict(group_top=0), dict(group_top=3), dict(score=2), dict(score=-1), dict(normalize=2),
                                  dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan)])
def test_route_groups_refuses(lib, over):
    assert route(lib, **over) == 1


def test_route_groups_refuses_pointers(lib):
    for i in (0, 2, 3):
        assert route(lib, ptrs=tuple(None if j == i else P for j in range(4))) == 1
    for i in range(4):
        assert route(lib, ptrs=tuple(ODD if j == i else P for j in range(4))) == 1
    assert route(lib, tokens=0, ptrs=(None,) * 4) == 0
    assert lib.bsgg_route_groups(None, P, P, P, P, None) == 1
    bw = lambda *a, **o: lib.bsgg_route_groups_backward(desc(ops.RouteGroupsDesc, ROUTE, o), *a, None)  # noqa: E731
    assert bw(P, P, P, None, None, 0, P) == 1
    assert bw(P, P, P, P, P, 0, P) == 1                               # rows without their number
    assert bw(P, P, P, P, None, 0, ODD) == 1
    assert bw(P, P, P, P, None, 0, P, scale=0.0) == 1
    assert bw(None, None, None, None, None, 0, None, tokens=0) == 0


# ------------------------------------------------------------------ norm
NORM = dict(tokens=4, hidden=64, m_pad=128, ld_x=64, ld_residual=64, ld_h=64, ld_y=64, token_format=0, weight_format=0, y_format=0,
            row_format=0, eps=1e-6)
NORM_PTRS = dict(x=P, residual=P, weight=P, h=P, y=P, rstd=P, a=P, sfa=P)


def norm(lib, ptrs=None, **over):
    return lib.bsgg_rms_norm(desc(ops.NormDesc, NORM, over), *{**NORM_PTRS, **(ptrs or {})}.values(), None)


@pytest.mark.parametrize("over", [dict(tokens=-1), dict(hidden=0), dict(hidden=60), dict(hidden=72, ld_x=72, ld_residual=72, ld_h=72, ld_y=72),
                                  dict(hidden=48, row_format=2), dict(ld_x=56), dict(ld_x=68), dict(ld_residual=56), dict(ld_residual=60),
                                  dict(ld_h=56), dict(ld_y=56), dict(ld_y=66), dict(token_format=3), dict(weight_format=-1), dict(y_format=4),
                                  dict(row_format=5), dict(row_format=6), dict(row_format=-1), dict(m_pad=0), dict(m_pad=130),
                                  dict(tokens=129), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan)])
def test_norm_refuses(lib, over):
    assert norm(lib, **over) == 1


def test_norm_refuses_pointers(lib):
    assert norm(lib, dict(x=None)) == 1 and norm(lib, dict(sfa=None)) == 1 and norm(lib, dict(a=None)) == 1
    assert norm(lib, dict(y=None, a=None, sfa=None)) == 1             # nothing wanted
    assert norm(lib, dict(residual=None)) == 1                         # h without a residual
    for name in NORM_PTRS:
        assert norm(lib, {name: ODD}) == 1
    assert norm(lib, hidden=65536, ld_x=65536, ld_residual=65536, ld_h=65536, ld_y=65536) == 2
    assert norm(lib, {n: None for n in NORM_PTRS}, tokens=0) == 0
    assert lib.bsgg_rms_norm(None, *[P] * 8, None) == 1


NORM_BWD = dict(tokens=4, hidden=64, ld_dy=64, ld_h=64, ld_dh=64, ld_dx=64, token_format=0, weight_format=0, y_format=0, reserved=0)


@pytest.mark.parametrize("over", [dict(tokens=-1), dict(hidden=4), dict(hidden=60), dict(ld_dy=60), dict(ld_h=56), dict(ld_dh=56),
                                  dict(ld_dx=56), dict(token_format=3), dict(weight_format=3), dict(y_format=3), dict(reserved=1)])
def test_norm_backward_refuses(lib, over):
    assert lib.bsgg_rms_norm_backward(desc(ops.NormBwdDesc, NORM_BWD, over), *[P] * 8, None) == 1


def test_norm_backward_refuses_pointers(lib):
    bw = lambda *a, **o: lib.bsgg_rms_norm_backward(desc(ops.NormBwdDesc, NORM_BWD, o), *a, None)  # noqa: E731
    for i in (0, 1, 3, 5, 7):                                          # dy, h, rstd, dx, the workspace
        a = [P] * 8
        a[i] = None
        assert bw(*a) == 1, i
    for i in range(8):
        a = [P] * 8
        a[i] = ODD
        assert bw(*a) == 1, i
    assert bw(*[None] * 8, tokens=0) == 0
    assert bw(*[P] * 8, hidden=32776, ld_dy=32776, ld_h=32776, ld_dh=32776, ld_dx=32776) == 2
    assert lib.bsgg_rms_norm_workspace_bytes(-1, 64) == 0 and lib.bsgg_rms_norm_workspace_bytes(4, 64) >= 4 * 64


# ------------------------------------------------------------------ adapters
ADAPT = dict(tokens=4, k=64, n=32, m_pad=128, ldx=64, ld_base=32, ldy=32, adapters=3, rank=16, format=0, reserved=0)


def adapt(lib, ptrs=None, **over):
    ok = dict(x=P, a=P, b=P, scales=P, off=P, row=P, slot=P, base=Q, u=P, y=P)
    return lib.bsgg_adapters(desc(ops.AdaptersDesc, ADAPT, over), *{**ok, **(ptrs or {})}.values(), None)


BAD = [dict(tokens=-1), dict(k=0), dict(k=60, ldx=64), dict(n=0), dict(n=36), dict(m_pad=0), dict(m_pad=100), dict(adapters=0),
       dict(adapters=1025), dict(rank=0), dict(rank=12), dict(rank=136), dict(format=2), dict(format=-1), dict(ldx=56), dict(ldx=66),
       dict(ld_base=24), dict(ld_base=36)]


@pytest.mark.parametrize("over", BAD + [dict(ldy=24), dict(ldy=36), dict(reserved=1)])
def test_adapters_refuses(lib, over):
    assert adapt(lib, **over) == 1


def test_adapters_refuses_pointers(lib):
    for name in ("x", "a", "b", "off", "row", "slot", "u", "y"):
        assert adapt(lib, {name: None}) == 1, name
    for name in ("x", "a", "b", "scales", "off", "row", "slot", "base", "u", "y"):
        assert adapt(lib, {name: ODD}) == 1, name
    assert adapt(lib, dict(base=P), ld_base=40) == 1                   # in place under another pitch
    assert adapt(lib, {n: None for n in ("x", "a", "b", "scales", "off", "row", "slot", "base", "u", "y")}, tokens=0) == 0
    assert lib.bsgg_adapters(None, *[P] * 10, None) == 1


ADAPT_BWD = dict(tokens=4, k=64, n=32, m_pad=128, ld_dy=32, ldx=64, ld_base=64, ld_dx=64, adapters=3, rank=16, format=0, grad_format=2)


def adapt_bwd(lib, ptrs=None, **over):
    ok = dict(dy=P, x=P, u=P, a=P, b=P, scales=P, off=P, row=P, slot=P, used=P, base=Q, du=P, dx=P, da=P, db=P, ws=P)
    return lib.bsgg_adapters_backward(desc(ops.AdaptersBwdDesc, ADAPT_BWD, over), *{**ok, **(ptrs or {})}.values(), None)


@pytest.mark.parametrize("over", [o for o in BAD if "ld_base" not in o] + [dict(ld_dy=24), dict(ld_dy=34), dict(ld_base=56), dict(ld_dx=56),
                                                                           dict(ld_dx=68), dict(grad_format=3), dict(grad_format=-1)])
def test_adapters_backward_refuses(lib, over):
    assert adapt_bwd(lib, **over) == 1


def test_adapters_backward_refuses_pointers(lib):
    for name in ("dy", "x", "u", "a", "b", "off", "row", "slot", "used", "du", "ws"):
        assert adapt_bwd(lib, {name: None}) == 1, name
    for name in ("dy", "x", "u", "a", "b", "scales", "off", "row", "slot", "used", "base", "du", "dx", "da", "db", "ws"):
        assert adapt_bwd(lib, {name: ODD}) == 1, name
    assert adapt_bwd(lib, dict(dx=None, da=None, db=None)) == 1        # nothing wanted
    assert adapt_bwd(lib, dict(ws=None)) == 1 and adapt_bwd(lib, dict(ws=None, da=None)) == 1
    need = lib.bsgg_adapters_workspace_bytes
    assert need(4, 64, 32, 128, 3, 16) > 0 and need(0, 64, 32, 128, 3, 16) == 0 and need(-1, 64, 32, 128, 3, 16) == 0
    # sums of segments on top of the terms, for many tokens
    assert need(100000, 4096, 14336, 2 ** 17, 3, 16) > 6 * 2 ** 17 * 32 + 4 * 16 * 18432
    assert adapt_bwd(lib, dict(base=P), ld_base=72) == 1               # in place under another pitch
    assert adapt_bwd(lib, dict(dy=None, da=None, db=None), tokens=0) == 0


# ------------------------------------------------------------------ binding
def test_binding_refuses_shapes_and_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, 1, dtype=torch.int32)
    tm = bsgg.TokenMap(i, i, i, i, i)
    for call in (lambda: bsgg.route_groups(x, 2), lambda: bsgg.route_groups_backward(x, i, x, x), lambda: bsgg.rms_norm(x),
                 lambda: bsgg.rms_norm_backward(x, x, None, x), lambda: bsgg.adapters(x, w, w, tm),
                 lambda: bsgg.adapters_backward(x, x, x, w, w, tm)):
        with pytest.raises(ValueError):
            call()


class OnGpu:
    """What the binding asks of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), 0

    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


T, H, L, K, M, N, S, r = 4, 64, 8, 2, 128, 16, 3, 8
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
MAP = dict(off=(I32, S), row=(I32, T, 1), slot=(I32, M))
map_of = lambda t: bsgg.TokenMap(t["off"], t["row"], t["slot"], None, t.get("used"))  # noqa: E731
CALLS = {
    "route_groups": (lambda t: bsgg.route_groups(t["logits"], K, bias=t["bias"], ids=t["ids"], weights=t["weights"]),
                     dict(logits=(F32, T, L), bias=(F32, L), ids=(I32, T, K), weights=(F32, T, K))),
    "route_groups_backward": (lambda t: bsgg.route_groups_backward(t["logits"], t["ids"], t["weights"], t["dweights"],
                                                                   row_of_slot=t["row"], dlogits=t["dlogits"]),
                              dict(logits=(F32, T, L), ids=(I32, T, K), weights=(F32, T, K), dweights=(F32, M), row=(I32, T, K),
                                   dlogits=(F32, T, L))),
    "rms_norm": (lambda t: bsgg.rms_norm(t["x"], t["w"], residual=t["res"], h=t["h"]),
                 dict(x=(BF, T, H), w=(BF, H), res=(BF, T, H), h=(BF, T, H))),
    "rms_norm_backward": (lambda t: bsgg.rms_norm_backward(t["dy"], t["h"], t["w"], t["rstd"], dh=t["dh"], dx=t["dx"]),
                          dict(dy=(BF, T, H), h=(BF, T, H), w=(BF, H), rstd=(F32, T), dh=(BF, T, H), dx=(BF, T, H))),
    "adapters": (lambda t: bsgg.adapters(t["x"], t["a"], t["b"], map_of(t), scales=t["s"], base=t["base"], out=t["out"]),
                 dict(x=(BF, T, H), a=(BF, S, r, H), b=(BF, S, r, N), s=(F32, S), base=(BF, T, N), out=(BF, T, N), **MAP)),
    "adapters_backward": (lambda t: bsgg.adapters_backward(t["dy"], t["x"], t["u"], t["a"], t["b"], map_of(t), scales=t["s"],
                                                           base=t["base"], dx=t["dx"]),
                          dict(dy=(BF, T, N), x=(BF, T, H), u=(F32, T, r), a=(BF, S, r, H), b=(BF, S, r, N), s=(F32, S),
                               base=(BF, T, H), dx=(BF, T, H), used=(I32, 1), **MAP)),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, tensors) in CALLS.items() for n in tensors])
def test_another_device_is_refused(call, name, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    run, tensors = CALLS[call]
    t = {n: OnGpu(*spec) for n, spec in tensors.items()}
    t[name].index = 1
    with pytest.raises(ValueError, match="cuda:1"):
        run(t)


# ------------------------------------------------------------------ the references' gradients
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_reference_route_gradient_against_differences(score, normalize):
    g = torch.Generator().manual_seed(3)
    l = torch.randn(5, 12, generator=g, dtype=torch.float64)
    ids, w = R.route_groups(l, 3, score=score, groups=3, topk_groups=2, normalize=normalize, scale=2.5)
    dw = torch.randn(5, 3, generator=g, dtype=torch.float64)
    want = R.route_groups_backward(l, ids, dw, score, normalize, 2.5)
    for e in range(12):
        step = torch.zeros_like(l)
        step[:, e] = 1e-6
        up, down = (R.weights_at(l + s * step, ids, score, normalize, 2.5) for s in (1, -1))
        # second-order differences: off by the third derivative times 1e-12, and 2^-52 / 1e-6
        assert torch.allclose(((up - down) * dw).sum(1) / 2e-6, want[:, e], rtol=0, atol=1e-8)


def test_reference_norm_gradient_against_differences():
    g = torch.Generator().manual_seed(4)
    h, dy, dh = (torch.randn(3, 16, generator=g, dtype=torch.float64) for _ in range(3))
    w = torch.randn(16, generator=g, dtype=torch.float64)
    f = lambda h, w: (R.rms_norm(h, w, 1e-3)[0] * dy).sum() + (h * dh).sum()  # noqa: E731
    dx, dw = R.rms_norm_backward(dy, h, w, R.rms_norm(h, w, 1e-3)[1], dh)
    for t in range(3):
        for c in range(16):
            s = torch.zeros_like(h)
            s[t, c] = 1e-6
            assert abs(float(f(h + s, w) - f(h - s, w)) / 2e-6 - float(dx[t, c])) < 1e-7
    for c in range(16):
        s = torch.zeros_like(w)
        s[c] = 1e-6
        assert abs(float(f(h, w + s) - f(h, w - s)) / 2e-6 - float(dw[c])) < 1e-7


def test_reference_adapters_gradient_against_differences():
    g = torch.Generator().manual_seed(5)
    x, a, b = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 8), (2, 3, 8), (2, 3, 6)))
    ids, scales, dy = torch.tensor([0, -1, 1, 1, 0]), torch.tensor([0.5, 2.0]), torch.randn(5, 6, generator=g, dtype=torch.float64)
    f = lambda x, a, b: (R.adapters(x, a, b, ids, scales, None)[0] * dy).sum()  # noqa: E731
    dx, da, db, _ = R.adapters_backward(dy, x, R.adapters(x, a, b, ids, scales, None)[1], a, b, ids, scales, None)
    for i, (v, d) in enumerate(((x, dx), (a, da), (b, db))):
        for at in range(v.numel()):
            s = torch.zeros(v.numel(), dtype=torch.float64)
            s[at] = 1e-6
            args = [[x, a, b], [x, a, b]]
            args[0][i], args[1][i] = v + s.view_as(v), v - s.view_as(v)
            assert abs(float(f(*args[0]) - f(*args[1])) / 2e-6 - float(d.reshape(-1)[at])) < 1e-7


# ------------------------------------------------------------------ wide layers
@pytest.mark.parametrize("k,n", [(4096, 14336), (4096, 105904), (4096, 112648), (4096, 128256), (8192, 151936), (2 ** 24, 2 ** 24)])
@pytest.mark.parametrize("tokens", [1, 2, 16, 4096, 65536])
def test_workspace_of_wide_layers(lib, tokens, k, n):
    """Beside an output head a single segment has more blocks than fill the chip.  The terms, in
    six bytes at the most, are there for any width; sums of segments only where there are several,
    of blocks that are 456 together at the most."""
    m_pad, adapters, rank = bsgg.sort_rows(tokens, 4), 4, 16
    need = lib.bsgg_adapters_workspace_bytes(tokens, k, n, m_pad, adapters, rank)
    terms = 2 * 6 * m_pad * 16
    assert terms <= need
    if tokens <= 128 or 2 * (-(-k // 256) - (-n // 256)) > 456:
        assert need <= terms + 2 * 4 * (adapters + m_pad // 64) + 6 * 16
    else:
        assert need >= terms + 2 * 4 * rank * (k + n)


def test_grids_past_31_bits_are_refused_before_anything_runs(lib):
    """(No GPU here: a launch would give another status.)"""
    wide = dict(tokens=2 ** 30, m_pad=2 ** 30)
    assert adapt(lib, n=2 ** 24, ld_base=2 ** 24, ldy=2 ** 24, **wide) == 2
    assert adapt_bwd(lib, dict(da=None, db=None), k=2 ** 24, ldx=2 ** 24, ld_base=2 ** 24, ld_dx=2 ** 24, **wide) == 2
    # one segment of 2^30 rows for each of the adapters
    assert adapt_bwd(lib, k=65536, n=65536, ld_dy=65536, ldx=65536, ld_base=65536, ld_dx=65536, adapters=1024, **wide) == 2

# ------------------------------------------------------------------ the norm's gradient
@pytest.mark.parametrize("hidden", [64, 512, 520, 1024, 1536, 2048, 4096, 4104, 5120, 7168, 8192, 8200, 12288, 16384, 32768])
def test_norm_gradient_has_as_many_blocks_on_each_sm(lib, hidden):
    """Its blocks walk rows until there are none: one more than fit at once would double the time."""
    parts = lib.bsgg_rms_norm_workspace_bytes(2 ** 20, hidden) // (4 * hidden)
    assert parts % 152 == 0 and parts >= 2 * 152
