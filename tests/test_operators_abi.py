"""What the operators around the grouped GEMM refuse, without a GPU: every
check runs on the host before any device call."""
import ctypes
import os
import re

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
from block_scaled_grouped_gb300 import build as bsgg_build
from block_scaled_grouped_gb300 import operators as ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bsgg.h")
P = ctypes.c_void_p(4096)        # never dereferenced: refused first
ODD = ctypes.c_void_p(4098)


@pytest.fixture(scope="module", autouse=True)
def lib():
    bsgg_build.build()
    return bsgg.lib()


@pytest.mark.parametrize("struct,cls", [("bsgg_route_desc", ops.RouteDesc), ("bsgg_tokens_desc", ops.TokensDesc),
                                        ("bsgg_linear_desc", ops.LinearDesc), ("bsgg_linear_bwd_desc", ops.LinearBwdDesc)])
def test_binding_structs_match_the_header(struct, cls):
    src = open(HEADER).read()
    end = src.index("} " + struct + ";")
    body = re.sub(r"/\*.*?\*/", "", src[src.rindex("typedef struct {", 0, end) + len("typedef struct {"):end], flags=re.S)
    fields = [(t, n.strip()) for t, names in re.findall(r"(int64_t|int32_t)\s+([^;]+);", body) for n in names.split(",")]
    ctype = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32}
    assert [(ctype[t], n) for t, n in fields] == [(t, n) for n, t in cls._fields_]


def route(lib, ptrs=(P, P, P), **over):
    d = dict(tokens=4, ld=8, num_experts=8, topk=2, logit_format=2, normalize=1)
    d.update(over)
    return lib.bsgg_route(ctypes.byref(ops.RouteDesc(*[d[n] for n, _ in ops.RouteDesc._fields_])), *ptrs, None)


@pytest.mark.parametrize("over", [dict(tokens=-1), dict(num_experts=0), dict(num_experts=1025, ld=2000), dict(topk=0),
                                  dict(topk=9), dict(topk=33, num_experts=64, ld=64), dict(ld=7), dict(logit_format=3),
                                  dict(normalize=2), dict(logit_format=-1)])
def test_route_refuses(lib, over):
    assert route(lib, **over) == 1


def test_route_refuses_pointers(lib):
    assert route(lib, ptrs=(None, P, P)) == 1 and route(lib, ptrs=(P, None, P)) == 1 and route(lib, ptrs=(P, P, None)) == 1
    assert route(lib, ptrs=(ODD, P, P)) == 1                      # float32 logits off their alignment
    assert route(lib, tokens=0, ptrs=(None, None, None)) == 0
    assert lib.bsgg_route(None, P, P, P, None) == 1
    d = ops.RouteDesc(4, 8, 8, 2, 2, 1)
    assert lib.bsgg_route_backward(ctypes.byref(d), P, P, P, None, None, 0, P, None) == 1
    assert lib.bsgg_route_backward(ctypes.byref(d), P, P, P, P, P, 0, P, None) == 1     # rows without their number


def test_sort_refuses(lib):
    assert [lib.bsgg_sort_rows(*a) for a in ((-1, 8), (4, 0), (4, 1025), (2 ** 31, 8))] == [-1] * 4
    ok = dict(slots=8, L=4, m_pad=512, ids=P, weights=None, off=P, row=P, slot=P, prob=None, used=None, ws=None, st=None)

    def sort(**over):
        return lib.bsgg_sort_tokens(*{**ok, **over}.values(), None)

    for over in (dict(slots=-1), dict(L=0), dict(L=1025), dict(m_pad=0), dict(m_pad=100), dict(m_pad=-128), dict(ids=None),
                 dict(off=None), dict(row=None), dict(slot=None), dict(ids=ODD), dict(prob=ODD), dict(st=ODD)):
        assert sort(**over) == 1, over
    many = 100000
    assert lib.bsgg_sort_workspace_bytes(8, 4) == 0 and lib.bsgg_sort_workspace_bytes(many, 4) > 0
    assert sort(slots=many, m_pad=128 * 1000) == 1                # the workspace is missing


def test_sort_rows_holds_every_split():
    """Against all splits of small numbers of slots."""
    def most(n, L):
        if L == 1:
            return -(-n // 128)
        return max(-(-c // 128) + most(n - c, L - 1) for c in sorted({0, 1, n} | set(range(1, n + 1, 128))) if c <= n)
    for n in (0, 1, 2, 127, 128, 129, 130, 257, 400):
        for L in (1, 2, 3):
            assert bsgg.sort_rows(n, L) == max(128, 128 * most(n, L)), (n, L)


def tokens_desc(**over):
    d = dict(tokens=4, hidden=64, m_pad=128, ld_token=64, ld_residual=0, topk=2, token_format=0, row_format=0, d_format=0)
    d.update(over)
    return ctypes.byref(ops.TokensDesc(*[d[n] for n, _ in ops.TokensDesc._fields_]))


BAD_TOKENS = [dict(tokens=-1), dict(hidden=0), dict(hidden=60, ld_token=64), dict(m_pad=0), dict(m_pad=130), dict(ld_token=56),
              dict(ld_token=68), dict(topk=0), dict(topk=33), dict(token_format=3), dict(tokens=2 ** 30, topk=4)]


@pytest.mark.parametrize("over", BAD_TOKENS + [dict(row_format=7), dict(row_format=-1), dict(hidden=72, ld_token=72),
                                                dict(hidden=48, ld_token=48, row_format=2)])
def test_dispatch_refuses(lib, over):
    assert lib.bsgg_dispatch(tokens_desc(**over), P, P, P, P, P, None) == 1


def test_dispatch_refuses_pointers(lib):
    good = [P] * 5
    for i in range(5):
        a = list(good)
        a[i] = None
        assert lib.bsgg_dispatch(tokens_desc(), *a, None) == 1
        a[i] = ODD
        assert lib.bsgg_dispatch(tokens_desc(), *a, None) == 1
    assert lib.bsgg_dispatch(tokens_desc(row_format=5), P, P, P, P, P, None) == 1      # scales of unscaled rows
    assert lib.bsgg_dispatch(None, *good, None) == 1


@pytest.mark.parametrize("over", BAD_TOKENS + [dict(d_format=4), dict(ld_residual=60), dict(ld_residual=68)])
def test_combine_refuses(lib, over):
    assert lib.bsgg_combine(tokens_desc(**{"ld_residual": 64, **over}), P, P, P, P, P, None) == 1


def test_combine_refuses_pointers(lib):
    for a in ((None, P, None, None, P), (P, None, None, None, P), (P, P, None, None, None), (ODD, P, None, None, P),
              (P, P, ODD, None, P), (P, P, None, None, ODD)):
        assert lib.bsgg_combine(tokens_desc(), *a, None) == 1
    assert lib.bsgg_combine(tokens_desc(tokens=0), P, P, None, None, P, None) == 0
    bw = lambda *a, **o: lib.bsgg_combine_backward(tokens_desc(**o), *a, None)  # noqa: E731
    assert bw(P, P, P, P, P, None, None, None) == 1                   # nothing wanted
    assert bw(P, None, P, P, P, P, P, P) == 1                         # dweights without D
    assert bw(P, P, P, None, P, P, P, P) == 1                         # dD without its map
    assert bw(P, P, P, P, P, P, None, P) == 1                         # quantized rows without scales
    assert bw(P, P, P, P, P, P, P, P, row_format=6) == 1              # scales of unscaled rows
    assert bw(P, P, P, P, P, None, P, P) == 1


def linear_desc(**over):
    d = dict(m=4, n=16, k=32, ldx=32, ldw=32, ld_residual=16, ldy=16, ldz=16, in_format=0, out_format=0, bias_format=2,
             activation=0)
    d.update(over)
    return ctypes.byref(ops.LinearDesc(*[d[n] for n, _ in ops.LinearDesc._fields_]))


@pytest.mark.parametrize("over", [dict(m=-1), dict(n=0), dict(k=0), dict(ldx=24), dict(ldx=36), dict(ldw=24), dict(ldw=33),
                                  dict(ld_residual=15), dict(ldy=15), dict(ldz=8), dict(in_format=2), dict(out_format=3),
                                  dict(bias_format=5), dict(activation=5), dict(activation=-1), dict(m=2 ** 25)])
def test_linear_refuses(lib, over):
    assert lib.bsgg_linear(linear_desc(**over), P, P, P, P, P, P, None, None) == 1


def test_linear_refuses_pointers(lib):
    for a in ((None, P, P, P, P, P), (P, None, P, P, P, P), (P, P, P, P, None, P), (ODD, P, P, P, P, P), (P, ODD, P, P, P, P),
              (P, P, ODD, P, P, P)):
        assert lib.bsgg_linear(linear_desc(), *a, None, None) == 1
    assert lib.bsgg_linear(linear_desc(), P, P, P, P, P, P, ODD, None) == 1
    assert lib.bsgg_linear(linear_desc(m=0), P, P, P, P, P, P, None, None) == 0


def bwd_desc(**over):
    d = dict(m=4, n=16, k=32, ld_dy=16, ldz=16, ld_dz=16, ldx=32, ldw=32, ld_dx=32, ld_dw=32, in_format=0, dx_format=0,
             dw_format=0, activation=3, accumulate_dw=0)
    d.update(over)
    return ctypes.byref(ops.LinearBwdDesc(*[d[n] for n, _ in ops.LinearBwdDesc._fields_]))


@pytest.mark.parametrize("over", [dict(m=-1), dict(n=0), dict(k=0), dict(ld_dy=8), dict(ld_dy=20), dict(ldz=20), dict(ld_dz=20),
                                  dict(ldx=36), dict(ldw=36), dict(ld_dx=31), dict(ld_dw=31), dict(in_format=2), dict(dx_format=3),
                                  dict(dw_format=3), dict(activation=9), dict(accumulate_dw=2)])
def test_linear_backward_refuses(lib, over):
    assert lib.bsgg_linear_backward(bwd_desc(**over), P, P, P, P, P, P, P, P, None, None) == 1


def test_linear_backward_refuses_pointers(lib):
    bw = lambda *a, **o: lib.bsgg_linear_backward(bwd_desc(**o), *a, None, None)  # noqa: E731
    assert bw(P, P, P, None, P, P, P, P) == 1 and bw(P, P, P, P, None, P, P, P) == 1      # z and dz of an activation
    assert bw(P, P, P, P, P, P, P, P, activation=0) == 1                                    # and of none
    assert bw(P, P, P, P, P, None, None, None) == 1                                         # nothing wanted
    assert bw(None, P, P, P, P, P, P, P) == 1 and bw(P, None, P, P, P, P, P, P) == 1 and bw(P, P, None, P, P, P, P, P) == 1
    assert bw(ODD, P, P, P, P, P, P, P) == 1
    assert lib.bsgg_query_status_word(None, None) == 1


def test_binding_refuses_shapes_and_types():
    """The binding's own checks (no GPU here: a CPU tensor is one of them)."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: bsgg.route(x, 2), lambda: bsgg.linear(x, x), lambda: bsgg.linear_backward(x, x, x),
                 lambda: bsgg.dispatch(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(128, dtype=torch.int32)),
                 lambda: bsgg.sort_tokens(torch.zeros(4, 2, dtype=torch.int32), 8),
                 lambda: bsgg.combine(x, torch.zeros(4, 2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(bsgg.BsggError):
        bsgg.sort_rows(-1, 4)
