"""Every operator of no tokens: an empty tensor has no address, and that is not an
absent one."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu
H, L, K, N, M = 64, 8, 2, 32, 128


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def maps():
    return empty(0, K, dtype=torch.int32), torch.full((M,), -1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("normalize", [True, False])
def test_route(normalize):
    ids, w = bsgg.route(empty(0, L), K, normalize=normalize)
    dl = bsgg.route_backward(empty(0, L), ids, w, w, normalize=normalize)
    assert ids.shape == w.shape == (0, K) and dl.shape == (0, L)


def test_rows():
    rs, sr = maps()
    tm = bsgg.sort_tokens(rs, L, weights=empty(0, K, dtype=torch.float32))
    assert (tm.slot_of_row == -1).all() and tm.rows_used.item() == 0
    a, sfa = bsgg.dispatch(empty(0, H), rs, sr)
    assert (a == 0).all() and (sfa == 127)[:M * 2].any()
    d = torch.ones(M, H, device="cuda")
    assert bsgg.combine(d, rs, residual=empty(0, H, dtype=torch.float32)).shape == (0, H)


@pytest.mark.parametrize("want_dd", [True, False])
@pytest.mark.parametrize("want_dweights", [True, False])
def test_combine_backward(want_dd, want_dweights):
    rs, sr = maps()
    dd, _, dw = bsgg.combine_backward(empty(0, H), torch.ones(M, H, device="cuda"), rs, sr, want_dd=want_dd,
                                      want_dweights=want_dweights)
    assert (dd == 0).all() if want_dd else dd is None
    assert dw.shape == (0, K) if want_dweights else dw is None


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("wanted", range(1, 8))
def test_linear_backward(wanted, act):
    dx, dw, db = bsgg.linear_backward(empty(0, N), empty(0, H), torch.ones(N, H, dtype=torch.bfloat16, device="cuda"),
                                      z=empty(0, N) if act != "none" else None, activation=act, want_dx=bool(wanted & 1),
                                      want_dw=bool(wanted & 2), want_dbias=bool(wanted & 4))
    assert dx.shape == (0, H) if wanted & 1 else dx is None
    assert (dw == 0).all() and dw.shape == (N, H) if wanted & 2 else dw is None
    assert (db == 0).all() and db.shape == (N,) if wanted & 4 else db is None
