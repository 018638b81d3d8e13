"""Gradients of dense layers with more columns than a grid's second extent has
groups of 64 (65535 of them: 4194240 columns)."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
from test_gpu_linear import DT, check_backward, gen, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("M,N", [(1, 4194240), (1, 4194248), (3, 5000008), (1, 2 ** 24)])
def test_wide_gradient(M, N, act):
    K = 8
    x, w, _, z = problem(M, N, K, "bf16", M + N)
    dy = (torch.randn(M, N, generator=gen(2)) * 0.3).to(DT["bf16"])
    dx, dw, db = bsgg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=z.cuda() if act != "none" else None, activation=act,
                                      want_dbias=True)
    check_backward(dy, x, w, z, act, dx, dw, db)
    assert bsgg.operators_status() == 0
