"""Gradients of dense layers whose width is no multiple of the eight columns that
the pass over dz takes at a time: columns past the last are neither used nor written."""
import ctypes
import math

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
from block_scaled_grouped_gb300 import operators as ops
from test_gpu_linear import DT, check_backward, gen, pitched, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "srelu", "none"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 2, 65, 700])
@pytest.mark.parametrize("N", [1, 7, 9, 33, 2049])
def test_ragged_gradient(M, N, dtype, act):
    K = 40
    x, w, _, z = problem(M, N, K, dtype, M + N)
    dy = (torch.randn(M, N, generator=gen(2)) * 0.3).to(DT[dtype])
    # a single row has exactly its own columns, more rows a pitch with NaN between them
    put = (lambda t: t.cuda()) if M == 1 else (lambda t: pitched(t, 8, 8))
    dx, dw, db = bsgg.linear_backward(put(dy), x.cuda(), w.cuda(), z=put(z) if act != "none" else None, activation=act,
                                      want_dbias=True)
    check_backward(dy, x, w, z, act, dx, dw, db)
    assert bsgg.operators_status() == 0


@pytest.mark.parametrize("M,N", [(1, 13), (70, 2049), (5, 64)])
def test_columns_past_the_last_are_not_written(M, N):
    K, ld = 16, (N + 7) // 8 * 8 + 16
    x, w, _, z = problem(M, N, K, "bf16", 3)
    dy = torch.randn(M, N, generator=gen(4)).bfloat16()
    dyp, zp, xd, wd = pitched(dy, 1, ld - N), pitched(z, 1, ld - N), x.cuda(), w.cuda()
    dz = torch.full((M, ld), math.inf, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    desc = ops.LinearBwdDesc(M, N, K, ld, ld, ld, K, K, K, K, 0, 0, 0, ops.ACTIVATIONS["silu"], 0)
    st = bsgg.lib().bsgg_linear_backward(ctypes.byref(desc), dyp.data_ptr(), xd.data_ptr(), wd.data_ptr(), zp.data_ptr(),
                                         dz.data_ptr(), dx.data_ptr(), None, None, None,
                                         torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert (dz[:, N:] == math.inf).all() and torch.isfinite(dz[:, :N]).all()
    check_backward(dy, x, w, z, "silu", dx, None, None)
