"""silu over the arguments where e^-z leaves what 32 bits hold, to float32.

The formula's own errors, in units of 2^-23 of the value: the hardware's
exponential 2 + 1.2 |z|, product and sum 1 together, quotient 2.  Values below
2^-126 may be flushed."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu


def arguments(dtype):
    z = torch.cat([torch.arange(-1200, 1000) / 8.0, torch.arange(-712, -690) / 8.0 - 0.0625, torch.tensor([0.0, -0.0])])
    return z.to(dtype).unique()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_silu(dtype):
    z = arguments(dtype)
    x = torch.zeros(z.numel(), 8, dtype=dtype)
    x[:, 0] = z                                          # z = x w^T exactly
    w = torch.zeros(3, 8, dtype=dtype)
    w[:, 0] = 1.0
    y, _ = bsgg.linear(x.cuda(), w.cuda(), activation="silu", out_format="f32")
    zd = z.double()
    want = zd / (1.0 + torch.exp(-zd))
    tol = want.abs() * (5.0 + 1.2 * zd.abs()) * 2.0 ** -23 + 2.0 ** -126
    assert ((y.cpu().double() - want[:, None]).abs() <= tol[:, None]).all()
    assert bsgg.operators_status() == 0
