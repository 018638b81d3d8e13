"""Long reductions of the dense products in float32: the tensor core cuts off what
an addition to its accumulator drops, which a sum over the whole reduction would
carry into the result.

The bound on the norm of the error: in a run of 512 elements the accumulator is
added to 32 times, each addition short by one unit in the last place, 2^-23 of the
sum so far, at most; that sum's norm grows as the square root of the length, so the
norm of what is cut is at most 2/3 * 32 * 2^-23 = 2.5e-6 of the run's, and the runs'
errors relate to the total as the runs do.  Their float32 additions round: 2^-24 each
of the sum so far, n^(1/2) of them in norm at most, 0.5e-6 for 56 runs.
"""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu

BOUND = 3.0e-6


def draw(seed, *shape, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def off(got, want):
    assert torch.isfinite(got).all()
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [
    (1, 4096, 14336), (1, 4096, 28672), (64, 1000, 28672), (227, 76, 12528), (333, 2049, 28672), (100, 8200, 14336),
    (700, 6144, 8192), (1030, 4104, 14336), (2048, 4096, 14336),
    # an end inside a run, inside a block, one block past a run, and one run alone
    (300, 2048, 4104), (130, 2048, 576), (2048, 4096, 520), (2048, 4096, 584), (2048, 4096, 512)])
def test_forward(m, n, k, dtype):
    x, w = draw(1, m, k, dtype=dtype), draw(2, n, k, dtype=dtype)
    b = draw(3, n, dtype=torch.float32)
    y, _ = bsgg.linear(x, w, bias=b, out_format="f32")
    assert off(y, x.double() @ w.double().t() + b.double()) <= BOUND


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [(8192, 256, 512), (14336, 64, 200), (16384, 1024, 1032), (8200, 4096, 2048)])
def test_weight_gradient(m, n, k, dtype):
    """dw sums over the tokens; into float32, where it may also be added to."""
    x, dy, w = draw(1, m, k, dtype=dtype), draw(2, m, n, dtype=dtype), draw(3, n, k, dtype=dtype)
    want = dy.double().t() @ x.double()
    _, dw, _ = bsgg.linear_backward(dy, x, w, dw_format="f32", want_dx=False)
    assert off(dw, want) <= BOUND
    start = draw(4, n, k, dtype=torch.float32) * m ** 0.5
    dw = start.clone()
    bsgg.linear_backward(dy, x, w, dw=dw, want_dx=False)
    assert off(dw, want + start.double()) <= BOUND


@pytest.mark.parametrize("m,n,k", [(64, 14336, 512), (1000, 8192, 4096)])
def test_input_gradient(m, n, k):
    dt = torch.bfloat16
    x, dy, w = draw(1, m, k, dtype=dt), draw(2, m, n, dtype=dt), draw(3, n, k, dtype=dt)
    dx, _, _ = bsgg.linear_backward(dy, x, w, dx_format="f32", want_dw=False)
    assert off(dx, dy.double() @ w.double()) <= BOUND


def test_longest_in_16_bits():
    """Where even the eight parts of a reduction are longer than a 16-bit output
    lets one sum be; the rounding to float16 is 2^-11 of a value at most."""
    x, w = draw(1, 8, 270008, dtype=torch.float16), draw(2, 128, 270008, dtype=torch.float16) * 0.01
    y, _ = bsgg.linear(x, w)
    assert off(y, x.double() @ w.double().t()) <= 2.0 ** -11 + BOUND


def test_the_same_bits_twice():
    x, w = draw(1, 1030, 14336, dtype=torch.bfloat16), draw(2, 4104, 14336, dtype=torch.bfloat16)
    first, _ = bsgg.linear(x, w, out_format="f32")
    for _ in range(5):
        y, _ = bsgg.linear(x, w, out_format="f32")
        assert torch.equal(y, first)
