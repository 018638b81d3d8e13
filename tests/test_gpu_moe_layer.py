"""The layer of examples/moe_layer.py, every operator together, against the same
layer in 64 bits.  The experts run in MXFP8 (three fraction bits, scales per 32),
so values of theirs are right to a few per cent of their size: the check is on the
norm of the difference."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def reference(layer, x, dy, ids):
    """The layer and its gradients by autograd in 64 bits, with the ids held."""
    T, H, I, L, k = layer.T, layer.H, layer.I, layer.L, layer.k
    x = x.double().requires_grad_()
    wr, s1, s2 = (w.double().requires_grad_() for w in (layer.w_router, layer.s1, layer.s2))
    w1 = layer.w1.double().view(L, I // 32, 2, 32, H)
    up, gate, w2 = w1[:, :, 0].reshape(L, I, H), w1[:, :, 1].reshape(L, I, H), layer.w2.double()
    p = torch.softmax((x @ wr.t()).gather(1, ids.long()), 1)
    y = x + torch.nn.functional.silu(x @ s1.t()) @ s2.t()
    for e in range(L):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = (x[t] @ up[e].t()) * torch.nn.functional.silu(x[t] @ gate[e].t()) * p[t, j][:, None]
        y = y.index_add(0, t, h @ w2[e].t())
    y.backward(dy.double())
    return y.detach(), {"x": x.grad, "w_router": wr.grad, "s1": s1.grad, "s2": s2.grad}


def far(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [(300, 256, 128, 4, 2), (1, 512, 256, 8, 2), (1024, 512, 512, 16, 4)])
def test_layer(tokens, hidden, inter, experts, topk):
    from moe_layer import MoELayer
    layer = MoELayer(tokens, hidden, inter, experts, topk)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    dy = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    y = layer.forward(x)
    grads = layer.backward(dy)
    assert layer.status() == [0] * 5
    want_y, want = reference(layer, x, dy, layer.ids)
    # E4M3 with a power-of-two scale: values off by up to 2^-4 of themselves, on
    # average 2^-5.3 or 2.6 %; two quantized operands per product and two or three
    # products in a row come to 2.6 % sqrt(6), which only part of y and dx carries
    assert far(y, want_y) < 0.065
    assert far(grads["x"], want["x"]) < 0.065
    assert far(grads["s1"], want["s1"]) < 0.01 and far(grads["s2"], want["s2"]) < 0.01     # bfloat16 all the way
    if topk > 1:
        assert far(grads["w_router"], want["w_router"]) < 0.2       # differences of experts' outputs
