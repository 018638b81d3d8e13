"""Dense products of every tiling on three streams at once: their blocks share the
SMs' tensor memory and shared memory, and every result has the bits it has alone."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu

# one row and a few (split single CTAs), many single CTAs, split pairs, pairs walking tiles
SHAPES = [(1, 4096, 7168), (40, 2048, 7168), (100, 8200, 1032), (300, 4096, 4160), (2048, 4096, 1024)]


def test_three_streams():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    work = []
    for m, n, k in SHAPES:
        x = torch.randn(m, k, generator=g, device="cuda").bfloat16()
        w = (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).bfloat16()
        for out in ("bf16", "f32"):
            work.append((x, w, out, bsgg.linear(x, w, activation="silu", out_format=out)[0]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(20):
        for j, s in enumerate(streams):
            for step in range(len(work)):
                x, w, out, want = work[(step * (j + 1) + i) % len(work)]
                with torch.cuda.stream(s):
                    got.append((bsgg.linear(x, w, activation="silu", out_format=out)[0], want))
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y, want in got)
        got.clear()
    assert bsgg.operators_status() == 0
