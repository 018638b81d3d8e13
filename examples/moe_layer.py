"""One mixture-of-experts layer, forward and backward, from the tokens to the
tokens: the operators of ``block_scaled_grouped_gb300`` around its grouped GEMM.

    y = x + shared(x) + sum_j w_j E_j(x)

    logits = linear(x, Wr)                 router projection, float32
    ids, w = route(logits, k)              softmax top-k
    map    = sort_tokens(ids, weights=w)   rows by expert, padded to 128; prob per row
    a, sfa = dispatch(x, map)              MXFP8 rows and scale factors
    C, h   = FC1 + SwiGLU * prob           grouped GEMM, E4M3 rows out, C kept
    d      = FC2                           grouped GEMM, bfloat16
    s      = linear(silu(linear(x, S1)), S2) + x       the shared expert, residual fused
    y      = combine(d, map) + s

and back: dispatch(dy) -> dSwiGLU grouped GEMM (its dprob is the routing weights'
gradient) -> grouped GEMM with W1 -> combine; route_backward and linear_backward for
the router and the shared expert.  (The experts' own weight gradients are products
over rows, which the library does not have.)

m_pad is the number of rows that always suffices, so every shape is fixed: the
layer needs no read-back of the routing and can be captured in a CUDA graph.

    python examples/moe_layer.py [--tokens 4096 --hidden 4096 --inter 2048 --experts 8 --topk 2]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_grouped_gb300 as bsgg  # noqa: E402
from block_scaled_grouped_gb300 import workloads  # noqa: E402


def mxfp8(w):
    """(L, rows, K) weights as MXFP8 codes and swizzled scale factors."""
    codes, scales = zip(*(workloads.quantize_mxfp8(e.float(), "mxfp8_e4m3") for e in w))
    return torch.stack(codes), bsgg.pack_sf(torch.stack(scales))


def interleave(gate, up):
    """(L, inter, H) gate and up projections as FC1's paired 32-column blocks [up | gate]."""
    L, n, h = gate.shape
    return torch.stack([up.view(L, n // 32, 32, h), gate.view(L, n // 32, 32, h)], 2).reshape(L, 2 * n, h)


class MoELayer:
    def __init__(self, tokens, hidden, inter, experts, topk, shared=None, device="cuda", seed=0):
        self.T, self.H, self.I, self.L, self.k = tokens, hidden, inter, experts, topk
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device) / shape[-1] ** 0.5

        shared = inter if shared is None else shared
        self.w_router = normal(experts, hidden).bfloat16()
        self.w1, self.w2 = interleave(normal(experts, inter, hidden), normal(experts, inter, hidden)), normal(experts, hidden, inter)
        self.s1, self.s2 = normal(shared, hidden).bfloat16(), normal(hidden, shared).bfloat16()
        # the grouped GEMMs' weights, laid out once: forward, and transposed for the gradient
        self.b1, self.sfb1 = mxfp8(self.w1)
        self.b2, self.sfb2 = mxfp8(self.w2)
        self.b1t, self.sfb1t = mxfp8(self.w1.transpose(1, 2))
        self.b2t, self.sfb2t = mxfp8(self.w2.transpose(1, 2))
        self.m_pad = m = bsgg.sort_rows(tokens * topk, experts)
        plan = dict(m_pad=m, num_groups=experts, in_format="mxfp8_e4m3")
        self.fc1 = bsgg.Plan(n=2 * inter, k=hidden, out_format="e4m3", epilogue="swiglu", c_format="bf16", **plan)
        self.fc2 = bsgg.Plan(n=hidden, k=inter, out_format="bf16", epilogue="gate", **plan)
        self.dfc2 = bsgg.Plan(n=inter, k=hidden, out_format="e4m3", epilogue="dswiglu", **plan)
        self.dfc1 = bsgg.Plan(n=hidden, k=2 * inter, out_format="bf16", epilogue="gate", **plan)
        f32 = dict(dtype=torch.float32, device=device)
        self.ones, self.row_ones, self.one = torch.ones(experts, **f32), torch.ones(m, **f32), torch.ones(1, **f32)
        u8 = dict(dtype=torch.uint8, device=device)
        self.h, self.sfh = torch.empty(m, inter, **u8), torch.empty(bsgg.sf_bytes(m, inter, 32), **u8)
        self.dc, self.sfdc = torch.empty(m, 2 * inter, **u8), torch.empty(bsgg.sf_bytes(m, 2 * inter, 32), **u8)
        self.c = torch.empty(m, 2 * inter, dtype=torch.bfloat16, device=device)
        self.d = torch.empty(m, hidden, dtype=torch.bfloat16, device=device)
        # bfloat16 logit gradients, rows 16 bytes apart or a multiple of it as products want them
        self.dl = torch.zeros(tokens, -(-experts // 8) * 8, dtype=torch.bfloat16, device=device)[:, :experts]
        self.dprob, self.amax = torch.empty(m, **f32), torch.empty(experts, **f32)

    def forward(self, x):
        """x (tokens, hidden) bfloat16 -> y; what the backward needs is kept."""
        self.x = x
        self.logits, _ = bsgg.linear(x, self.w_router, out_format="f32")
        self.ids, self.weights = bsgg.route(self.logits, self.k)
        self.map = t = bsgg.sort_tokens(self.ids, self.L, m_pad=self.m_pad, weights=self.weights)
        a, sfa = bsgg.dispatch(x, t.row_of_slot, t.slot_of_row)
        common = dict(padded_offsets=t.padded_offsets, alpha=self.ones)
        self.fc1.run(a=a, sfa=sfa, b=self.b1, sfb=self.sfb1, prob=t.prob, norm_const=self.one, d=self.h, sfd_row=self.sfh,
                     c=self.c, **common)
        self.fc2.run(a=self.h, sfa=self.sfh, b=self.b2, sfb=self.sfb2, prob=self.row_ones, d=self.d, amax=self.amax, **common)
        self.sh, self.sz = bsgg.linear(x, self.s1, activation="silu", want_z=True)
        s, _ = bsgg.linear(self.sh, self.s2, residual=x)
        return bsgg.combine(self.d, t.row_of_slot, residual=s)

    def backward(self, dy):
        """dy (tokens, hidden) bfloat16 -> the gradients of x, the router and the
        shared expert."""
        t = self.map
        common = dict(padded_offsets=t.padded_offsets, alpha=self.ones)
        # shared expert: s = silu(x S1^T) S2^T + x
        dsh, ds2, _ = bsgg.linear_backward(dy, self.sh, self.s2)
        dxs, ds1, _ = bsgg.linear_backward(dsh, self.x, self.s1, z=self.sz, activation="silu")
        # experts: rows of dy, through FC2 and the SwiGLU, then through FC1
        g, sfg = bsgg.dispatch(dy, t.row_of_slot, t.slot_of_row)
        self.dprob.zero_()
        self.dfc2.run(a=g, sfa=sfg, b=self.b2t, sfb=self.sfb2t, prob=t.prob, norm_const=self.one, saved_c=self.c,
                      beta=self.ones, dprob=self.dprob, d=self.dc, sfd_row=self.sfdc, **common)
        self.dfc1.run(a=self.dc, sfa=self.sfdc, b=self.b1t, sfb=self.sfb1t, prob=self.row_ones, d=self.d, amax=self.amax, **common)
        # router: dprob is the weights' gradient, row by row
        dlogits = bsgg.route_backward(self.logits, self.ids, self.weights, self.dprob, row_of_slot=t.row_of_slot)
        self.dl.copy_(dlogits)
        dxr, dwr, _ = bsgg.linear_backward(self.dl, self.x, self.w_router)
        # x: the residual, the shared expert, the router and the experts
        dx = bsgg.combine(self.d, t.row_of_slot, residual=dy + dxs + dxr)
        return {"x": dx, "w_router": dwr, "s1": ds1, "s2": ds2}

    def status(self):
        """Device status of every part (0 = ok); synchronizes."""
        return [p.device_status() for p in (self.fc1, self.fc2, self.dfc2, self.dfc1)] + [bsgg.operators_status()]


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 4096), ("inter", 2048), ("experts", 8), ("topk", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    layer = MoELayer(a.tokens, a.hidden, a.inter, a.experts, a.topk)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()
    dy = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").bfloat16()

    def step():
        layer.forward(x)
        return layer.backward(dy)

    for _ in range(3):
        step()
    torch.cuda.synchronize()
    assert not any(layer.status()), layer.status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for what, run in (("calls", step), ("graph", graph.replay)):
        run()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(10):
            run()
        end.record()
        torch.cuda.synchronize()
        print(f"{what}: {begin.elapsed_time(end) / 10 * 1e3:.0f} us per forward and backward "
              f"({a.tokens} tokens, {a.hidden} -> {a.inter}, top-{a.topk} of {a.experts})")


if __name__ == "__main__":
    main()
