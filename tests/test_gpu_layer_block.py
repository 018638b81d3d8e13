"""The operators in front of an expert layer and beside its dense layers together, as a
training step has them: norm with the residual, router, adapters beside a projection,
and back, against the same step by autograd in 64 bits; captured, replayed on other
inputs, and on two streams."""
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg

pytestmark = pytest.mark.gpu
T, H, N, L, K, S, R = 260, 256, 384, 32, 4, 3, 16
HOW = dict(score="sigmoid", normalize=True, scale=2.5)
EPS = 1e-5


def problem(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    ids = torch.randint(-1, S, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    return dict(x=normal(T, H), res=normal(T, H), wn=(1 + normal(H, scale=0.2).float()).bfloat16(), wr=normal(L, H, scale=H ** -0.5),
                w=normal(N, H, scale=H ** -0.5), a=normal(S, R, H, scale=H ** -0.5), b=normal(S, R, N, scale=R ** -0.5),
                bias=torch.randn(L, generator=g, device="cuda") * 0.1, scales=torch.rand(S, generator=g, device="cuda") + 0.5,
                ids=ids, dy=normal(T, N), dh=normal(T, H), dw=torch.randn(T, K, generator=g, device="cuda"))


def step(p):
    """y = adapters(linear(norm(x + res))), top-k of the router on the same norm; the gradients
    of everything from dy, dh (the residual stream's) and dw (the routing weights')."""
    n = bsgg.rms_norm(p["x"], p["wn"], residual=p["res"], eps=EPS, row_format="mxfp8_e4m3")
    logits, _ = bsgg.linear(n.y, p["wr"], out_format="f32")
    ids, weights = bsgg.route_groups(logits, K, bias=p["bias"], groups=8, topk_groups=4, **HOW)
    t = bsgg.sort_tokens(p["ids"], S)
    base, _ = bsgg.linear(n.y, p["w"])
    y, u = bsgg.adapters(n.y, p["a"], p["b"], t, scales=p["scales"], base=base, out=base)
    dlogits = bsgg.route_groups_backward(logits, ids, weights, p["dw"], **HOW)
    dn, dw, _ = bsgg.linear_backward(p["dy"], n.y, p["w"])
    dnr, dwr, _ = bsgg.linear_backward(dlogits.bfloat16(), n.y, p["wr"])
    dn, da, db = bsgg.adapters_backward(p["dy"], n.y, u, p["a"], p["b"], t, scales=p["scales"], base=dn, dx=dn)
    dx, dwn = bsgg.rms_norm_backward(dn + dnr, n.h, p["wn"], n.rstd, dh=p["dh"])
    return dict(h=n.h, y=y, rows=n.a, sf=n.sfa, ids=ids, weights=weights, dx=dx, dwn=dwn, dw=dw, dwr=dwr, da=da, db=db)


def reference(p, ids):
    d = {k: v.double() for k, v in p.items() if v.is_floating_point()}
    leaves = {k: d[k].requires_grad_() for k in ("x", "wn", "wr", "w", "a", "b")}
    h = d["x"] + d["res"]
    n = h * (h.square().mean(1, keepdim=True) + EPS) ** -0.5 * d["wn"]
    s = torch.sigmoid(n @ d["wr"].t()).gather(1, ids.long())
    weights = HOW["scale"] * s / s.sum(1, keepdim=True)
    mine = (p["ids"] == torch.arange(S, device="cuda")).double()
    u = torch.einsum("th,srh->tsr", n, d["a"]) * mine[:, :, None]
    y = n @ d["w"].t() + torch.einsum("tsr,s,srn->tn", u, d["scales"], d["b"])
    ((y * d["dy"]).sum() + (h * d["dh"]).sum() + (weights * d["dw"]).sum()).backward()
    return dict(h=h, y=y, weights=weights, dx=leaves["x"].grad, dwn=leaves["wn"].grad, dw=leaves["w"].grad, dwr=leaves["wr"].grad,
                da=leaves["a"].grad, db=leaves["b"].grad)


def test_a_step_against_64_bits():
    p = problem(1)
    got = step(p)
    want = {k: v.detach() for k, v in reference(p, got["ids"]).items()}
    far = lambda g, w: float((g.double() - w).norm() / w.norm())  # noqa: E731
    # each result carries a few roundings to bfloat16 (2^-9.2 in norm): of h, of the norm, of
    # the layer's output or gradient, and its own; up to eight of them in dx
    for name, steps in dict(h=1, y=4, weights=4, dw=4, da=6, db=5, dwr=6, dx=8, dwn=8).items():
        assert far(got[name], want[name]) < steps ** 0.5 * 2.0 ** -8.5, name
    # the chosen experts are those of the router's own logits, checked where it is tested; here
    # that every row has K different ones
    assert (got["ids"].sort(1).values.diff(dim=1) > 0).all() and bsgg.operators_status() == 0


def test_captured_and_on_two_streams():
    p, q = problem(2), problem(3)
    want_p = {k: v.clone() for k, v in step(p).items()}
    want_q = {k: v.clone() for k, v in step(q).items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    live = {k: v.clone() for k, v in p.items()}
    with torch.cuda.graph(graph):
        out = step(live)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want_p[k]) for k in out)
    for k in live:
        live[k].copy_(q[k])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want_q[k]) for k in out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, inputs in zip(streams, (p, q)):
        with torch.cuda.stream(s):
            got.append([step(inputs) for _ in range(3)][-1])
    torch.cuda.synchronize()
    for g, want in zip(got, (want_p, want_q)):
        assert all(torch.equal(g[k], want[k]) for k in g)


def test_two_captured_graphs_in_turn():
    """Graphs with workspaces of their own, replayed one between the other's replays."""
    ps = [problem(4), problem(5)]
    want = [{k: v.clone() for k, v in step(p).items()} for p in ps]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(p))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(o[k], w[k]) for k in o)
