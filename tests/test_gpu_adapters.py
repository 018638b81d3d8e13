"""Low-rank adapters on the GPU against 64-bit references: ranks, widths and adapters'
shares of the tokens from one up, tokens without an adapter, adapters without a token,
both types, pitches, in place, and gradients."""
import math

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
import layer_operator_refs as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def pitched(t, extra):
    """t on the GPU as a view of a wider buffer (extra columns, poisoned)."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), math.nan, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]]


def rounding(ref, dtype):
    return ref.abs() * ROUND[dtype] + TINY[dtype]


def product_error(depth):
    """Bound on |error| / sum |a b| of a product accumulated in 32 bits: steps of 16 products,
    each added with one rounding or truncation of 2^-23, and as much again for the joins."""
    return (depth / 16 + 32) * 2.0 ** -23


# u's and du's terms: two of bfloat16 hold them to 2^-17 (2^-16 where both are rounded up), two
# of float16 to 2^-21 of the row's largest, three of bfloat16 to 2^-24
TERMS = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -20}


def problem(T, S, r, K, N, dtype, kind, seed):
    g = gen(seed)
    dt = DT[dtype]
    if kind == "one":
        ids = torch.full((T,), S - 1)
    elif kind == "none":
        ids = torch.full((T,), -1)
    else:
        ids = torch.randint(-1, S, (T,), generator=g)
        if kind == "runs":
            ids = ids[torch.cummax(torch.where(torch.rand(T, generator=g) < 0.02, torch.arange(T), torch.zeros(T, dtype=torch.long)), 0).values]
    return dict(ids=ids.to(torch.int32), x=torch.randn(T, K, generator=g).to(dt), a=(torch.randn(S, r, K, generator=g) / K ** 0.5).to(dt),
                b=(torch.randn(S, r, N, generator=g) / r ** 0.5).to(dt), scales=torch.rand(S, generator=g) + 0.5,
                base=torch.randn(T, N, generator=g).to(dt), dy=torch.randn(T, N, generator=g).to(dt), basex=torch.randn(T, K, generator=g).to(dt))


def map_of(p, S, m_pad=None):
    return bsgg.sort_tokens(p["ids"].cuda().view(-1, 1), S, m_pad=m_pad)


# tokens, adapters, rank, k, n, type, tokens' adapters
CASES = [(1, 1, 8, 8, 8, "bf16", "one"), (1, 4, 16, 2048, 512, "f16", "any"), (3, 2, 16, 64, 72, "bf16", "any"), (17, 1, 24, 136, 520, "f16", "one"),
         (16, 3, 32, 256, 1024, "bf16", "any"), (40, 1, 8, 4096, 64, "bf16", "one"), (33, 1, 40, 72, 200, "bf16", "one"),
         (64, 5, 64, 320, 1032, "f16", "any"), (65, 1, 128, 128, 136, "bf16", "one"), (130, 1, 128, 200, 600, "f16", "one"),
         (70, 1, 56, 1000, 264, "bf16", "one"), (100, 2, 72, 88, 520, "bf16", "any"), (128, 64, 16, 512, 640, "bf16", "any"),
         (300, 3, 16, 256, 512, "f16", "runs"), (600, 2, 32, 128, 2056, "bf16", "runs"), (20, 1, 120, 64, 64, "f16", "one"),
         (9, 3, 16, 64, 64, "bf16", "none"), (25, 1, 8, 512, 96, "f16", "one"), (90, 1, 24, 1024, 160, "bf16", "one"),
         (20, 1, 56, 200, 80, "bf16", "one"), (31, 2, 104, 72, 304, "f16", "one"), (50, 1000, 8, 64, 64, "f16", "any"), (120, 1, 112, 640, 1096, "bf16", "one")]


@pytest.mark.parametrize("case", CASES)
def test_adapters(case):
    T, S, r, K, N, dtype, kind = case
    p = problem(*case, seed=T + r)
    t = map_of(p, S)
    want, want_u = R.adapters(p["x"], p["a"], p["b"], p["ids"], p["scales"], p["base"])
    dev = dict(scales=p["scales"].cuda(), base=pitched(p["base"], 8))
    y, u = bsgg.adapters(pitched(p["x"], 24), p["a"].cuda(), p["b"].cuda(), t, **dev)
    at = p["ids"].clamp(min=0).long()
    sizes = torch.einsum("tk,trk->tr", p["x"].double().abs(), p["a"].double().abs()[at])
    utol = sizes * product_error(K)
    assert ((u.cpu().double() - want_u).abs() <= utol + 1e-38).all()
    dt = DT[dtype]
    # of the row's largest |u| for the terms; b's products in up to 8 steps of 16
    largest = want_u.abs().amax(1, keepdim=True)
    f = p["scales"].double()[at][:, None]
    bs = p["b"].double().abs()[at]
    tol = f * (torch.einsum("tr,trn->tn", utol + largest * TERMS[dt], bs) +
               torch.einsum("tr,trn->tn", want_u.abs(), bs) * product_error(2 * r))
    tol = torch.where((p["ids"] >= 0)[:, None], tol, torch.zeros_like(tol))
    assert ((y.cpu().double() - want).abs() <= tol + want.abs() * 2.0 ** -23 + rounding(want, dt)).all()
    none = p["ids"] < 0
    assert torch.equal(y.cpu()[none], p["base"][none]) and (u.cpu()[none] == 0).all()
    # in place, and into a wider buffer
    into = pitched(p["base"], 8)
    same, _ = bsgg.adapters(p["x"].cuda(), p["a"].cuda(), p["b"].cuda(), t, scales=dev["scales"], base=into, out=into)
    assert same is into and torch.equal(into, y)
    out = pitched(torch.zeros_like(p["base"]), 16)
    bsgg.adapters(p["x"].cuda(), p["a"].cuda(), p["b"].cuda(), t, out=out, **dev)
    assert torch.equal(out, y) and torch.isnan(out._base[:, N:].float()).all()
    # neither base nor scales
    want, _ = R.adapters(p["x"], p["a"], p["b"], p["ids"], None, None)
    z, _ = bsgg.adapters(p["x"].cuda(), p["a"].cuda(), p["b"].cuda(), t)
    assert ((z.cpu().double() - want).abs() <= tol / f + want.abs() * 2.0 ** -23 + rounding(want, dt)).all()
    # a map with more rows than it needs
    wide = map_of(p, S, m_pad=bsgg.sort_rows(T, S) + 384)
    assert torch.equal(bsgg.adapters(p["x"].cuda(), p["a"].cuda(), p["b"].cuda(), wide, **dev)[0], y)


@pytest.mark.parametrize("grads", [None, "f32"])
@pytest.mark.parametrize("case", CASES)
def test_adapters_backward(case, grads):
    T, S, r, K, N, dtype, kind = case
    p = problem(*case, seed=T + r + 1)
    t = map_of(p, S)
    dt = DT[dtype]
    gt = DT[dtype] if grads is None else torch.float32
    u = R.adapters(p["x"], p["a"], p["b"], p["ids"], None, None)[1].float()
    want_dx, want_da, want_db, want_du = R.adapters_backward(p["dy"], p["x"], u, p["a"], p["b"], p["ids"], p["scales"], p["basex"])
    args = (pitched(p["dy"], 8), pitched(p["x"], 16), u.cuda(), p["a"].cuda(), p["b"].cuda(), t)
    how = dict(scales=p["scales"].cuda(), base=p["basex"].cuda(), grad_format=grads)
    dx, da, db = bsgg.adapters_backward(*args, **how)
    assert da.dtype == gt and db.dtype == gt
    on = (p["ids"] >= 0)[:, None]
    at = p["ids"].clamp(min=0).long()
    f = p["scales"].double()[at][:, None]
    zero = torch.zeros((), dtype=torch.float64)
    dutol = torch.where(on, f * torch.einsum("tn,trn->tr", p["dy"].double().abs(), p["b"].double().abs()[at]) * product_error(N), zero)
    one = torch.nn.functional.one_hot(at, S).double() * on
    terms = 2.0 ** -23 if gt == torch.float32 and dt == torch.bfloat16 else TERMS[dt]
    largest = want_du.abs().amax(1, keepdim=True)
    as_ = p["a"].double().abs()[at]
    tol = torch.einsum("tr,trk->tk", dutol + largest * TERMS[dt], as_) + torch.einsum("tr,trk->tk", want_du.abs(), as_) * product_error(2 * r)
    assert ((dx.cpu().double() - want_dx).abs() <= tol + want_dx.abs() * 2.0 ** -23 + rounding(want_dx, dt)).all()
    # float16's terms are of the block's largest
    most = want_du.abs().max() if dt == torch.float16 else zero
    x = p["x"].double().abs()
    tol = torch.einsum("ts,tr,tk->srk", one, dutol + want_du.abs() * (terms + product_error(3 * T)) + most * TERMS[dt], x)
    assert ((da.cpu().double() - want_da).abs() <= tol + rounding(want_da, gt)).all()
    most = u.double().abs().max() if dt == torch.float16 else zero
    tol = torch.einsum("ts,tr,tn->srn", one * p["scales"].double(), u.double().abs() * (terms + product_error(3 * T)) + most * TERMS[dt],
                       p["dy"].double().abs())
    assert ((db.cpu().double() - want_db).abs() <= tol + want_db.abs() * 2.0 ** -23 + rounding(want_db, gt)).all()
    # an adapter without tokens has zeros, a token without an adapter its base
    unused = [i for i in range(S) if not (p["ids"] == i).any()]
    assert (da[unused] == 0).all() and (db[unused] == 0).all()
    none = p["ids"] < 0
    assert torch.equal(dx.cpu()[none], p["basex"][none])
    # each alone
    for i, name in enumerate(("want_dx", "want_da", "want_db")):
        only = bsgg.adapters_backward(*args, **{**dict(want_dx=False, want_da=False, want_db=False), name: True}, **how)
        assert [v is not None for v in only] == [j == i for j in range(3)] and torch.equal(only[i], (dx, da, db)[i])
    # the dense layer's own dx updated where it is
    into = p["basex"].cuda()
    assert bsgg.adapters_backward(*args, **{**how, "base": into}, dx=into, want_da=False, want_db=False)[0] is into and torch.equal(into, dx)


def test_gradients_are_those_of_the_forward_by_differences():
    """Adapters are linear in A, in B and in x, so differences are exact up to rounding."""
    T, S, r, K, N = 24, 2, 16, 64, 48
    p = problem(T, S, r, K, N, "f16", "any", 3)
    t = map_of(p, S)
    x, a, b, s, dy = (p[n].cuda() for n in ("x", "a", "b", "scales", "dy"))
    f = lambda x, a, b: (bsgg.adapters(x, a, b, t, scales=s)[0].double() * dy.double()).sum()  # noqa: E731
    u = bsgg.adapters(x, a, b, t, scales=s)[1]
    grads = bsgg.adapters_backward(dy, x, u, a, b, t, scales=s, grad_format="f32")
    y_size = bsgg.adapters(x.abs(), a.abs(), b.abs(), t, scales=s)[0].double()
    for i, v in enumerate((x, a, b)):
        d = torch.randn(v.shape, generator=gen(i)).to(v.dtype).cuda() * 0.25
        args = [[x, a, b], [x, a, b]]
        args[0][i], args[1][i] = v + d, v - d
        moved = (args[0][i].double() - args[1][i].double())
        want = float((grads[i].double() * moved).sum())
        # the two y are rounded to float16 (and dx is): |dy| 2^-11 of their sizes
        tol = 4 * float((dy.double().abs() * (y_size * 2 + 1)).sum()) * 2.0 ** -11 / (T * N) ** 0.5 * 6
        assert abs(float(f(*args[0]) - f(*args[1])) - want) <= tol


@pytest.mark.parametrize("T,S,r,K,N,dtype", [(3000, 3, 32, 1024, 1536, "bf16"), (2500, 5, 16, 4096, 2048, "f16"), (1100, 2, 64, 512, 8192, "bf16"),
                                             (2000, 2, 128, 256, 768, "f16"), (700, 40, 24, 512, 264, "bf16")])
def test_many_tokens_of_few_adapters(T, S, r, K, N, dtype):
    """Several tiles and segments of an adapter, long sums, against the same in 64 bits by products."""
    p = problem(T, S, r, K, N, dtype, "runs", 7)
    t = map_of(p, S)
    x, a, b, base, dy = (p[n].cuda() for n in ("x", "a", "b", "base", "dy"))
    y, u = bsgg.adapters(x, a, b, t, base=base)
    dx, da, db = bsgg.adapters_backward(dy, x, u, a, b, t, grad_format="f32")
    far = lambda g, w: float((g.double() - w).norm() / w.norm())  # noqa: E731
    ids = p["ids"].cuda()
    want_y, want_dx, want_da, want_db = base.double(), torch.zeros(T, K, dtype=torch.float64, device="cuda"), [], []
    for i in range(S):
        m = (ids == i).double()[:, None]
        ui, dui = m * (x.double() @ a[i].double().t()), m * (dy.double() @ b[i].double().t())
        want_y = want_y + ui @ b[i].double()
        want_dx += dui @ a[i].double()
        want_da.append(dui.t() @ x.double())
        want_db.append(ui.t() @ dy.double())
    # 16-bit results carry their own rounding, 2^-9.2 in norm; those in 32 bits the sums' 2^-19
    half = 2.0 ** -8.5 if dtype == "bf16" else 2.0 ** -11.5
    assert far(y, want_y) < half and far(dx, want_dx) < half
    assert far(da, torch.stack(want_da)) < 2.0 ** -19 and far(db, torch.stack(want_db)) < 2.0 ** -19
    for _ in range(2):                                # no order depends on timing
        again = bsgg.adapters_backward(dy, x, u, a, b, t, grad_format="f32")
        assert torch.equal(again[0], dx) and torch.equal(again[1], da) and torch.equal(again[2], db)


def test_float16_keeps_small_and_large_values():
    """du far below float16's smallest number and u far above its largest."""
    T, S, r, K, N = 20, 1, 16, 64, 64
    p = problem(T, S, r, K, N, "f16", "one", 9)
    t = map_of(p, S)
    a, b = (p["a"] * 2.0 ** -4).half(), (p["b"] * 2.0 ** -4).half()
    dy = (p["dy"].double() * 2.0 ** -13).half()
    u = torch.randn(T, r, generator=gen(1))
    dx, da, db = bsgg.adapters_backward(dy.cuda(), p["x"].cuda(), (u * 1e9).cuda(), a.cuda(), b.cuda(), t, grad_format="f32",
                                        scales=torch.full((1,), 2.0 ** -13).cuda())
    want = R.adapters_backward(dy, p["x"], u.double() * 1e9, a, b, p["ids"], torch.tensor([2.0 ** -13]), None)
    for g, w in ((da, want[1]), (db, want[2])):
        assert float((g.cpu().double() - w).norm() / w.norm()) < 2.0 ** -18
    x = (p["x"].double() * 2.0 ** 15).clamp(-60000, 60000).half()
    big = torch.full((1, r, K), 60000.0).half()
    tiny = torch.full((1, r, N), 2.0 ** -24).half()
    y, uu = bsgg.adapters(x.cuda(), big.cuda(), tiny.cuda(), t, scales=torch.full((1,), 2.0 ** -14).cuda())
    want, _ = R.adapters(x, big, tiny, p["ids"], torch.tensor([2.0 ** -14]), None)
    assert float(uu.abs().max()) > 1e6
    assert float((y.cpu().double() - want).norm() / want.norm()) < 2.0 ** -10


def test_streams_and_graph():
    """A captured step, replayed on new inputs; two streams at once."""
    T, S, r, K, N = 130, 4, 16, 256, 512
    p, q = problem(T, S, r, K, N, "bf16", "any", 5), problem(T, S, r, K, N, "bf16", "runs", 6)
    dev = {n: v.cuda() for n, v in p.items()}
    ids = dev["ids"].view(-1, 1)

    def step(ids, d):
        t = bsgg.sort_tokens(ids, S)
        y, u = bsgg.adapters(d["x"], d["a"], d["b"], t, scales=d["scales"], base=d["base"])
        return (y, u) + bsgg.adapters_backward(d["dy"], d["x"], u, d["a"], d["b"], t, scales=d["scales"], base=d["basex"])

    want_p = [v.clone() for v in step(ids, dev)]
    other = {n: v.cuda() for n, v in q.items()}
    want_q = [v.clone() for v in step(other["ids"].view(-1, 1), other)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ids, dev)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want_p))
    for n in dev:
        dev[n].copy_(other[n])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want_q))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(step(ids, dev))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want_q))


def test_offsets_past_32_bits():
    """Rows of x, base and y that lie more than 2^31 elements from the first."""
    K = N = 16384
    T = 2 ** 31 // K + 40
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T, 1), -1, dtype=torch.int32)
    last = [T - 1, T - 2, T - 17, 5]
    ids[last] = 1
    g = gen(3)
    rows = torch.randn(len(last), K, generator=g).bfloat16()
    x[last] = rows.cuda()
    a, b = (torch.randn(2, 8, K, generator=g) / K ** 0.5).bfloat16(), torch.randn(2, 8, N, generator=g).bfloat16()
    t = bsgg.sort_tokens(ids.cuda(), 2)
    y, u = bsgg.adapters(x, a.cuda(), b.cuda(), t, base=x)
    want, want_u = R.adapters(rows, a, b, [1] * len(last), None, rows)
    got = y[last].cpu().double()
    assert ((got - want).abs() <= 2.0 ** -6 + rounding(want, torch.bfloat16)).all()
    assert torch.equal(y[:5], x[:5]) and torch.equal(y[T - 16:T - 2], x[T - 16:T - 2]) and (u[:5] == 0).all()
    dx, da, db = bsgg.adapters_backward(y, x, u, a.cuda(), b.cuda(), t, grad_format="f32")
    assert (da[0] == 0).all() and (db[0] == 0).all()
    w = u[last].double().t() @ y[last].double()
    assert float((db[1].double() - w).norm() / w.norm()) < 2.0 ** -18
    w = (y[last].double() @ b[1].cuda().double().t()) @ a[1].cuda().double()
    assert float((dx[last].double() - w).norm() / w.norm()) < 2.0 ** -8.5 and (dx[:5] == 0).all()


def test_no_tokens():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    a, b = (torch.zeros(2, 8, n, dtype=torch.bfloat16, device="cuda") for n in (64, 32))
    t = bsgg.sort_tokens(torch.empty(0, 1, dtype=torch.int32, device="cuda"), 2)
    y, u = bsgg.adapters(x, a, b, t)
    assert y.shape == (0, 32) and u.shape == (0, 8)
    dx, da, db = bsgg.adapters_backward(y, x, u, a, b, t)
    assert dx.shape == (0, 64) and (da == 0).all() and (db == 0).all()


def test_a_map_with_too_few_rows():
    """Tokens that the sort had no row for are tokens without an adapter, of an adapter cut
    in the middle and of one that is left out as a whole."""
    T, S, r, K, N = 1200, 4, 16, 128, 192
    p = problem(T, S, r, K, N, "bf16", "any", seed=5)
    t = map_of(p, S, m_pad=384)
    assert bsgg.operators_status() == 5
    cut = p["ids"].clone()
    cut[t.row_of_slot.view(-1).cpu() < 0] = -1
    sizes = [int((cut == i).sum()) for i in range(S)]
    assert 128 < sizes[0] <= 256 and sizes[1:] == [128, 0, 0] and int((p["ids"] == 1).sum()) > 128
    whole = map_of({"ids": cut}, S)
    dev = {k: p[k].cuda() for k in ("x", "a", "b", "scales", "base", "dy", "basex")}
    y, u = bsgg.adapters(dev["x"], dev["a"], dev["b"], t, scales=dev["scales"], base=dev["base"])
    want = bsgg.adapters(dev["x"], dev["a"], dev["b"], whole, scales=dev["scales"], base=dev["base"])
    assert torch.equal(y, want[0]) and torch.equal(u, want[1])
    got, want = (bsgg.adapters_backward(dev["dy"], dev["x"], u, dev["a"], dev["b"], m, scales=dev["scales"], base=dev["basex"])
                 for m in (t, whole))
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_offsets_that_the_sort_does_not_write():
    """Offsets out of order, negative, past the map or off the multiples of 128 give some
    gradient, of no memory but the arguments' own."""
    T, S, r, K, N = 700, 3, 24, 64, 136
    p = problem(T, S, r, K, N, "bf16", "any", seed=6)
    t = map_of(p, S)
    dev = {k: p[k].cuda() for k in ("x", "a", "b", "base", "dy")}
    m = t.slot_of_row.numel()
    for offsets, used in (([5, 261, m - 3], m + 7), ([m, -128, 384], m), ([1 << 30, 1 << 30, 1 << 30], 1 << 30), ([-5, -5, -5], -1)):
        bad = t._replace(padded_offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                         rows_used=torch.tensor([used], dtype=torch.int32, device="cuda"))
        y, u = bsgg.adapters(dev["x"], dev["a"], dev["b"], bad, base=dev["base"])
        for grads in (None, "f32"):
            bsgg.adapters_backward(dev["dy"], dev["x"], u, dev["a"], dev["b"], bad, grad_format=grads)
    torch.cuda.synchronize()
    # what a good map gives is what it gave
    first = bsgg.adapters_backward(dev["dy"], dev["x"], u, dev["a"], dev["b"], t)
    again = bsgg.adapters_backward(dev["dy"], dev["x"], u, dev["a"], dev["b"], t)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("grads", [None, "f32"])
@pytest.mark.parametrize("T,S,r,K,N,dtype", [(16, 1, 8, 64, 128256, "bf16"), (1, 2, 16, 64, 128256, "bf16"), (40, 3, 24, 128256, 72, "f16"),
                                             (300, 2, 72, 64, 128256, "bf16"), (500, 1, 40, 151936, 136, "f16")])
def test_gradients_of_wide_layers(T, S, r, K, N, dtype, grads):
    """Beside an output head: so wide that a segment of all tokens has more blocks than fill the
    chip, from one token up, several chunks of an adapter's rows among them."""
    p = problem(T, S, r, K, N, dtype, "any" if S > 1 else "one", seed=T + r)
    p["ids"][0] = S - 1                                  # a token, where there is one
    t = map_of(p, S)
    dt, gt = DT[dtype], DT[dtype] if grads is None else torch.float32
    x, a, b, s, dy, base = (p[n].cuda() for n in ("x", "a", "b", "scales", "dy", "basex"))
    u = torch.randn(T, r, generator=gen(r)).cuda()
    dx, da, db = bsgg.adapters_backward(dy, x, u, a, b, t, scales=s, base=base, grad_format=grads)
    ids = p["ids"].cuda()
    want_dx, tol_dx = base.double(), torch.zeros(T, K, dtype=torch.float64, device="cuda")
    terms = 2.0 ** -23 if gt == torch.float32 and dt == torch.bfloat16 else TERMS[dt]
    for i in range(S):
        m, f = (ids == i).double()[:, None], float(s[i])
        dui, ui = f * m * (dy.double() @ b[i].double().t()), f * m * u.double()
        err = f * m * (dy.double().abs() @ b[i].double().abs().t()) * product_error(N)
        # float16's terms are of the largest: of the row for dx, of the segment for the gradients
        size = dui.abs().amax(1, keepdim=True) if dt == torch.float16 else dui.abs()
        want_dx = want_dx + dui @ a[i].double()
        tol_dx += (err + size * TERMS[dt] + dui.abs() * product_error(2 * r)) @ a[i].double().abs()
        for got, g, e, v in ((da[i], dui, err, x), (db[i], ui, torch.zeros_like(err), dy)):
            want = g.t() @ v.double()
            size = g.abs().max() if dt == torch.float16 else g.abs()
            tol = (e + size * terms * m + g.abs() * product_error(3 * T)).t() @ v.double().abs()
            assert ((got.double() - want).abs() <= tol + want.abs() * 2.0 ** -23 + rounding(want, gt)).all()
    assert ((dx.double() - want_dx).abs() <= tol_dx + want_dx.abs() * 2.0 ** -23 + rounding(want_dx, dt)).all()


def gradients_in_64_bits(p, u, S):
    """(du, da, db) by products in 64 bits on the GPU, scales none."""
    ids, x, b, dy = (p[n].cuda() for n in ("ids", "x", "b", "dy"))
    da, db, du = [], [], torch.zeros(u.shape, dtype=torch.float64, device="cuda")
    for i in range(S):
        m = (ids == i).double()[:, None]
        di = m * (dy.double() @ b[i].double().t())
        du += di
        da.append(di.t() @ x.double())
        db.append((m * u.double()).t() @ dy.double())
    return du, da, db


@pytest.mark.parametrize("T,S,r,K,N,dtype", [(3000, 3, 64, 1024, 1536, "bf16"), (2000, 2, 128, 256, 768, "f16"), (1100, 2, 64, 512, 8192, "f16"),
                                             (3000, 3, 32, 1024, 1536, "bf16"), (2500, 5, 16, 4096, 2048, "f16"), (2600, 2, 88, 1032, 520, "bf16"),
                                             (4100, 1, 128, 2048, 264, "bf16"), (1900, 3, 40, 4096, 8192, "f16")])
def test_gradients_into_16_bits_of_several_segments(T, S, r, K, N, dtype):
    """da and db in the tokens' own type, of adapters whose tokens lie in several segments."""
    p = problem(T, S, r, K, N, dtype, "runs" if S > 1 else "one", 11)
    t = map_of(p, S)
    x, a, b, dy = (p[n].cuda() for n in ("x", "a", "b", "dy"))
    u = torch.randn(T, r, generator=gen(r)).cuda()
    dt = DT[dtype]
    _, da, db = bsgg.adapters_backward(dy, x, u, a, b, t, want_dx=False)
    assert da.dtype == dt and db.dtype == dt
    du, want_da, want_db = gradients_in_64_bits(p, u, S)
    ids = p["ids"].cuda()
    for i in range(S):
        m = (ids == i).double()[:, None]
        err = m * (dy.double().abs() @ b[i].double().abs().t()) * product_error(N)
        for got, g, e, v, want in ((da[i], m * du, err, x, want_da[i]), (db[i], m * u.double(), 0 * err, dy, want_db[i])):
            # bfloat16's two terms are of each value, float16's of the largest
            size = g.abs() if dt == torch.bfloat16 else g.abs().max() * m
            tol = (e + size * TERMS[dt] + g.abs() * product_error(3 * T)).t() @ v.double().abs()
            assert ((got.double() - want).abs() <= tol + rounding(want, dt)).all()
    for _ in range(2):                                # no order depends on timing
        again = bsgg.adapters_backward(dy, x, u, a, b, t, want_dx=False)
        assert torch.equal(again[1], da) and torch.equal(again[2], db)


@pytest.mark.parametrize("T,r,dtype,grads", [(32768, 64, "bf16", "bf16"), (32768, 64, "f16", "f16"), (32768, 40, "f16", "f16"), (8192, 128, "f16", "f16"),
                                             (32768, 128, "bf16", "bf16"), (16384, 64, "bf16", "f16"), (32768, 32, "f16", "f16")])
def test_long_sums_of_one_sign_into_16_bits(T, r, dtype, grads):
    """A segment of 8192 to 32768 tokens of one adapter, all products of one sign: what the additions
    drop adds up, and stays under an eighth of the rounding to 16 bits."""
    K, N = 16384, 45056                                # 240 blocks of columns: one segment
    dt, gt = DT[dtype], DT[grads]
    g = torch.Generator(device="cuda").manual_seed(r)
    some = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    x, dy = (some(T, K) + 0.25).to(dt), (some(T, N) + 0.25).to(dt)
    u = some(T, r) + 0.25
    a = torch.zeros(1, r, K, dtype=dt, device="cuda")
    b = (some(1, r, N) / N).to(dt)
    t = bsgg.sort_tokens(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1)
    _, da, db = bsgg.adapters_backward(dy, x, u, a, b, t, want_dx=False, grad_format=grads)
    # (columns of the first and the last blocks)
    at_k, at_n = (torch.cat([torch.arange(300), torch.arange(w - 300, w)]).cuda() for w in (K, N))
    du = torch.cat([part.double() @ b[0].double().t() for part in dy.split(4096)])
    for got, g, v in ((da[0][:, at_k], du, x[:, at_k]), (db[0][:, at_n], u.double(), dy[:, at_n])):
        want = g.t() @ v.double()
        off = (got.double() - want) / want
        # du's own sums are in runs, a rounding for each; float16's terms are of the largest, up to 8
        # times the value
        terms = TERMS[dt] * (8 if dt == torch.float16 else 1) + product_error(512) + N / 512 * 2.0 ** -24
        assert (off.abs() <= 1.125 * ROUND[gt] + terms).all()
        # roundings to 16 bits are of either sign: their mean over n values is within 6 of their
        # own standard errors
        assert abs(float(off.mean())) <= 0.125 * ROUND[gt] + terms + 6 * ROUND[gt] / off.numel() ** 0.5
