"""Routing, sort by expert, dispatch and combine on the GPU against 64-bit
references: sizes from one token up, odd ones, pitches wider than the rows,
masked experts, masked tokens, ties, infinities and NaN."""
import math

import numpy as np
import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
import operator_refs as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def pitched(t, extra):
    """t on the GPU as a view of a wider buffer (extra columns, poisoned)."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), math.nan, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]]


# ------------------------------------------------------------------ route
ROUTE = [(1, 1, 1, "f32"), (1, 8, 2, "bf16"), (5, 33, 8, "f16"), (128, 64, 8, "bf16"), (67, 128, 4, "f32"),
         (9, 129, 3, "f32"), (31, 300, 32, "f16"), (3, 1024, 6, "bf16"), (257, 60, 4, "bf16")]


def logits_of(T, L, dtype, seed):
    l = torch.randn(T, L, generator=gen(seed)).to(DT[dtype])
    if L > 2:
        l[:, L // 2] = l[:, L // 2 - 1]              # a tie in every row
    if T > 2:
        l[1, :] = -math.inf                          # nothing left
        l[2, 1:] = -math.inf                         # one expert left
    if T > 4:
        l[4, ::2] = -math.inf
        l[3, :] = torch.finfo(DT[dtype]).min         # a mask of the type's lowest value: all equal
    return l


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,L,k,dtype", ROUTE)
def test_route(T, L, k, dtype, normalize):
    l = logits_of(T, L, dtype, 3 * T + L)
    want_ids, want_w = R.route(l, k, normalize)
    dev = pitched(l, 3)
    ids, w = bsgg.route(dev, k, normalize=normalize)
    assert torch.equal(ids.cpu(), want_ids)
    # exp(l - m): 2 ulp, its argument rounded once; a sum of up to L terms
    fin = l.double()[torch.isfinite(l) & (l > torch.finfo(l.dtype).min)]
    spread = float(fin.max() - fin.min()) if fin.numel() else 0.0
    tol = want_w * 2.0 ** -24 * (16 + L / 32 + k + 2 * spread)
    assert ((w.cpu().double() - want_w).abs() <= tol + 1e-38).all()

    g = torch.randn(T, k, generator=gen(7))
    dl = bsgg.route_backward(dev, ids, w, g.cuda(), normalize=normalize)
    want = R.route_backward(l, want_ids, g, normalize)
    scale = (g.double().abs() * want_w).sum(1, keepdim=True)
    p = R.route_weights_at(l.double(), torch.arange(L).expand(T, L), False) if not normalize else \
        torch.zeros(T, L, dtype=torch.float64).scatter_add_(1, want_ids.clamp(min=0).long(), want_w)
    big = torch.zeros(T, L, dtype=torch.float64).scatter_add_(1, want_ids.clamp(min=0).long(),
                                                                g.double().abs() * want_w) + p * scale
    tol = big * 2.0 ** -24 * (32 + L / 32 + 2 * k + 4 * spread) + R.rounding(want, l.dtype)
    assert ((dl.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("normalize", [True, False])
def test_route_gradient_against_differences(normalize):
    T, L, k = 6, 24, 5
    l = torch.randn(T, L, generator=gen(11))
    l[2, 3:20] = -math.inf
    g = torch.randn(T, k, generator=gen(12))
    dev = l.cuda()
    ids, w = bsgg.route(dev, k, normalize=normalize)
    dl = bsgg.route_backward(dev, ids, w, g.cuda(), normalize=normalize).cpu().double()
    ids = ids.cpu()
    h = 1e-5
    for i in range(L):
        if i == 3 or i == 10:
            pass
        step = torch.zeros(T, L, dtype=torch.float64)
        step[:, i] = h
        up = R.route_weights_at(l.double() + step, ids, normalize)
        dn = R.route_weights_at(l.double() - step, ids, normalize)
        diff = ((up - dn) * g.double()).sum(1) / (2 * h)
        # differences of second order: h^2 times third derivatives below 1, and 1e-16 / h
        assert ((dl[:, i] - diff).abs() <= 1e-9 + 1e-6 * g.double().abs().sum(1)).all()


def test_route_nan_and_infinity():
    l = torch.randn(4, 20, generator=gen(5))
    l[0, 7] = math.nan
    l[1, 3] = math.inf
    ids, w = bsgg.route(l.cuda(), 4)
    ids, w = ids.cpu(), w.cpu()
    assert ids[0, 0] == 7 and torch.isnan(w[0]).all()
    assert ids[1, 0] == 3 and torch.isnan(w[1, 0])        # inf - inf
    want_ids, want_w = R.route(l[2:], 4, True)
    assert torch.equal(ids[2:], want_ids) and torch.allclose(w[2:].double(), want_w, rtol=1e-5)


def test_route_backward_of_a_row_gradient():
    """dweights taken per row (the backward GEMM's dprob) through row_of_slot."""
    T, L, k = 50, 16, 4
    l = torch.randn(T, L, generator=gen(8))
    l[5] = -math.inf
    ids, w = bsgg.route(l.cuda(), k)
    tm = bsgg.sort_tokens(ids, L)
    dprob = torch.randn(tm.slot_of_row.numel(), generator=gen(9)).cuda()
    row = tm.row_of_slot.long()
    g = torch.where(row >= 0, dprob[row.clamp(min=0)], torch.zeros((), device="cuda"))
    a = bsgg.route_backward(l.cuda(), ids, w, dprob, row_of_slot=tm.row_of_slot)
    b = bsgg.route_backward(l.cuda(), ids, w, g)
    assert torch.equal(a, b)


def test_route_of_no_tokens():
    ids, w = bsgg.route(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


# ------------------------------------------------------------------ sort
def ids_of(T, L, k, seed, masked):
    g = gen(seed)
    like = torch.randn(L, generator=g)
    ids = torch.sort(torch.randn(T, L, generator=g) + like, dim=1, descending=True).indices[:, :k].to(torch.int32)
    if masked:
        ids[::3, 0] = -1
        ids[1::7] = L + 5                    # another process's expert
    return ids


SORT = [(1, 8, 1, False), (1, 64, 8, False), (128, 64, 8, False), (333, 5, 2, True), (1000, 1024, 8, True),
        (4096, 8, 2, False), (1025, 128, 4, True), (8191, 64, 8, True), (20000, 60, 4, True)]


@pytest.mark.parametrize("T,L,k,masked", SORT)
def test_sort_tokens(T, L, k, masked):
    ids = ids_of(T, L, k, T + L, masked)
    w = torch.rand(T, k, generator=gen(1))
    m_pad = bsgg.sort_rows(T * k, L)
    tm = bsgg.sort_tokens(ids.cuda(), L, weights=w.cuda())
    offsets, row_of_slot, slot_of_row, used = R.sort_tokens(ids, L, m_pad)
    assert tm.padded_offsets.cpu().tolist() == offsets
    assert tm.row_of_slot.cpu().reshape(-1).tolist() == row_of_slot
    assert tm.slot_of_row.cpu().tolist() == slot_of_row
    assert tm.rows_used.cpu().tolist() == [used]
    s = torch.tensor(slot_of_row)
    want = torch.where(s >= 0, w.reshape(-1)[s.clamp(min=0)], torch.zeros(()))
    assert torch.equal(tm.prob.cpu(), want)
    assert bsgg.operators_status() == 0
    # the least m_pad gives the same rows
    if 0 < used < m_pad:
        tight = bsgg.sort_tokens(ids.cuda(), L, m_pad=used)
        assert tight.slot_of_row.cpu().tolist() == slot_of_row[:used]
        assert bsgg.operators_status() == 0


@pytest.mark.parametrize("T,L,k", [(1, 7, 1), (1, 8, 3), (5, 3, 1), (3001, 5, 3)])
def test_sort_outputs_are_aligned(T, L, k):
    """Every output where the grouped GEMM accepts it: 16-byte aligned."""
    tm = bsgg.sort_tokens(ids_of(T, L, k, 3, False).cuda(), L)
    assert all(t.data_ptr() % 16 == 0 for t in tm)


def test_sort_of_nothing():
    for ids in (torch.full((7, 3), -1, dtype=torch.int32), torch.empty(0, 3, dtype=torch.int32)):
        tm = bsgg.sort_tokens(ids.cuda(), 6)
        assert tm.padded_offsets.cpu().tolist() == [0] * 5 + [bsgg.sort_rows(ids.numel(), 6)]
        assert (tm.slot_of_row == -1).all() and (tm.row_of_slot == -1).all() and (tm.prob == 0).all()
        assert tm.rows_used.item() == 0


@pytest.mark.parametrize("T", [300, 9000])
def test_sort_into_too_few_rows_is_reported(T):
    ids = ids_of(T, 8, 2, 1, False)
    m_pad = 256
    tm = bsgg.sort_tokens(ids.cuda(), 8, m_pad=m_pad)
    assert bsgg.operators_status() == 5
    assert bsgg.operators_status() == 0           # read and cleared
    offsets, row_of_slot, slot_of_row, _ = R.sort_tokens(ids, 8, m_pad)
    assert tm.padded_offsets.cpu().tolist() == offsets
    assert tm.row_of_slot.cpu().reshape(-1).tolist() == row_of_slot
    assert tm.slot_of_row.cpu().tolist() == slot_of_row


def test_sort_prob_without_weights_is_one():
    tm = bsgg.sort_tokens(ids_of(70, 4, 2, 2, True).cuda(), 4)
    assert torch.equal(tm.prob, (tm.slot_of_row >= 0).float())


# ------------------------------------------------------------------ dispatch
def tokens_of(T, H, dtype, seed):
    x = torch.randn(T, H, generator=gen(seed))
    x[:, ::37] *= 30.0
    x *= torch.exp2(torch.randint(-12, 8, (T, 1), generator=gen(seed + 1)).float())
    x[0, :min(H, 32)] = 0.0                                   # a block of zeros
    if T > 1:
        x[1, 0], x[1, 5] = 448.0, -448.0                      # a maximum at the top of the scale
    if T > 3:
        x[3, :] = 0.0
        x[3, 0] = 2.0 ** -24                                  # the smallest scales
    return x.to(DT[dtype])


DISPATCH = [("mxfp8_e4m3", "bf16", 1, 7168, 8, 64), ("mxfp8_e4m3", "f32", 37, 48, 2, 5), ("mxfp8_e5m2", "f16", 130, 272, 4, 9),
            ("nvfp4", "bf16", 65, 544, 2, 8), ("nvfp4", "f32", 20, 32, 3, 4), ("fp4_ue8m0_16", "f16", 33, 96, 1, 3),
            ("mxfp4", "bf16", 50, 2080, 2, 8), ("bf16", "f32", 40, 24, 2, 6), ("f16", "f16", 40, 1032, 2, 6),
            ("bf16", "bf16", 300, 8, 8, 16), ("mxfp8_e4m3", "bf16", 700, 4096, 2, 8)]


@pytest.mark.parametrize("fmt,dtype,T,H,k,L", DISPATCH)
def test_dispatch(fmt, dtype, T, H, k, L):
    x = tokens_of(T, H, dtype, T + H)
    ids = ids_of(T, L, k, T, T > 10)
    m_pad = bsgg.sort_rows(T * k, L)
    _, row_of_slot, slot_of_row, _ = R.sort_tokens(ids, L, m_pad)
    dev = pitched(x, 16)
    rs = torch.tensor(row_of_slot, dtype=torch.int32).view(T, k).cuda()
    sr = torch.tensor(slot_of_row, dtype=torch.int32).cuda()
    a, sfa = bsgg.dispatch(dev, rs, sr, in_format=fmt)
    s = torch.tensor(slot_of_row)
    token = (s.clamp(min=0) // k)
    on = s >= 0
    if fmt in ("bf16", "f16"):
        want = torch.where(on[:, None], x.float()[token], torch.zeros(())).to(DT[fmt])
        assert sfa is None and torch.equal(a.cpu().view(torch.int16), want.view(torch.int16))
        return
    codes, scodes = R.quantize(x.double(), fmt)
    one = 0x38 if fmt == "nvfp4" else 127
    want = torch.where(on[:, None], R.pack_codes(codes, fmt)[token], torch.zeros((), dtype=torch.uint8))
    wsf = torch.where(on[:, None], scodes[token], torch.full((), one, dtype=torch.uint8))
    assert torch.equal(a.cpu(), want)
    assert torch.equal(sfa.cpu(), R.swizzle(wsf))


@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp8_e5m2", "nvfp4", "mxfp4"])
def test_dispatch_infinity_and_nan(fmt):
    """A block with one gets the NaN scale and zero codes, its neighbours nothing;
    a token without a row may hold anything."""
    x = torch.randn(6, 128, generator=gen(3))
    x[0, 40] = math.nan
    x[1, 100] = -math.inf
    x[2, :] = math.nan
    ids = torch.tensor([[0], [1], [-1], [0], [1], [0]], dtype=torch.int32)
    _, row_of_slot, slot_of_row, _ = R.sort_tokens(ids, 2, 256)
    a, sfa = bsgg.dispatch(x.cuda(), torch.tensor(row_of_slot, dtype=torch.int32).view(6, 1).cuda(),
                           torch.tensor(slot_of_row, dtype=torch.int32).cuda(), in_format=fmt)
    s = torch.tensor(slot_of_row)
    on, token = s >= 0, s.clamp(min=0)
    codes, scodes = R.quantize(x.double(), fmt)
    one = 0x38 if fmt == "nvfp4" else 127
    assert torch.equal(a.cpu(), torch.where(on[:, None], R.pack_codes(codes, fmt)[token], torch.zeros((), dtype=torch.uint8)))
    assert torch.equal(sfa.cpu(), R.swizzle(torch.where(on[:, None], scodes[token], torch.full((), one, dtype=torch.uint8))))


def test_dispatch_feeds_the_grouped_gemm():
    """sort -> dispatch -> the gated grouped GEMM -> combine equals the tokens'
    own products, prob applied in the GEMM's epilogue."""
    T, L, k, K, N = 200, 4, 2, 256, 256
    g = gen(2)
    x = torch.randn(T, K, generator=g).bfloat16()
    wts = torch.randn(L, N, K, generator=g) / 16
    ids = ids_of(T, L, k, 4, False)
    pr = torch.rand(T, k, generator=g)
    from block_scaled_grouped_gb300 import workloads as W
    b, sfb = zip(*[W.quantize_mxfp8(wts[e], "mxfp8_e4m3") for e in range(L)])
    tm = bsgg.sort_tokens(ids.cuda(), L, weights=pr.cuda())
    m_pad = tm.slot_of_row.numel()
    a, sfa = bsgg.dispatch(x.cuda(), tm.row_of_slot, tm.slot_of_row)
    plan = bsgg.Plan(m_pad=m_pad, n=N, k=K, num_groups=L, in_format="mxfp8_e4m3", out_format="f32", epilogue="gate")
    d = torch.empty(m_pad, N, device="cuda")
    plan.run(a=a, sfa=sfa, b=torch.stack(b).cuda(), sfb=bsgg.pack_sf(torch.stack(sfb).cuda()),
             padded_offsets=tm.padded_offsets, alpha=torch.ones(L, device="cuda"), prob=tm.prob, d=d)
    assert plan.device_status() == 0
    y = bsgg.combine(d, tm.row_of_slot)
    codes, sc = R.quantize(x.double(), "mxfp8_e4m3")
    deq = lambda c, s: c.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).repeat_interleave(32, -1)  # noqa: E731
    xq = deq(codes, sc)
    wq = deq(torch.stack(b), torch.stack(sfb))
    want = torch.zeros(T, N, dtype=torch.float64)
    size = torch.zeros(T, N, dtype=torch.float64)
    for j in range(k):
        e = ids[:, j].long()
        want += pr[:, j, None].double() * torch.einsum("tk,tnk->tn", xq, wq[e])
        size += pr[:, j, None].double() * torch.einsum("tk,tnk->tn", xq.abs(), wq[e].abs())
    assert ((y.cpu().double() - want).abs() <= R.product_error(K) * size).all()


# ------------------------------------------------------------------ combine
COMBINE = [(1, 8, 1, 2, "bf16", "bf16", True), (1, 7168, 8, 64, "bf16", "bf16", True), (37, 264, 3, 5, "f16", "f32", True),
           (100, 1032, 4, 8, "f32", "bf16", False), (513, 4096, 2, 8, "bf16", "f16", True), (60, 24, 8, 16, "f32", "f32", True)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,H,k,L,dk,yk,res", COMBINE)
def test_combine(T, H, k, L, dk, yk, res, weighted):
    ids = ids_of(T, L, k, H, T > 10)
    m_pad = bsgg.sort_rows(T * k, L)
    _, row_of_slot, slot_of_row, _ = R.sort_tokens(ids, L, m_pad)
    g = gen(T + H)
    d = torch.randn(m_pad, H, generator=g).to(DT[dk])
    d[torch.tensor(slot_of_row) < 0] = math.nan               # padding rows are not read
    w = torch.rand(T, k, generator=g)
    residual = torch.randn(T, H, generator=g).to(DT[yk]) if res else None
    rs = torch.tensor(row_of_slot, dtype=torch.int32).view(T, k)
    out = pitched(torch.zeros(T, H, dtype=DT[yk]), 8)
    y = bsgg.combine(d.cuda(), rs.cuda(), weights=w.cuda() if weighted else None,
                     residual=pitched(residual, 24) if res else None, out_format=yk, out=out)
    assert y is out
    want = residual.double() if res else torch.zeros(T, H, dtype=torch.float64)
    size = want.abs()
    for j in range(k):
        r = rs[:, j].long()
        v = torch.where((r >= 0)[:, None], d.double()[r.clamp(min=0)], torch.zeros((), dtype=torch.float64))
        v = v * (w[:, j, None].double() if weighted else 1.0)
        want, size = want + v, size + v.abs()
    tol = size * (k + 2) * 2.0 ** -24 + R.rounding(want, DT[yk])
    assert ((y.cpu().double() - want).abs() <= tol).all()
    # rows past the end of each row of `out` stay
    assert torch.isnan(out.as_strided((T, 8), (H + 8, 1), H)).all()

    # the gradient, rows in 16 bits
    dy = torch.randn(T, H, generator=g).to(DT[yk])
    fmt = "f16" if dk == "f16" else "bf16"
    sr = torch.tensor(slot_of_row, dtype=torch.int32).cuda()
    dd, sf, dw = bsgg.combine_backward(pitched(dy, 8), d.cuda(), rs.cuda(), sr, weights=w.cuda() if weighted else None,
                                       out_format=fmt)
    s = torch.tensor(slot_of_row)
    on = (s >= 0)[:, None]
    ws = w.reshape(-1)[s.clamp(min=0)][:, None] if weighted else torch.ones(())
    want_dd = torch.where(on, dy.float()[s.clamp(min=0) // k] * ws, torch.zeros(()))
    assert sf is None and torch.equal(dd.cpu(), want_dd.to(DT[fmt]))
    r = rs.long()
    picked = torch.where((r >= 0)[..., None], d.double()[r.clamp(min=0)], torch.zeros((), dtype=torch.float64))
    want_dw = (picked * dy.double()[:, None, :]).sum(-1)
    size = (picked * dy.double()[:, None, :]).abs().sum(-1)
    assert ((dw.cpu().double() - want_dw).abs() <= size * (H / 32 + 8) * 2.0 ** -24).all()


@pytest.mark.parametrize("fmt", ["mxfp8_e5m2", "nvfp4", "mxfp8_e4m3"])
def test_combine_backward_into_quantized_rows(fmt):
    T, H, k, L = 90, 320, 3, 6
    ids = ids_of(T, L, k, 3, True)
    m_pad = bsgg.sort_rows(T * k, L)
    _, row_of_slot, slot_of_row, _ = R.sort_tokens(ids, L, m_pad)
    dy, w = torch.randn(T, H, generator=gen(1)), torch.rand(T, k, generator=gen(2))
    dd, sf, dw = bsgg.combine_backward(dy.cuda(), None, torch.tensor(row_of_slot, dtype=torch.int32).view(T, k).cuda(),
                                       torch.tensor(slot_of_row, dtype=torch.int32).cuda(), weights=w.cuda(),
                                       out_format=fmt, want_dweights=False)
    s = torch.tensor(slot_of_row)
    rows = torch.where((s >= 0)[:, None], dy[s.clamp(min=0) // k] * w.reshape(-1)[s.clamp(min=0)][:, None], torch.zeros(()))
    codes, sc = R.quantize(rows.double(), fmt)
    assert dw is None
    on = (s >= 0)[:, None]
    # the sign of a padding row's zeros is plus
    codes = torch.where(on, codes, torch.zeros((), dtype=torch.uint8))
    assert torch.equal(dd.cpu(), R.pack_codes(codes, fmt)) and torch.equal(sf.cpu(), R.swizzle(sc))


def test_combine_gradient_against_differences():
    T, H, k, L = 20, 64, 2, 4
    ids = ids_of(T, L, k, 6, True)
    m_pad = bsgg.sort_rows(T * k, L)
    _, row_of_slot, slot_of_row, _ = R.sort_tokens(ids, L, m_pad)
    g = gen(4)
    d, w, dy = torch.randn(m_pad, H, generator=g), torch.rand(T, k, generator=g), torch.randn(T, H, generator=g)
    rs = torch.tensor(row_of_slot, dtype=torch.int32).view(T, k)
    _, _, dw = bsgg.combine_backward(dy.cuda(), d.cuda(), rs.cuda(), torch.tensor(slot_of_row, dtype=torch.int32).cuda(),
                                     weights=w.cuda(), out_format="bf16")

    def loss(dd, ww):
        r = rs.long()
        picked = torch.where((r >= 0)[..., None], dd[r.clamp(min=0)], torch.zeros((), dtype=torch.float64))
        return ((picked * ww[..., None]).sum(1) * dy.double()).sum()

    dirw = torch.randn(T, k, generator=g).double()
    diff = (loss(d.double(), w.double() + dirw) - loss(d.double(), w.double() - dirw)) / 2     # linear in w
    assert abs((dw.cpu().double() * dirw).sum() - diff) <= 1e-5 * (dw.cpu().double() * dirw).abs().sum()
    # dispatch's adjoint is combine without weights: <dispatch(x), v> = <x, combine(v)>
    x = torch.randn(T, H, generator=g).bfloat16()
    v = torch.randn(m_pad, H, generator=g)
    a, _ = bsgg.dispatch(x.cuda(), rs.cuda(), torch.tensor(slot_of_row, dtype=torch.int32).cuda(), in_format="bf16")
    left = (a.cpu().double() * v.double()).sum()
    back = bsgg.combine(v.cuda(), rs.cuda()).cpu().double()
    assert abs(left - (x.double() * back).sum()) <= 1e-6 * (a.cpu().double() * v.double()).abs().sum()


def test_maps_out_of_range_count_as_no_row():
    """row_of_slot / slot_of_row entries outside their ranges touch nothing."""
    T, H, k, m_pad = 4, 32, 2, 128
    rs = torch.tensor([[0, 128], [-5, 2 ** 31 - 1], [1, -1], [2, 3]], dtype=torch.int32)
    sr = torch.full((m_pad,), -1, dtype=torch.int32)
    sr[0], sr[1], sr[2], sr[3], sr[4] = 0, 4, 6, 7, 8                  # 8 = tokens * topk
    x = torch.randn(T, H, generator=gen(1))
    a, _ = bsgg.dispatch(x.cuda(), rs.cuda(), sr.cuda(), in_format="bf16")
    want = torch.zeros(m_pad, H)
    want[0], want[1], want[2], want[3] = x[0], x[2], x[3], x[3]
    assert torch.equal(a.cpu(), want.bfloat16())
    y = bsgg.combine(want.cuda(), rs.cuda()).cpu()
    assert torch.equal(y, torch.stack([x[0], torch.zeros(H), x[2], x[3] + x[3]]))


def test_offsets_past_32_bits():
    """Rows whose elements lie past 2^31: written, padded and read where they are."""
    T, H, k, m_pad = 6, 8448, 2, 262144                            # 2.2e9 elements
    g = gen(51)
    rs = torch.randint(m_pad - 100000, m_pad, (T, k), generator=g, dtype=torch.int32)
    rs[0, 0], rs[1, 1], rs[2, 0] = m_pad - 1, -1, 3
    assert len(set(rs.reshape(-1).tolist())) == T * k
    sr = torch.full((m_pad,), -1, dtype=torch.int32)
    for s, r in enumerate(rs.reshape(-1).tolist()):
        if r >= 0:
            sr[r] = s
    x = torch.randn(T, H, generator=g).bfloat16()
    w = torch.rand(T, k, generator=g)
    a, sfa = bsgg.dispatch(x.cuda(), rs.cuda(), sr.cuda())
    codes, sc = R.quantize(x.double(), "mxfp8_e4m3")
    real = torch.nonzero(sr >= 0)[:, 0]
    token = sr[real].long() // k
    assert torch.equal(a[real.cuda()].cpu(), codes[token])
    assert int((a != 0).any(1).sum()) == real.numel()               # every padding row is zero
    kq = H // 128
    full = sfa.view(m_pad // 128, kq, 32, 4, 4)
    got = full[(real // 128).cuda(), :, (real % 32).cuda(), (real % 128 // 32).cuda()].reshape(real.numel(), -1).cpu()
    assert torch.equal(got, sc[token])
    assert int((sfa != 127).sum()) == int((got != 127).sum())        # and its scales one
    del a, sfa
    d = torch.zeros(m_pad, H, dtype=torch.bfloat16, device="cuda")
    d[real.cuda()] = x[token].cuda()
    y = bsgg.combine(d, rs.cuda(), weights=w.cuda(), out_format="f32").cpu().double()
    total = torch.where(rs >= 0, w, torch.zeros(())).double().sum(1, keepdim=True)
    assert ((y - total * x.double()).abs() <= 4 * 2.0 ** -24 * (total * x.double()).abs()).all()
    dd, _, dw = bsgg.combine_backward(x.cuda(), d, rs.cuda(), sr.cuda(), weights=w.cuda())
    ws = w.reshape(-1)[sr[real].long()][:, None]
    assert torch.equal(dd[real.cuda()].cpu(), (x[token].float() * ws).bfloat16())
    sq = (x.double() ** 2).sum(1, keepdim=True) * (rs >= 0)
    assert ((dw.cpu().double() - sq).abs() <= sq * (H / 32 + 8) * 2.0 ** -24).all()


def test_other_stream_and_graph():
    """The chain on a stream of its own, then captured in a graph and replayed on
    new values."""
    T, H, k, L = 128, 256, 4, 16
    g = gen(21)
    logits, x = torch.randn(T, L, generator=g), torch.randn(T, H, generator=g)

    def chain(l, t, stream):
        ids, w = bsgg.route(l, k, stream=stream)
        tm = bsgg.sort_tokens(ids, L, stream=stream)
        a, _ = bsgg.dispatch(t, tm.row_of_slot, tm.slot_of_row, in_format="bf16", stream=stream)
        return bsgg.combine(a, tm.row_of_slot, weights=w, out_format="f32", stream=stream)

    dl, dx = logits.cuda(), x.cuda()
    want = chain(dl, dx, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = chain(dl, dx, side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(dl, dx, None)
    for seed in (1, 2):
        dl.copy_(torch.randn(T, L, generator=gen(seed)))
        dx.copy_(torch.randn(T, H, generator=gen(seed + 9)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, chain(dl, dx, None))
