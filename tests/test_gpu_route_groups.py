"""The router with scores, a bias and groups on the GPU against 64-bit references:
every choice of score, bias, groups and weights, sizes from one token and one expert
up, masked experts and groups, ties, near ties and scores that leave 32 bits."""
import math

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
import layer_operator_refs as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def pitched(t, extra):
    """t on the GPU as a view of a wider buffer (extra columns, poisoned)."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), math.nan, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]]


def logits_of(T, L, dtype, seed):
    l = torch.randn(T, L, generator=gen(seed)).to(DT[dtype])
    if L > 2:
        l[:, L // 2] = l[:, L // 2 - 1]              # a tie in every row
    if T > 4:
        l[1, :] = -math.inf                          # nothing left
        l[2, 1:] = -math.inf                         # one expert left
        l[3, :] = torch.finfo(DT[dtype]).min         # a mask of the type's lowest value: all equal
        l[4, ::2] = -math.inf
    if T > 6:
        l[5, : L // 2] = -math.inf                   # groups without an expert
        l[6, :] = 0.0
    return l


def tolerance(l, ids, want, normalize):
    """Of the weights: an exponential is off by 2 units (2^-22) and its argument by half a unit of
    the row's spread, the division and the score's own sum add three roundings, sums have up
    to 69 terms in a row, and the factor one rounding."""
    fin = torch.where(torch.isfinite(l.double()) & (l > torch.finfo(l.dtype).min), l.double(), torch.zeros((), dtype=torch.float64))
    spread = (fin.amax(1) - fin.amin(1))[:, None]
    return want.abs() * 2.0 ** -24 * (2 * (4 + 3) + 69 + 2 + 2 * spread) + 2.0 ** -148


# tokens, experts, topk, groups, topk_groups, group_top
SHAPES = [(1, 1, 1, 1, 1, 1), (7, 8, 2, 1, 1, 2), (128, 64, 8, 8, 4, 2), (33, 256, 8, 8, 4, 2), (9, 60, 6, 5, 2, 1), (17, 33, 5, 3, 1, 2),
          (12, 64, 4, 32, 7, 2), (10, 1024, 32, 16, 3, 2), (8, 1023, 7, 31, 30, 1), (7, 1000, 4, 1, 1, 1), (9, 4, 4, 4, 4, 2),
          (8, 48, 3, 24, 2, 2)]


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("score,biased", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("shape", SHAPES)
def test_route_groups(shape, score, biased, normalize):
    T, L, k, groups, kept, top = shape
    dtype = ["f32", "bf16", "f16"][(T + L + normalize) % 3]
    l = logits_of(T, L, dtype, 7 * T + L)
    bias = torch.randn(L, generator=gen(L)) * (0.1 if score == "sigmoid" else 0.3 / L) if biased else None
    if biased and L > 8:
        bias[3] = -math.inf                          # an expert that is off
        bias[5], bias[6] = bias[4], bias[4]
    how = dict(score=score, normalize=normalize, scale=2.5)
    where = dict(groups=groups, topk_groups=kept, group_top=top)
    want_ids, want_w = R.route_groups(l, k, bias=bias, **where, **how)
    dev = pitched(l, 3)
    ids, w = bsgg.route_groups(dev, k, bias=None if bias is None else bias.cuda(), **where, **how)
    assert torch.equal(ids.cpu(), want_ids)
    assert ((w.cpu().double() - want_w).abs() <= tolerance(l, want_ids, want_w, normalize)).all()


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,L,k,dtype", [(1, 1, 1, "f32"), (9, 33, 8, "f16"), (128, 64, 8, "bf16"), (67, 256, 4, "f32"), (10, 1000, 32, "f32")])
def test_route_groups_backward(T, L, k, dtype, score, normalize):
    l = logits_of(T, L, dtype, T + L)
    l[l == torch.finfo(l.dtype).min] = -3.0
    how = dict(score=score, normalize=normalize, scale=1.5)
    ids, w = R.route_groups(l, k, **how)
    g = torch.randn(T, k, generator=gen(1))
    want = R.route_groups_backward(l, ids, g, **how)
    dev = pitched(l, 5)
    args = (dev, ids.cuda(), w.float().cuda())
    got = bsgg.route_groups_backward(*args, g.cuda(), **how)
    # the weights (rounded), 1 - s (2^-21) and inner, a sum of up to 32 products with five
    # roundings, each to 2^-20 of the terms' sizes; softmax over all: as the forward's scores
    on = ids >= 0
    gw = torch.where(on, g.double().abs() * w, torch.zeros_like(w))
    inner = gw.sum(1, keepdim=True) / 1.5
    sizes = torch.zeros(T, L, dtype=torch.float64).scatter_add_(1, ids.clamp(min=0).long(), gw + torch.where(on, w * inner, torch.zeros_like(w)))
    if score == "softmax" and not normalize:
        sizes += 1.5 * R.scores(l.double(), None, score)[0] * inner
    tol = sizes * 2.0 ** -17 + want.abs() * ROUND[l.dtype] + TINY[l.dtype]
    assert ((got.cpu().double() - want).abs() <= tol).all()
    # the same from a per-row gradient; slots without a row have none
    m_pad = 128 * (-(-T * k // 128))
    rows = torch.randperm(m_pad, generator=gen(2))[:T * k].to(torch.int32).view(T, k)
    per_row = torch.full((m_pad,), math.nan)
    per_row[rows.reshape(-1).long()] = g.reshape(-1)
    rows[0, 0] = -1
    g0 = g.clone()
    g0[0, 0] = 0.0
    out = pitched(torch.zeros(T, L, dtype=l.dtype), 5)
    same = bsgg.route_groups_backward(*args, per_row.cuda(), row_of_slot=rows.cuda(), dlogits=out, **how)
    assert same.data_ptr() == out.data_ptr()
    assert torch.equal(same, bsgg.route_groups_backward(*args, g0.cuda(), **how))
    # where the logits are
    assert torch.equal(bsgg.route_groups_backward(*args, g.cuda(), dlogits=dev, **how), got) and torch.isnan(dev._base[:, L:].float()).all()


def test_gradient_is_that_of_the_formula_by_differences():
    """The kernel's own weights, moved by differences (float32, so a coarse step)."""
    T, L, k = 16, 24, 4
    l = torch.randn(T, L, generator=gen(5)) * 0.5
    b = torch.randn(L, generator=gen(6)).cuda() * 3.0        # the choice stays where it is
    how = dict(score="sigmoid", normalize=True, scale=2.0)
    run = lambda x: bsgg.route_groups(x.cuda(), k, bias=b, groups=4, topk_groups=2, **how)  # noqa: E731
    ids, w = run(l)
    g = torch.randn(T, k, generator=gen(7))
    got = bsgg.route_groups_backward(l.cuda(), ids, w, g.cuda(), **how).cpu().double()
    step = 2.0 ** -6
    for e in range(L):
        d = torch.zeros_like(l)
        d[:, e] = step
        (iu, up), (io, down) = run(l + d), run(l - d)
        assert torch.equal(iu, ids) and torch.equal(io, ids)
        diff = ((up - down).cpu().double() * g.double()).sum(1) / (2 * step)
        # a third derivative of at most 2 sum |g|, times step^2 / 6; weights off by 2^-22 each
        tol = 2 * g.abs().double().sum(1) * (step ** 2 / 6 + 2.0 ** -21 / step)
        assert ((diff - got[:, e]).abs() <= tol).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_near_ties_are_decided_in_64_bits(score):
    """Scores that differ by less than 32 bits hold, in every row: bias and score add up to
    nearly the same for all experts, and so do the groups."""
    T, L, k = 64, 64, 6
    l = torch.randn(T, L, generator=gen(11)) * 0.5
    l[1:] = l[0] + torch.randn(T - 1, 1, generator=gen(12)) * 1e-7          # rows that differ in the last bits
    s = R.scores(l[:1].double(), None, score)[0][0]
    bias = (0.75 - s).float()                                                # c = 0.75 up to a rounding of 2^-25
    for groups, kept, top in ((1, 1, 1), (8, 3, 2), (8, 3, 1)):
        want, _ = R.route_groups(l, k, score=score, bias=bias, groups=groups, topk_groups=kept, group_top=top)
        ids, _ = bsgg.route_groups(l.cuda(), k, score=score, bias=bias.cuda(), groups=groups, topk_groups=kept, group_top=top)
        assert torch.equal(ids.cpu(), want), (groups, top)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_groups_without_a_bias_near_ties(score):
    """Sums of two scores that are equal, or nearly so, in another order."""
    T, L = 32, 32
    l = torch.zeros(T, L)
    base = torch.randn(T, 4, generator=gen(13))
    for q in range(8):                               # eight groups of four, the same logits in another order
        l[:, 4 * q: 4 * q + 4] = base[:, [(q + i) % 4 for i in range(4)]]
    l[::2, 20] += 1e-6                               # a group that leads by less than 32 bits of the sum show
    want, _ = R.route_groups(l, 5, score=score, groups=8, topk_groups=3, group_top=2)
    ids, _ = bsgg.route_groups(l.cuda(), 5, score=score, groups=8, topk_groups=3, group_top=2)
    assert torch.equal(ids.cpu(), want)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_ties_of_logits_of_few_bits(score, dtype):
    """bfloat16 logits with a bias of zeros, as training starts: equal scores in most rows,
    of experts and of groups."""
    T, L = 500, 64
    l = (torch.randn(T, L, generator=gen(29)) * 0.3).to(DT[dtype])
    l = torch.round(l.float() * 8).div(8).to(DT[dtype])
    for bias in (None, torch.zeros(L), torch.full((L,), 0.25)):
        for groups, kept, top in ((1, 1, 1), (8, 4, 2), (8, 4, 1), (4, 1, 2)):
            where = dict(score=score, groups=groups, topk_groups=kept, group_top=top)
            want, _ = R.route_groups(l, 6, bias=bias, **where)
            ids, _ = bsgg.route_groups(l.cuda(), 6, bias=None if bias is None else bias.cuda(), **where)
            assert torch.equal(ids.cpu(), want), (groups, top)


def test_a_router_of_zeros():
    """Logits and biases that are all the same: the first groups, the first experts; and groups
    of which some have a single expert left."""
    l = torch.zeros(40, 32)
    l[10:20, 1:8] = -math.inf
    l[20:30, ::2] = -math.inf
    for bias in (torch.zeros(32), torch.full((32,), 0.3)):
        for top in (1, 2):
            where = dict(groups=8, topk_groups=3, group_top=top)
            want, _ = R.route_groups(l, 6, bias=bias, **where)
            ids, _ = bsgg.route_groups(l.cuda(), 6, bias=bias.cuda(), **where)
            assert torch.equal(ids.cpu(), want)


def test_biases_larger_than_scores():
    """Groups whose terms cancel: large biases of both signs."""
    T, L = 64, 32
    l = torch.randn(T, L, generator=gen(31))
    bias = torch.randn(L, generator=gen(32)) * 30.0
    bias[::2] = bias[1::2] * -1.0
    for top in (1, 2):
        where = dict(groups=8, topk_groups=3, group_top=top)
        want, _ = R.route_groups(l, 5, bias=bias, **where)
        ids, _ = bsgg.route_groups(l.cuda(), 5, bias=bias.cuda(), **where)
        assert torch.equal(ids.cpu(), want)


def test_offsets_past_32_bits():
    T, L = 2 ** 21 + 3, 1024
    l = torch.zeros(T, L, dtype=torch.bfloat16, device="cuda")
    l[-1] = torch.randn(L, generator=gen(33)).bfloat16().cuda()
    ids, w = bsgg.route_groups(l, 3, score="sigmoid", groups=16, topk_groups=2)
    want, want_w = R.route_groups(l[-1:].cpu(), 3, groups=16, topk_groups=2)
    assert torch.equal(ids[-1:].cpu(), want) and (ids[:-1] == torch.arange(3, device="cuda", dtype=torch.int32)).all()
    dl = bsgg.route_groups_backward(l, ids, w, torch.ones_like(w), normalize=False)
    assert float(dl[-1, int(want[0, 0])]) != 0.0 and (dl[0, 3:] == 0).all()


def test_scores_below_the_smallest_number_keep_their_ratios():
    l = torch.tensor([[-200.0, -201.0, -300.0, -202.0], [90.0, 100.0, 95.0, -95.0], [-88.0, -89.0, -104.0, -87.0]])
    for score in ("sigmoid", "softmax"):
        want_ids, want = R.route_groups(l, 2, score=score, scale=3.0)
        ids, w = bsgg.route_groups(l.cuda(), 2, score=score, scale=3.0)
        assert torch.equal(ids.cpu(), want_ids)
        assert ((w.cpu().double() - want).abs() <= want * 2.0 ** -20).all()


def test_infinities_and_nan():
    """A NaN logit is the largest and makes the row's weights NaN; a bias of -inf turns an
    expert off, one of +inf forces it."""
    l = torch.randn(4, 16, generator=gen(17))
    l[0, 9] = math.nan
    l[2, 3] = math.inf
    ids, w = bsgg.route_groups(l.cuda(), 3, score="sigmoid", normalize=True)
    assert int(ids[0, 0]) == 9 and torch.isnan(w[0]).all() and int(ids[2, 0]) == 3
    assert torch.isfinite(w[1:]).all()
    bias = torch.zeros(16)
    bias[2], bias[12] = -math.inf, math.inf
    ids, w = bsgg.route_groups(l[1:].cuda(), 14, score="sigmoid", bias=bias.cuda(), groups=4, topk_groups=4)
    assert (ids[:, 0] == 12).all() and not (ids == 2).any() and torch.isfinite(w).all()
    ids, _ = bsgg.route_groups(l[:1].cuda(), 3, score="sigmoid", bias=torch.zeros(16).cuda(), groups=4, topk_groups=1)
    assert int(ids[0, 0]) == 9 and ((ids >= 8) & (ids < 12)).all()


def test_without_bias_and_groups_it_is_the_softmax_router():
    l = torch.randn(300, 96, generator=gen(19)).bfloat16().cuda()
    for normalize in (True, False):
        ids, w = bsgg.route(l, 6, normalize=normalize)
        got_ids, got = bsgg.route_groups(l, 6, score="softmax", normalize=normalize)
        assert torch.equal(ids, got_ids)
        assert torch.allclose(w, got, rtol=2.0 ** -18, atol=0)


def test_many_tokens_and_given_outputs():
    """More tokens than a wave of blocks, two streams, outputs the caller's."""
    T, L, k = 20000, 128, 4
    l = torch.randn(T, L, generator=gen(23))
    bias = torch.randn(L, generator=gen(24)) * 0.1
    dev, b = l.cuda(), bias.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        torch.cuda.synchronize()
        got = bsgg.route_groups(dev, k, bias=b, groups=8, topk_groups=3, ids=ids, weights=w, stream=s)
        assert got[0] is ids and got[1] is w
        outs.append(got)
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    s = torch.sigmoid(l.double())
    c = s + bias.double()
    best = c.view(T, 8, 16).sort(dim=2, descending=True).values[:, :, :2].sum(2)
    kept = best.sort(dim=1, descending=True, stable=True).indices[:, :3]
    mask = torch.zeros(T, 8, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(16, 1)
    want = torch.where(mask, c, torch.full_like(c, -math.inf)).sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(outs[0][0].cpu().long(), want)


def test_no_tokens():
    l = torch.empty(0, 16, device="cuda")
    ids, w = bsgg.route_groups(l, 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)
    assert bsgg.route_groups_backward(l, ids, w, w).shape == (0, 16)


@pytest.mark.parametrize("L,groups,kept", [(32, 8, 3), (256, 8, 4), (60, 5, 2)])
def test_sigmoids_at_the_end_of_the_range(L, groups, kept):
    """Scores near the smallest normal number, where the quotient of the choice's sigmoid is
    already 0: groups of them are in the order of their sums all the same."""
    T = 64
    l = -88.0 + torch.rand(T, L, generator=gen(41)) * 1.5                  # -88 to -86.5
    l[1::4, : L // 2] = -87.9 + torch.rand(T // 4, L // 2, generator=gen(42)) * 0.5
    l[2::4, -(L // groups):] -= 30.0                                       # a group that is 0 in 32 bits
    l[3::4] = torch.round(l[3::4] * 64) / 64
    want, _ = R.route_groups(l, 4, groups=groups, topk_groups=kept, group_top=2)
    ids, w = bsgg.route_groups(l.cuda(), 4, groups=groups, topk_groups=kept, group_top=2)
    assert torch.equal(ids.cpu(), want) and torch.isfinite(w).all()
