"""The dense layer and its gradient on the GPU against 64-bit references: one
row to many, odd sizes, wide pitches, each type and activation, the gradient
also against differences."""
import math

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


def pitched(t, multiple=1, extra=0):
    """t on the GPU, its row pitch a multiple plus extra columns, poisoned."""
    ld = -(-t.shape[1] // multiple) * multiple + extra
    buf = torch.full((t.shape[0], ld), math.nan, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]]


def problem(M, N, K, dtype, seed):
    g = gen(seed)
    x = torch.randn(M, K, generator=g).to(DT[dtype])
    w = (torch.randn(N, K, generator=g) / math.sqrt(K)).to(DT[dtype])
    b = torch.randn(N, generator=g) * 0.5
    r = torch.randn(M, N, generator=g).to(DT[dtype])
    return x, w, b, r


def layer(x, w, b, r, act):
    """z, y and the size sum |x w| of every element."""
    z = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if b is not None:
        z, size = z + b.double(), size + b.double().abs()
    y = R.act(z, act)
    return z, y if r is None else y + r.double(), size


def check_forward(x, w, b, r, act, y, z, want_z):
    zr, yr, size = layer(x, w, b, r, act)
    K = x.shape[1]
    ez = R.product_error(K) * size
    if want_z:
        assert ((z.cpu().double() - zr).abs() <= ez + R.rounding(zr, z.dtype)).all()
    # the activation: z's error times the largest slope near it, and 16 units of
    # 2^-24 of the values formed on the way (for gelu and silu |z| e^|..| stays below |z|)
    slope = 2 * (zr.abs() + ez) + ez if act == "srelu" else torch.full_like(zr, 1.13)
    ey = slope * ez + 16 * 2.0 ** -24 * (R.act(zr, act).abs() + 1e-3 * zr.abs()) + R.rounding(yr, y.dtype)
    if r is not None:
        ey = ey + 2.0 ** -24 * yr.abs() + 2.0 ** -24 * r.double().abs()
    bad = (y.cpu().double() - yr).abs() > ey
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}"


SIZES = [(1, 1, 1), (1, 4096, 1024), (1, 33, 7168), (2, 257, 129), (7, 64, 4096), (16, 1000, 520), (17, 128, 64), (33, 130, 72),
         (64, 2048, 256), (100, 96, 1000), (128, 128, 128), (129, 255, 65), (200, 640, 2048), (256, 256, 64),
         (300, 513, 777), (512, 1024, 512), (1000, 60, 4096), (1025, 2049, 136)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_sizes(M, N, K, dtype):
    x, w, b, r = problem(M, N, K, dtype, M + N + K)
    y, z = bsgg.linear(pitched(x, 8), pitched(w, 8), bias=b.cuda(), residual=pitched(r), activation="silu", want_z=True)
    check_forward(x, w, b, r, "silu", y, z, True)
    assert bsgg.operators_status() == 0


@pytest.mark.parametrize("dtype,act", [("bf16", "gelu"), ("f16", "silu")])
def test_linear_many_tiles(dtype, act):
    """Enough 256 x 256 tiles for CTA pairs to walk several each, ragged both ways."""
    M, N, K = 2500, 5001, 328
    x, w, b, r = problem(M, N, K, dtype, 77)
    y, z = bsgg.linear(x.cuda(), w.cuda(), bias=b.cuda(), residual=r.cuda(), activation=act, want_z=True)
    check_forward(x, w, b, r, act, y, z, True)
    assert bsgg.operators_status() == 0


@pytest.mark.parametrize("act", ["none", "relu", "srelu", "silu", "gelu"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(3, 70, 264), (150, 300, 328), (260, 520, 200)])
def test_linear_types_and_activations(M, N, K, act, out):
    dtype = "f16" if out == "f16" else "bf16"
    x, w, b, r = problem(M, N, K, dtype, 5)
    b = b.to(DT[out])
    for bias, res in ((b, r), (None, None), (b, None), (None, r)):
        y, z = bsgg.linear(x.cuda(), w.cuda(), bias=bias.cuda() if bias is not None else None, activation=act,
                           residual=res.cuda() if res is not None else None, want_z=bias is None, out_format=out)
        check_forward(x, w, bias, res, act, y, z, bias is None)
        assert (z is None) == (bias is not None)
    assert bsgg.operators_status() == 0


@pytest.mark.parametrize("M,N,K", [(5, 40, 72), (140, 264, 96)])
def test_linear_pitches_and_in_place_residual(M, N, K):
    """Pitches wider than the rows (their padding untouched), odd output pitch,
    and the residual updated in place."""
    x, w, b, r = problem(M, N, K, "bf16", 9)
    out = pitched(r, 1, 3)
    y, _ = bsgg.linear(pitched(x, 8, 8), pitched(w, 8, 16), bias=b.cuda(), activation="gelu", residual=out, out=out)
    assert y is out
    check_forward(x, w, b, r, "gelu", y, None, False)
    assert torch.isnan(out.as_strided((M, 3), (N + 3, 1), N)).all()


def test_linear_infinity_and_nan_stay_in_their_rows_and_columns():
    M, N, K = 150, 140, 200
    x, w, _, _ = problem(M, N, K, "bf16", 13)
    x[7, 3], x[90, 199], w[11, 0] = math.nan, math.inf, math.nan
    y, _ = bsgg.linear(x.cuda(), w.cuda(), activation="silu")
    y = y.cpu()
    bad = torch.isnan(y)
    keep = torch.ones(M, N, dtype=torch.bool)
    keep[7], keep[90], keep[:, 11] = False, False, False
    assert not bad[keep].any() and bad[7].all() and bad[:, 11].all()


def test_linear_of_no_rows():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    y, _ = bsgg.linear(x, w)
    assert y.shape == (0, 32)
    dy = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    dx, dw, db = bsgg.linear_backward(dy, x, w, want_dbias=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    kept = torch.ones(32, 64, dtype=torch.bfloat16, device="cuda")
    _, dw, _ = bsgg.linear_backward(dy, x, w, dw=kept)
    assert dw is kept and (kept == 1).all()


@pytest.mark.parametrize("M,N,K", [(3, 4096, 7168), (40, 2048, 7168), (100, 4096, 4160), (300, 4096, 4160), (600, 4096, 4160)])
def test_linear_back_to_back(M, N, K):
    """Launches that follow one another at once, each set up under the one before,
    on operands that come from memory: every one's result."""
    n = 6
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    xs = [torch.randn(M, K, generator=g, device="cuda").bfloat16() for _ in range(n)]
    ws = [(torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).bfloat16() for _ in range(n)]
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    flush.fill_(1)                                              # out of L2
    ys = [bsgg.linear(xs[i % n], ws[i % n], out_format="f32")[0] for i in range(4 * n)]
    assert bsgg.operators_status() == 0
    for i in range(n):
        want = xs[i].double() @ ws[i].double().t()
        tol = R.product_error(K) * (xs[i].double().abs() @ ws[i].double().abs().t()) + R.rounding(want, torch.float32)
        for y in ys[i::n]:
            assert ((y.double() - want).abs() <= tol).all()


def test_linear_offsets_past_32_bits():
    """An output of 2.3e9 elements, its pre-activation and residual: rows at both ends."""
    M, N, K = 147456, 15616, 72
    g = gen(61)
    x, w = torch.randn(M, K, generator=g).bfloat16(), (torch.randn(N, K, generator=g) / 8).bfloat16()
    res = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    res[-3:] = 2.0
    y, z = bsgg.linear(x.cuda(), w.cuda(), activation="relu", residual=res, want_z=True)
    for rows in (slice(0, 5), slice(M // 2, M // 2 + 3), slice(M - 5, M)):
        check_forward(x[rows], w, None, res[rows].cpu(), "relu", y[rows], z[rows], True)
    assert bsgg.operators_status() == 0


# ------------------------------------------------------------------ gradient
BWD = [(1, 8, 8), (1, 256, 4096), (3, 40, 24), (17, 136, 264), (64, 64, 512), (100, 1000, 72), (129, 264, 520), (257, 512, 256),
       (300, 60 * 8, 1000), (1000, 128, 200)]


def check_backward(dy, x, w, z, act, dx, dw, db, dw0=None):
    g = dy.double()
    if act != "none":
        slope = R.act_slope(z.double(), act)
        g = g * slope
        # one rounding to the input type of dy act'(z), formed in 32 bits
        eg = R.rounding(g, dy.dtype) + dy.double().abs() * 16 * 2.0 ** -24 * (1 + z.double().abs())
        eb = dy.double().abs() * 16 * 2.0 ** -24 * (1 + z.double().abs())
    else:
        eg = eb = torch.zeros_like(g)
    M, N = g.shape
    if dx is not None:
        ref = g @ w.double()
        tol = R.product_error(N) * (g.abs() @ w.double().abs()) + eg @ w.double().abs() + R.rounding(ref, dx.dtype)
        assert ((dx.cpu().double() - ref).abs() <= tol).all()
    if dw is not None:
        ref = g.t() @ x.double()
        tol = R.product_error(M) * (g.abs().t() @ x.double().abs()) + eg.t() @ x.double().abs()
        if dw0 is not None:
            ref, tol = ref + dw0.double(), tol + 2.0 ** -23 * (dw0.double().abs() + ref.abs())
        assert ((dw.cpu().double() - ref).abs() <= tol + R.rounding(ref, dw.dtype)).all()
    if db is not None:
        ref = g.sum(0)
        tol = (M / 8 + 16) * 2.0 ** -24 * g.abs().sum(0) + eb.sum(0)
        assert ((db.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("M,N,K", BWD)
def test_linear_backward_sizes(M, N, K, act):
    dtype = "bf16" if M % 2 else "f16"
    x, w, _, z = problem(M, N, K, dtype, M * 3 + N)
    dy = (torch.randn(M, N, generator=gen(2)) * 0.3).to(DT[dtype])
    dx, dw, db = bsgg.linear_backward(pitched(dy, 8, 8), pitched(x, 8), pitched(w, 8, 8), z=pitched(z, 8) if act != "none" else None,
                                      activation=act, want_dbias=True)
    check_backward(dy, x, w, z, act, dx, dw, db)
    assert bsgg.operators_status() == 0


def test_linear_rounds_with_a_split_remainder():
    """More tiles than pairs, the last round short and the reduction long, so that
    the remainder's reduction is split."""
    M, N, K = 2304, 2304, 8200                                      # 81 tiles of 256 x 256
    x, w, b, r = problem(M, N, K, "bf16", 79)
    y, z = bsgg.linear(x.cuda(), w.cuda(), bias=b.cuda(), residual=r.cuda(), activation="silu", want_z=True)
    check_forward(x, w, b, r, "silu", y, z, True)
    assert bsgg.operators_status() == 0


def test_linear_backward_many_tiles():
    M, N, K = 2310, 2408, 2504
    x, w, _, z = problem(M, N, K, "bf16", 78)
    dy = torch.randn(M, N, generator=gen(9)).bfloat16()
    dx, dw, db = bsgg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=z.cuda(), activation="silu", want_dbias=True)
    check_backward(dy, x, w, z, "silu", dx, dw, db)
    assert bsgg.operators_status() == 0


@pytest.mark.parametrize("act", ["relu", "srelu", "gelu"])
@pytest.mark.parametrize("fmt", ["f32", "bf16"])
def test_linear_backward_activations_and_accumulation(act, fmt):
    M, N, K = 150, 72, 136
    x, w, _, z = problem(M, N, K, "bf16", 31)
    dy = torch.randn(M, N, generator=gen(3)).bfloat16()
    dw0 = torch.randn(N, K, generator=gen(4)).to(DT[fmt])
    kept = pitched(dw0, 1, 5)
    dx, dw, db = bsgg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=z.cuda(), activation=act, want_dbias=True, dx_format=fmt,
                                      dw=kept)
    assert dw is kept
    check_backward(dy, x, w, z, act, dx, dw, db, dw0)
    dx, dw, db = bsgg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=z.cuda(), activation=act, want_dx=False, dw_format=fmt)
    assert dx is None and db is None
    check_backward(dy, x, w, z, act, None, dw, None)
    dx, dw, db = bsgg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=z.cuda(), activation=act, want_dw=False, want_dx=False,
                                      want_dbias=True)
    assert dx is None and dw is None
    check_backward(dy, x, w, z, act, None, None, db)


@pytest.mark.parametrize("act", ["silu", "gelu", "srelu"])
def test_linear_gradient_against_differences(act):
    """<grad, direction> against differences of the 64-bit layer's loss."""
    M, N, K = 40, 48, 64
    x, w, b, _ = problem(M, N, K, "f16", 17)
    dy = torch.randn(M, N, generator=gen(5)).half()
    _, z = bsgg.linear(x.cuda(), w.cuda(), bias=b.cuda(), activation=act, want_z=True)
    dx, dw, db = bsgg.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=z, activation=act, want_dbias=True, dx_format="f32",
                                      dw_format="f32")
    g = gen(6)
    ux, uw, ub = (torch.randn(M, K, generator=g).double(), torch.randn(N, K, generator=g).double(),
                  torch.randn(N, generator=g).double())

    def loss(t):
        zz = (x.double() + t * ux) @ (w.double() + t * uw).t() + b.double() + t * ub
        return (R.act(zz, act) * dy.double()).sum()

    h = 1e-5
    diff = (loss(h) - loss(-h)) / (2 * h)
    parts = [(dx.cpu().double() * ux), (dw.cpu().double() * uw), (db.cpu().double() * ub)]
    got = sum(p.sum() for p in parts)
    # z and dz are rounded to 11 bits: independent errors of 2^-12 on M N terms
    zz = x.double() @ w.double().t() + b.double()
    per = dy.double().abs() * (ux @ w.double().t() + x.double() @ uw.t() + ub).abs() * (1 + zz.abs())
    assert abs(got - diff) <= 6 * 2.0 ** -11 * per.pow(2).sum().sqrt() + 1e-4


def test_linear_gradients_are_repeatable():
    M, N, K = 700, 264, 520
    x, w, _, z = problem(M, N, K, "bf16", 41)
    dy = torch.randn(M, N, generator=gen(8)).bfloat16()
    args = (dy.cuda(), x.cuda(), w.cuda())
    first = bsgg.linear_backward(*args, z=z.cuda(), activation="silu", want_dbias=True)
    again = bsgg.linear_backward(*args, z=z.cuda(), activation="silu", want_dbias=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
