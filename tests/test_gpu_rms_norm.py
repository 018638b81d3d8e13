"""The RMS norm with the residual's addition and its gradient on the GPU against 64-bit
references: every pair of types, every row format, widths from 8 to the largest,
one token and many, pitches wider than the rows, sums in place."""
import ctypes
import math
import threading

import pytest
import torch

import block_scaled_grouped_gb300 as bsgg
import layer_operator_refs as R
import operator_refs as Q

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


def stream_of(T, H, dtype, seed):
    x = torch.randn(T, H, generator=gen(seed))
    x[:, ::61] *= 8.0
    return x.to(DT[dtype])


def rounding(ref, dtype):
    return ref.abs() * ROUND[dtype] + TINY[dtype]


# rstd: a sum of squares with up to 16 x 4 products, 5 and 16 additions in a row (half of it
# under the root), its mean, the root, the quotient; y: two more products
RSTD = 2.0 ** -24 * ((16 * 4 + 4 + 5 + 16) / 2 + 4)
WIDTHS = [8, 64, 96, 512, 520, 1024, 1032, 2048, 4096, 4104, 7168, 8192, 8200, 12288, 32768]


@pytest.mark.parametrize("dtype,wtype,ytype", [("bf16", "bf16", None), ("f16", "f32", "f32"), ("f32", "bf16", "f16"), ("f32", "f32", None),
                                               ("bf16", "f32", "f16")])
@pytest.mark.parametrize("H", WIDTHS)
def test_rms_norm(H, dtype, wtype, ytype):
    T = 5 if H > 2000 else 9
    x, r = stream_of(T, H, dtype, H), stream_of(T, H, dtype, H + 1)
    w = (1 + 0.2 * torch.randn(H, generator=gen(3))).to(DT[wtype])
    yt = DT[ytype or dtype]
    h = (x.double() + r.double()).to(torch.float32).to(DT[dtype])      # in 32 bits, then rounded, as documented
    n = bsgg.rms_norm(pitched(x, 16), w.cuda(), residual=pitched(r, 8), eps=1e-5, out_format=ytype)
    assert torch.equal(n.h.cpu(), h) and n.a is None and n.sfa is None
    want, rstd = R.rms_norm(h, w, 1e-5)
    assert ((n.rstd.cpu().double() - rstd).abs() <= rstd * RSTD).all()
    assert n.y.dtype == yt
    assert ((n.y.cpu().double() - want).abs() <= want.abs() * (RSTD + 2.0 ** -23) + rounding(want, yt)).all()
    # without residual, weight and rstd
    n = bsgg.rms_norm(x.cuda(), eps=1e-5, want_rstd=False)
    want, _ = R.rms_norm(x, None, 1e-5)
    assert n.h is None and n.rstd is None
    assert ((n.y.cpu().double() - want).abs() <= want.abs() * (RSTD + 2.0 ** -23) + rounding(want, DT[dtype])).all()


@pytest.mark.parametrize("fmt", ["mxfp8_e4m3", "mxfp8_e5m2", "nvfp4", "fp4_ue8m0_16", "mxfp4"])
@pytest.mark.parametrize("T,H,dtype", [(1, 32, "bf16"), (130, 96, "f16"), (3, 1024, "f32"), (5, 1056, "bf16"), (2, 7168, "bf16"), (2, 8224, "f16")])
def test_quantized_rows_are_those_of_y(T, H, dtype, fmt):
    """The rows are the quantization of the values before they are rounded to y: those come
    out whole in float32, and are quantized as dispatch documents, bit for bit."""
    x, r = stream_of(T, H, dtype, 5), stream_of(T, H, dtype, 6)
    x[0, :32] = 0                                     # a block of zeros
    r[0, :32] = 0
    w = (1 + 0.2 * torch.randn(H, generator=gen(3))).to(DT[dtype])
    n = bsgg.rms_norm(pitched(x, 8), w.cuda(), residual=r.cuda(), out_format="f32", row_format=fmt)
    rows = 128 * -(-T // 128)
    codes, scodes = Q.quantize(n.y.cpu().double(), fmt)
    want = torch.zeros(rows, codes.shape[1], dtype=torch.uint8)
    want[:T] = codes
    sf = torch.full((rows, scodes.shape[1]), 0x38 if fmt == "nvfp4" else 127, dtype=torch.uint8)
    sf[:T] = scodes
    got = n.a.cpu()
    assert torch.equal(got, Q.pack_codes(want, fmt))
    assert torch.equal(n.sfa.cpu(), Q.swizzle(sf))
    # alone, with more padding rows, and with 16-bit values beside them
    m = bsgg.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), want_y=False, row_format=fmt, m_pad=rows + 256)
    assert m.y is None and torch.equal(m.a[:rows].cpu(), got)
    assert torch.equal(m.a[rows:].cpu(), torch.zeros_like(m.a[rows:].cpu())) and torch.equal(m.h, n.h)
    b = bsgg.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), out_format="bf16", row_format=fmt)
    assert torch.equal(b.a, n.a) and torch.equal(b.sfa, n.sfa) and torch.equal(b.y, n.y.bfloat16())


def test_rows_are_those_of_dispatch():
    """A norm into rows is a norm into float32 and a dispatch of it."""
    T, H = 200, 512
    x = stream_of(T, H, "bf16", 9).cuda()
    n = bsgg.rms_norm(x, out_format="f32", row_format="mxfp8_e4m3")
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    t = bsgg.sort_tokens(ids, 1, m_pad=256)
    a, sfa = bsgg.dispatch(n.y, t.row_of_slot, t.slot_of_row)
    assert torch.equal(a, n.a) and torch.equal(sfa, n.sfa)


def test_nan_infinity_and_zeros():
    x = stream_of(4, 256, "f32", 11)
    x[0] = 0.0
    x[1, 7] = math.nan
    x[2, 9] = math.inf
    n = bsgg.rms_norm(x.cuda(), eps=1e-6, row_format="mxfp8_e4m3")
    y = n.y.cpu()
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and math.isnan(float(y[2, 9])) and (y[2, :9] == 0).all()
    assert torch.isfinite(y[3]).all() and float(n.rstd[2]) == 0.0
    # a block with a NaN has the NaN scale and zero codes
    sf = n.sfa.cpu().view(1, 2, 32, 4, 4)
    assert (sf[0, :, 1, 0, :] == 255).all() and (n.a[1].cpu() == 0).all() and int(sf[0, 0, 2, 0, 0]) == 255
    assert (sf[0, :, 0, 0, :] == 127).all()


@pytest.mark.parametrize("H", [64, 4096])
def test_sums_in_place(H):
    """The residual stream updated where it is, and where the new part is."""
    x, r = stream_of(40, H, "bf16", 12).cuda(), stream_of(40, H, "bf16", 13).cuda()
    want = bsgg.rms_norm(x, residual=r)
    for into in (x.clone(), r.clone()):
        a, b = (into, r) if torch.equal(into, x) else (x, into)
        n = bsgg.rms_norm(a, residual=b, h=into)
        assert n.h is into and torch.equal(into, want.h) and torch.equal(n.y, want.y)


BWD = [("bf16", "bf16", "bf16"), ("f16", "f32", "f16"), ("f32", "f32", "f32"), ("bf16", "f32", "f32"), ("f32", "bf16", "f16")]


@pytest.mark.parametrize("dtype,wtype,ytype", BWD)
@pytest.mark.parametrize("T,H", [(1, 8), (70, 64), (5, 520), (33, 1024), (7, 1032), (700, 4096), (5, 4104), (40, 7168), (3, 12288), (2, 32768)])
def test_rms_norm_backward(T, H, dtype, wtype, ytype):
    h, dy = stream_of(T, H, dtype, T + H), torch.randn(T, H, generator=gen(2)).to(DT[ytype])
    dh = torch.randn(T, H, generator=gen(4)).to(DT[dtype])
    w = (1 + 0.2 * torch.randn(H, generator=gen(3))).to(DT[wtype])
    rstd = R.rms_norm(h, None, 1e-6)[1].float()
    want, want_dw = R.rms_norm_backward(dy, h, w, rstd, dh)
    dx, dw = bsgg.rms_norm_backward(pitched(dy, 8), pitched(h, 16), w.cuda(), rstd.cuda(), dh=pitched(dh, 24))
    assert dx.dtype == h.dtype and dw.dtype == torch.float32
    n, g = h.double() * rstd.double()[:, None], dy.double() * w.double()
    # the mean of up to 64 products, 5 and 16 additions in a row, each product three roundings
    mean = (g * n).abs().mean(1, keepdim=True) * 2.0 ** -24 * (64 + 21 + 6)
    tol = rstd.double()[:, None] * (n.abs() * mean + (g.abs() + n.abs() * (g * n).mean(1, keepdim=True).abs()) * 2.0 ** -21)
    assert ((dx.cpu().double() - want).abs() <= tol + (want.abs() + dh.double().abs()) * 2.0 ** -23 + rounding(want, h.dtype)).all()
    # rows in a row of a block, the blocks' parts in eight runs, each product two roundings
    terms = (dy.double() * n).abs().sum(0)
    assert ((dw.cpu().double() - want_dw).abs() <= terms * 2.0 ** -24 * (min(T, -(-T // 304) + 4 + 304 / 8 + 8) + 2) + 1e-38).all()
    # alone: no gradient past the norm, no weight, no gradient of it
    dx, none = bsgg.rms_norm_backward(dy.cuda(), h.cuda(), None, rstd.cuda(), want_dweight=False)
    want, _ = R.rms_norm_backward(dy, h, None, rstd, None)
    g = dy.double()
    mean = (g * n).abs().mean(1, keepdim=True) * 2.0 ** -24 * (64 + 21 + 6)
    tol = rstd.double()[:, None] * (n.abs() * mean + (g.abs() + n.abs() * (g * n).mean(1, keepdim=True).abs()) * 2.0 ** -21)
    assert none is None
    assert ((dx.cpu().double() - want).abs() <= tol + rounding(want, h.dtype)).all()


def test_backward_in_place_and_repeated():
    T, H = 300, 1024
    h, dy, dh = (stream_of(T, H, "bf16", s).cuda() for s in (1, 2, 3))
    w = torch.ones(H, device="cuda").bfloat16()
    rstd = bsgg.rms_norm(h).rstd
    dx, dw = bsgg.rms_norm_backward(dy, h, w, rstd, dh=dh)
    for _ in range(3):                                # no order depends on timing
        again = bsgg.rms_norm_backward(dy, h, w, rstd, dh=dh)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    into = dh.clone()
    assert bsgg.rms_norm_backward(dy, h, w, rstd, dh=into, dx=into)[0] is into and torch.equal(into, dx)


def test_gradient_by_differences():
    """The kernels' own y in float32 against their own gradient."""
    T, H = 2, 24
    h = torch.randn(T, H, generator=gen(21))
    w = 1 + 0.2 * torch.randn(H, generator=gen(22))
    dy = torch.randn(T, H, generator=gen(23))
    f = lambda h, w: (bsgg.rms_norm(h.cuda(), w.cuda()).y.cpu().double() * dy.double()).sum(1)  # noqa: E731
    dx, dw = bsgg.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), bsgg.rms_norm(h.cuda()).rstd)
    step = 2.0 ** -7
    size = float(dy.abs().sum(1).max()) * 4
    for c in range(H):
        d = torch.zeros_like(h)
        d[:, c] = step
        diff = (f(h + d, w) - f(h - d, w)) / (2 * step)
        # third derivatives of size sum|dy| |y|, times step^2; values off by 2^-22 of themselves
        assert ((diff - dx[:, c].cpu().double()).abs() <= size * (step ** 2 + 2.0 ** -21 / step)).all()
        d = torch.zeros_like(w)
        d[c] = step
        diff = float((f(h, w + d) - f(h, w - d)).sum() / (2 * step))
        assert abs(diff - float(dw[c])) <= 2 * size * 2.0 ** -21 / step


def test_no_tokens():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    n = bsgg.rms_norm(x, residual=x, row_format="mxfp8_e4m3")
    assert n.y.shape == (0, 64) and n.a.shape == (128, 64) and (n.a == 0).all() and (n.sfa.view(1, 1, 32, 4, 4)[..., :2] == 127).all()
    dx, dw = bsgg.rms_norm_backward(x, x, None, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()
    assert bsgg.rms_norm(x).y.shape == (0, 64)


def test_many_rows_and_long_offsets():
    """More rows than 32 bits of elements: the last ones are right, on a stream of their own."""
    H = 32768
    T = 2 ** 31 // H + 3
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(H, device="cuda").bfloat16()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    n = bsgg.rms_norm(x, residual=x, eps=0.0, row_format="mxfp8_e4m3", stream=s)
    s.synchronize()
    want, _ = R.rms_norm(2 * x[-2:].cpu(), None, 0.0)
    assert ((n.y[-2:].cpu().double() - want).abs() <= want.abs() * (RSTD + 2.0 ** -23) + rounding(want, torch.bfloat16)).all()
    assert torch.equal(n.a[T - 2].cpu(), n.a[0].cpu()) and (n.a[T:] == 0).all()


def test_widths_in_two_threads():
    """Rows above 8192 columns keep sums in shared memory, more of it the wider they are: calls of
    two widths from two host threads, on streams of their own."""
    lib, codes = bsgg.lib(), [[], []]
    torch.cuda.synchronize()

    def calls(i, H):
        s = torch.cuda.Stream()
        h = torch.ones(1, H, dtype=torch.bfloat16, device="cuda")
        rstd, dx = torch.ones(1, device="cuda"), torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        d = bsgg.operators.NormBwdDesc(1, H, H, H, H, H, 0, 0, 0, 0)
        args = (ctypes.byref(d), h.data_ptr(), h.data_ptr(), None, rstd.data_ptr(), None, dx.data_ptr(), None, None, s.cuda_stream)
        codes[i] = [lib.bsgg_rms_norm_backward(*args) for _ in range(60000)]
        s.synchronize()
        assert (dx == 0).all()                       # g - n mean(g n) of ones

    threads = [threading.Thread(target=calls, args=a) for a in enumerate((16384, 32768))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [(len(c), sum(c)) for c in codes] == [(60000, 0)] * 2
