"""Plain 64-bit references of the operators around the grouped GEMM, on CPU
tensors, written from their formulas."""
import math

import torch

# Rounding to nearest with p significant bits is off by at most 2^-p of the value
# (8, 11 and 24 bits), or by half the subnormal spacing.
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
QMAX = {"mxfp8_e4m3": 448.0, "mxfp8_e5m2": 57344.0, "nvfp4": 6.0, "fp4_ue8m0_16": 6.0, "mxfp4": 6.0}
VEC = {"mxfp8_e4m3": 32, "mxfp8_e5m2": 32, "nvfp4": 16, "fp4_ue8m0_16": 16, "mxfp4": 32}


def rounding(ref, dtype):
    """The largest error of one rounding of `ref` to dtype."""
    return ref.abs() * ROUND[dtype] + TINY[dtype]


# ------------------------------------------------------------------ routing
def route(logits, k, normalize):
    """logits (T, L) -> ids (T, k), weights float64 (T, k)."""
    l = logits.double()
    T, L = l.shape
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        row = l[t].tolist()
        key = lambda e: (0 if math.isnan(row[e]) else 1, -row[e] if not math.isnan(row[e]) else 0.0, e)  # noqa: E731
        order = [e for e in sorted(range(L), key=key) if row[e] != -math.inf][:k]
        if not order:
            continue
        m = row[order[0]]
        if math.isnan(m):
            ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
            w[t, :len(order)] = math.nan
            continue
        over = order if normalize else [e for e in range(L) if row[e] != -math.inf]
        total = sum(math.exp(row[e] - m) for e in over)
        for j, e in enumerate(order):
            ids[t, j], w[t, j] = e, math.exp(row[e] - m) / total
    return ids, w


def route_weights_at(l, ids, normalize):
    """The weights as a smooth function of the logits (float64), ids held."""
    m = l.amax(1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(l - m)
    on = ids >= 0
    picked = torch.where(on, e.gather(1, ids.clamp(min=0).long()), torch.zeros((), dtype=l.dtype))
    total = picked.sum(1, keepdim=True) if normalize else e.sum(1, keepdim=True)
    return picked / torch.where(total > 0, total, torch.ones_like(total))


def route_backward(logits, ids, g, normalize):
    l = logits.double()
    w = route_weights_at(l, ids, normalize)
    on = ids >= 0
    gw = torch.where(on, g.double() * w, torch.zeros((), dtype=torch.float64))
    inner = gw.sum(1, keepdim=True)
    pick = torch.zeros_like(l).scatter_add_(1, ids.clamp(min=0).long(), gw)
    if normalize:
        p = torch.zeros_like(l).scatter_add_(1, ids.clamp(min=0).long(), torch.where(on, w, torch.zeros_like(w)))
    else:
        m = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
        tot = e.sum(1, keepdim=True)
        p = e / torch.where(tot > 0, tot, torch.ones_like(tot))
    return pick - p * inner


# ------------------------------------------------------------------ sort
def sort_tokens(ids, L, m_pad):
    """ids (T, k) -> offsets, row_of_slot, slot_of_row, used (lists)."""
    flat = ids.reshape(-1).tolist()
    members = [[] for _ in range(L)]
    for s, e in enumerate(flat):
        if 0 <= e < L:
            members[e].append(s)
    rows, offsets = [], []
    for e in range(L):
        rows += members[e] + [-1] * (-len(members[e]) % 128)
        offsets.append(len(rows))
    used = len(rows)
    offsets = [min(o, m_pad) for o in offsets[:-1]] + [m_pad]
    rows = (rows + [-1] * m_pad)[:m_pad]
    row_of_slot = [-1] * len(flat)
    for r, s in enumerate(rows):
        if s >= 0:
            row_of_slot[s] = r
    return offsets, row_of_slot, rows, used


# ------------------------------------------------------------------ quantization
def _float_codes(fmt):
    """Every finite value of an 8-bit format in order of its positive codes."""
    man, bias, last = (3, 7, 0x7E) if fmt == "e4m3" else (2, 15, 0x7B)
    out = []
    for c in range(last + 1):
        e, m = c >> man, c & ((1 << man) - 1)
        out.append(m * 2.0 ** (1 - bias - man) if e == 0 else (1 + m / 2 ** man) * 2.0 ** (e - bias))
    return torch.tensor(out, dtype=torch.float64)


def nearest_code(y, values):
    """Index of the value nearest to |y| (float64), ties to the even index,
    saturating."""
    a = y.abs().contiguous()
    hi = torch.searchsorted(values, a).clamp(max=len(values) - 1)
    lo = (hi - 1).clamp(min=0)
    dlo, dhi = a - values[lo], values[hi] - a
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    return torch.where(up | (a >= values[-1]), hi, lo)


def quantize(x, fmt):
    """x float64 (R, H) -> (codes uint8 (R, H), one per value, scale codes uint8
    (R, ceil(H / v)))."""
    R, H = x.shape
    v, q = VEC[fmt], QMAX[fmt]
    kb = -(-H // v)
    xb = torch.nn.functional.pad(x, (0, kb * v - H)).view(R, kb, v)
    amax = xb.abs().amax(-1)
    bad = ~torch.isfinite(xb).all(-1)
    amax = torch.where(bad, torch.zeros_like(amax), amax)
    if fmt == "nvfp4":
        # amax / 6 in 32 bits, as the framework's quantization recipe forms it
        s32 = (amax.float() / torch.full_like(amax, 6.0).float()).double()
        values = _float_codes("e4m3")
        scode = nearest_code(s32, values).to(torch.uint8)
        scode = torch.where(scode == 0, torch.full_like(scode, 0x38), scode)
        scale = values[scode.long()]
        scode = torch.where(bad, torch.full_like(scode, 0x7F), scode)
    else:
        e = torch.zeros_like(amax)
        for i in torch.nonzero(amax > 0):
            i = tuple(i.tolist())
            a = amax[i].item()
            m, ex = math.frexp(a / q)          # an estimate, made exact below
            while math.ldexp(q, ex) < a:
                ex += 1
            while math.ldexp(q, ex - 1) >= a:
                ex -= 1
            e[i] = max(-127, ex)
        scale = torch.ldexp(torch.ones_like(e), e.to(torch.int32))
        scode = (e + 127).to(torch.uint8)
        scode = torch.where(bad, torch.full_like(scode, 255), scode)
    values = torch.tensor(E2M1, dtype=torch.float64) if q == 6.0 else _float_codes(fmt[6:])
    y = torch.where(bad[..., None], torch.zeros_like(xb), xb / scale[..., None])
    code = nearest_code(y, values).to(torch.uint8)
    sign = torch.signbit(y).to(torch.uint8) << (3 if q == 6.0 else 7)
    return (code | sign).view(R, kb * v)[:, :H].contiguous(), scode


def pack_codes(codes, fmt):
    """One code per value -> the row buffer's bytes."""
    if QMAX[fmt] != 6.0:
        return codes
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def swizzle(scodes):
    """Row-major scale codes (R, kb), R a multiple of 128, in the swizzled
    layout, padding 0."""
    R, kb = scodes.shape
    kq = -(-kb // 4)
    out = torch.zeros(R * kq * 4, dtype=torch.uint8)
    r = torch.arange(R)[:, None]
    b = torch.arange(kb)[None, :]
    at = (r // 128 * kq + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    out[at.reshape(-1)] = scodes.reshape(-1)
    return out


# ------------------------------------------------------------------ dense layer
def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "srelu":
        return z.clamp(min=0) ** 2
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z


def act_slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "srelu":
        return 2 * z.clamp(min=0)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def product_error(depth):
    """Bound on |error| / sum |a b| of a product accumulated in 32 bits: groups
    of 16 products (one matrix instruction's step), each added with one rounding
    or truncation of 2^-23, and as much again for the joins and the epilogue."""
    return (depth / 16 + 16) * 2.0 ** -23
