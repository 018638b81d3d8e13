"""Cases of the operators in front of an expert layer and beside its dense layers.

Three operators, each in its forward and its backward direction:

route_groups  routing with softmax or sigmoid scores, a bias per expert that only
              steers the choice, experts in groups of which the best few are kept,
              and top-k weights from the unbiased scores; and its gradient
rms_norm      root-mean-square norm with the residual's addition, out in 16 bits
              and, in the same pass, in 8 bits with scale factors as the grouped
              GEMM's A operand; and its gradient
adapters      low-rank adapters of many requests at once beside a dense layer:
              y = base + s_i (x A_i^T) B_i, i the token's own adapter; and its gradient

Sizes are those of the expert-layer workloads: 4096 and 14336 wide, 7168 wide, 8192
tokens, 64 and 128 experts, decode steps of 128 tokens; ranks 16 to 64 are generic.
"""
import math

import torch

own = False          # False: the plain form; True: the framework's operators

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SCALE_BITS = {"mxfp8_e4m3": (torch.float8_e4m3fn, 448.0), "mxfp8_e5m2": (torch.float8_e5m2, 57344.0)}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's router, 64 experts in 8 groups of which 4 are kept: latency of the smallest launch
        {"name": "route_decode", "op": "route", "dir": "fwd", "T": 128, "L": 64, "groups": 8, "kept": 4, "top": 2, "k": 8,
         "score": "sigmoid", "bias": True, "normalize": True, "scale": 2.5, "dtype": "f32", "masked": False},
        # a prompt's router over 256 experts, bfloat16 logits, an expert that is off and padding tokens
        {"name": "route_prefill", "op": "route", "dir": "fwd", "T": 8192, "L": 256, "groups": 8, "kept": 4, "top": 2, "k": 8,
         "score": "sigmoid", "bias": True, "normalize": True, "scale": 2.5, "dtype": "bf16", "masked": True},
        # a training step's router, forward and gradient
        {"name": "route_train", "op": "route", "dir": "train", "T": 16384, "L": 128, "groups": 8, "kept": 3, "top": 2, "k": 4,
         "score": "sigmoid", "bias": True, "normalize": True, "scale": 1.0, "dtype": "f32", "masked": True},
        # softmax scores, groups by their best expert, weights not renormalised; an odd number of groups
        {"name": "route_softmax_train", "op": "route", "dir": "train", "T": 8191, "L": 60, "groups": 5, "kept": 2, "top": 1, "k": 6,
         "score": "softmax", "bias": False, "normalize": False, "scale": 16.0, "dtype": "bf16", "masked": False},
        # a decode step's norm: both forms of the output
        {"name": "norm_decode", "op": "norm", "dir": "fwd", "T": 128, "H": 7168, "dtype": "bf16", "residual": True, "y": True,
         "format": "mxfp8_e4m3"},
        # the fine-grained layer's tokens, a prompt: 16 bits for the router, 8 for the experts' product; the largest
        {"name": "norm_prefill", "op": "norm", "dir": "fwd", "T": 8192, "H": 7168, "dtype": "bf16", "residual": True, "y": True,
         "format": "mxfp8_e4m3"},
        # a ragged prompt of an odd width, float16
        {"name": "norm_ragged", "op": "norm", "dir": "fwd", "T": 333, "H": 4104, "dtype": "f16", "residual": True, "y": True,
         "format": "none"},
        # the gradient over a training batch, with the residual stream's and the weight's
        {"name": "norm_train", "op": "norm", "dir": "bwd", "T": 8192, "H": 4096, "dtype": "bf16", "residual": True},
        # one token with its adapter beside a down projection: latency
        {"name": "adapters_token", "op": "adapters", "dir": "fwd", "T": 1, "S": 4, "r": 16, "K": 14336, "N": 4096,
         "dtype": "bf16", "requests": "tokens"},
        # a decode step: every token with an adapter of its own out of 64
        {"name": "adapters_decode", "op": "adapters", "dir": "fwd", "T": 128, "S": 64, "r": 16, "K": 4096, "N": 14336,
         "dtype": "bf16", "requests": "tokens"},
        # prompts of several requests in one batch, ragged, some without an adapter
        {"name": "adapters_prefill", "op": "adapters", "dir": "fwd", "T": 4096, "S": 8, "r": 64, "K": 4096, "N": 14336,
         "dtype": "bf16", "requests": "prompts"},
        # training of a few adapters at once beside the up projection
        {"name": "adapters_train", "op": "adapters", "dir": "bwd", "T": 4096, "S": 4, "r": 32, "K": 4096, "N": 14336,
         "dtype": "bf16", "requests": "prompts"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "adapters"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 3, 4, 5, 8, 8, 16])
        L = groups * max(2, _log(rng, 4, 256) // groups)
        kept = rng.randint(1, groups)
        return {"op": op, "dir": rng.choice(["fwd", "train"]), "T": _log(rng, 1, 16384), "L": L, "groups": groups, "kept": kept,
                "top": rng.choice([1, 2]), "k": rng.randint(1, min(8, L // groups * kept)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "normalize": rng.random() < 0.5,
                "scale": rng.choice([1.0, 2.5, 16.0]), "dtype": rng.choice(["bf16", "f16", "f32"]), "masked": rng.random() < 0.5}
    if op == "norm":
        bwd = rng.random() < 0.4
        fmt = "none" if bwd else rng.choice(["none", "mxfp8_e4m3", "mxfp8_e5m2"])
        H = 8 * _log(rng, 16, 1024)
        if fmt != "none":
            H = -(-H // 16) * 16
        T = max(1, min(_log(rng, 1, 16384), 8192 * 4096 // H))
        c = {"op": op, "dir": "bwd" if bwd else "fwd", "T": T, "H": H, "dtype": rng.choice(["bf16", "f16", "f32"]),
             "residual": rng.random() < 0.7}
        return c if bwd else c | {"y": fmt == "none" or rng.random() < 0.5, "format": fmt}
    bwd = rng.random() < 0.4
    r, K, N = 8 * _log(rng, 1, 12), 8 * _log(rng, 16, 1792), 8 * _log(rng, 16, 1792)
    T = max(1, min(_log(rng, 1, 4096), 4096 * (4096 + 14336) // (K + N)))
    S = _log(rng, 1, max(2, min(64, 64 * 16 * 18432 // (r * (K + N)))))
    return {"op": op, "dir": "bwd" if bwd else "fwd", "T": T, "S": S, "r": r, "K": K, "N": N,
            "dtype": rng.choice(["bf16", "f16"]), "requests": rng.choice(["tokens", "prompts"])}


# ------------------------------------------------------------------ sizes
def _padded(T):
    return -(-T // 128) * 128


def _rows(c):
    """Rows that always suffice: the adapters' counts of tokens rounded up to 128."""
    a = min(c["S"], c["T"])
    return max(128, 128 * (a + (c["T"] - a) // 128))


def work(c):
    es = DTYPES[c["dtype"]].itemsize
    if c["op"] == "route":
        T, L, k = c["T"], c["L"], c["k"]
        b, train = T * L * es + T * k * 8 + (4 * L if c["bias"] else 0), c["dir"] == "train"
        if train:
            b += T * k * 4 + T * L * es
        return {"bytes": b, "flops": (16 if train else 8) * T * L}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        if c["dir"] == "bwd":
            return {"bytes": T * H * es * (4 if c["residual"] else 3) + T * 4 + H * (es + 4), "flops": 12 * T * H}
        b = T * H * es * (3 if c["residual"] else 1) + H * es + T * 4 + (T * H * es if c["y"] else 0)
        if c["format"] != "none":
            b += _padded(T) * (H + -(-H // 128) * 4)
        return {"bytes": b, "flops": 6 * T * H}
    T, S, r, K, N = c["T"], c["S"], c["r"], c["K"], c["N"]
    weights, used = r * (K + N) * es, min(S, T)
    if c["dir"] == "fwd":
        return {"bytes": es * T * (K + 2 * N) + used * weights + T * r * 4 + T * 4, "flops": 2 * T * r * (K + N)}
    return {"bytes": es * T * (3 * K + N) + (used + S) * weights + T * r * 4 + T * 4, "flops": 4 * T * r * (K + N)}


# ------------------------------------------------------------------ inputs
def _token_adapters(c, g):
    """Each token's adapter, -1 for none.  Decoding: a request per token, one in
    eight without an adapter; prompts: runs of tokens of ragged lengths."""
    T, S = c["T"], c["S"]
    pick = torch.randint(0, S, (T,), generator=g, device="cuda")
    off = torch.rand(T, generator=g, device="cuda") < 0.125
    ids = torch.where(off & (T > 1), torch.full_like(pick, -1), pick)
    if c["requests"] == "prompts":
        starts = torch.rand(T, generator=g, device="cuda") < 1.0 / 300.0
        first = torch.cummax(torch.where(starts, torch.arange(T, device="cuda"), torch.zeros_like(pick)), 0).values
        ids = ids[first]
    return ids.to(torch.int32)


def _sorted_tokens(ids, S, m_pad):
    """Tokens in order of adapter, then of token; each adapter's rows padded to 128,
    the last one's to m_pad: (padded_offsets, row of each token, token of each row, ones, rows used)."""
    T = ids.numel()
    key = torch.where(ids >= 0, ids.long(), torch.full((), S, device=ids.device))
    counts = torch.zeros(S + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    ends = torch.cumsum((counts[:S] + 127) // 128 * 128, 0)
    start = torch.cat([torch.zeros_like(ends[:1]), ends])
    order = torch.sort(key, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    at = key[order]
    row_sorted = torch.where(at < S, start[at] + torch.arange(T, device=ids.device) - first[at], torch.full_like(at, -1))
    row = torch.empty_like(row_sorted)
    row[order] = row_sorted
    token = torch.full((m_pad + 1,), -1, dtype=torch.int32, device=ids.device)
    token[torch.where(row >= 0, row, torch.full_like(row, m_pad))] = torch.arange(T, dtype=torch.int32, device=ids.device)
    token = token[:m_pad].contiguous()
    offsets = torch.cat([ends[:-1], torch.full_like(ends[:1], m_pad)]).to(torch.int32)
    return offsets, row.to(torch.int32)[:, None].contiguous(), token, (token >= 0).float(), ends[-1:].to(torch.int32)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(c)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "route":
        T, L = c["T"], c["L"]
        s["logits"] = (normal(T, L) + normal(L, scale=0.7)).to(dt)
        if c["masked"]:        # an expert that is off, and padding tokens whose every expert is
            s["logits"][:, L // 2] = -math.inf
            s["logits"][7::8] = -math.inf
        # steered by as much as the scores differ
        s["b"] = normal(L, scale=0.1 if c["score"] == "sigmoid" else 0.5 / L) if c["bias"] else None
        if c["dir"] == "train":
            s["dweights"] = normal(T, c["k"])
    elif c["op"] == "norm":
        T, H = c["T"], c["H"]
        # a residual stream with a few large channels
        h = normal(T, H)
        h[:, ::61] *= 8.0
        s["w"] = (1.0 + normal(H, scale=0.2)).to(dt)
        if c["dir"] == "fwd":
            s["x"] = normal(T, H, dtype=dt, scale=0.3) if c["residual"] else h.to(dt)
            s["res"] = h.to(dt) if c["residual"] else None
        else:
            s["h"] = h.to(dt)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
            s["dy"] = normal(T, H, dtype=dt, scale=0.1)
            s["dh"] = normal(T, H, dtype=dt, scale=0.1) if c["residual"] else None
    else:
        T, S, r, K, N = c["T"], c["S"], c["r"], c["K"], c["N"]
        s["ids"] = _token_adapters(c, g)
        s["map"] = _sorted_tokens(s["ids"], S, _rows(c))     # once per step, for every layer's adapters
        s["a"] = normal(S, r, K, dtype=dt, scale=1.0 / math.sqrt(K))
        s["b"] = normal(S, r, N, dtype=dt, scale=0.5 / math.sqrt(r))
        s["scales"] = 0.5 + torch.rand(S, generator=g, device="cuda")
        s["x"] = normal(T, K, dtype=dt)
        if c["dir"] == "fwd":
            s["base"] = normal(T, N, dtype=dt)
        else:
            s["dy"] = normal(T, N, dtype=dt, scale=0.1)
            s["base"] = normal(T, K, dtype=dt, scale=0.1)
            of = torch.randn(T, r, generator=g, device="cuda")    # the forward's x A^T
            s["u"] = torch.where(s["ids"][:, None] >= 0, of, torch.zeros_like(of))
    return s


# ------------------------------------------------------------------ the plain form
def _route_plain(s):
    k, L, G = s["k"], s["L"], s["groups"]
    # the order of experts depends on differences near the borders of the choice: 64 bits
    l = s["logits"].double()
    T = l.shape[0]
    on = l > -math.inf
    m = l.amax(1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    e = torch.exp(l - m)
    total = e.sum(1, keepdim=True)
    total = torch.where(total > 0, total, torch.ones_like(total))
    score = e / total if s["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    c = score if s["b"] is None else score + s["b"].double()
    c = torch.where(on, c, torch.full_like(c, -math.inf))
    best = torch.sort(c.view(T, G, L // G), dim=2, descending=True).values[:, :, :s["top"]]
    alive = best[:, :, 0] > -math.inf
    group = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
    group = torch.where(alive, group, torch.full_like(group, -math.inf))
    kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :s["kept"]]
    allowed = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
    c = torch.where(allowed.repeat_interleave(L // G, 1), c, torch.full_like(c, -math.inf))
    order = torch.sort(c, dim=1, descending=True, stable=True)
    chosen = order.values[:, :k] > -math.inf
    ids = torch.where(chosen, order.indices[:, :k], torch.full_like(order.indices[:, :k], -1))
    at = ids.clamp(min=0)
    sc = torch.where(chosen, score.gather(1, at), torch.zeros((), dtype=l.dtype, device=l.device))
    w = sc
    if s["normalize"]:
        sum_ = sc.sum(1, keepdim=True)
        w = sc / torch.where(sum_ > 0, sum_, torch.ones_like(sum_))
    out = {"ids": ids.to(torch.int32), "weights": (s["scale"] * w).float()}
    if s["dir"] == "fwd":
        return out
    g = torch.where(chosen, s["dweights"].double(), torch.zeros((), dtype=l.dtype, device=l.device))
    inner = (g * w).sum(1, keepdim=True)
    if s["score"] == "sigmoid":
        d = w * (1.0 - sc) * ((g - inner) if s["normalize"] else g)
        dl = torch.zeros_like(l).scatter_add_(1, at, d)
    elif s["normalize"]:
        dl = torch.zeros_like(l).scatter_add_(1, at, w * (g - inner))
    else:
        dl = torch.zeros_like(l).scatter_add_(1, at, w * g) - score * inner
    out["dlogits"] = (s["scale"] * dl).to(s["logits"].dtype)
    return out


def _quantize_plain(x, fmt):
    """Codes and power-of-two scales per 32 columns: 2^ceil(log2(amax / qmax))."""
    dt, qmax = SCALE_BITS[fmt]
    T, H = x.shape
    kb = -(-H // 32)
    xb = torch.nn.functional.pad(x, (0, kb * 32 - H)).view(T, kb, 32)
    amax = xb.abs().amax(-1)
    mant, ex = torch.frexp(amax / torch.full_like(amax, qmax))   # a scalar divisor would be multiplied by its reciprocal
    e = torch.where(mant == 0.5, ex - 1, ex)
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-127, 127)
    # 2^e from its bits (2^-127 is the subnormal 2^22 units): a power function need not be exact
    bits = torch.where(e == -127, torch.full_like(e, 1 << 22), (e + 127).clamp(min=1) << 23)
    scale = bits.to(torch.int32).view(torch.float32)
    q = (xb / scale[..., None]).clamp(-qmax, qmax).to(dt).view(T, kb * 32)[:, :H]
    return q.contiguous(), (e + 127).to(torch.uint8)


def _swizzle(codes):
    """Row-major scale codes (rows, kb) in the layout (rows/128, kb/4, 32, 4, 4)."""
    rows, kb = codes.shape
    kq = -(-kb // 4)
    full = torch.nn.functional.pad(codes, (0, kq * 4 - kb))
    return full.view(rows // 128, 4, 32, kq, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _norm_plain(s):
    T, H = s["T"], s["H"]
    dt, w = DTYPES[s["dtype"]], s["w"].float()
    if s["dir"] == "bwd":
        xh = s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * w
        dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dw": (dy * xh).sum(0)}
    out = {}
    h = s["x"]
    if s["res"] is not None:
        # the sum is kept in the tokens' type, and what is kept is normed
        out["h"] = h = (s["x"].float() + s["res"].float()).to(dt)
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(1) + EPS)
    y = hf * rstd[:, None] * w
    out["rstd"] = rstd
    if s["y"]:
        out["y"] = y.to(dt)
    if s["format"] != "none":
        q, e = _quantize_plain(y, s["format"])
        rows = _padded(T)
        a = torch.zeros(rows, H, dtype=torch.uint8, device=y.device)
        sf = torch.full((rows, e.shape[1]), 127, dtype=torch.uint8, device=y.device)
        a[:T], sf[:T] = q.view(torch.uint8), e
        out["a"] = a.view(q.dtype)
        out["sfa"] = _swizzle(sf).view(torch.float8_e8m0fnu)
    return out


def _adapters_plain(s):
    """All adapters' products at once, each token's own kept: (x A^T) masked, times B."""
    T, S, r = s["T"], s["S"], s["r"]
    dt = DTYPES[s["dtype"]]
    a, b = s["a"].float().view(S * r, -1), s["b"].float().view(S * r, -1)
    mine = (s["ids"][:, None] == torch.arange(S, device=a.device)).float()      # (T, S)
    x = s["x"].float()
    if s["dir"] == "fwd":
        u = (x @ a.t()).view(T, S, r) * mine[:, :, None]
        y = s["base"].float() + (u * s["scales"][:, None]).view(T, S * r) @ b
        return {"y": y.to(dt), "u": u.sum(1)}
    dy = s["dy"].float()
    mine = mine * s["scales"]
    du = ((dy @ b.t()).view(T, S, r) * mine[:, :, None]).view(T, S * r)
    u = (s["u"][:, None, :] * mine[:, :, None]).view(T, S * r)
    dx = s["base"].float() + du @ a
    return {"dx": dx.to(dt), "da": (du.t() @ x).to(dt).view(S, r, -1), "db": (u.t() @ dy).to(dt).view(S, r, -1)}


# ------------------------------------------------------------------ the framework's operators
def _route_own(s):
    import block_scaled_grouped_gb300 as bsgg
    how = dict(score=s["score"], normalize=s["normalize"], scale=s["scale"])
    ids, w = bsgg.route_groups(s["logits"], s["k"], bias=s["b"], groups=s["groups"], topk_groups=s["kept"],
                               group_top=s["top"], **how)
    out = {"ids": ids, "weights": w}
    if s["dir"] == "train":
        out["dlogits"] = bsgg.route_groups_backward(s["logits"], ids, w, s["dweights"], **how)
    return out


def _norm_own(s):
    import block_scaled_grouped_gb300 as bsgg
    if s["dir"] == "bwd":
        dx, dw = bsgg.rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    fmt = None if s["format"] == "none" else s["format"]
    n = bsgg.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS, want_y=s["y"], row_format=fmt)
    out = {"rstd": n.rstd}
    if s["res"] is not None:
        out["h"] = n.h
    if s["y"]:
        out["y"] = n.y
    if fmt is not None:
        out["a"], out["sfa"] = n.a.view(SCALE_BITS[fmt][0]), n.sfa.view(torch.float8_e8m0fnu)
    return out


def _adapters_own(s):
    import block_scaled_grouped_gb300 as bsgg
    tokens = bsgg.TokenMap(*s["map"])
    if s["dir"] == "fwd":
        y, u = bsgg.adapters(s["x"], s["a"], s["b"], tokens, scales=s["scales"], base=s["base"])
        return {"y": y, "u": u}
    dx, da, db = bsgg.adapters_backward(s["dy"], s["x"], s["u"], s["a"], s["b"], tokens, scales=s["scales"], base=s["base"])
    return {"dx": dx, "da": da, "db": db}


def run(s):
    table = {"route": (_route_plain, _route_own), "norm": (_norm_plain, _norm_own), "adapters": (_adapters_plain, _adapters_own)}
    return table[s["op"]][1 if own else 0](s)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _take_best(values, count):
    """The `count` largest of each row one after the other, the lowest index first among equals; -1 where
    only -inf is left."""
    T, n = values.shape
    left = values.clone()
    index = torch.arange(n, device=values.device).expand(T, n)
    got = []
    for _ in range(count):
        top = left.amax(1, keepdim=True)
        at = torch.where((left == top) & (top > -math.inf), index, torch.full_like(index, n)).amin(1)
        left = left.masked_fill(index == at[:, None], -math.inf)
        got.append(torch.where(at < n, at, torch.full_like(at, -1)))
    return torch.stack(got, 1)


def _exact_route(s):
    l = s["logits"].double()
    T, L = l.shape
    G, size, k = s["groups"], L // s["groups"], s["k"]
    alive = torch.isfinite(l)
    if s["score"] == "softmax":
        p = torch.zeros_like(l)
        some = alive.any(1)
        p[some] = torch.softmax(l[some], dim=1)
    else:
        p = torch.sigmoid(l)
    c = p if s["b"] is None else p + s["b"].double()[None, :]
    c = c.masked_fill(~alive, -math.inf)
    sums = []
    for q in range(G):
        part = c[:, q * size:(q + 1) * size]
        at = _take_best(part, min(s["top"], size))
        v = torch.where(at >= 0, part.gather(1, at.clamp(min=0)), torch.zeros((), dtype=l.dtype, device=l.device))
        total = v[:, 0]
        for j in range(1, v.shape[1]):
            total = total + v[:, j]
        sums.append(torch.where(at[:, 0] >= 0, total, torch.full_like(total, -math.inf)))
    kept = _take_best(torch.stack(sums, 1), s["kept"])
    ok = torch.zeros(T, L, dtype=torch.bool, device=l.device)
    for j in range(s["kept"]):
        ok |= (torch.arange(L, device=l.device)[None, :] // size) == kept[:, j:j + 1]
    ids = _take_best(c.masked_fill(~ok, -math.inf), k)
    on = ids >= 0
    v = torch.where(on, p.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=l.dtype, device=l.device))
    part = v / v.sum(1, keepdim=True).clamp(min=1e-300) if s["normalize"] else v
    w = s["scale"] * part
    out = {"ids": ids.to(torch.int32), "weights": w}
    if s["dir"] == "train":
        # the Jacobian of the weights, choice by choice
        dl = torch.zeros_like(l)
        for j in range(k):
            g = torch.where(on[:, j], s["dweights"].double()[:, j], torch.zeros((), dtype=l.dtype, device=l.device))
            if s["score"] == "softmax" and not s["normalize"]:
                dl -= (g * w[:, j])[:, None] * p
            for i in range(k):
                # d w_j / d l_i through the chosen scores
                slope = 1 - v[:, i] if s["score"] == "sigmoid" else torch.ones_like(g)
                if s["normalize"]:
                    d = g * w[:, j] * ((1.0 if i == j else 0.0) - part[:, i]) * slope
                else:
                    d = g * w[:, j] * slope if i == j else torch.zeros_like(g)
                rows = torch.nonzero(on[:, i])[:, 0]
                dl[rows, ids[rows, i]] += d[rows]
        out["dlogits"] = dl
    return out


def _two_to(e):
    """2^e in 64 bits, from its bits (whole e, -1022 to 1023)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_to(v, man, emin):
    """v to the nearest number with `man` fraction bits and exponents from emin, ties to even."""
    _, ex = torch.frexp(v)
    step = _two_to((ex - 1).clamp(min=emin) - man)
    return torch.round(v / step) * step


def _exact_norm(s):
    T, H = s["T"], s["H"]
    w = s["w"].double()
    if s["dir"] == "bwd":
        xh = s["h"].double() * s["rstd"].double()[:, None]
        g = s["dy"].double() * w
        dx = (g - xh * (torch.einsum("th,th->t", g, xh) / H)[:, None]) * s["rstd"].double()[:, None]
        dx = dx if s["dh"] is None else dx + s["dh"].double()
        return {"dx": dx, "dw": torch.einsum("th,th->h", s["dy"].double(), xh)}
    out = {}
    h = s["x"].double()
    if s["res"] is not None:
        h = (h + s["res"].double()).to(s["x"].dtype).double()
        out["h"] = h
    rstd = (torch.einsum("th,th->t", h, h) / H + EPS) ** -0.5
    y = torch.einsum("th,t,h->th", h, rstd, w)
    out["rstd"] = rstd
    if s["y"]:
        out["y"] = y
    if s["format"] != "none":
        man, emin, qmax = (3, -6, 448.0) if s["format"] == "mxfp8_e4m3" else (2, -14, 57344.0)
        rows, kb = _padded(T), -(-H // 32)
        values = torch.zeros(T, kb * 32, dtype=torch.float64, device=y.device)
        values[:, :H] = y
        amax = values.abs().view(T, kb, 32).amax(2)
        e = torch.ceil(torch.log2(amax.clamp(min=1e-40) / qmax))
        e = torch.where(_two_to(e - 1) * qmax >= amax, e - 1, e)
        e = torch.where(_two_to(e) * qmax < amax, e + 1, e).clamp(-127, 127)
        scale = torch.where(amax > 0, _two_to(e), torch.ones_like(amax))
        a = torch.zeros(rows, H, dtype=torch.float64, device=y.device)
        a[:T] = _round_to(values / scale.repeat_interleave(32, 1), man, emin)[:, :H]
        sf = torch.ones(rows, kb, dtype=torch.float64, device=y.device)
        sf[:T] = scale
        kq = -(-kb // 4)
        # position of (row, block): tile of 128 rows, group of 4 blocks, row % 32, row % 128 / 32, block % 4
        r = torch.arange(rows, device=y.device)[:, None]
        b = torch.arange(kb, device=y.device)[None, :]
        at = (r // 128 * kq + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
        flat = torch.full((rows * kq * 4,), 2.0 ** -127, dtype=torch.float64, device=y.device)   # code 0 outside
        flat[at.reshape(-1)] = sf.reshape(-1)
        out["a"], out["sfa"] = a, flat
    return out


def _exact_adapters(s):
    T, S, r = s["T"], s["S"], s["r"]
    x = s["x"].double()
    fwd = s["dir"] == "fwd"
    out = s["base"].double()
    u = torch.zeros(T, r, dtype=torch.float64, device=x.device)
    da, db = torch.zeros(s["a"].shape, dtype=torch.float64, device=x.device), torch.zeros(s["b"].shape, dtype=torch.float64, device=x.device)
    for i in range(S):
        t = torch.nonzero(s["ids"] == i)[:, 0]
        if not t.numel():
            continue
        a, b, scale = s["a"][i].double(), s["b"][i].double(), s["scales"][i].double()
        if fwd:
            u[t] = torch.einsum("tk,rk->tr", x[t], a)
            out[t] += scale * torch.einsum("tr,rn->tn", u[t], b)
        else:
            dy = s["dy"][t].double()
            du = scale * torch.einsum("tn,rn->tr", dy, b)
            out[t] += torch.einsum("tr,rk->tk", du, a)
            da[i] = torch.einsum("tr,tk->rk", du, x[t])
            db[i] = scale * torch.einsum("tr,tn->rn", s["u"][t].double(), dy)
    return {"y": out, "u": u} if fwd else {"dx": out, "da": da, "db": db}


def exact(c, seed):
    s = prepare(c, seed)
    return {"route": _exact_route, "norm": _exact_norm, "adapters": _exact_adapters}[c["op"]](s)
