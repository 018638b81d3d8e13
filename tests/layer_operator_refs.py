"""Plain 64-bit references of the router with scores and groups, the RMS norm and
the low-rank adapters, on CPU tensors, written from their formulas."""
import math

import torch


# ------------------------------------------------------------------ routing
def scores(l, bias, score):
    """s and c = s + bias of logits (T, L) float64."""
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
        t = e.sum(1, keepdim=True)
        s = e / torch.where(t > 0, t, torch.ones_like(t))
    return s, (s if bias is None else s + bias.double())


def route_groups(logits, k, score="sigmoid", bias=None, groups=1, topk_groups=1, group_top=2, normalize=True, scale=1.0):
    """ids int32 (T, k), weights float64 (T, k).  Logits without NaN."""
    l = logits.double()
    T, L = l.shape
    size = L // groups
    s, c = scores(l, bias, score)
    # without a bias the order is that of the logits, which scores near 1 cannot tell apart
    order_by = l if bias is None else c
    off = (l == -math.inf) | (torch.zeros_like(l, dtype=torch.bool) if bias is None else (bias.double() == -math.inf)[None, :])
    ids = torch.full((T, k), -1, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        live = [e for e in range(L) if not off[t, e]]
        by = {e: (-float(order_by[t, e]), e) for e in live}
        best = []
        for g in range(groups):
            members = sorted((e for e in live if e // size == g), key=by.get)
            if members:
                # one expert a group: its order is enough
                value = float(order_by[t, members[0]]) if group_top == 1 else sum(float(c[t, e]) for e in members[:2])
                best.append((-value, g))
        kept = {g for _, g in sorted(best)[:topk_groups]}
        chosen = sorted((e for e in live if e // size in kept), key=by.get)[:k]
        if not chosen:
            continue
        ids[t, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        w[t, :len(chosen)] = weights_at(l[t:t + 1], torch.tensor([chosen]), score, normalize, scale)[0]
    return ids, w


def weights_at(l, ids, score, normalize, scale):
    """The weights as a smooth function of the logits (float64), ids held (-1: none)."""
    on = ids >= 0
    at = ids.clamp(min=0).long()
    if not normalize:
        s, _ = scores(l, None, score)
        p = torch.where(on, s.gather(1, at), torch.zeros((), dtype=l.dtype))
        return scale * p
    # logarithms, so that scores below the smallest number keep their ratios
    picked = l.gather(1, at)
    logs = torch.nn.functional.logsigmoid(picked) if score == "sigmoid" else picked
    logs = torch.where(on, logs, torch.full_like(logs, -math.inf))
    m = logs.amax(1, keepdim=True)
    e = torch.exp(logs - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    t = e.sum(1, keepdim=True)
    return scale * e / torch.where(t > 0, t, torch.ones_like(t))


def route_groups_backward(logits, ids, g, score, normalize, scale):
    l = logits.double()
    T, L = l.shape
    on = ids >= 0
    at = ids.clamp(min=0).long()
    zero = torch.zeros((), dtype=torch.float64)
    s, _ = scores(l, None, score)
    w = torch.where(on, weights_at(l, ids, score, normalize, scale), zero)
    g = torch.where(on, g.double(), zero)
    inner = (g * w).sum(1, keepdim=True) / scale
    out = torch.zeros_like(l)
    sc = s.gather(1, at)
    if score == "sigmoid":
        d = w * (1.0 - sc) * ((g - inner) if normalize else g)
        return out.scatter_add_(1, at, torch.where(on, d, zero))
    if normalize:
        return out.scatter_add_(1, at, w * (g - inner))
    return out.scatter_add_(1, at, w * g) - scale * s * inner


# ------------------------------------------------------------------ norm
def rms_norm(h, weight, eps):
    """h (T, H) as it is kept -> y, rstd in float64."""
    h = h.double()
    rstd = (h.square().mean(1) + eps) ** -0.5
    y = h * rstd[:, None]
    return (y if weight is None else y * weight.double()), rstd


def rms_norm_backward(dy, h, weight, rstd, dh):
    n = h.double() * rstd.double()[:, None]
    g = dy.double() if weight is None else dy.double() * weight.double()
    dx = rstd.double()[:, None] * (g - n * (g * n).mean(1, keepdim=True))
    return (dx if dh is None else dx + dh.double()), (dy.double() * n).sum(0)


# ------------------------------------------------------------------ adapters
def adapters(x, a, b, ids, scales, base):
    """y, u in float64; ids (T) of the tokens' adapters, -1 (or any other outside) for none."""
    x, a, b = x.double(), a.double(), b.double()
    T, S, r = x.shape[0], a.shape[0], a.shape[1]
    u = torch.zeros(T, r, dtype=torch.float64)
    y = torch.zeros(T, b.shape[2], dtype=torch.float64) if base is None else base.double().clone()
    for t in range(T):
        i = int(ids[t])
        if 0 <= i < S:
            u[t] = a[i] @ x[t]
            y[t] += (1.0 if scales is None else float(scales[i])) * (u[t] @ b[i])
    return y, u


def adapters_backward(dy, x, u, a, b, ids, scales, base):
    dy, x, u, a, b = dy.double(), x.double(), u.double(), a.double(), b.double()
    T, S = x.shape[0], a.shape[0]
    dx = torch.zeros_like(x) if base is None else base.double().clone()
    da, db, du = torch.zeros_like(a), torch.zeros_like(b), torch.zeros_like(u)
    for t in range(T):
        i = int(ids[t])
        if 0 <= i < S:
            f = 1.0 if scales is None else float(scales[i])
            du[t] = f * (b[i] @ dy[t])
            dx[t] += du[t] @ a[i]
            da[i] += torch.outer(du[t], x[t])
            db[i] += f * torch.outer(u[t], dy[t])
    return dx, da, db, du
