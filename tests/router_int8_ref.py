"""The router with balance and groups, the row cast to 8-bit integers and the experts'
products in them, in 64 bits, from their formulas (include/moe_route.h).

Tolerances, derived from the arithmetic and not from any run.  The selection and the
integers are fixed by the definition: they have to be equal.  The router's weights and
gradients go through exp, reciprocals, sums of at most 32 lanes and at most 1024 terms
and a few products, each within 2 ulp: block_ref's U = 128 * 2^-24 of the terms'
magnitude.  A product's sum of integers is exact while the sum of its terms' absolute
values is below 2^24; two f32 products follow, and with the SwiGLU an exp, a division
and a product: 16 * 2^-24 of the result (and of the gate's own slope, see matmul).
"""
import torch

from tests.block_ref import cpu64

INF = float("inf")


def scores(x, func):
    x = cpu64(x)
    if func == "sigmoid":
        return torch.sigmoid(x)
    m = x.max(1, keepdim=True).values
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    ex = torch.exp(x - m)
    z = ex.sum(1, keepdim=True)
    return ex / torch.where(z == 0, torch.ones_like(z), z)


def gate(x, k, func, bias, G, g, group_score, renorm, scale):
    """-> idx [T, k], w [T, k], one token after the other by plain comparisons."""
    T, E = x.shape
    s = scores(x, func)
    xs = cpu64(x)
    # without a bias the order of c is that of x, also where s has left f64's range
    c = xs.clone() if bias is None else s + cpu64(bias)
    c[xs == -INF] = -INF
    gc = (s if bias is None else s + cpu64(bias)).clone()
    gc[xs == -INF] = -INF
    if bias is None and group_score == "max":
        gc = c
    n = E // G
    idx = torch.empty(T, k, dtype=torch.int64)
    for t in range(T):
        vals = []
        for i in range(G):
            v = sorted(gc[t, i * n:(i + 1) * n].tolist(), reverse=True)
            two = group_score == "top2" and n > 1 and v[1] > -INF
            vals.append(v[0] + v[1] if two else v[0])
        kept = sorted(range(G), key=lambda i: (-vals[i], i))[:g]
        open_ = [e for i in sorted(kept) for e in range(i * n, (i + 1) * n)]
        row = c[t].tolist()
        idx[t] = torch.tensor(sorted(open_, key=lambda e: (-row[e], e))[:k])
    return idx, weights(x, idx, func, renorm, scale)


def weights(x, idx, func, renorm, scale):
    x = cpu64(x)
    if not renorm:
        return scale * scores(x, func).gather(1, idx)
    sel = x.gather(1, idx)
    # the log of the score, so that the ratio keeps its digits
    ls = torch.nn.functional.logsigmoid(sel) if func == "sigmoid" else sel
    w = torch.softmax(ls, 1).nan_to_num(nan=0.0)
    return scale * w


def gate_grad(x, idx, gw, func, renorm, scale, add):
    """-> gradient and the magnitude of its terms."""
    xs, gw = cpu64(x), cpu64(gw)
    E = x.shape[1]
    idx = idx.cpu().long()
    ok = (idx >= 0) & (idx < E)
    at = idx.clamp(0, E - 1)
    out = torch.zeros_like(xs) if add is None else cpu64(add).clone()
    mag = out.abs()
    gw = torch.where(ok, gw, 0.0)
    if renorm:
        sel = xs.gather(1, at)
        ls = torch.nn.functional.logsigmoid(sel) if func == "sigmoid" else sel
        w = torch.softmax(torch.where(ok, ls, -INF), 1).nan_to_num(nan=0.0)
    else:
        w = torch.where(ok, scores(x, func).gather(1, at), 0.0)
    dot, adot = (gw * w).sum(1, keepdim=True), (gw * w).abs().sum(1, keepdim=True)
    tail = torch.sigmoid(-xs.gather(1, at)) if func == "sigmoid" else torch.ones_like(w)
    if renorm:
        d, m = scale * w * (gw - dot) * tail, scale * w * (gw.abs() + adot) * tail
    elif func == "sigmoid":
        d, m = scale * w * gw * tail, (scale * w * gw * tail).abs()
    else:
        d, m = scale * w * gw, (scale * w * gw).abs()
        s = scores(x, func)
        out = out - s * scale * dot
        mag = mag + s * abs(scale) * adot
    d, m = torch.where(ok, d, 0.0), torch.where(ok, m, 0.0)
    return out.scatter_add(1, at, d), mag.scatter_add(1, at, m.abs())


def cast(x):
    """The definition's f32 steps, which 64 bits hold exactly before each rounding."""
    v = cpu64(x)
    a = v.abs().max(1).values.clamp(min=2.0 ** -96)
    sf = (a / 127).float()
    inv = (127 / a).float().double()
    q = torch.round((v * inv[:, None]).float())
    return q.to(torch.int8), sf


def matmul(x, x_sf, w, w_sf, offsets, src, k, swiglu):
    """-> out [R, N] (NaN where no row is written), its magnitude, and the largest sum of
    absolute terms."""
    X, WT = x.cpu().double(), w.cpu().double()
    E, M = w.shape[:2]
    R = x.shape[0] if src is None else src.shape[0]
    ends = [0, R] if offsets is None else offsets.cpu().tolist()
    N = M // 2 if swiglu else M
    out = torch.full((R, N), float("nan"), dtype=torch.float64)
    mag = torch.ones_like(out)
    largest = 0.0
    for e in range(E):
        lo, hi = max(ends[e], 0), min(ends[e + 1], R)
        if hi <= lo:
            continue
        at = torch.arange(lo, hi) if src is None else torch.div(
            src[lo:hi].cpu().long(), k, rounding_mode="floor")
        keep = (at >= 0) & (at < X.shape[0])
        if src is not None:
            keep &= src[lo:hi].cpu() >= 0
        at = at.clamp(0, X.shape[0] - 1)
        rows = X[at] * keep[:, None]
        if rows.numel():
            largest = max(largest, float((rows.abs() @ WT[e].abs().T).max()))
        o = (rows @ WT[e].T) * cpu64(x_sf)[at][:, None] * cpu64(w_sf)[e]
        if swiglu:
            gt, up = o[:, :N], o[:, N:]
            sig = torch.sigmoid(gt)
            out[lo:hi] = gt * sig * up
            # an error of the gate relative to it grows by |g silu'(g)| / |silu(g)| <= 1 + |g|
            mag[lo:hi] = out[lo:hi].abs() * (1 + gt.abs())
        else:
            out[lo:hi] = o
            mag[lo:hi] = o.abs()
    return out, mag, largest
