"""The operators around the routed experts, in 64 bits, from their formulas
(include/moe_route.h), with the magnitude of the terms behind every output.

Tolerances, derived from the arithmetic and not from any run: every kernel sums
in f32, each thread at most a few dozen terms in sequence and then trees of at
most 2 x 5 steps, uses exp, log, sqrt and the division of at most 2 ulp each,
and rounds once to the output type.  U = 128 * 2^-24 bounds that chain relative
to the sum of the absolute values of the terms (`mag`).  A bf16 output must be
the nearest bf16 of some value within that bound: it adds half the spacing of
the bf16 numbers (8 significant bits) around the output.
"""
import torch

U = 128 * 2.0 ** -24
TINY = 1e-30


def check(got, want, mag, what):
    """|got - want| <= U mag (+ half a bf16 spacing at got for bf16)."""
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)} vs {tuple(want.shape)}"
    tol = U * mag.abs() + TINY
    g = got.detach().cpu().double()
    if got.dtype == torch.bfloat16:
        # |g| = m 2^e with 1/2 <= m < 1: spacing 2^(e - 8), subnormals 2^-133
        e = torch.frexp(g).exponent.double()
        tol = tol + torch.pow(2.0, torch.clamp(e - 9, min=-134.0))
    err = (g - want).abs()
    if not bool((err <= tol).all()):
        worst = (err / tol).nan_to_num(nan=float("inf")).argmax()
        raise AssertionError(f"{what}: {int((~(err <= tol)).sum())} of {err.numel()} off; worst "
                             f"{g.flatten()[worst]} for {want.flatten()[worst]}, "
                             f"tolerance {tol.flatten()[worst]}")


def cpu64(t):
    return None if t is None else t.detach().cpu().double()


def norm_forward(residual, y, post_w, gate, act, scale, pre_w, eps):
    """-> {name: (value, magnitude)}"""
    r, y, post_w, gate, pre_w = map(cpu64, (residual, y, post_w, gate, pre_w))
    out = {}
    h, mag = r, r.abs()
    if y is not None:
        z = y
        if post_w is not None:
            rho = (y.square().mean(1) + eps).rsqrt()
            out["rstd_post"] = (rho, rho)
            z = y * rho[:, None] * post_w
        if gate is not None:
            z = z * (torch.sigmoid(gate) if act == "sigmoid" else gate)
        h = r + scale * z
        mag = r.abs() + (scale * z).abs()
        out["h"] = (h, mag)
    if pre_w is not None:
        rho = (h.square().mean(1) + eps).rsqrt()
        # h's own error, up to U mag, enters the norm relative to its rms
        grow = 1 + (mag.square().mean(1).sqrt() * rho)
        out["rstd_pre"] = (rho, rho * grow)
        out["n"] = (h * rho[:, None] * pre_w,
                    (h.abs() * grow[:, None] + mag) * rho[:, None] * pre_w.abs())
    return out


def norm_backward(gh, gn, h, y, post_w, gate, act, scale, pre_w, rstd_post, rstd_pre):
    shape = h.shape
    H = shape[1]
    gh, gn, h, y, post_w, gate, pre_w, rp, rn = map(
        cpu64, (gh, gn, h, y, post_w, gate, pre_w, rstd_post, rstd_pre))
    out = {}
    d = torch.zeros(shape, dtype=torch.float64) if gh is None else gh
    mag = d.abs()
    if pre_w is not None:
        r = rn[:, None]
        u = gn * pre_w
        d = d + r * u - h * r ** 3 * (u * h).mean(1, keepdim=True)
        mag = mag + (r * u).abs() + h.abs() * r ** 3 * (u * h).abs().mean(1, keepdim=True)
        out["grad_pre_weight"] = ((gn * h * r).sum(0), (gn * h * r).abs().sum(0))
    out["grad_residual"] = (d, mag)
    if y is None:
        return out
    g = torch.ones((), dtype=torch.float64)
    g1 = g
    if gate is not None:
        g = torch.sigmoid(gate) if act == "sigmoid" else gate
        g1 = g * (1 - g) if act == "sigmoid" else torch.ones_like(g)
    r = torch.ones(shape[0], 1, dtype=torch.float64) if rp is None else rp[:, None]
    w = torch.ones(H, dtype=torch.float64) if post_w is None else post_w
    z = y * r * w
    if gate is not None:
        dg, mg = scale * d * z * g1, (scale * mag * z * g1).abs()
        if gate.dim() == 1:
            dg, mg = dg.sum(0), mg.sum(0)
        elif gate.shape == (shape[0], 1) and H != 1:
            dg, mg = dg.sum(1, keepdim=True), mg.sum(1, keepdim=True)
        out["grad_gate"] = (dg, mg)
    b, mb = scale * g * d, (scale * g).abs() * mag
    if post_w is None:
        out["grad_y"] = (b.expand(shape), mb.expand(shape))
    else:
        out["grad_post_weight"] = ((b * y * r).sum(0), (mb * (y * r).abs()).sum(0))
        out["grad_y"] = (r * b * w - y * r ** 3 * (b * w * y).mean(1, keepdim=True),
                         r * mb * w.abs() + y.abs() * r ** 3
                         * (mb * (w * y).abs()).mean(1, keepdim=True))
    return out


def _tokens(scores, seq, mask):
    """Sequence of each token (-1: in none, or it does not count)."""
    T = scores.shape[0]
    seg = torch.full((T,), -1)
    ends = [0, T] if seq is None else seq.cpu().tolist()
    for i in range(len(ends) - 1):
        seg[ends[i]:ends[i + 1]] = i
    if mask is not None:
        seg[~mask.cpu().bool()] = -1
    # a token that does not count may hold anything
    x = torch.where((seg >= 0)[:, None], scores.cpu().double(), 0.0)
    dead = x.max(1).values == -float("inf")
    seg[dead] = -1
    x = torch.where((seg >= 0)[:, None], x, 0.0)
    return seg, x, len(ends) - 1


def _probs(x, func):
    if func == "softmax":
        return torch.softmax(x, 1)
    ls = torch.nn.functional.logsigmoid(x)
    return torch.softmax(ls, 1)


def balance_forward(scores, idx, func, seq, mask):
    seg, x, S = _tokens(scores, seq, mask)
    E, k = x.shape[1], idx.shape[1]
    p = _probs(x, func)
    lse = torch.logsumexp(x, 1)
    zmag = x.nan_to_num(neginf=0.0).abs().max(1).values + torch.log(torch.tensor(float(E))) + 1
    bal, z, zm = (torch.zeros(S, dtype=torch.float64) for _ in range(3))
    probs = torch.zeros(S, E, dtype=torch.float64)
    counts = torch.zeros(S, E, dtype=torch.int32)
    tokens = torch.zeros(S, dtype=torch.int32)
    idx = idx.cpu().long()
    for i in range(S):
        rows = (seg == i).nonzero()[:, 0]
        n = rows.numel()
        if n == 0:
            continue
        e = idx[rows].flatten()
        e = e[(e >= 0) & (e < E)]
        counts[i] = torch.bincount(e, minlength=E)
        tokens[i] = n
        probs[i] = p[rows].mean(0)
        z[i] = lse[rows].square().mean()
        zm[i] = zmag[rows].square().mean()
        bal[i] = (counts[i].double() * E / (k * n) * probs[i]).sum()
    return dict(balance=(bal, 2 * bal), z=(z, 2 * zm), probs=(probs, probs)), counts, tokens


def balance_backward(scores, counts, tokens, gb, gz, func, seq, mask, idx, w, gw, k):
    seg, x, S = _tokens(scores, seq, mask)
    T, E = x.shape
    p, q, lse = _probs(x, func), torch.softmax(x, 1), torch.logsumexp(x, 1)
    zmag = x.nan_to_num(neginf=0.0).abs().max(1).values + torch.log(torch.tensor(float(E))) + 1
    d = torch.zeros(T, E, dtype=torch.float64)
    mag = torch.zeros(T, E, dtype=torch.float64)
    counts, tokens = counts.cpu().double(), tokens.cpu().double()
    for i in range(S):
        rows = (seg == i).nonzero()[:, 0]
        n = float(tokens[i])
        if rows.numel() == 0 or n == 0:
            continue
        pr, qr = p[rows], q[rows]
        if gb is not None:
            a = float(gb[i]) * counts[i] * E / (k * n) / n
            dot = (pr * a).sum(1, keepdim=True)
            t = pr * (a - dot)
            m = pr * (a.abs() + (pr * a).abs().sum(1, keepdim=True))
            if func == "sigmoid":
                t, m = t * torch.sigmoid(-x[rows]), m * torch.sigmoid(-x[rows])
            d[rows] += t
            mag[rows] += m
        if gz is not None:
            c = 2 * float(gz[i]) / n
            d[rows] += c * lse[rows, None] * qr
            mag[rows] += abs(c) * zmag[rows, None] * qr
    if gw is not None:
        w, gw = w.cpu().double(), gw.cpu().double()
        live = (seg >= 0)[:, None]
        w, gw = torch.where(live, w, 0.0), torch.where(live, gw, 0.0)
        sel = idx.cpu().long().clamp(0, E - 1)
        dot = (w * gw).sum(1, keepdim=True)
        d.scatter_add_(1, sel, torch.where(live, w * (gw - dot), 0.0))
        mag.scatter_add_(1, sel, torch.where(
            live, w * (gw.abs() + (w * gw).abs().sum(1, keepdim=True)), 0.0))
    d[seg < 0] = 0
    mag[seg < 0] = 0
    return d, mag


def combine_backward(go, y, w, pos):
    """-> (gy, mag, named rows), (gw, mag)"""
    go, y, w, pos = go.cpu().double(), y.cpu().double(), w.cpu().double(), pos.cpu().long()
    gy = torch.zeros_like(y)
    named = torch.zeros(y.shape[0], dtype=torch.bool)
    gw, mw = torch.zeros_like(w), torch.zeros_like(w)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            r = int(pos[t, j])
            if 0 <= r < y.shape[0]:
                gy[r] = w[t, j] * go[t]
                named[r] = True
                gw[t, j] = (go[t] * y[r]).sum()
                mw[t, j] = (go[t] * y[r]).abs().sum()
    return (gy, gy.abs(), named), (gw, mw)


E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def dequant(w, sf, group):
    """[E, M, K/2] codes and [E, M, K/group] scales -> [E, M, K] float64."""
    w, sf = w.cpu(), sf.cpu()
    code = torch.stack([w & 15, w >> 4], -1).flatten(-2).long()
    v = E2M1[code & 7] * torch.where(code >= 8, -1.0, 1.0).double()
    s = torch.pow(2.0, sf.double() - 127) if sf.dtype == torch.uint8 else sf.double()
    return v * s.repeat_interleave(group, -1)


def expert_matvec(x, w, sf, group, offsets, src, k, swiglu, R):
    """-> (out, mag, rows written)"""
    d = dequant(w, sf, group)
    E, M, _ = d.shape
    ends = [0, R] if offsets is None else offsets.cpu().tolist()
    x = x.cpu().double()
    o = torch.zeros(R, M, dtype=torch.float64)
    m = torch.zeros(R, M, dtype=torch.float64)
    written = torch.zeros(R, dtype=torch.bool)
    for e in range(E):
        for r in range(max(ends[e], 0), min(ends[e + 1], R)):
            written[r] = True
            s = r if src is None else int(src[r])
            if src is not None:
                s = s // k if s >= 0 else -1
            if 0 <= s < x.shape[0]:
                o[r] = d[e] @ x[s]
                m[r] = d[e].abs() @ x[s].abs()
    if not swiglu:
        return o, m, written
    N = M // 2
    g, u, mg, mu = o[:, :N], o[:, N:], m[:, :N], m[:, N:]
    act = g * torch.sigmoid(g)
    # |silu'| <= 1.1; a product of two values, each off by U times its magnitude
    return act * u, (act * u).abs() + 1.1 * mg * u.abs() + act.abs() * mu + U * 1.1 * mg * mu, \
        written
