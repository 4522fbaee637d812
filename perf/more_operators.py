"""The router with balance and groups, and the experts' 8-bit integer products, as they are measured.

Three operators, each with the cases it meets in use:

* ``gate``    the router: softmax or sigmoid scores, a bias for balance, groups,
              top-k, renormalised and scaled weights; forward, and its gradient;
* ``cast``    rows to 8-bit integers with one scale per row;
* ``matmul``  products of routed 8-bit rows with their expert's 8-bit weights, one
              scale per token and one per output channel, with or without SwiGLU.

``own`` selects the framework's kernels; otherwise ``run`` computes the same
outputs from elementary torch operations in 32 bits, rounded once at the end
(the router's selection, which is by comparison, in 64).  ``exact`` computes them
in 64 bits from the definitions.

Sizes come from the framework's workloads (hidden 256, 4096, 7168; E = 16 or
256, k = 2 or 8; expert width 2048; up to 65536 tokens) and, for the ragged
cases, from between them.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FLOOR = 2.0 ** -96      # smallest row maximum of the cast's scale


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the router of a small decode batch: launch latency
        dict(name="gate_decode", op="gate", dir="fwd", T=16, E=256, k=8, G=8, g=4, func="sigmoid",
             score="top2", bias=True, renorm=True, scale=2.5, limited=False),
        # the same router over a prompt or a training batch
        dict(name="gate_prefill", op="gate", dir="fwd", T=65536, E=256, k=8, G=8, g=4,
             func="sigmoid", score="top2", bias=True, renorm=True, scale=2.5, limited=False),
        # an older form: softmax over all experts, the groups' maxima, no bias, weights
        # not renormalised; some tokens see only some of the experts (-inf)
        dict(name="gate_ragged", op="gate", dir="fwd", T=4099, E=160, k=6, G=8, g=3,
             func="softmax", score="max", bias=False, renorm=False, scale=16.0, limited=True),
        # the training step's gradient, added onto the balance losses' gradient
        dict(name="gate_grad", op="gate", dir="bwd", T=65536, E=256, k=8, G=8, g=4,
             func="sigmoid", score="top2", bias=True, renorm=True, scale=2.5, limited=False,
             add=True),
        # a decode batch's activations
        dict(name="cast_decode", op="cast", T=16, H=7168, x="bf16"),
        # a prompt's activations
        dict(name="cast_prefill", op="cast", T=65536, H=7168, x="bf16"),
        # weight rows from f32 masters of an odd width
        dict(name="cast_ragged", op="cast", T=4097, H=1155, x="f32"),
        # one decoded token's gate and up products with the SwiGLU
        dict(name="matmul_one", op="matmul", T=1, K=7168, N=2048, E=256, k=8, swiglu=True,
             gather=True, align=1, out="bf16"),
        # a decode batch's down products: nearly every expert is read
        dict(name="matmul_batch", op="matmul", T=64, K=2048, N=7168, E=256, k=8, swiglu=False,
             gather=False, align=1, out="bf16"),
        # a prompt's gate and up products over many experts
        dict(name="matmul_prefill", op="matmul", T=8192, K=7168, N=2048, E=256, k=8, swiglu=True,
             gather=True, align=1, out="bf16"),
        # a prompt's products over few experts with many rows each
        dict(name="matmul_few", op="matmul", T=8192, K=4096, N=4096, E=16, k=2, swiglu=False,
             gather=True, align=1, out="bf16"),
        # ragged sizes, a padded layout, f32 results
        dict(name="matmul_ragged", op="matmul", T=333, K=1040, N=1001, E=16, k=2, swiglu=False,
             gather=True, align=16, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate", "cast", "cast", "matmul", "matmul", "matmul"])
    if op == "gate":
        G = rng.choice([1, 1, 4, 8, 8, rng.randint(2, 16)])
        E = rng.choice([256, 64, 16 * G, G * rng.randint(1, 48)])
        E = max(2 if G == 1 else 1, min(E, 512) // G) * G
        g = rng.randint(1, G)
        most = min(8, E // G * g)
        # one selected expert's renormalised weight is a constant
        renorm = most > 1 and rng.random() < 0.6
        k = rng.randint(2 if renorm else 1, most)
        T = _log_int(rng, 1, min(65536, (16 << 20) // E))
        return dict(op="gate", dir=rng.choice(["fwd", "fwd", "bwd"]), T=T, E=E, k=k, G=G, g=g,
                    func=rng.choice(["sigmoid", "softmax"]), score=rng.choice(["top2", "max"]),
                    bias=rng.random() < 0.6, renorm=renorm,
                    scale=rng.choice([1.0, 2.5]), limited=rng.random() < 0.3,
                    add=rng.random() < 0.5)
    if op == "cast":
        H = rng.choice([_log_int(rng, 1, 16384), 16 * _log_int(rng, 1, 1024), 256, 4096, 7168])
        T = _log_int(rng, 1, max(1, min(65536, (256 << 20) // H)))
        return dict(op="cast", T=T, H=H, x=rng.choice(["bf16", "bf16", "f32"]))
    E = rng.choice([1, 8, 16, 64, 256])
    k = 1 if E == 1 else rng.randint(1, 8)
    case = dict(op="matmul", T=_log_int(rng, 1, 8192), K=16 * _log_int(rng, 2, 448),
                N=rng.choice([256, 2048, 4096, _log_int(rng, 1, 7168)]), E=E, k=k,
                swiglu=rng.random() < 0.5, gather=rng.random() < 0.6,
                align=rng.choice([1, 1, 1, 16, 128]), out=rng.choice(["bf16", "bf16", "f32"]))
    if E == 1:
        case["align"] = 1
    # no more work and no more memory than the largest listed case
    while work(case)["flops"] > 2e12 or case["E"] * case["K"] * case["N"] > 3e9:
        if case["T"] > 64:
            case["T"] //= 2
        else:
            case["N"] = (case["N"] + 1) // 2
    return case


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    return {"gate": _prepare_gate, "cast": _prepare_cast, "matmul": _prepare_matmul}[case["op"]](
        case, g)


def _prepare_gate(case, g):
    T, E, k, G = case["T"], case["E"], case["k"], case["G"]
    # router logits, with experts of uneven popularity; the bias works against it
    pop = _randn((E,), g, std=0.3)
    scores = _randn((T, E), g) + pop
    s = dict(case=case, bias=(-0.2 * pop + _randn((E,), g, std=0.02)) if case["bias"] else None)
    if case["limited"]:
        # about a third of the experts is closed to a token, never all of them
        shut = torch.rand((T, E), generator=g, device=DEV) < 0.33
        shut[:, 0] = False
        scores = torch.where(shut, torch.full_like(scores, -math.inf), scores)
    s["scores"] = scores
    if case["dir"] == "bwd":
        # what the forward pass left
        s["topk_idx"] = (scores + (0 if s["bias"] is None else s["bias"])).topk(
            k, dim=1).indices.to(torch.int32)
        s["grad_w"] = _randn((T, k), g, std=0.02)
        s["add"] = _randn((T, E), g, std=1e-4) if case["add"] else None
    return s


def _prepare_cast(case, g):
    T, H = case["T"], case["H"]
    # activations: a few channels are much larger than the others
    x = torch.randn((T, H), generator=g, device=DEV, dtype=torch.float32)
    x *= torch.where(torch.rand((H,), generator=g, device=DEV) < 0.005, 8.0, 1.0)
    return dict(case=case, x=x.to(DTYPES[case["x"]]))


def _normal_int8(shape, g):
    """Normal values in 8 bits, as a row of a few thousand scaled by its largest gives them."""
    out = torch.empty(shape, dtype=torch.int8, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.shape, generator=g, device=DEV).mul_(32.0).round_().clamp_(
            -127.0, 127.0))
    return out


def _prepare_matmul(case, g):
    T, K, N, E, k, align = (case[n] for n in ("T", "K", "N", "E", "k", "align"))
    M = N * (2 if case["swiglu"] else 1)
    s = dict(case=case)
    s["offsets"] = s["sorted_src"] = None
    R = T * k
    s["ends"] = [0, R]
    if E > 1:
        # each token's distinct experts, of uneven popularity; rows sorted by expert, every
        # expert's rows rounded up to `align`
        scores = _randn((T, E), g) + _randn((E,), g, std=0.3)
        flat = scores.topk(k, dim=1).indices.reshape(-1)
        order = flat.argsort(stable=True)
        counts = torch.bincount(flat, minlength=E)
        padded = (counts + align - 1) // align * align
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), padded.cumsum(0)])
        first = counts.cumsum(0) - counts
        e = flat[order]
        row = offsets[:-1][e] + torch.arange(R, device=DEV) - first[e]
        R = int(offsets[-1])
        src = torch.full((R,), -1, dtype=torch.int32, device=DEV)
        src[row] = order.to(torch.int32)
        s["offsets"], s["sorted_src"] = offsets.to(torch.int32), src
        s["ends"] = offsets.tolist()
    gather = case["gather"] and E > 1
    X = T if gather else R
    s["x"] = _normal_int8((X, K), g)
    s["x_sf"] = (0.7 + 0.6 * torch.rand((X,), generator=g, device=DEV)) / 32.0
    s["gather"] = gather
    if not gather and align == 1:
        s["sorted_src"] = None
    elif not gather:
        # the rows are in place already; a padding row is zero
        s["x"][s["sorted_src"] < 0] = 0
        s["sorted_src"] = None
    s["w"] = _normal_int8((E, M, K), g)
    # weights of variance 1/K
    s["w_sf"] = (0.7 + 0.6 * torch.rand((E, M), generator=g, device=DEV)) / (32.0 * math.sqrt(K))
    return s


# ---------------------------------------------------------------- the passes

def run(state):
    if own:
        return _run_own(state)
    return {"gate": _plain_gate, "cast": _plain_cast, "matmul": _plain_matmul}[
        state["case"]["op"]](state)


def _run_own(s):
    from moe_routing_precision_gb300 import ops
    c = s["case"]
    if c["op"] == "gate":
        if c["dir"] == "fwd":
            idx, w = ops.router_gate(s["scores"], c["k"], score_func=c["func"], bias=s["bias"],
                                     num_groups=c["G"], topk_groups=c["g"],
                                     group_score=c["score"], renormalize=c["renorm"],
                                     scale=c["scale"])
            return dict(idx=idx, w=w)
        return ops.router_gate_backward(s["scores"], s["topk_idx"], s["grad_w"],
                                        score_func=c["func"], renormalize=c["renorm"],
                                        scale=c["scale"], add=s["add"])
    if c["op"] == "cast":
        q, sf = ops.cast_int8(s["x"])
        return dict(q=q, sf=sf)
    return ops.expert_matmul_int8(s["x"], s["x_sf"], s["w"], s["w_sf"], s["offsets"],
                                  sorted_src=s["sorted_src"], k=c["k"], swiglu=c["swiglu"],
                                  out_dtype=DTYPES[c["out"]])


def _plain_scores(x, func):
    """Every expert's score; 0 where x is -inf (a row of -inf: all 0)."""
    if func == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.max(1, keepdim=True).values
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    ex = torch.exp(x - m)
    tot = ex.sum(1, keepdim=True)
    return ex / torch.where(tot == 0, torch.ones_like(tot), tot)


def _plain_gate(s):
    c = s["case"]
    T, E, k, G, g = (c[n] for n in ("T", "E", "k", "G", "g"))
    x = s["scores"]
    if c["dir"] == "bwd":
        return _plain_gate_grad(s)
    # the choice lies next to a border: 64 bits
    sc = _plain_scores(x.double(), c["func"])
    live = x > -math.inf
    choice = sc if s["bias"] is None else sc + s["bias"].double()
    low = torch.full_like(choice, -math.inf)
    choice = torch.where(live, choice, low)
    if G > 1:
        per = choice.view(T, G, E // G).sort(dim=2, descending=True).values
        gs = per[:, :, 0]
        if c["score"] == "top2" and E // G > 1:
            gs = torch.where(per[:, :, 1] > -math.inf, gs + per[:, :, 1], gs)
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, :g]
        open_ = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, best, True)
        open_ = open_.repeat_interleave(E // G, 1)
        # a closed expert of an open group comes after every other one of the open groups
        choice = torch.where(open_, choice.clamp(min=-1e300), low)
    idx = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = sc.gather(1, idx)
    if c["renorm"]:
        tot = w.sum(1, keepdim=True)
        w = w / torch.where(tot == 0, torch.ones_like(tot), tot)
    return dict(idx=idx.to(torch.int32), w=(w * c["scale"]).float())


def _plain_gate_grad(s):
    c = s["case"]
    x, idx, gw = s["scores"], s["topk_idx"].long(), s["grad_w"]
    out = torch.zeros_like(x) if s["add"] is None else s["add"].clone()
    sc = _plain_scores(x, c["func"])
    sel = sc.gather(1, idx)
    if c["renorm"]:
        tot = sel.sum(1, keepdim=True)
        w = sel / torch.where(tot == 0, torch.ones_like(tot), tot)
        d = c["scale"] * w * (gw - (gw * w).sum(1, keepdim=True))
        if c["func"] == "sigmoid":
            d = d * (1.0 / (1.0 + torch.exp(x.gather(1, idx))))
    else:
        d = c["scale"] * gw * sel
        if c["func"] == "sigmoid":
            d = d * (1.0 / (1.0 + torch.exp(x.gather(1, idx))))
        else:
            out = out - sc * d.sum(1, keepdim=True)
    return out.scatter_add_(1, idx, d)


def _plain_cast(s):
    x = s["x"].float()
    amax = x.abs().max(1).values.clamp(min=FLOOR)
    top = torch.full_like(amax, 127.0)      # a tensor: divided, not multiplied by an inverse
    sf = amax / top
    q = torch.round(x * (top / amax)[:, None])
    return dict(q=q.to(torch.int8), sf=sf)


def _plain_matmul(s):
    c = s["case"]
    N, E, k = c["N"], c["E"], c["k"]
    ends = s["ends"]
    R = ends[-1]
    out = torch.empty((R, N), dtype=DTYPES[c["out"]], device=DEV)
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        w = s["w"][e].float().T
        for a in range(lo, hi, 16384):
            b = min(hi, a + 16384)
            if s["sorted_src"] is None:
                o = (s["x"][a:b].float() @ w) * s["x_sf"][a:b, None]
            else:
                src = s["sorted_src"][a:b]
                row = src.clamp(min=0).long() // k
                keep = (src >= 0).float()[:, None]
                o = (s["x"][row].float() @ w) * (s["x_sf"][row][:, None] * keep)
            o = o * s["w_sf"][e]
            if c["swiglu"]:
                o = o[:, :N] / (1.0 + torch.exp(-o[:, :N])) * o[:, N:]
            out[a:b] = o.to(out.dtype)
    return out


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "cast": _exact_cast, "matmul": _exact_matmul}[case["op"]](s)


def _exact_gate(s):
    c = s["case"]
    T, E, k, G, g = (c[n] for n in ("T", "E", "k", "G", "g"))
    x = s["scores"].double()
    shut = torch.isneginf(x)
    if c["func"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(x, 1).nan_to_num(nan=0.0)
    if c["dir"] == "bwd":
        # the Jacobian of the weights, row by row of the selected experts
        idx, gw = s["topk_idx"].long(), s["grad_w"].double() * c["scale"]
        sel = torch.gather(p, 1, idx)
        if c["renorm"]:
            tot = sel.sum(1, keepdim=True).clamp(min=1e-300)
            ds = gw / tot - (gw * sel).sum(1, keepdim=True) / tot.square()
        else:
            ds = gw
        dp = torch.zeros_like(p).scatter_add_(1, idx, ds)
        if c["func"] == "sigmoid":
            grad = dp * p * torch.sigmoid(-x)
        else:
            grad = p * (dp - (p * dp).sum(1, keepdim=True))
        return grad if s["add"] is None else grad + s["add"].double()
    key = p.clone() if s["bias"] is None else p + s["bias"].double()
    rows = torch.arange(T, device=DEV)
    if G > 1:
        rest = key.masked_fill(shut, -math.inf).view(T, G, -1).clone()
        score = rest.amax(2)
        if c["score"] == "top2" and E // G > 1:
            rest.scatter_(2, rest.argmax(2, keepdim=True), -math.inf)
            second = rest.amax(2)
            score = score + second.masked_fill(torch.isneginf(second), 0.0)
        taken = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        for _ in range(g):
            # the first of the largest among those not taken (all of them may be -inf)
            left = score.masked_fill(taken, -math.inf)
            top = left.amax(1, keepdim=True)
            first = ((left == top) & ~taken).int().argmax(1)
            taken[rows, first] = True
        gone = ~taken.repeat_interleave(E // G, 1)
    else:
        gone = torch.zeros(T, E, dtype=torch.bool, device=DEV)
    idx = torch.empty(T, k, dtype=torch.int64, device=DEV)
    for j in range(k):
        left = key.masked_fill(shut | gone, -math.inf)
        top = left.amax(1, keepdim=True)
        idx[:, j] = ((left == top) & ~gone).int().argmax(1)
        gone[rows, idx[:, j]] = True
    w = torch.gather(p.masked_fill(shut, 0.0), 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return dict(idx=idx.to(torch.int32), w=w * c["scale"])


def _exact_cast(s):
    """The cast's definition has two f32 roundings, the scale and its inverse; then x times
    the inverse, rounded to f32 and to the nearest integer, ties to even.  The integers
    have to be equal, so the roundings are the definition's too."""
    x = s["x"].float().cpu().numpy()
    q = np.empty(x.shape, dtype=np.int8)
    sfs = np.empty(x.shape[0], dtype=np.float64)
    step = max(1, (1 << 26) // x.shape[1])
    for a in range(0, x.shape[0], step):
        part = x[a:a + step].astype(np.float64)
        top = np.maximum(np.max(np.abs(part), axis=1), FLOOR)
        sf = (top / 127.0).astype(np.float32).astype(np.float64)
        inv = (127.0 / top).astype(np.float32).astype(np.float64)
        part *= inv[:, None]
        q[a:a + step] = np.rint(part.astype(np.float32)).astype(np.int8)
        sfs[a:a + step] = sf
    return dict(q=torch.from_numpy(q), sf=torch.from_numpy(sfs))


def _exact_matmul(s):
    c = s["case"]
    if work(c)["flops"] > 6e12:
        return None
    N, k = c["N"], c["k"]
    out = torch.zeros(s["ends"][-1], N, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        rows = torch.arange(s["ends"][e], s["ends"][e + 1], device=DEV)
        if rows.numel() == 0:
            continue
        at = rows
        if s["sorted_src"] is not None:
            src = s["sorted_src"][rows].long()
            rows, src = rows[src >= 0], src[src >= 0]
            at = torch.div(src, k, rounding_mode="floor")
        o = torch.einsum("rc,mc->rm", s["x"][at].double() * s["x_sf"][at, None].double(),
                         s["w"][e].double() * s["w_sf"][e, :, None].double())
        if c["swiglu"]:
            o = o[:, :N] * torch.sigmoid(o[:, :N]) * o[:, N:]
        out[rows] = o
    return out


# -------------------------------------------------------------------- the work

def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    op = case["op"]
    T = case["T"]
    if op == "gate":
        E, k = case["E"], case["k"]
        if case["dir"] == "fwd":
            return {"bytes": T * E * 4 + (4 * E if case["bias"] else 0) + T * k * 8,
                    "flops": T * E * 6}
        dense = case["func"] == "softmax" and not case["renorm"]
        b = T * E * 4 * (1 + (1 if case["add"] else 0)) + T * k * 8
        # the selected scores, or all where the gradient reaches all
        return {"bytes": b + (T * E * 4 if dense else T * k * 4),
                "flops": T * (E * 6 if dense else k * 12)}
    if op == "cast":
        H = case["H"]
        return {"bytes": T * H * (1 + (2 if case["x"] == "bf16" else 4)) + 4 * T,
                "flops": T * H * 3}
    K, N, E, k = case["K"], case["N"], case["E"], case["k"]
    M = N * (2 if case["swiglu"] else 1)
    R = T * k
    # experts that T tokens with k distinct experts each are expected to use
    used = E * (1.0 - (1.0 - min(1.0, k / E)) ** T)
    X = T if case["gather"] and E > 1 else R
    b = used * M * (K + 4) + X * (K + 4) + R * N * (2 if case["out"] == "bf16" else 4)
    return {"bytes": int(b), "flops": 2 * R * M * K}
