"""The operators around the routed experts, as they are measured.

Four operators, each with the cases it meets in use:

* ``norm``      the norms before and after a block, with the block's gate and
                residual scale: forward (serving and training) and backward;
* ``balance``   the router's balance loss, z-loss and per-expert counts over
                packed sequences: forward, and the router's whole score gradient;
* ``combine``   the backward pass of the weighted combine;
* ``matvec``    products of routed rows with 4-bit expert weights (E2M1 codes,
                one scale per group), for decode batches.

``own`` selects the framework's kernels; otherwise ``run`` computes the same
outputs from elementary torch operations in 32 bits, rounded once at the end.
``exact`` computes them in 64 bits from the definitions.

Sizes come from the framework's workloads (hidden 256, 4096, 7168; E = 16 or
256, k = 2 or 8; expert width 2048; up to 65536 tokens) and, for the ragged
cases, from between them.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token between two layers of a hidden-4096 model: residual
        # add, post-norm and the next pre-norm; latency is all that counts
        dict(name="norm_decode", op="norm", dir="fwd", T=1, H=4096, stream="bf16", block="bf16",
             gate="none", act="none", post=True, pre=True),
        # a prefill batch at hidden 7168, each token's branch gated by a sigmoid
        dict(name="norm_prefill", op="norm", dir="fwd", T=16384, H=7168, stream="bf16",
             block="bf16", gate="token", act="sigmoid", post=True, pre=True),
        # the training backward at hidden 7168: f32 residual stream, bf16 block,
        # a learned gate per channel (its gradient summed over all tokens)
        dict(name="norm_train", op="norm", dir="bwd", T=8192, H=7168, stream="f32", block="bf16",
             gate="channel", act="none", post=True, pre=True),
        # a ragged micro-batch of an odd width with an elementwise gate, all f32
        dict(name="norm_ragged", op="norm", dir="bwd", T=1001, H=1155, stream="f32", block="f32",
             gate="element", act="sigmoid", post=True, pre=True),
        # the smallest router: one tiny batch, one sequence; launch latency
        dict(name="balance_tiny", op="balance", dir="fwd", T=64, E=16, k=2, S=1, func="softmax",
             mask=False, limited=False),
        # a training step's packed batch: 33 sequences of uneven lengths, padding masked
        dict(name="balance_train", op="balance", dir="fwd", T=65536, E=256, k=8, S=33,
             func="softmax", mask=True, limited=False),
        # its backward: the score gradient from both losses and the top-k weights,
        # for a sigmoid router whose tokens see only some of the expert groups
        dict(name="balance_grad", op="balance", dir="bwd", T=65536, E=256, k=8, S=33,
             func="sigmoid", mask=True, limited=True),
        # the combine's backward in a training step, hidden 7168
        dict(name="combine_train", op="combine", T=8192, H=7168, E=256, k=8, grad="bf16", align=1,
             drop=0.0),
        # a ragged batch into a padded layout with copies over capacity dropped
        dict(name="combine_padded", op="combine", T=999, H=1000, E=16, k=2, grad="f32", align=128,
             drop=0.05),
        # one decoded token's gate and up products with the SwiGLU
        dict(name="matvec_one", op="matvec", T=1, K=7168, N=2048, E=256, k=8, group=32,
             scale="ue8m0", swiglu=True, gather=True, out="bf16"),
        # a decode batch's down products: nearly every expert is read
        dict(name="matvec_batch", op="matvec", T=64, K=2048, N=7168, E=256, k=8, group=128,
             scale="f32", swiglu=False, gather=False, out="bf16"),
        # ragged sizes: 16 experts with several rows each, the smallest groups
        dict(name="matvec_ragged", op="matvec", T=29, K=1056, N=1001, E=16, k=2, group=16,
             scale="f32", swiglu=False, gather=True, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "balance", "balance", "combine", "matvec", "matvec"])
    if op == "norm":
        H = rng.choice([_log_int(rng, 1, 8192), 8 * _log_int(rng, 8, 1024), 256, 4096, 7168])
        T = _log_int(rng, 1, max(1, min(65536, (40 << 20) // H)))
        y = rng.random() < 0.85
        post = y and rng.random() < 0.8
        return dict(op="norm", dir=rng.choice(["fwd", "bwd"]), T=T, H=H,
                    stream=rng.choice(["bf16", "f32"]), block=rng.choice(["bf16", "f32"]),
                    gate=rng.choice(["none", "channel", "token", "element"]) if y else "none",
                    act=rng.choice(["none", "sigmoid"]) if y else "none", post=post,
                    pre=(not y) or rng.random() < 0.8, y=y)
    if op == "balance":
        E = rng.choice([16, 64, 256, rng.randint(1, 512)])
        T = _log_int(rng, 1, min(65536, (16 << 20) // E))
        return dict(op="balance", dir=rng.choice(["fwd", "bwd"]), T=T, E=E,
                    k=rng.randint(1, min(8, E)), S=rng.choice([1, rng.randint(1, 64)]),
                    func=rng.choice(["softmax", "sigmoid"]), mask=rng.random() < 0.5,
                    limited=rng.random() < 0.4)
    if op == "combine":
        E = rng.choice([16, 256, rng.randint(8, 300)])
        k = rng.randint(1, 8)
        H = 8 * rng.choice([_log_int(rng, 1, 1024), 32, 512, 896])
        T = _log_int(rng, 1, max(1, min(8192, (400 << 20) // (H * k))))
        return dict(op="combine", T=T, H=H, E=E, k=k, grad=rng.choice(["bf16", "f32"]),
                    align=rng.choice([1, 1, 16, 128]), drop=rng.choice([0.0, 0.0, 0.1]))
    group = rng.choice([16, 32, 64, 128])
    E = rng.choice([1, 8, 16, 64, 256])
    K = max(group, 32) * rng.randint(1, 7168 // max(group, 32))
    N = rng.choice([256, 2048, 4096, _log_int(rng, 1, 4096)])
    swiglu = rng.random() < 0.5
    k = 1 if E == 1 else rng.randint(1, 8)
    case = dict(op="matvec", T=_log_int(rng, 1, 32 if E == 1 else 64), K=K, N=N, E=E, k=k,
                group=group, scale=rng.choice(["f32", "ue8m0"]), swiglu=swiglu,
                gather=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    # no more weights than the largest listed batch reads
    while work(case)["bytes"] > 1.6e9:
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
    return {"norm": _prepare_norm, "balance": _prepare_balance, "combine": _prepare_combine,
            "matvec": _prepare_matvec}[case["op"]](case, g)


def _prepare_norm(case, g):
    T, H = case["T"], case["H"]
    rt, yt = DTYPES[case["stream"]], DTYPES[case["block"]]
    has_y = case.get("y", True)
    s = dict(case=case, scale=0.5, eps=EPS)
    # a residual stream grows along the layers; the block's outputs are of order one
    s["residual"] = _randn((T, H), g, rt, 3.0)
    s["y"] = _randn((T, H), g, yt) if has_y else None
    s["post_weight"] = 1.0 + _randn((H,), g, std=0.2) if case["post"] else None
    s["pre_weight"] = 1.0 + _randn((H,), g, std=0.2) if case["pre"] else None
    kind = case["gate"]
    s["gate"] = (None if kind == "none" else _randn((H,), g) if kind == "channel"
                 else _randn((T, 1), g) if kind == "token" else _randn((T, H), g, yt))
    s["act"] = case["act"] if kind != "none" else "none"
    if case["dir"] == "bwd":
        # what the forward pass left: h and the two rows of inverse norms
        s["grad_h"] = _randn((T, H), g, rt)
        s["grad_n"] = _randn((T, H), g, yt) if case["pre"] else None
        h = s["residual"].float()
        s["rstd_post"] = None
        if has_y:
            y = s["y"].float()
            z = y
            if case["post"]:
                s["rstd_post"] = torch.rsqrt(y.square().mean(1) + EPS)
                z = y * s["rstd_post"][:, None] * s["post_weight"]
            if s["gate"] is not None:
                gt = s["gate"].float()
                z = z * (torch.sigmoid(gt) if s["act"] == "sigmoid" else gt)
            h = h + s["scale"] * z
        s["rstd_pre"] = torch.rsqrt(h.square().mean(1) + EPS) if case["pre"] else None
        s["h"] = h.to(rt)
        del s["residual"]
    return s


def _pick_experts(T, E, k, g, bias_std=0.3):
    """Distinct experts of each token, in descending score order, and the scores."""
    scores = _randn((T, E), g) + _randn((E,), g, std=bias_std)
    return scores, scores.topk(k, dim=1).indices.to(torch.int32)


def _prepare_balance(case, g):
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    scores = _randn((T, E), g) + _randn((E,), g, std=0.3)
    if case["limited"] and E >= 2 * k and E >= 4:
        # each token may use half of the experts, in blocks of a quarter: the rest are -inf
        q = (E + 3) // 4
        keep = torch.rand((T, 4), generator=g, device=DEV).argsort(1) < 2
        ok = keep.repeat_interleave(q, 1)[:, :E]
        ok = ok & (ok.sum(1, keepdim=True) >= k) | ~(ok.sum(1, keepdim=True) >= k)
        scores = torch.where(ok, scores, torch.full_like(scores, -math.inf))
    idx = scores.topk(k, dim=1).indices.to(torch.int32)
    s = dict(case=case, scores=scores, topk_idx=idx)
    cuts = torch.rand((S - 1,), generator=g, device=DEV).sort().values * T
    s["seq_offsets"] = torch.cat([torch.zeros(1, device=DEV), cuts.floor(),
                                  torch.full((1,), T, device=DEV)]).to(torch.int32)
    s["token_mask"] = (torch.rand((T,), generator=g, device=DEV) < 0.9) if case["mask"] else None
    if case["dir"] == "bwd":
        seg, keep = _segments(s)
        s["counts"] = torch.zeros((S, E), dtype=torch.int32, device=DEV)
        s["counts"].view(-1).index_add_(
            0, (seg[:, None] * E + idx.long()).reshape(-1),
            keep[:, None].expand(T, k).to(torch.int32).reshape(-1))
        s["tokens"] = torch.zeros(S, dtype=torch.int32, device=DEV).index_add_(
            0, seg, keep.to(torch.int32))
        s["topk_weights"] = torch.softmax(torch.gather(scores, 1, idx.long()), 1)
        s["grad_topk_weights"] = _randn((T, k), g, std=0.02)
        s["grad_balance"] = torch.rand((S,), generator=g, device=DEV) * 0.01 / S
        s["grad_z"] = torch.rand((S,), generator=g, device=DEV) * 0.001 / S
    return s


def _prepare_combine(case, g):
    T, H, E, k, align = case["T"], case["H"], case["E"], case["k"], case["align"]
    _, idx = _pick_experts(T, E, k, g)
    kept = torch.rand((T, k), generator=g, device=DEV) >= case["drop"]
    flat = torch.where(kept, idx, torch.full_like(idx, E)).reshape(-1).long()
    order = flat.argsort(stable=True)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    padded = (counts + align - 1) // align * align
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(counts, 0) - counts
    e = flat[order]
    n = int(counts.sum())
    e, order = e[:n], order[:n]
    row = start[e] + torch.arange(n, device=DEV) - first[e]
    R = max(1, int(padded.sum()))
    pos = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    pos[order] = row.to(torch.int32)
    src = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    src[row] = order.to(torch.int32)
    w = torch.softmax(_randn((T, k), g), 1)
    return dict(case=case, pos=pos.view(T, k), topk_weights=w,
                sorted_src=src if (align > 1 or n == 0) else None,
                y=_randn((R, H), g, torch.bfloat16),
                grad_out=_randn((T, H), g, DTYPES[case["grad"]], 0.02))


def _normal_codes(shape, g):
    """Random E2M1 codes with the frequencies of a normal weight scaled to +-6, two per byte."""
    q = torch.linspace(0.5 / 256, 1 - 0.5 / 256, 256, dtype=torch.float64, device=DEV)
    v = (math.sqrt(2.0) * torch.erfinv(2 * q - 1) * 2.2).float()
    lut = (v[:, None] - torch.tensor(E2M1, device=DEV)[None, :]).abs().argmin(1).to(torch.uint8)
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    for e in range(shape[0]):
        r = torch.randint(0, 256, (2,) + tuple(shape[1:]), generator=g, device=DEV)
        out[e] = lut[r[0]] | (lut[r[1]] << 4)
    return out


def _prepare_matvec(case, g):
    T, K, N, E, k, group = (case[n] for n in ("T", "K", "N", "E", "k", "group"))
    R, M = T * k, N * (2 if case["swiglu"] else 1)
    s = dict(case=case)
    if E == 1:
        s["offsets"] = s["sorted_src"] = None
    else:
        _, idx = _pick_experts(T, E, k, g)
        flat = idx.reshape(-1).long()
        s["sorted_src"] = flat.argsort(stable=True).to(torch.int32)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV),
                                  torch.bincount(flat, minlength=E).cumsum(0)]).to(torch.int32)
        s["expert_of_row"] = flat[s["sorted_src"].long()]
    gather = case["gather"] and E > 1
    s["x"] = _randn((T if gather else R, K), g, torch.bfloat16)
    if not gather:
        s["sorted_src"] = None
    s["w"] = _normal_codes((E, M, K // 2), g)
    # group scales of weights of variance 1/K
    std = 1.0 / (2.2 * math.sqrt(K))
    sf = std * (0.7 + 0.6 * torch.rand((E, M, K // group), generator=g, device=DEV))
    if case["scale"] == "ue8m0":
        sf = torch.floor(torch.log2(sf)).add_(127.0).to(torch.uint8)
    s["w_sf"] = sf
    return s


# ---------------------------------------------------------------- the passes

def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "balance": _plain_balance, "combine": _plain_combine,
            "matvec": _plain_matvec}[state["case"]["op"]](state)


def _run_own(s):
    from moe_routing_precision_gb300 import ops
    c = s["case"]
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            h, n, rp, rn = ops.block_norm(s["residual"], s["y"], post_weight=s["post_weight"],
                                          gate=s["gate"], gate_act=s["act"], scale=s["scale"],
                                          pre_weight=s["pre_weight"], eps=s["eps"],
                                          block_dtype=DTYPES[c["block"]])
            return dict(h=h if s["y"] is not None else None, n=n, rstd_post=rp, rstd_pre=rn)
        gr, gy, gpw, gg, gw = ops.block_norm_backward(
            s["grad_h"], s["grad_n"], s["h"], y=s["y"], post_weight=s["post_weight"],
            gate=s["gate"], gate_act=s["act"], scale=s["scale"], pre_weight=s["pre_weight"],
            rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"])
        return dict(grad_residual=gr, grad_y=gy, grad_post_weight=gpw, grad_gate=gg,
                    grad_pre_weight=gw)
    if c["op"] == "balance":
        kw = dict(score_func=c["func"], seq_offsets=s["seq_offsets"], token_mask=s["token_mask"])
        if c["dir"] == "fwd":
            b, z, counts, probs, tokens = ops.balance_loss(s["scores"], s["topk_idx"], **kw)
            return dict(balance=b, z=z, counts=counts, probs=probs, tokens=tokens)
        return ops.balance_loss_backward(
            s["scores"], s["counts"], s["tokens"], s["grad_balance"], s["grad_z"],
            topk_idx=s["topk_idx"], topk_weights=s["topk_weights"],
            grad_topk_weights=s["grad_topk_weights"], **kw)
    if c["op"] == "combine":
        gy, gw = ops.combine_backward(s["grad_out"], s["y"], s["topk_weights"], s["pos"],
                                      sorted_src=s["sorted_src"])
        return dict(grad_y=gy, grad_topk_weights=gw)
    return ops.expert_matvec_fp4(s["x"], s["w"], s["w_sf"], s["offsets"],
                                 sorted_src=s["sorted_src"], k=c["k"], group=c["group"],
                                 swiglu=c["swiglu"], out_dtype=DTYPES[c["out"]])


def _plain_norm(s):
    c = s["case"]
    gate = None
    if s["gate"] is not None:
        gate = s["gate"].float()
        if s["act"] == "sigmoid":
            gate = 1.0 / (1.0 + torch.exp(-gate))
    rt, yt = DTYPES[c["stream"]], DTYPES[c["block"]]
    if c["dir"] == "fwd":
        h = s["residual"].float()
        rstd_post = rstd_pre = n = None
        if s["y"] is not None:
            z = s["y"].float()
            if c["post"]:
                rstd_post = 1.0 / torch.sqrt((z * z).mean(1) + s["eps"])
                z = z * rstd_post[:, None] * s["post_weight"]
            if gate is not None:
                z = z * gate
            h = h + s["scale"] * z
        if c["pre"]:
            rstd_pre = 1.0 / torch.sqrt((h * h).mean(1) + s["eps"])
            n = (h * rstd_pre[:, None] * s["pre_weight"]).to(yt)
        return dict(h=h.to(rt) if s["y"] is not None else None, n=n, rstd_post=rstd_post,
                    rstd_pre=rstd_pre)
    d = s["grad_h"].float()
    out = dict(grad_residual=None, grad_y=None, grad_post_weight=None, grad_gate=None,
               grad_pre_weight=None)
    if c["pre"]:
        r = s["rstd_pre"][:, None]
        hn = s["h"].float() * r
        gn = s["grad_n"].float()
        out["grad_pre_weight"] = (gn * hn).sum(0)
        u = gn * s["pre_weight"]
        d = d + r * (u - hn * (u * hn).mean(1, keepdim=True))
    out["grad_residual"] = d.to(rt)
    if s["y"] is None:
        return out
    y = s["y"].float()
    yn = y * s["rstd_post"][:, None] if c["post"] else y
    z = yn * s["post_weight"] if c["post"] else yn
    dz = s["scale"] * d
    if gate is not None:
        dg = dz * z
        if c["gate"] == "channel":
            dg = dg.sum(0)
        elif c["gate"] == "token":
            dg = dg.sum(1, keepdim=True)
        if s["act"] == "sigmoid":
            dg = dg * gate * (1.0 - gate)
        out["grad_gate"] = dg.to(s["gate"].dtype)
        dz = dz * gate
    if c["post"]:
        out["grad_post_weight"] = (dz * yn).sum(0)
        u = dz * s["post_weight"]
        dz = s["rstd_post"][:, None] * (u - yn * (u * yn).mean(1, keepdim=True))
    out["grad_y"] = dz.to(yt)
    return out


def _segments(s):
    """Each token's sequence, and whether it counts."""
    T = s["scores"].shape[0]
    seg = torch.bucketize(torch.arange(T, dtype=torch.int32, device=DEV), s["seq_offsets"][1:],
                          right=True)
    keep = s["scores"].max(1).values > -math.inf
    if s["token_mask"] is not None:
        keep = keep & s["token_mask"]
    return seg, keep


def _plain_probs(s):
    x = s["scores"]
    m = x.max(1, keepdim=True).values
    ex = torch.exp(x - m)
    tot = ex.sum(1, keepdim=True)
    lse = (m + torch.log(tot))[:, 0]
    if s["case"]["func"] == "softmax":
        return ex / tot, lse, None
    sg = 1.0 / (1.0 + torch.exp(-x))
    return sg / sg.sum(1, keepdim=True), lse, sg


def _plain_balance(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    seg, keep = _segments(s)
    p, lse, sg = _plain_probs(s)
    if c["dir"] == "fwd":
        p = torch.where(keep[:, None], p, 0.0)
        z = torch.where(keep, lse * lse, 0.0)
        tokens = torch.zeros(S, dtype=torch.int32, device=DEV).index_add_(0, seg,
                                                                         keep.to(torch.int32))
        counts = torch.zeros(S * E, dtype=torch.int32, device=DEV).index_add_(
            0, (seg[:, None] * E + s["topk_idx"]).reshape(-1),
            keep[:, None].expand(T, k).to(torch.int32).reshape(-1)).view(S, E)
        n = tokens.float().clamp(min=1.0)
        probs = torch.zeros((S, E), device=DEV).index_add_(0, seg, p) / n[:, None]
        zs = torch.zeros(S, device=DEV).index_add_(0, seg, z) / n
        bal = (counts.float() * probs).sum(1) * (E / k) / n
        return dict(balance=bal, z=zs, counts=counts, probs=probs, tokens=tokens)
    n = s["tokens"].float().clamp(min=1.0)
    f = s["counts"].float() * (E / k) / n[:, None]
    a = (s["grad_balance"] / n)[:, None] * f
    a = a[seg]
    d = p * (a - (p * a).sum(1, keepdim=True))
    if sg is not None:
        d = d * (1.0 - sg)
        x = s["scores"]
        q = torch.exp(x - lse[:, None])
    else:
        q = p
    d = d + (2.0 * s["grad_z"] / n)[seg][:, None] * lse[:, None] * q
    w, gw = s["topk_weights"], s["grad_topk_weights"]
    d.scatter_add_(1, s["topk_idx"].long(), w * (gw - (w * gw).sum(1, keepdim=True)))
    return torch.where(keep[:, None], d, 0.0)


def _plain_combine(s):
    pos, w = s["pos"], s["topk_weights"]
    T, k = pos.shape
    R, H = s["y"].shape
    go = s["grad_out"].float()
    gy = torch.zeros((R + 1, H), dtype=torch.bfloat16, device=DEV)
    gw = torch.empty((T, k), device=DEV)
    for j in range(k):
        r = pos[:, j].long()
        ok = r >= 0
        yj = s["y"][r.clamp(min=0)].float()
        gw[:, j] = torch.where(ok, (go * yj).sum(1), 0.0)
        gy[torch.where(ok, r, R)] = (w[:, j:j + 1] * go).to(torch.bfloat16)
    return dict(grad_y=gy[:R], grad_topk_weights=gw)


def _scale_values(s, rows, dtype):
    sf = s["w_sf"][rows]
    if sf.dtype == torch.uint8:
        return torch.exp2(sf.to(dtype) - 127.0)
    return sf.to(dtype)


def _plain_matvec(s):
    c = s["case"]
    T, K, N, E, k, group = (c[n] for n in ("T", "K", "N", "E", "k", "group"))
    R, M = T * k, s["w"].shape[1]
    table = torch.tensor(E2M1, device=DEV)
    e = s["expert_of_row"] if E > 1 else torch.zeros(R, dtype=torch.int64, device=DEV)
    src = torch.arange(R, device=DEV) if s["sorted_src"] is None else s["sorted_src"].long() // k
    x = s["x"].float()
    out = torch.empty((R, N), dtype=DTYPES[c["out"]], device=DEV)
    # rows whose dequantised weights together stay within about 2 GB
    step = max(1, (1 << 29) // (M * K)) if E > 1 else R
    for r0 in range(0, R, step):
        rows = e[r0:r0 + step] if E > 1 else e[:1]
        b = s["w"][rows]
        v = torch.stack([table[(b & 15).int()], table[(b >> 4).int()]], -1)
        v = v.view(len(rows), M, K // group, group) * _scale_values(s, rows,
                                                                   torch.float32)[..., None]
        v = v.view(len(rows), M, K)
        xr = x[src[r0:r0 + step]]
        if E > 1:
            o = (v * xr[:, None, :]).sum(2)
        else:
            o = torch.stack([(v[0] * xr[i]).sum(1) for i in range(R)])
        if c["swiglu"]:
            gt, up = o[:, :N], o[:, N:]
            o = gt / (1.0 + torch.exp(-gt)) * up
        out[r0:r0 + step] = o.to(out.dtype)
    return out


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "balance": _exact_balance, "combine": _exact_combine,
            "matvec": _exact_matvec}[case["op"]](s)


def _f64(t):
    return None if t is None else t.double()


def _exact_norm(s):
    c = s["case"]
    H = c["H"]
    gate, dgate = _f64(s["gate"]), None
    if gate is not None and s["act"] == "sigmoid":
        gate = torch.sigmoid(gate)
        dgate = gate * (1 - gate)
    post_w, pre_w = _f64(s["post_weight"]), _f64(s["pre_weight"])
    y = _f64(s["y"])
    if c["dir"] == "fwd":
        out = dict(h=None, n=None, rstd_post=None, rstd_pre=None)
        h = _f64(s["residual"])
        if y is not None:
            b = y
            if c["post"]:
                out["rstd_post"] = (y.pow(2).sum(1) / H + s["eps"]).pow(-0.5)
                b = torch.einsum("th,t,h->th", y, out["rstd_post"], post_w)
            h = h + s["scale"] * (b if gate is None else b * gate)
            out["h"] = h
        if c["pre"]:
            out["rstd_pre"] = (h.pow(2).sum(1) / H + s["eps"]).pow(-0.5)
            out["n"] = torch.einsum("th,t,h->th", h, out["rstd_pre"], pre_w)
        return out
    # gradients of L = <grad_h, h> + <grad_n, n>, term by term
    gh = _f64(s["grad_h"])
    out = dict(grad_residual=None, grad_y=None, grad_post_weight=None, grad_gate=None,
               grad_pre_weight=None)
    if c["pre"]:
        h, gn, r = _f64(s["h"]), _f64(s["grad_n"]), _f64(s["rstd_pre"])
        out["grad_pre_weight"] = torch.einsum("th,th,t->h", gn, h, r)
        dot = torch.einsum("th,th,h->t", gn, h, pre_w)
        gh = gh + torch.einsum("th,h,t->th", gn, pre_w, r) - h * (r.pow(3) * dot / H)[:, None]
    out["grad_residual"] = gh
    if y is None:
        return out
    db = s["scale"] * gh
    r = _f64(s["rstd_post"])
    b = y if r is None else torch.einsum("th,t,h->th", y, r, post_w)
    if gate is not None:
        dg = db * b
        if c["gate"] == "channel":
            dg = dg.sum(0)
        elif c["gate"] == "token":
            dg = dg.sum(1, keepdim=True)
        out["grad_gate"] = dg if dgate is None else dg * dgate
        db = db * gate
    if c["post"]:
        out["grad_post_weight"] = torch.einsum("th,th,t->h", db, y, r)
        dot = torch.einsum("th,th,h->t", db, y, post_w)
        db = torch.einsum("th,h,t->th", db, post_w, r) - y * (r.pow(3) * dot / H)[:, None]
    out["grad_y"] = db
    return out


def _exact_balance(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    x = s["scores"].double()
    keep = torch.isfinite(x.amax(1))
    if s["token_mask"] is not None:
        keep &= s["token_mask"]
    lse = torch.logsumexp(x, 1)
    if c["func"] == "softmax":
        p = torch.softmax(x, 1)
    else:
        p = torch.softmax(torch.nn.functional.logsigmoid(x), 1)
    ends = s["seq_offsets"].tolist()
    if c["dir"] == "fwd":
        bal, zs = torch.zeros(2, S, dtype=torch.float64, device=DEV)
        probs = torch.zeros(S, E, dtype=torch.float64, device=DEV)
        counts = torch.zeros(S, E, dtype=torch.int32, device=DEV)
        tokens = torch.zeros(S, dtype=torch.int32, device=DEV)
        for i in range(S):
            rows = torch.arange(ends[i], ends[i + 1], device=DEV)
            rows = rows[keep[rows]]
            n = rows.numel()
            if n == 0:
                continue
            tokens[i] = n
            counts[i] = torch.bincount(s["topk_idx"][rows].reshape(-1).long(), minlength=E)
            probs[i] = p[rows].mean(0)
            zs[i] = lse[rows].square().mean()
            bal[i] = torch.dot(counts[i].double() * E / (k * n), probs[i])
        return dict(balance=bal, z=zs, counts=counts, probs=probs, tokens=tokens)
    grad = torch.zeros(T, E, dtype=torch.float64, device=DEV)
    for i in range(S):
        lo, hi = ends[i], ends[i + 1]
        n = int(s["tokens"][i])
        if hi == lo or n == 0:
            continue
        f = s["counts"][i].double() * E / (k * n)
        pi, xi = p[lo:hi], x[lo:hi]
        d = pi * (f - pi @ f[:, None]) * (s["grad_balance"][i].double() / n)
        if c["func"] == "sigmoid":
            d = d * torch.sigmoid(-xi)
        soft = torch.softmax(xi, 1)
        grad[lo:hi] = d + soft * lse[lo:hi, None] * (2 * s["grad_z"][i].double() / n)
    w, gw = s["topk_weights"].double(), s["grad_topk_weights"].double()
    grad.scatter_add_(1, s["topk_idx"].long(), w * gw - w * (w * gw).sum(1, keepdim=True))
    grad[~keep] = 0
    return grad


def _exact_combine(s):
    pos, w, y = s["pos"].long(), s["topk_weights"].double(), s["y"]
    go = s["grad_out"].double()
    gy = torch.zeros(y.shape, dtype=torch.float64, device=DEV)
    gw = torch.zeros(pos.shape, dtype=torch.float64, device=DEV)
    for j in range(pos.shape[1]):
        t = (pos[:, j] >= 0).nonzero()[:, 0]
        r = pos[t, j]
        gy[r] = go[t] * w[t, j, None]
        gw[t, j] = torch.einsum("th,th->t", go[t], y[r].double())
    return dict(grad_y=gy, grad_topk_weights=gw)


def _exact_matvec(s):
    c = s["case"]
    T, K, N, E, k, group = (c[n] for n in ("T", "K", "N", "E", "k", "group"))
    R = T * k
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=DEV) / 2
    ends = [0, R] if E == 1 else s["offsets"].tolist()
    out = torch.zeros(R, N, dtype=torch.float64, device=DEV)
    for e in range(E):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        b = s["w"][e].int()
        code = torch.stack((b % 16, b // 16), 2).reshape(b.shape[0], K)
        w = mag[code % 8] * (1 - 2 * (code // 8)).double()
        w = w * _scale_values(s, e, torch.float64).repeat_interleave(group, 1)
        rows = torch.arange(lo, hi, device=DEV)
        if s["sorted_src"] is not None:
            rows = s["sorted_src"][rows].long() // k
        o = s["x"][rows].double() @ w.T
        if c["swiglu"]:
            o = o[:, :N] * torch.sigmoid(o[:, :N]) * o[:, N:]
        out[lo:hi] = o
    return out


# -------------------------------------------------------------------- the work

def work(case):
    """What one pass cannot do without: inputs read once, outputs written once."""
    op = case["op"]
    T = case["T"]
    if op == "norm":
        H = case["H"]
        sr, sb = (2 if case[n] == "bf16" else 4 for n in ("stream", "block"))
        has_y, pre, post = case.get("y", True), case["pre"], case["post"]
        gate = {"none": 0, "channel": 4 * H, "token": 4 * T, "element": sb * T * H}[case["gate"]]
        vec = 4 * H * (int(pre) + int(post)) + 4 * T * (int(pre) + int(post))
        if case["dir"] == "fwd":
            b = T * H * (sr + (sr + sb if has_y else 0) + (sb if pre else 0)) + gate + vec
            return {"bytes": b, "flops": T * H * 10}
        b = T * H * (2 * sr + (sr + sb if pre else 0) + (2 * sb if has_y else 0))
        b += 2 * gate + vec + 4 * H * (int(pre) + int(post))
        return {"bytes": b, "flops": T * H * 25}
    if op == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        mask = T if case["mask"] else 0
        if case["dir"] == "fwd":
            return {"bytes": T * E * 4 + T * k * 4 + mask + S * (8 * E + 16), "flops": T * E * 6}
        return {"bytes": 2 * T * E * 4 + T * k * 12 + mask + S * (4 * E + 16), "flops": T * E * 12}
    if op == "combine":
        H, k = case["H"], case["k"]
        g = 2 if case["grad"] == "bf16" else 4
        R = int(T * k * (1.0 - case["drop"]))
        return {"bytes": T * H * g + 2 * R * H * 2 + T * k * 12, "flops": 3 * R * H}
    K, N, E, k = case["K"], case["N"], case["E"], case["k"]
    M = N * (2 if case["swiglu"] else 1)
    R = T * k
    # experts that T tokens with k distinct experts each are expected to use
    used = E * (1.0 - (1.0 - min(1.0, k / E)) ** T)
    per = M * (K // 2 + (K // case["group"]) * (4 if case["scale"] == "f32" else 1))
    b = used * per + (T if case["gather"] and E > 1 else R) * K * 2 + R * N * (
        2 if case["out"] == "bf16" else 4)
    return {"bytes": int(b), "flops": 2 * R * M * K}
