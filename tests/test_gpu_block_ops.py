"""GPU parity of the operators around the routed experts against 64-bit plain
implementations (tests/block_ref.py, where the tolerances are derived)."""
import math

import pytest
import torch


from moe_routing_precision_gb300 import ops
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_routing_precision_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    assert ops.device_status() == 0
    yield
    assert ops.device_status() == 0


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(shape, g, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def shifted(t, by=1):
    """The same values in a tensor that starts `by` elements past an aligned address."""
    if t is None:
        return None
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------------- norms

def norm_inputs(T, H, sd, bd, gate, seed, y=True, post=True, pre=True):
    g = gen(seed)
    s = dict(residual=randn((T, H), g, sd, 3.0), y=randn((T, H), g, bd) if y else None,
             post_w=1 + randn((H,), g, std=0.2) if post and y else None,
             pre_w=1 + randn((H,), g, std=0.2) if pre else None)
    s["gate"] = {"none": lambda: None, "channel": lambda: randn((H,), g),
                 "token": lambda: randn((T, 1), g),
                 "element": lambda: randn((T, H), g, bd)}[gate if y else "none"]()
    return s


def run_norm(s, act, scale=0.5, eps=1e-6, bd=None, **kw):
    return ops.block_norm(s["residual"], s["y"], post_weight=s["post_w"], gate=s["gate"],
                          gate_act=act, scale=scale, pre_weight=s["pre_w"], eps=eps,
                          block_dtype=bd, **kw)


def check_norm(s, act, got, scale=0.5, eps=1e-6):
    h, n, rp, rn = got
    want = ref.norm_forward(s["residual"], s["y"], s["post_w"], s["gate"], act, scale, s["pre_w"],
                            eps)
    for name, t in (("h", h), ("n", n), ("rstd_post", rp), ("rstd_pre", rn)):
        if name in want:
            ref.check(t, *want[name], name)
        elif name != "h":
            assert t is None


def run_check_backward(s, act, seed, gh_none=False, scale=0.5, eps=1e-6, bd=None, **kw):
    g = gen(seed)
    sd = s["residual"].dtype
    T, H = s["residual"].shape
    h, n, rp, rn = run_norm(s, act, scale, eps, bd)
    gh = None if gh_none else randn((T, H), g, sd)
    gn = None if n is None else randn((T, H), g, n.dtype)
    got = ops.block_norm_backward(gh, gn, h, y=s["y"], post_weight=s["post_w"], gate=s["gate"],
                                  gate_act=act, scale=scale, pre_weight=s["pre_w"], rstd_post=rp,
                                  rstd_pre=rn, **kw)
    want = ref.norm_backward(gh, gn, h, s["y"], s["post_w"], s["gate"], act, scale, s["pre_w"], rp,
                             rn)
    for name, t in zip(("grad_residual", "grad_y", "grad_post_weight", "grad_gate",
                        "grad_pre_weight"), got):
        if name in want:
            ref.check(t, *want[name], name)
        else:
            assert t is None, name
    return got


NORM_SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 8), (2, 1155), (33, 256), (7, 1000), (9, 7168),
               (4, 8200), (2, 16384), (3, 16383), (130, 72), (700, 40)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("sd,bd", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_norm_shapes_and_types(T, H, sd, bd):
    s = norm_inputs(T, H, sd, bd, "channel", T * 31 + H)
    check_norm(s, "sigmoid", run_norm(s, "sigmoid"))
    run_check_backward(s, "sigmoid", H)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("act", ["none", "sigmoid"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T,H", [(37, 520), (19, 333)])
def test_norm_options(gate, act, post, pre, T, H):
    if gate == "none" and act == "sigmoid":
        pytest.skip("no gate to act on")
    s = norm_inputs(T, H, BF, BF, gate, 5, post=post, pre=pre)
    check_norm(s, act, run_norm(s, act, scale=-1.25), scale=-1.25)
    run_check_backward(s, act, 6, scale=-1.25)


@pytest.mark.parametrize("T,H", [(5, 4096), (300, 64), (6, 101)])
@pytest.mark.parametrize("sd", [BF, F32])
def test_norm_alone_before_a_block(T, H, sd):
    s = norm_inputs(T, H, sd, BF, "none", 8, y=False)
    got = run_norm(s, "none")
    assert got[0] is s["residual"] and got[2] is None
    check_norm(s, "none", got)
    run_check_backward(s, "none", 9)
    run_check_backward(s, "none", 9, gh_none=True)
    s32 = dict(s)
    got = run_norm(s32, "none", bd=F32)
    assert got[1].dtype == F32
    check_norm(s32, "none", got)


@pytest.mark.parametrize("H", [512, 513])
def test_norm_in_place_streams_and_unaligned_views(H):
    s = norm_inputs(21, H, F32, BF, "element", 3)
    want = run_norm(s, "sigmoid")
    keep = s["residual"].clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    n = torch.empty_like(want[1])
    got = run_norm(s, "sigmoid", out=(s["residual"], n), stream=st)
    st.synchronize()
    assert got[0] is s["residual"]
    assert torch.equal(got[0], want[0]) and torch.equal(n, want[1])
    s["residual"] = keep
    check_norm(s, "sigmoid", want)
    # tensors that start off any 16-byte boundary
    v = {k: shifted(t) for k, t in s.items()}
    check_norm(v, "sigmoid", run_norm(v, "sigmoid"))
    run_check_backward(v, "sigmoid", 4)


@pytest.mark.parametrize("H", [256, 2048, 2304, 3584, 4096, 4608, 5120, 5632, 6144, 6656, 7168,
                               7680, 8192, 2312, 5128, 7176])
@pytest.mark.parametrize("gate", ["none", "element"])
def test_norm_backward_wide_rows_several_per_block(H, gate):
    for T, sd, bd in ((700, BF, BF), (467, F32, F32), (3, F32, BF), (463, BF, F32)):
        s = norm_inputs(T, H, sd, bd, gate, H)
        run_check_backward(s, "sigmoid" if gate != "none" else "none", T)
    run_check_backward(s, "none", T, gh_none=True)
    run_check_backward(norm_inputs(470, H, F32, BF, gate, H, pre=False), "none", 5)
    run_check_backward(norm_inputs(470, H, F32, BF, gate, H, post=False), "none", 6)


@pytest.mark.parametrize("H", [256, 512, 1024, 2560, 4096, 4608, 5120, 6144, 6656, 7168, 7680, 8192])
@pytest.mark.parametrize("gate", ["token", "element"])
def test_norm_wide_rows_several_per_block(H, gate):
    T = (2 << 20) // H + 701                   # an odd last row for two rows per turn
    T += 1 - T % 2
    for sd, bd in ((BF, BF), (F32, BF), (F32, F32)):
        s = norm_inputs(T, H, sd, bd, gate, H)
        check_norm(s, "sigmoid", run_norm(s, "sigmoid"))
    s = norm_inputs(T, H, BF, BF, gate, H, post=False)
    check_norm(s, "none", run_norm(s, "none"))


def test_norm_zero_rows_and_extremes():
    s = norm_inputs(6, 264, BF, BF, "none", 1)
    s["y"][0] = 0
    s["residual"][0] = 0                     # a row of zeros: rstd = eps^-1/2
    s["y"][1] *= 2.0 ** 40
    s["residual"][2] *= 2.0 ** 50
    s["y"][3] *= 2.0 ** -60                  # below eps: the norm is linear there
    got = run_norm(s, "none")
    check_norm(s, "none", got)
    assert float(got[2][0]) == pytest.approx(1e3, rel=1e-5)
    run_check_backward(s, "none", 2)


def test_norm_backward_is_deterministic_and_zero_tokens():
    s = norm_inputs(501, 1032, F32, BF, "channel", 12)
    a = run_check_backward(s, "sigmoid", 13)
    b = run_check_backward(s, "sigmoid", 13)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    z = norm_inputs(0, 72, F32, BF, "channel", 1)
    h, n, rp, rn = run_norm(z, "none")
    assert h.shape == n.shape == (0, 72)
    gr, gy, gpw, gg, gnw = ops.block_norm_backward(
        h, n, h, y=z["y"], post_weight=z["post_w"], gate=z["gate"], scale=0.5,
        pre_weight=z["pre_w"], rstd_post=rp, rstd_pre=rn)
    assert gr.shape == (0, 72) and not gpw.any() and not gg.any() and not gnw.any()


def test_norm_backward_against_differences():
    """Directional differences of the forward (f32), along random directions
    in every input: the change of L = <A, h> + <B, n>."""
    T, H = 3, 40
    s = norm_inputs(T, H, F32, F32, "element", 21)
    g = gen(22)
    A, B = randn((T, H), g), randn((T, H), g)
    h, n, rp, rn = run_norm(s, "sigmoid")
    gr, gy, gpw, gg, gnw = ops.block_norm_backward(A, B, h, y=s["y"], post_weight=s["post_w"],
                                                   gate=s["gate"], gate_act="sigmoid", scale=0.5,
                                                   pre_weight=s["pre_w"], rstd_post=rp,
                                                   rstd_pre=rn)
    step = 2.0 ** -7
    for name, grad in (("residual", gr), ("y", gy), ("post_w", gpw), ("gate", gg), ("pre_w", gnw)):
        v = randn(tuple(s[name].shape), g)
        L = []
        for sgn in (1, -1):
            p = dict(s)
            p[name] = s[name] + sgn * step * v
            hh, nn, _, _ = run_norm(p, "sigmoid")
            L.append(float((A.double() * hh.double()).sum() + (B.double() * nn.double()).sum()))
        slope = (L[0] - L[1]) / (2 * step)
        want = float((grad.double() * v.double()).sum())
        # central differences: third derivatives of order |L| step^2, and f32
        # rounding of L (about 2^-24 sum |terms|) over the step
        terms = float(A.abs().sum() * h.abs().max() + B.abs().sum() * n.abs().max())
        assert abs(slope - want) <= terms * (step ** 2 * 0.5 + 2.0 ** -22 / step), name


def test_norm_past_32_bit_offsets():
    T, H = 270000, 16000                       # 4.3e9 elements
    x = torch.zeros((T, H), dtype=BF, device=DEV)
    g = gen(2)
    rows = randn((3, H), g, BF)
    x[0], x[T // 2], x[T - 1] = rows[0], rows[1], rows[2]
    w = 1 + randn((H,), g, std=0.2)
    _, n, _, rn = ops.block_norm(x, pre_weight=w)
    pick = torch.tensor([0, T // 2, T - 1], device=DEV)
    want = ref.norm_forward(rows, None, None, None, "none", 1.0, w, 1e-6)
    ref.check(n[pick], *want["n"], "n")
    ref.check(rn[pick], *want["rstd_pre"], "rstd_pre")
    assert not n[1].any() and not n[T - 2].any()


# ------------------------------------------------------------ balance loss

def balance_inputs(T, E, k, S, seed, mask=True, limited=False, levels=False):
    g = gen(seed)
    x = torch.randn(T, E, generator=g) * 2
    if levels:
        x = torch.randint(-2, 3, (T, E), generator=g).float()
    idx = x.topk(k, 1).indices.to(torch.int32) if T else torch.zeros(0, k, dtype=torch.int32)
    if limited:                                   # some experts closed to some tokens
        closed = torch.rand(T, E, generator=g) < 0.4
        closed.scatter_(1, idx.long(), False)
        x[closed] = -math.inf
    m = (torch.rand(T, generator=g) < 0.8) if mask else None
    if m is not None:                             # what is masked may hold anything
        x[~m] = math.nan
        idx[~m] = -7
    cuts = (torch.rand(S - 1, generator=g) * T).long().sort().values
    seq = torch.cat([torch.zeros(1, dtype=torch.long), cuts,
                     torch.tensor([T])]).to(torch.int32)
    return (x.to(DEV), idx.to(DEV), seq.to(DEV), None if m is None else m.to(DEV))


def check_balance(x, idx, func, seq, mask):
    bal, z, counts, probs, tokens = ops.balance_loss(x, idx, score_func=func, seq_offsets=seq,
                                                     token_mask=mask)
    want, wc, wt = ref.balance_forward(x, idx, func, seq, mask)
    assert torch.equal(counts.cpu(), wc) and torch.equal(tokens.cpu(), wt)
    for name, t in (("balance", bal), ("z", z), ("probs", probs)):
        ref.check(t, *want[name], name)
    return counts, tokens


def check_balance_grad(x, idx, func, seq, mask, counts, tokens, seed, selected=True, gb=True,
                       gz=True):
    g = gen(seed)
    T, k = idx.shape
    S = tokens.numel()
    gb = randn((S,), g) if gb else None
    gz = randn((S,), g) if gz else None
    w = gw = None
    if selected:
        w = torch.softmax(randn((T, k), g), 1)
        gw = randn((T, k), g)
        if mask is not None:
            gw[~mask.bool()] = math.nan
    got = ops.balance_loss_backward(x, counts, tokens, gb, gz, score_func=func, seq_offsets=seq,
                                    token_mask=mask, topk_idx=idx, topk_weights=w,
                                    grad_topk_weights=gw)
    d, mag = ref.balance_backward(x, counts, tokens, gb, gz, func, seq, mask, idx, w, gw, k)
    ref.check(got, d, 2 * mag, "grad_scores")


BAL_SHAPES = [(1, 1, 1), (1, 16, 2), (64, 16, 2), (5, 7, 3), (300, 8, 1), (33, 30, 4), (700, 33, 5),
              (40, 64, 6), (257, 100, 8), (1000, 128, 8), (90, 129, 9), (600, 256, 8), (50, 300, 8),
              (70, 511, 7), (21, 513, 32), (33, 1000, 8), (19, 1024, 32), (5000, 24, 2)]


@pytest.mark.parametrize("T,E,k", BAL_SHAPES)
@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
def test_balance_shapes(T, E, k, func):
    for S, mask, limited in ((1, False, False), (5, True, E > k)):
        x, idx, seq, m = balance_inputs(T, E, k, S, T + E, mask, limited)
        c, t = check_balance(x, idx, func, seq, m)
        check_balance_grad(x, idx, func, seq, m, c, t, E)
    c, t = check_balance(x, idx, func, None, m)
    check_balance_grad(x, idx, func, None, m, c, t, E, selected=False)
    check_balance_grad(x, idx, func, None, m, c, t, E, gb=False)
    check_balance_grad(x, idx, func, None, m, c, t, E, gz=False)


@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
def test_balance_many_short_sequences_gaps_and_empty(func):
    T, E, k = 400, 32, 4
    x, idx, _, _ = balance_inputs(T, E, k, 1, 3, mask=False)
    # sequences of length 0, 1 and more; tokens before the first and past the last in none
    ends = [9, 9, 10, 11, 11, 40, 41, 41, 41, 300, 301, 333]
    seq = torch.tensor(ends, dtype=torch.int32, device=DEV)
    c, t = check_balance(x, idx, func, seq, None)
    check_balance_grad(x, idx, func, seq, None, c, t, 4)
    seq = torch.arange(T + 1, dtype=torch.int32, device=DEV)     # one token each
    c, t = check_balance(x, idx, func, seq, None)
    check_balance_grad(x, idx, func, seq, None, c, t, 4)
    # nothing counts: all masked, rows of -inf
    m = torch.zeros(T, dtype=torch.uint8, device=DEV)
    c, t = check_balance(x, idx, func, None, m)
    assert not t.any()
    check_balance_grad(x, idx, func, None, m, c, t, 4)
    x[::3] = -math.inf
    c, t = check_balance(x, idx, func, None, None)
    check_balance_grad(x, idx, func, None, None, c, t, 4)
    x[:] = -math.inf
    c, t = check_balance(x, idx, func, None, None)
    check_balance_grad(x, idx, func, None, None, c, t, 4)


@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-500.0, -60.0, 60.0, 500.0])
def test_balance_scores_far_from_zero(func, shift):
    x, idx, seq, m = balance_inputs(50, 20, 3, 2, 9, mask=False)
    x += shift
    x[7, 3] = torch.finfo(F32).min               # the type's lowest value as a mask
    idx[7] = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    c, t = check_balance(x, idx, func, seq, m)
    check_balance_grad(x, idx, func, seq, m, c, t, 1)


@pytest.mark.parametrize("T,E,S", [(162, 64, 52), (15, 309, 40), (40, 16, 300), (1, 8, 70),
                                   (2048, 8, 130), (2049, 8, 130), (700, 16, 63)])
def test_balance_more_sequences_than_warps(T, E, S):
    x, idx, _, m = balance_inputs(T, E, 3, 1, T + S, mask=True)
    cuts = torch.randint(0, T + 1, (S + 1,), generator=torch.Generator().manual_seed(T))
    cuts, _ = torch.sort(cuts)  # gaps at both ends, empty sequences
    seq = cuts.to(torch.int32).to(DEV)
    for func in ("softmax", "sigmoid"):
        c, t = check_balance(x, idx, func, seq, m)
        check_balance_grad(x, idx, func, seq, m, c, t, S)


def test_balance_determinism_errors_and_views():
    x, idx, seq, m = balance_inputs(3000, 256, 8, 7, 11, mask=False)
    a = ops.balance_loss(x, idx, seq_offsets=seq)
    b = ops.balance_loss(x, idx, seq_offsets=seq)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    xs = shifted(x)
    c, t = check_balance(xs, idx, "softmax", seq, None)
    check_balance_grad(xs, idx, "softmax", seq, None, c, t, 5)
    bad = idx.clone()
    bad[5, 0], bad[6, 1] = 256, -1
    _, _, counts, _, _ = ops.balance_loss(x, bad, seq_offsets=seq)
    assert ops.device_status() == ops.MOE_DEVERR_EXPERT_RANGE
    assert int(counts.sum()) == 3000 * 8 - 2
    z = ops.balance_loss(x[:0], idx[:0], seq_offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
    for p in z:
        assert p.shape[0] == 3 and not p.any()
    assert ops.balance_loss_backward(x[:0], z[2], z[4], k=8,
                                     seq_offsets=torch.zeros(4, dtype=torch.int32,
                                                             device=DEV)).shape == (0, 256)


@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
def test_balance_backward_against_differences(func):
    T, E, k = 6, 10, 2
    x, idx, seq, _ = balance_inputs(T, E, k, 2, 14, mask=False)
    g = gen(15)
    gb, gz = randn((2,), g), randn((2,), g)
    gw = randn((T, k), g)
    pick = idx.long()
    w = torch.softmax(x.gather(1, pick), 1)
    _, _, counts, _, tokens = ops.balance_loss(x, idx, score_func=func, seq_offsets=seq)
    grad = ops.balance_loss_backward(x, counts, tokens, gb, gz, score_func=func, seq_offsets=seq,
                                     topk_idx=idx, topk_weights=w, grad_topk_weights=gw)
    v = randn((T, E), g)
    step, L = 2.0 ** -7, []
    for sgn in (1, -1):
        p = x + sgn * step * v
        bal, z, _, _, _ = ops.balance_loss(p, idx, score_func=func, seq_offsets=seq)
        wp = torch.softmax(p.gather(1, pick).double(), 1)
        L.append(float((gb.double() * bal.double()).sum() + (gz.double() * z.double()).sum()
                       + (gw.double() * wp).sum()))
    slope, want = (L[0] - L[1]) / (2 * step), float((grad.double() * v.double()).sum())
    terms = 40.0 * (1 + float(gb.abs().sum() + gz.abs().sum() + gw.abs().sum()))
    assert abs(slope - want) <= terms * (step ** 2 * 0.5 + 2.0 ** -22 / step)


# -------------------------------------------------------- combine backward

@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (1, 7168, 8), (5, 1000, 2), (33, 256, 9), (17, 4096, 32),
                                   (50, 264, 17), (130, 24, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("padded", [False, True])
def test_combine_backward(T, H, k, dtype, padded):
    g = gen(T + H + k)
    R = T * k + (13 if padded else 0)
    perm = torch.randperm(R, generator=g)[:T * k].to(torch.int32)
    pos = perm.view(T, k).clone()
    if padded:
        pos[torch.rand(T, k, generator=g) < 0.2] = -1
    src = torch.full((R,), -1, dtype=torch.int32)
    live = pos.flatten() >= 0
    src[pos.flatten()[live].long()] = torch.arange(T * k, dtype=torch.int32)[live]
    go, y = randn((T, H), g, dtype), randn((R, H), g, BF)
    w = torch.softmax(randn((T, k), g), 1)
    pos, src = pos.to(DEV), src.to(DEV)
    if padded:                     # rows no copy lands on may hold anything
        y[src < 0] = math.nan
    buf = torch.full((R, H), 7.0, dtype=BF, device=DEV)
    gy, gw = ops.combine_backward(go, y, w, pos, sorted_src=src if padded else None,
                                  out=(buf, torch.empty_like(w)))
    (wy, my, named), (ww, mw) = ref.combine_backward(go, y.nan_to_num(), w, pos)
    ref.check(gy, wy, my, "grad_y")
    ref.check(gw, ww, mw, "grad_topk_weights")
    if padded:
        gy, _ = ops.combine_backward(go, y, w, pos, out=(torch.full_like(buf, 7.0), gw))
        assert bool((gy[~named.to(DEV)] == 7.0).all())
        ref.check(gy[named.to(DEV)], wy[named], my[named], "named rows")


def test_combine_backward_matches_combine_by_differences_and_reports():
    """combine is linear in y and in w, so differences are exact up to rounding."""
    T, H, k = 7, 64, 3
    g = gen(3)
    pos = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k).to(DEV)
    y, w, go = randn((T * k, H), g, BF), torch.softmax(randn((T, k), g), 1), randn((T, H), g)
    gy, gw = ops.combine_backward(go, y, w, pos)
    dy, dw = randn((T * k, H), g, BF), randn((T, k), g)
    base = ops.combine(y, w, pos, F32).double()
    by_w = ((ops.combine(y, w + dw, pos, F32).double() - base) * go.double()).sum()
    want = (gw.double() * dw.double()).sum()
    assert abs(float(by_w - want)) <= 1e-4 * float(go.abs().sum())
    by_y = (ops.combine(dy, w, pos, F32).double() * go.double()).sum()
    want = (gy.double() * dy.double()).sum()
    tol = 2.0 ** -8 * float((gy.abs().double() * dy.abs().double()).sum())
    assert abs(float(by_y - want)) <= tol
    bad = pos.clone()
    bad[2, 1] = T * k
    gy2, gw2 = ops.combine_backward(go, y, w, bad)
    assert ops.device_status() == ops.MOE_DEVERR_POS_RANGE and float(gw2[2, 1]) == 0.0
    e = ops.combine_backward(go[:0], y, w[:0], pos[:0],
                             sorted_src=torch.full((T * k,), -1, dtype=torch.int32, device=DEV))
    assert not e[0].any() and e[1].shape == (0, k)


# ----------------------------------------------------- 4-bit expert products

def weights(E, M, K, group, ue8m0, g):
    w = torch.randint(0, 256, (E, M, K // 2), generator=g).to(torch.uint8).to(DEV)
    if ue8m0:
        sf = torch.randint(110, 130, (E, M, K // group), generator=g).to(torch.uint8).to(DEV)
    else:
        sf = (torch.rand((E, M, K // group), generator=g) * 0.1 + 0.01).to(DEV)
    return w, sf


def check_matvec(x, w, sf, offsets, src, k, group, swiglu, dtype, R):
    M = w.shape[1]
    N = M // 2 if swiglu else M
    buf = torch.full((R, N), 7.0, dtype=dtype, device=DEV)
    got = ops.expert_matvec_fp4(x, w, sf, offsets, sorted_src=src, k=k, group=group,
                                swiglu=swiglu, out_dtype=dtype, out=buf)
    want, mag, written = ref.expert_matvec(x, w, sf, group, offsets, src, k, swiglu, R)
    ref.check(got[written.to(DEV)], want[written], mag[written], "out")
    assert bool((got[~written.to(DEV)] == 7.0).all())


@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K,N,R", [(128, 1, 1), (384, 17, 2), (1152, 40, 5), (2048, 100, 8),
                                   (640, 33, 9), (128, 64, 23)])
def test_matvec_one_expert(group, ue8m0, swiglu, K, N, R):
    g = gen(K + N + R)
    w, sf = weights(1, N * (2 if swiglu else 1), K, group, ue8m0, g)
    x = randn((R, K), g, BF)
    check_matvec(x, w, sf, None, None, 1, group, swiglu, BF if R % 2 else F32, R)


@pytest.mark.parametrize("T,E,k,K,N,group", [(1, 16, 2, 256, 64, 32), (1, 256, 8, 512, 48, 32),
                                             (29, 16, 2, 1056, 101, 16), (64, 8, 4, 224, 33, 32),
                                             (40, 5, 5, 320, 7, 64), (3, 1024, 32, 128, 24, 128),
                                             (16, 64, 8, 7168, 20, 128), (9, 2, 1, 16384, 9, 16),
                                             (3, 2, 1, 16352, 8, 32)])
@pytest.mark.parametrize("gather", [False, True])
def test_matvec_routed(T, E, k, K, N, group, gather):
    g = gen(T + E + K)
    scores = torch.randn(T, E, generator=g)
    if E < 20:
        scores[:, 1] += 5                      # most rows with one expert
        scores[:, 0] -= 50                     # and one expert with none
    idx = scores.topk(k, 1).indices.to(torch.int32).to(DEV)
    _, offsets, pos, src = ops.route_map(idx, E)
    x = randn((T if gather else T * k, K), g, BF)
    w, sf = weights(E, 2 * N, K, group, group == 32, g)
    check_matvec(x, w, sf, offsets, src if gather else None, k, group, True, F32, T * k)
    check_matvec(x, w, sf, offsets, src if gather else None, k, group, False, BF, T * k)


def test_matvec_padded_layout_and_bad_rows():
    T, E, k, K, N, group = 9, 4, 2, 96, 30, 16
    g = gen(4)
    idx = torch.randn(T, E, generator=g).topk(k, 1).indices.to(torch.int32).to(DEV)
    _, offsets, pos, src = ops.route_map_aligned(idx, E, 8)
    x = randn((T, K), g, BF)
    w, sf = weights(E, N, K, group, False, g)
    check_matvec(x, w, sf, offsets, src, k, group, False, F32, src.numel())
    assert ops.device_status() == 0
    far = src.clone()
    far[0] = T * k                             # past the last row of x: a row of zeros
    check_matvec(x, w, sf, offsets, far, k, group, False, F32, src.numel())
    assert ops.device_status() == ops.MOE_DEVERR_POS_RANGE
    over = offsets.clone()
    over[E] = src.numel() + 5                  # past the output: clipped
    check_matvec(x, w, sf, over, src, k, group, False, F32, src.numel())
    assert ops.device_status() == ops.MOE_DEVERR_POS_RANGE
    assert ops.expert_matvec_fp4(x[:0], w, sf, torch.zeros(E + 1, dtype=torch.int32, device=DEV),
                                 group=16).shape == (0, N)


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** -10, 2.0 ** 40])
def test_matvec_wide_range_of_x_and_scales(scale):
    """Rows whose channels span many binades, and rows far from one."""
    K, N, R, group = 512, 20, 3, 32
    g = gen(7)
    x = torch.randn(R, K, generator=g) * torch.pow(2.0, torch.randint(-30, 1, (R, K), generator=g))
    x = (x * scale).to(BF).to(DEV)
    x[1, 128:256] = 0
    w, sf = weights(1, N, K, group, True, g)
    sf[:, ::2] = 40                            # scales of 2^-87 beside ordinary ones
    check_matvec(x, w, sf, None, None, 1, group, False, F32, R)


def test_matvec_of_weights_cast_by_the_framework():
    """Weights from expand_cast_fp4 and activations through the route map:
    every E2M1 code and both scale layouts, as a user would have them."""
    T, E, k, K, N = 6, 4, 2, 256, 24
    g = gen(8)
    dense = randn((E * N, K), g, BF, 0.1)
    rows = torch.arange(E * N, dtype=torch.int32, device=DEV).view(-1, 1)
    idx = torch.randn(T, E, generator=g).topk(k, 1).indices.to(torch.int32).to(DEV)
    _, offsets, pos, src = ops.route_map(idx, E)
    x = randn((T, K), g, BF)
    for flags in (0, ops.SF_POW2 | ops.SF_UE8M0):
        q, sf = ops.expand_cast_fp4(dense, rows, group=32, sf_flags=flags)
        check_matvec(x, q.view(E, N, K // 2), sf.view(E, N, K // 32), offsets, src, k, 32, False,
                     F32, T * k)


def test_matvec_past_32_bit_offsets():
    E, M, K = 200, 4096, 7168                  # 2.9e9 bytes of codes
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    w = torch.randint(0, 256, (E, M, K // 2), generator=g, dtype=torch.uint8, device=DEV)
    sf = torch.full((E, M, K // 32), 120, dtype=torch.uint8, device=DEV)
    x = torch.randn((2, K), generator=g, device=DEV).to(BF)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = 1
    offsets[E] = 2                             # the first and the last expert, one row each
    got = ops.expert_matvec_fp4(x, w, sf, offsets, out_dtype=F32)
    for r, e in ((0, 0), (1, E - 1)):
        want, mag, _ = ref.expert_matvec(x[r:r + 1], w[e:e + 1], sf[e:e + 1], 32, None, None, 1,
                                         False, 1)
        ref.check(got[r:r + 1], want, mag, f"expert {e}")


@pytest.mark.parametrize("T,H", [(512, 8), (700, 40), (5000, 264), (1300, 512), (900, 1024), (601, 4096),
                                 (640, 7168), (513, 8192)])
@pytest.mark.parametrize("sd,bd", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("gate", ["channel", "element"])
def test_norm_many_tokens(T, H, sd, bd, gate):
    """Enough rows that every block of the ring takes several."""
    s = norm_inputs(T, H, sd, bd, gate, T * 31 + H)
    check_norm(s, "sigmoid", run_norm(s, "sigmoid"))
    run_check_backward(s, "sigmoid", H)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
@pytest.mark.parametrize("post,pre,y", [(True, True, True), (True, False, True), (False, True, True),
                                        (False, False, True), (False, True, False)])
@pytest.mark.parametrize("H", [256, 1032])
def test_norm_many_tokens_options(gate, post, pre, y, H):
    s = norm_inputs(1500, H, F32, BF, gate, 5, post=post, pre=pre, y=y)
    act = "sigmoid" if s["gate"] is not None else "none"
    check_norm(s, act, run_norm(s, act, scale=0.75), scale=0.75)
    run_check_backward(s, act, 6, scale=0.75)
    run_check_backward(s, act, 7, gh_none=True, scale=0.75)
    a = run_norm(s, act)
    n = None if a[1] is None else torch.empty_like(a[1])
    if y:
        b = run_norm(s, act, out=(s["residual"], n))          # in place
        assert torch.equal(a[0], b[0]) and (n is None or torch.equal(a[1], n))


@pytest.mark.parametrize("T,H", [(513, 1), (700, 3), (1001, 33), (515, 250), (900, 1155), (640, 2050), (517, 4099),
                                 (514, 7161), (530, 8191)])
@pytest.mark.parametrize("sd,bd", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
def test_norm_many_tokens_of_odd_widths(T, H, sd, bd):
    """Rows that start and end inside 16-byte pieces, the last one included."""
    for gate in ("token", "element"):
        s = norm_inputs(T, H, sd, bd, gate, T * 31 + H)
        check_norm(s, "sigmoid", run_norm(s, "sigmoid"))
        run_check_backward(s, "sigmoid", H)


@pytest.mark.parametrize("T", [1, 2, 3, 151, 153, 305, 511])
@pytest.mark.parametrize("H", [1024, 1027])
def test_norm_backward_of_few_tokens(T, H):
    s = norm_inputs(T, H, F32, BF, "channel", T)
    run_check_backward(s, "sigmoid", T)
