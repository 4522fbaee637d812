"""The operators around the routed experts where f32's range ends, where a row holds
a NaN, and where sizes or addresses select another form: against the 64-bit
references of tests/block_ref.py, with the tolerances derived there."""
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


def at_bytes(t, by):
    """The same values in a tensor that starts `by` bytes past an aligned address."""
    if t is None:
        return None
    n = by // t.element_size()
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    v = buf[n:].view(t.shape)
    v.copy_(t)
    return v


# ------------------------------------------------------------ score gradient

@pytest.mark.parametrize("top", [46.0, 50.0, 52.0, 56.0, 60.0])
@pytest.mark.parametrize("E", [16, 17, 256])
def test_sigmoid_gradient_of_saturated_scores(top, E):
    """The balance loss alone: p (a - sum p a) (1 - sigmoid), where 1 - sigmoid is e^-x."""
    T, k = 40, 2
    x = torch.randn(T, E, generator=gen(E))
    x = (x - x.max(1, keepdim=True).values + top).to(DEV)
    idx = x.topk(k, 1).indices.to(torch.int32)
    _, _, counts, _, tokens = ops.balance_loss(x, idx, score_func="sigmoid")
    gb = torch.full((1,), 100.0, device=DEV)
    got = ops.balance_loss_backward(x, counts, tokens, gb, k=k, score_func="sigmoid")
    d, mag = ref.balance_backward(x, counts, tokens, gb, None, "sigmoid", None, None, None, None,
                                  None, k)
    ref.check(got, d, 2 * mag, "grad_scores")


@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(16, 2), (37, 3), (256, 8)])
@pytest.mark.parametrize("top", [66.0, 70.0, 75.0, 79.0, 80.0])
def test_score_gradient_of_large_scores(func, E, k, top):
    """Coefficients from tiny (small losses over many tokens) to large (a loss scale)."""
    T = 24
    x = torch.randn(T, E, generator=gen(E))
    x = (x - x.max(1, keepdim=True).values + top).to(DEV)
    for n, scale in ((65536, 1e-8), (65536, 1e-4), (65536, 1.0), (1, 1.0), (1, 65536.0)):
        counts = torch.randint(0, 2 * n * k // E + 2, (1, E), generator=gen(3)).to(torch.int32)
        counts, tokens = counts.to(DEV), torch.full((1,), n, dtype=torch.int32, device=DEV)
        g = torch.full((1,), scale, device=DEV)
        for gb, gz in ((g, None), (None, g), (g, g)):
            got = ops.balance_loss_backward(x, counts, tokens, gb, gz, k=k, score_func=func)
            d, mag = ref.balance_backward(x, counts, tokens, gb, gz, func, None, None, None, None,
                                          None, k)
            ref.check(got, d, 2 * mag, f"grad_scores, n = {n}, upstream {scale}")


# ------------------------------------------------------------------ NaN rows

@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(96, 16), (60, 24), (50, 64), (40, 256), (30, 300), (2500, 24)])
@pytest.mark.parametrize("far", [False, True])
def test_a_row_with_a_nan_does_not_count(func, T, E, far):
    """Alone, beside -inf, beside ordinary scores, and beside rows far from zero; the
    other rows are as without it."""
    g, k = gen(T + E), 3
    x = torch.randn(T, E, generator=g)
    idx = x.topk(k, 1).indices.to(torch.int32).to(DEV)
    if far:
        x[::5] += 300.0
    keep = torch.ones(T, dtype=torch.bool)
    for i, t in enumerate(range(1, T, 7)):
        keep[t] = False
        if i % 3 == 0:
            x[t] = math.nan
        elif i % 3 == 1:
            x[t, :] = -math.inf
            x[t, i % E] = math.nan
        else:
            x[t, (5 * i) % E] = math.nan
    x = x.to(DEV)
    seq = torch.tensor([0, T // 3, T], dtype=torch.int32, device=DEV)
    bal, z, counts, probs, tokens = ops.balance_loss(x, idx, score_func=func, seq_offsets=seq)
    want, wc, wt = ref.balance_forward(x, idx, func, seq, keep)
    assert torch.equal(counts.cpu(), wc) and torch.equal(tokens.cpu(), wt)
    for name, t in (("balance", bal), ("z", z), ("probs", probs)):
        ref.check(t, *want[name], name)
    gb, gz = randn((2,), g), randn((2,), g)
    w, gw = torch.softmax(randn((T, k), g), 1), randn((T, k), g)
    got = ops.balance_loss_backward(x, counts, tokens, gb, gz, score_func=func, seq_offsets=seq,
                                    topk_idx=idx, topk_weights=w, grad_topk_weights=gw)
    d, mag = ref.balance_backward(x, counts, tokens, gb, gz, func, seq, keep, idx, w, gw, k)
    ref.check(got, d, 2 * mag, "grad_scores")
    assert not got[~keep.to(DEV)].any()


# ------------------------------------------------- log of sums that are near one

@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [1, 16, 64, 256, 300])
@pytest.mark.parametrize("many", [False, True])
def test_z_of_rows_with_one_open_expert(func, E, many):
    """log sum exp is that score exactly, however small: each output is off by no more
    than the bound relative to itself."""
    small = [1e-3, -2e-3, 0.1, -0.3, 1e-5, 0.6, -0.69, 3.0, 0.0, 7e-7]
    T = len(small)
    x = torch.full((T, E), -math.inf)
    at = torch.arange(T) * 7 % E
    x[torch.arange(T), at] = torch.tensor(small)
    if many:                      # more scores than the form with a block per sequence takes
        pad = torch.randn(40000 // E, E, generator=gen(1))
        x = torch.cat([x, pad])
    idx = torch.zeros((x.shape[0], 1), dtype=torch.int32, device=DEV)
    seq = torch.arange(T + 1, dtype=torch.int32, device=DEV)       # a sequence per token
    v = torch.tensor(small, dtype=F32).double()
    x = x.to(DEV)
    _, z, counts, _, tokens = ops.balance_loss(x, idx, score_func=func, seq_offsets=seq)
    ref.check(z, v.square(), 2 * v.square(), "z")
    got = ops.balance_loss_backward(x, counts, tokens, None, torch.ones(T, device=DEV), k=1,
                                    score_func=func, seq_offsets=seq)
    ref.check(got[torch.arange(T), at.to(DEV)], 2 * v, 2 * v.abs(), "grad_scores")


# --------------------------------------------------- forms chosen by the sizes

@pytest.mark.parametrize("E,T", [(1, 16384), (1, 500), (3, 5461), (5, 700), (17, 963), (33, 496),
                                 (16, 1024), (16, 1025), (64, 256), (24, 300)])
@pytest.mark.parametrize("func", ["softmax", "sigmoid"])
def test_balance_of_narrow_and_odd_rows(E, T, func):
    """Sizes on both sides of the limits of one block per sequence, 16-byte aligned rows
    and not, with as much workspace as the library names."""
    g, k = gen(E + T), min(2, E)
    x = randn((T, E), g)
    idx = x.topk(k, 1).indices.to(torch.int32)
    need = ops.balance_loss_workspace_bytes(T, E, 3)
    seq = torch.tensor([0, T // 4, T // 4, T], dtype=torch.int32, device=DEV)
    for xs in (x, at_bytes(x, 4)):
        guard = torch.full((need + 512,), 77, dtype=torch.uint8, device=DEV)
        bal, z, counts, probs, tokens = ops.balance_loss(xs, idx, score_func=func,
                                                         seq_offsets=seq,
                                                         workspace=guard[:need] if need else None)
        assert bool((guard[need:] == 77).all())
        want, wc, wt = ref.balance_forward(x, idx, func, seq, None)
        assert torch.equal(counts.cpu(), wc) and torch.equal(tokens.cpu(), wt)
        for name, t in (("balance", bal), ("z", z), ("probs", probs)):
            ref.check(t, *want[name], name)


# ---------------------------------------------------------- norms out of range

@pytest.mark.parametrize("T,H", [(6, 264), (5, 33), (4, 9000), (1100, 4096), (2100, 1001)])
@pytest.mark.parametrize("sd", [BF, F32])
def test_norm_of_rows_whose_squares_overflow(T, H, sd):
    """A sum of squares past f32's range has the inverse root 0, as 1/sqrt gives it."""
    g = gen(H)
    r, y = randn((T, H), g, sd), randn((T, H), g, BF)
    r0, y0 = r.clone(), y.clone()
    r[1] *= 2.0 ** 70
    y[3] *= 2.0 ** 70
    w = 1 + randn((H,), g, std=0.2)
    h, n, rp, rn = ops.block_norm(r, y, post_weight=w, pre_weight=w, scale=0.5)
    assert float(rp[3]) == 0.0 and float(rn[1]) == 0.0
    assert torch.equal(h[3], r[3]) and not n[1].any() and bool(torch.isfinite(h[1]).all())
    want = ref.norm_forward(r0, y0, w, None, "none", 0.5, w, 1e-6)
    rest = torch.ones(T, dtype=torch.bool)
    rest[1] = rest[3] = False
    ref.check(n[rest.to(DEV)], want["n"][0][rest], want["n"][1][rest], "n")
    gr, gy, _, _, _ = ops.block_norm_backward(r0, y0, h, y=y, post_weight=w, scale=0.5,
                                              pre_weight=w, rstd_post=rp, rstd_pre=rn)
    assert torch.equal(gr[1], r0[1])              # the norm of that row is constant: 0
    assert not gy[3].any()


@pytest.mark.parametrize("T,H", [(8, 264), (7, 33), (5, 9000), (700, 4096), (600, 1155)])
@pytest.mark.parametrize("bd", [BF, F32])
@pytest.mark.parametrize("eps", [1e-6, 1e-30])
def test_norm_backward_of_large_and_tiny_rows(T, H, bd, eps):
    """Rows whose inverse norm cubed leaves f32's range, with no other gradient that
    would hide the terms: rows of 2^45 to 2^60, and (eps = 1e-30) rows of zeros."""
    g = gen(T + H)
    r, y = randn((T, H), g), randn((T, H), g, bd)
    for i, e in enumerate((45, 50, 60)):
        r[i] *= 2.0 ** e
    y[3] *= 2.0 ** 48
    y[4] *= 2.0 ** 60
    if eps < 1e-20:
        r[2] = 0
        y[2] = 0
        y[0] = 0
    w, v = 1 + randn((H,), g, std=0.2), 1 + randn((H,), g, std=0.2)
    # the post-norm's rows are of order one: h is as large as r
    h, n, rp, rn = ops.block_norm(r, y, post_weight=w, pre_weight=v, scale=0.5, eps=eps)
    gn = randn((T, H), g, bd)
    got = ops.block_norm_backward(None, gn, h, y=y, post_weight=w, scale=0.5, pre_weight=v,
                                  rstd_post=rp, rstd_pre=rn)
    want = ref.norm_backward(None, gn, h, y, w, None, "none", 0.5, v, rp, rn)
    for name, t in zip(("grad_residual", "grad_y", "grad_post_weight"), got[:3]):
        val, mag = want[name]
        if t.dim() == 1:
            ref.check(t, val, mag, name)
            continue
        # row by row, so that no row hides behind another's size; those below 1e-30 are
        # compared times 2^60
        s = torch.where(val.abs().max(1, keepdim=True).values < 1e-12, 2.0 ** 60, 1.0).double()
        if t.dtype == BF:
            s = torch.ones_like(s)
        ref.check((t.double() * s.to(DEV)).to(F32 if t.dtype == F32 else BF), val * s, mag * s, name)


@pytest.mark.parametrize("T,H", [(9, 512), (1500, 512), (700, 4096), (560, 7168), (4100, 520)])
@pytest.mark.parametrize("sd,bd", [(BF, BF), (F32, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("by", [16, 48])
def test_norm_of_views_at_16_bytes(T, H, sd, bd, by):
    """Tensors that start at an odd multiple of 16 bytes, below and at sizes that take
    the ring of staged rows."""
    g = gen(T + H)
    r, y, gate = randn((T, H), g, sd, 3.0), randn((T, H), g, bd), randn((T, H), g, bd)
    w, v = 1 + randn((H,), g, std=0.2), 1 + randn((H,), g, std=0.2)
    r, y, gate, w, v = (at_bytes(t, by) for t in (r, y, gate, w, v))
    out = (at_bytes(torch.empty_like(r), by), at_bytes(torch.empty_like(y), by))
    got = ops.block_norm(r, y, post_weight=w, gate=gate, gate_act="sigmoid", scale=0.5,
                         pre_weight=v, out=out)
    want = ref.norm_forward(r, y, w, gate, "sigmoid", 0.5, v, 1e-6)
    for name, t in zip(("h", "n", "rstd_post", "rstd_pre"), got):
        ref.check(t, *want[name], name)
    h = got[0]
    gh, gn = at_bytes(randn((T, H), g, sd), by), at_bytes(randn((T, H), g, bd), by)
    grads = ops.block_norm_backward(gh, gn, h, y=y, post_weight=w, gate=gate, gate_act="sigmoid",
                                    scale=0.5, pre_weight=v, rstd_post=got[2], rstd_pre=got[3])
    want = ref.norm_backward(gh, gn, h, y, w, gate, "sigmoid", 0.5, v, got[2], got[3])
    for name, t in zip(("grad_residual", "grad_y", "grad_post_weight", "grad_gate",
                        "grad_pre_weight"), grads):
        ref.check(t, *want[name], name)


def test_inverse_root_and_sigmoid_to_a_few_ulp():
    """rstd of rows of one channel is 1 / sqrt(y^2 + eps); h of a token-gated row of ones
    on zeros is the sigmoid.  The root's argument has two roundings (each half an ulp of
    it, a quarter of the result), the inverse root at most 2 ulp: 2.5 ulp of 2^-23.  The
    sigmoid: e^-|x| 2 ulp, the sum and the reciprocal 1.5, the product 0.5: 4 ulp."""
    T = 20000
    e = torch.rand(T, generator=gen(1)) * 100 - 50
    y = torch.pow(2.0, e)[:, None].to(DEV)
    _, _, rp, _ = ops.block_norm(torch.zeros_like(y), y, post_weight=torch.ones(1, device=DEV),
                                 eps=1e-38)
    want = (y.cpu().double()[:, 0].square() + 1e-38).rsqrt()
    assert bool(((rp.cpu().double() - want).abs() <= 2.5 * 2.0 ** -23 * want).all())
    x = (torch.randn(T, generator=gen(2)) * 20).clamp(-80, 80)[:, None].to(DEV)
    one = torch.ones(T, 1, device=DEV)
    h, _, _, _ = ops.block_norm(torch.zeros_like(one), one, gate=x, gate_act="sigmoid")
    want = torch.sigmoid(x.cpu().double())
    assert bool(((h.cpu().double() - want).abs() <= 4 * 2.0 ** -23 * want).all())


# ------------------------------------------------------- 4-bit expert products

@pytest.mark.parametrize("group", [16, 32, 64, 128])
@pytest.mark.parametrize("K", [128, 384, 640, 1152])
def test_matvec_rows_beside_a_row_without_scales(K, group):
    """UE8M0 scales of 255 (NaN) in one weight row reach that row's output alone."""
    g, N, R = gen(K + group), 40, 3
    w = torch.randint(0, 256, (2, N, K // 2), generator=g).to(torch.uint8).to(DEV)
    sf = torch.randint(110, 130, (2, N, K // group), generator=g).to(torch.uint8).to(DEV)
    x = randn((2 * R, K), g, BF)
    offsets = torch.tensor([0, R, 2 * R], dtype=torch.int32, device=DEV)
    for n in (0, 9, N - 1):
        s = sf.clone()
        s[:, n] = 255
        got = ops.expert_matvec_fp4(x, w, s, offsets, group=group, out_dtype=F32)
        want, mag, _ = ref.expert_matvec(x, w, sf, group, offsets, None, 1, False, 2 * R)
        rest = torch.arange(N) != n
        ref.check(got[:, rest.to(DEV)], want[:, rest], mag[:, rest], f"row {n} without scales")
