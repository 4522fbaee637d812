"""The router with balance and groups, the row cast to 8-bit integers and the experts'
products in them against plain 64-bit arithmetic (router_int8_ref.py, where the
tolerances are derived)."""
import pytest
import torch

from moe_routing_precision_gb300 import ops
from tests import router_int8_ref as ref
from tests.block_ref import check, cpu64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_routing_precision_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    assert ops.device_status() == 0
    yield
    assert ops.device_status() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ the router

def run_gate(x, k, func="sigmoid", bias=None, G=1, g=None, gs="top2", renorm=True, scale=1.0):
    g = G if g is None else g
    idx, w = ops.router_gate(x.to(DEV), k, score_func=func,
                             bias=None if bias is None else bias.to(DEV), num_groups=G,
                             topk_groups=g, group_score=gs, renormalize=renorm, scale=scale)
    ri, rw = ref.gate(x, k, func, bias, G, g, gs, renorm, scale)
    bad = (idx.cpu().long() != ri).any(1).nonzero().flatten().tolist()
    assert not bad, (len(bad), bad[:3], idx[bad[0]].tolist(), ri[bad[0]].tolist())
    check(w, rw, rw, "weights")
    return idx, w


SHAPES = [  # T, E, k, G, g
    (1, 256, 8, 8, 4), (37, 256, 8, 8, 4), (33, 256, 8, 1, 1), (19, 256, 32, 1, 1),
    (21, 256, 8, 4, 1), (9, 256, 6, 32, 3), (17, 160, 6, 8, 3), (11, 72, 4, 6, 2),
    (13, 16, 2, 1, 1), (13, 16, 4, 16, 5), (7, 1, 1, 1, 1), (5, 33, 3, 11, 2), (6, 128, 8, 8, 3),
    (6, 64, 8, 4, 2), (5, 512, 8, 16, 4), (3, 1024, 32, 32, 32), (4, 1000, 5, 25, 7),
    (3, 384, 8, 1, 1), (5, 20, 20, 2, 2), (3, 1024, 32, 8, 1), (4, 480, 30, 15, 2),
]


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gate(shape, func):
    T, E, k, G, g = shape
    r = gen(E * k + T)
    x = torch.randn(T, E, generator=r)
    b = torch.randn(E, generator=r) * 0.1
    for gs in ("top2", "max"):
        for bias in (None, b):
            for renorm in (True, False):
                run_gate(x, k, func, bias, G, g, gs, renorm, 2.5)


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
def test_gate_ties(func, bias):
    """Equal scores, scores of few values, neighbours in f32: the lower index, or f64."""
    r = gen(7)
    E, k, G, g = 256, 8, 8, 3
    flat = torch.zeros(5, E)
    few = torch.randint(0, 3, (40, E), generator=r).float()
    bits = torch.full((40, E), 1.0) + torch.randint(0, 4, (40, E), generator=r) * 2.0 ** -23
    bf = torch.randn(60, E, generator=r).to(BF).float()
    b = None
    if bias:
        b = torch.randint(0, 4, (E,), generator=r) * 2.0 ** -24 + 0.25
    for x in (flat, few, bits, bf):
        run_gate(x, k, func, b)
        run_gate(x, 32, func, b, G, g, "top2")
        run_gate(x, k, func, b, G, g, "max", False)


def test_gate_saturated_and_small():
    """Sigmoids that f32 rounds to 1 or to 0 still order their experts and share out the
    weights."""
    r = gen(3)
    for shift in (30.0, -60.0, -200.0):
        x = torch.randn(9, 64, generator=r) + shift
        run_gate(x, 6, "sigmoid")
        run_gate(x, 6, "sigmoid", None, 8, 3, "max")
    x = torch.randn(9, 64, generator=r) * 30
    run_gate(x, 6, "softmax")
    run_gate(x, 6, "softmax", torch.randn(64, generator=r) * 0.01, 8, 3, "top2")
    run_gate(x, 6, "sigmoid", torch.randn(64, generator=r) * 0.01, 8, 3, "top2", False)


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
def test_gate_closed_experts(func):
    r = gen(11)
    T, E, k, G, g = 40, 64, 8, 8, 2
    x = torch.randn(T, E, generator=r)
    x[torch.rand(T, E, generator=r) < 0.5] = -INF
    x[0] = -INF                       # nothing is open: the first experts, weights 0
    x[1, :], x[1, 37] = -INF, 0.5     # one expert
    x[2, 8:] = -INF                   # one group
    x[3] = torch.where(torch.arange(E) % 8 == 3, x[3].clamp(min=-2), -INF)  # one per group
    for bias in (None, torch.randn(E, generator=r) * 0.1):
        for gs in ("top2", "max"):
            idx, w = run_gate(x, k, func, bias, G, g, gs)
            assert (w[0] == 0).all() and idx[0].tolist() == list(range(k))
            assert abs(float(w[1].sum()) - 1) < 1e-6
            run_gate(x, k, func, bias, G, g, gs, False)
            run_gate(x, k, func, bias)


def test_gate_many_tokens_and_unaligned_rows():
    r = gen(5)
    x = torch.randn(3001, 256, generator=r)
    b = torch.randn(256, generator=r) * 0.05
    run_gate(x, 8, "sigmoid", b, 8, 4)
    base = torch.empty(3001 * 256 + 1, device=DEV)
    view = base[1:].view(3001, 256)
    view.copy_(x)
    a = ops.router_gate(view, 8, score_func="sigmoid", bias=b.to(DEV), num_groups=8, topk_groups=4)
    c = ops.router_gate(x.to(DEV), 8, score_func="sigmoid", bias=b.to(DEV), num_groups=8,
                        topk_groups=4)
    assert torch.equal(a[0], c[0])
    check(a[1], cpu64(c[1]), cpu64(c[1]), "weights")


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("shape", [(1, 256, 8), (33, 256, 8), (17, 160, 6), (9, 33, 5), (5, 1, 1),
                                   (6, 1024, 32), (7, 18, 18)])
def test_gate_backward(shape, func, renorm):
    T, E, k = shape
    r = gen(T * E)
    x = torch.randn(T, E, generator=r) * 3
    if E > 8:
        x[0, 2:5] = -INF
    idx = torch.rand(T, E, generator=r).argsort(1)[:, :k].to(I32).contiguous()
    gw = torch.randn(T, k, generator=r)
    add = torch.randn(T, E, generator=r) * 0.1
    for a in (None, add):
        want, mag = ref.gate_grad(x, idx, gw, func, renorm, 2.5, a)
        got = ops.router_gate_backward(x.to(DEV), idx.to(DEV), gw.to(DEV), score_func=func,
                                       renormalize=renorm, scale=2.5,
                                       add=None if a is None else a.to(DEV))
        check(got, want, mag, "grad_scores")
    same = add.to(DEV)
    got = ops.router_gate_backward(x.to(DEV), idx.to(DEV), gw.to(DEV), score_func=func,
                                   renormalize=renorm, scale=2.5, add=same, out=same)
    assert got is same
    check(got, want, mag, "in place")


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_backward_against_differences(func, renorm):
    """The weights' derivative by central differences of the 64-bit formula."""
    r = gen(2)
    T, E, k = 3, 12, 4
    x = torch.randn(T, E, generator=r)
    idx, _ = ops.router_gate(x.to(DEV), k, score_func=func, renormalize=renorm, scale=1.5)
    gw = torch.randn(T, k, generator=r)
    got = cpu64(ops.router_gate_backward(x.to(DEV), idx, gw.to(DEV), score_func=func,
                                         renormalize=renorm, scale=1.5))
    h = 1e-4
    for e in range(E):
        d = torch.zeros(E, dtype=torch.float64)
        d[e] = h
        f = [(ref.weights(x.double() + s * d, idx.cpu().long(), func, renorm, 1.5)
              * gw.double()).sum(1) for s in (1, -1)]
        # the difference's own error: h^2 / 6 of a third derivative below 10
        assert torch.allclose(got[:, e], (f[0] - f[1]) / (2 * h), rtol=0, atol=1e-6)


def test_gate_backward_reports_bad_indices():
    x = torch.randn(3, 16, device=DEV)
    idx = torch.tensor([[0, 1], [16, 2], [3, -1]], dtype=I32, device=DEV)
    gw = torch.randn(3, 2, device=DEV)
    got = ops.router_gate_backward(x, idx, gw, score_func="sigmoid")
    assert ops.device_status() == ops.MOE_DEVERR_EXPERT_RANGE
    want, mag = ref.gate_grad(x, idx, gw, "sigmoid", True, 1.0, None)
    check(got, want, mag, "grad_scores")


# -------------------------------------------------------------------- the cast

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 8), (2, 250), (9, 256), (4, 264), (3, 1024),
                                 (2, 1155), (3, 2056), (5, 4096), (3, 7168), (2, 7161),
                                 (2, 8200), (2, 16384), (1, 20008), (2, 16385), (700, 64)])
def test_cast(T, H, dtype):
    r = gen(T + H)
    x = (torch.randn(T, H, generator=r) * torch.randn(T, 1, generator=r).exp()).to(dtype)
    q, sf = ops.cast_int8(x.to(DEV))
    rq, rs = ref.cast(x)
    assert torch.equal(sf.cpu(), rs) and torch.equal(q.cpu(), rq)


def test_cast_corners():
    """Zero rows, the smallest and largest magnitudes, exact halves, one nonzero value."""
    H = 64
    x = torch.zeros(8, H)
    x[1, 5] = 1e-38
    x[2, :2] = torch.tensor([3e38, -1.5e38])
    x[3] = torch.arange(H) - 31.5
    x[3, 0] = 127.0
    x[4, 63] = -2.0 ** -90
    x[5] = 2.0 ** -100
    x[6] = torch.linspace(-1, 1, H)
    x[7, :] = -127.0
    x[7, 1:] = torch.arange(H - 1) + 0.5
    for dt in (F32, BF):
        q, sf = ops.cast_int8(x.to(dt).to(DEV))
        rq, rs = ref.cast(x.to(dt))
        assert torch.equal(sf.cpu(), rs) and torch.equal(q.cpu(), rq)
    assert (q[0] == 0).all() and sf[0] > 0


def test_cast_views_and_outputs():
    """Addresses that rule out wide accesses; out= is written and nothing beside it."""
    r = gen(1)
    base = torch.randn(3 * 256 + 1, generator=r).to(BF).to(DEV)
    x = base[1:].view(3, 256)
    rq, rs = ref.cast(x)
    buf = torch.full((3 * 256 + 64,), 77, dtype=torch.int8, device=DEV)
    for off in (0, 3, 8, 16):
        buf.fill_(77)
        for src in (x, x.clone()):
            q, sf = ops.cast_int8(src, out=buf[off:off + 768].view(3, 256))
            assert torch.equal(q.cpu(), rq) and torch.equal(sf.cpu(), rs)
        assert (buf[:off] == 77).all() and (buf[off + 768:] == 77).all()


# --------------------------------------------------------------- the products

def problem(T, E, k, K, M, seed, *, align=1, gather=True, skew=False, lim=127, absent=0.0):
    r = gen(seed)
    s = torch.rand(T, E, generator=r)
    if skew:
        s[:, : max(1, min(k, E))] += 1
    flat = s.argsort(1, descending=True)[:, :k].reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    order = flat.argsort(stable=True)
    padded = (counts + align - 1) // align * align
    off = torch.cat([torch.zeros(1, dtype=torch.int64), padded.cumsum(0)])
    R = int(off[-1])
    src = torch.full((R,), -1, dtype=I32)
    first = counts.cumsum(0) - counts
    e = flat[order]
    src[off[:-1][e] + torch.arange(T * k) - first[e]] = order.to(I32)
    if absent:
        src[torch.rand(R, generator=r) < absent] = -1
    X = T if gather else R
    x = torch.randint(-lim, lim + 1, (X, K), generator=r, dtype=torch.int32).to(torch.int8)
    w = torch.randint(-lim, lim + 1, (E, M, K), generator=r, dtype=torch.int32).to(torch.int8)
    xs = torch.rand(X, generator=r) * 0.02 + 0.01
    ws = (torch.rand(E, M, generator=r) + 0.5) / (lim * K ** 0.5)
    return x, xs, w, ws, off.to(I32), (src if gather else None)


def run_matmul(x, xs, w, ws, off, src, k, swiglu, out_dtype, out=None):
    put = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    got = ops.expert_matmul_int8(put(x), put(xs), put(w), put(ws), put(off), sorted_src=put(src),
                                 k=k, swiglu=swiglu, out_dtype=out_dtype, out=out)
    want, mag, largest = ref.matmul(x, xs, w, ws, off, src, k, swiglu)
    assert largest < 2 ** 24      # the sums are exact: see the reference's tolerances
    written = ~want.isnan()
    check(got.cpu()[written], want[written], mag[written] / 8, "products")
    return got, written


CASES = [  # T, E, k, K, N, swiglu
    (1, 8, 2, 64, 32, False), (1, 1, 1, 16, 1, False), (1, 256, 8, 512, 64, True),
    (5, 4, 2, 48, 7, False), (5, 4, 2, 48, 7, True), (64, 16, 2, 256, 130, False),
    (33, 3, 2, 1040, 257, True), (300, 2, 1, 144, 300, False), (700, 2, 2, 128, 65, True),
    (129, 1, 1, 2048, 128, False), (40, 16, 4, 1024, 256, True), (257, 5, 3, 80, 129, False),
    (2, 2, 1, 7168, 40, True), (9, 64, 6, 272, 96, False), (1000, 7, 1, 32, 24, True),
    (150, 4, 4, 400, 384, False), (17, 1, 1, 4096, 520, True),
]


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("case", CASES)
def test_matmul(case, out_dtype):
    T, E, k, K, N, sw = case
    lim = 127 if K <= 1024 else 40
    p = problem(T, E, k, K, N * (2 if sw else 1), T + K, lim=lim)
    run_matmul(*p, k, sw, out_dtype)


@pytest.mark.parametrize("case", CASES[2:10])
def test_matmul_rows_in_place(case):
    T, E, k, K, N, sw = case
    p = problem(T, E, k, K, N * (2 if sw else 1), T + K + 1, gather=False, lim=40)
    run_matmul(*p, 1, sw, BF)


@pytest.mark.parametrize("align", [16, 128])
def test_matmul_padded(align):
    """Padding rows and dropped copies are zero rows; empty experts leave nothing."""
    for sw in (False, True):
        p = problem(70, 9, 2, 192, 88, 5, align=align, skew=True, absent=0.1)
        got, _ = run_matmul(*p, 2, sw, F32)
        assert (got[(p[5] < 0).to(DEV)] == 0).all()


def test_matmul_rows_behind_the_last_expert():
    x, xs, w, ws, off, src = problem(20, 4, 2, 64, 48, 6)
    src = torch.cat([src, torch.full((30,), 5, dtype=I32)])
    out = torch.full((70 + 3, 48), 7.0, device=DEV)
    run_matmul(x, xs, w, ws, off, src, 2, False, F32, out=out[:70])
    assert (out[40:] == 7).all()


def test_matmul_one_matrix_without_offsets():
    x, xs, w, ws, _, _ = problem(77, 1, 1, 320, 200, 8)
    for sw in (False, True):
        run_matmul(x, xs, w, ws, None, None, 1, sw, BF)
    run_matmul(x, xs, w, ws, torch.tensor([0, 77], dtype=I32),
               torch.arange(77, dtype=I32).flip(0), 1, False, BF)


def test_matmul_extreme_integers():
    """-128 and 127 everywhere: partial sums reach 2^24 in 1024 channels, exactly."""
    for K in (1024, 1008):
        x = torch.full((20, K), -128, dtype=torch.int8)
        x[1::2] = 127
        x[3, ::2] = -128
        w = torch.full((1, 130, K), -128, dtype=torch.int8)
        w[0, 1::3] = 127
        w[0, 5, ::2] = 1
        ones, wo = torch.ones(20), torch.ones(1, 130)
        got = ops.expert_matmul_int8(x.to(DEV), ones.to(DEV), w.to(DEV), wo.to(DEV),
                                     out_dtype=F32)
        assert torch.equal(cpu64(got), x.double() @ w[0].double().T)


def test_matmul_long_sums_of_one_sign():
    """Sums far past 2^24: a sum of f32 in K / 16 steps, each off by an ulp at most."""
    K = 7168
    x = torch.randint(100, 128, (9, K), generator=gen(1), dtype=torch.int32).to(torch.int8)
    w = torch.randint(100, 128, (1, 140, K), generator=gen(2), dtype=torch.int32).to(torch.int8)
    got = ops.expert_matmul_int8(x.to(DEV), torch.ones(9, device=DEV), w.to(DEV),
                                 torch.ones(1, 140, device=DEV), out_dtype=F32)
    want = x.double() @ w[0].double().T
    assert ((cpu64(got) - want).abs() <= want * (K / 16 + 4) * 2.0 ** -23).all()


def test_matmul_reports_bad_rows():
    x, xs, w, ws, off, src = problem(20, 4, 2, 64, 48, 9)
    bad = src.clone()
    bad[[3, 17]] = 40 * 2          # token 40 of 20
    got = ops.expert_matmul_int8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), off.to(DEV),
                                 sorted_src=bad.to(DEV), k=2, out_dtype=F32)
    assert ops.device_status() == ops.MOE_DEVERR_POS_RANGE
    want, mag, _ = ref.matmul(x, xs, w, ws, off, bad, 2, False)
    check(got, want, mag / 8, "products")
    assert (got[3] == 0).all() and (got[17] == 0).all()
    far = off.clone()
    far[4] = 60                    # beyond the 40 rows
    got = ops.expert_matmul_int8(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), far.to(DEV),
                                 sorted_src=src.to(DEV), k=2, out_dtype=F32)
    assert ops.device_status() == ops.MOE_DEVERR_POS_RANGE
    want, mag, _ = ref.matmul(x, xs, w, ws, off, src, 2, False)
    check(got, want, mag / 8, "products")


def test_matmul_nothing_to_do():
    e = torch.empty(0, 64, dtype=torch.int8, device=DEV)
    w = torch.zeros(4, 8, 64, dtype=torch.int8, device=DEV)
    out = ops.expert_matmul_int8(e, torch.empty(0, device=DEV), w, torch.ones(4, 8, device=DEV),
                                 torch.zeros(5, dtype=I32, device=DEV))
    assert out.shape == (0, 8)
    # rows, but none of any expert
    x = torch.ones(6, 64, dtype=torch.int8, device=DEV)
    out = torch.full((6, 8), 3.0, device=DEV)
    ops.expert_matmul_int8(x, torch.ones(6, device=DEV), w, torch.ones(4, 8, device=DEV),
                           torch.zeros(5, dtype=I32, device=DEV), out_dtype=F32, out=out)
    assert (out == 3).all()
