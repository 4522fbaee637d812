"""The router with balance and groups and the 8-bit experts as a program uses them: a whole
block, its router's gradient with the balance losses' against autograd in 64 bits, captured
graphs, other streams, guarded outputs, weights that come cold from memory, and the
debug-bounds library.  Tolerances: router_int8_ref.py and block_ref.py."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from moe_routing_precision_gb300 import _build, ops
from tests import router_int8_ref as ref
from tests.block_ref import check, cpu64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    torch.cuda.set_device(0)
    assert ops.device_status() == 0
    yield
    assert ops.device_status() == 0


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("moe_block",
                                                  os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["moe_block"] = m      # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def block(T, E, k, H, N, seed, G=1, g=1):
    """A block's inputs: logits, rows, experts already in 8 bits."""
    r = gen(seed)
    scores = torch.randn(T, E, generator=r).to(DEV)
    bias = (torch.randn(E, generator=r) * 0.05).to(DEV)
    x = torch.randn(T, H, generator=r).to(BF).to(DEV)
    up, up_sf = ops.cast_int8((torch.randn(E * 2 * N, H, generator=r) * H ** -0.5).to(DEV))
    down, down_sf = ops.cast_int8((torch.randn(E * H, N, generator=r) * N ** -0.5).to(DEV))
    return dict(scores=scores, bias=bias, x=x, up=up.view(E, 2 * N, H), up_sf=up_sf.view(E, 2 * N),
                down=down.view(E, H, N), down_sf=down_sf.view(E, H), k=k, G=G, g=g)


def run_block(b):
    idx, w = ops.router_gate(b["scores"], b["k"], score_func="sigmoid", bias=b["bias"],
                             num_groups=b["G"], topk_groups=b["g"], scale=2.5)
    _, offsets, pos, src = ops.route_map(idx, b["scores"].shape[1])
    xq, xs = ops.cast_int8(b["x"])
    act = ops.expert_matmul_int8(xq, xs, b["up"], b["up_sf"], offsets, sorted_src=src, k=b["k"],
                                 swiglu=True)
    aq, as_ = ops.cast_int8(act)
    y_e = ops.expert_matmul_int8(aq, as_, b["down"], b["down_sf"], offsets)
    out = ops.combine(y_e, w, pos, F32)
    return dict(idx=idx, w=w, offsets=offsets, pos=pos, src=src, xq=xq, xs=xs, act=act, aq=aq,
                as_=as_, y_e=y_e, out=out)


@pytest.mark.parametrize("T,E,k,H,N,G,g", [(1, 16, 4, 256, 96, 4, 2), (37, 16, 4, 256, 96, 4, 2),
                                           (700, 4, 2, 640, 160, 1, 1)])
def test_a_block_step_by_step(T, E, k, H, N, G, g):
    """Every step against the formula on the tensors that the step before left."""
    b = block(T, E, k, H, N, T, G, g)
    s = run_block(b)
    ri, rw = ref.gate(b["scores"].cpu(), k, "sigmoid", b["bias"].cpu(), G, g, "top2", True, 2.5)
    assert torch.equal(s["idx"].cpu().long(), ri)
    check(s["w"], rw, rw, "weights")
    q, sf = ref.cast(b["x"])
    assert torch.equal(s["xq"].cpu(), q) and torch.equal(s["xs"].cpu(), sf)
    want, mag, largest = ref.matmul(s["xq"], s["xs"], b["up"], b["up_sf"], s["offsets"], s["src"],
                                    k, True)
    assert largest < 2 ** 24
    check(s["act"], want, mag / 8, "act")
    q, sf = ref.cast(s["act"])
    assert torch.equal(s["aq"].cpu(), q) and torch.equal(s["as_"].cpu(), sf)
    want, mag, largest = ref.matmul(s["aq"], s["as_"], b["down"], b["down_sf"], s["offsets"], None,
                                    1, False)
    assert largest < 2 ** 24
    check(s["y_e"], want, mag / 8, "y_e")
    rows = cpu64(s["y_e"])[s["pos"].cpu().long()]
    want = (rows * cpu64(s["w"])[..., None]).sum(1)
    check(s["out"], want, (rows * cpu64(s["w"])[..., None]).abs().sum(1), "out")


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
def test_router_gradient_with_the_losses_against_autograd(func):
    T, E, k, S = 50, 16, 4, 3
    r = gen(4)
    x = torch.randn(T, E, generator=r)
    cuts = [0, 20, 21, T]
    seq = torch.tensor(cuts, dtype=I32, device=DEV)
    bias = torch.randn(E, generator=r) * 0.1
    idx, w = ops.router_gate(x.to(DEV), k, score_func=func, bias=bias.to(DEV), num_groups=4,
                             topk_groups=2, scale=1.5)
    _, _, counts, _, tokens = ops.balance_loss(x.to(DEV), idx, score_func=func, seq_offsets=seq)
    gw = torch.randn(T, k, generator=r)
    gb, gz = torch.rand(S, generator=r), torch.rand(S, generator=r) * 0.1
    g = ops.balance_loss_backward(x.to(DEV), counts, tokens, gb.to(DEV), gz.to(DEV),
                                  score_func=func, seq_offsets=seq, k=k)
    ops.router_gate_backward(x.to(DEV), idx, gw.to(DEV), score_func=func, scale=1.5, add=g, out=g)
    x64 = x.double().requires_grad_()
    p = torch.sigmoid(x64) if func == "sigmoid" else torch.softmax(x64, 1)
    pn = p / p.sum(1, keepdim=True)
    sel = p.gather(1, idx.cpu().long())
    total = (gw.double() * 1.5 * sel / sel.sum(1, keepdim=True)).sum()
    for i in range(S):
        a, e = cuts[i], cuts[i + 1]
        f = counts[i].cpu().double() * E / (k * (e - a))
        total = total + gb[i].double() * (f * pn[a:e].mean(0)).sum()
        total = total + gz[i].double() * torch.logsumexp(x64[a:e], 1).square().mean()
    total.backward()
    # three terms of order one per entry, each within U of its own
    assert ((cpu64(g) - x64.grad).abs() <= 128 * 2.0 ** -24 * (4 * x64.grad.abs() + 4)).all()


def test_example_trains_and_serves(ex):
    b = ex.Block(H=64, N=32, E=8, k=2, router="sigmoid", groups=4, topk_groups=2, route_scale=2.0)
    history = ex.train(b, steps=2, tokens=48, say=lambda *a: None)
    assert len(history) == 2 and all(torch.isfinite(torch.tensor(history)))
    q = ex.quantise_int8(b)
    for T in (1, 130):
        r = torch.randn(T, b.H, generator=gen(T)).to(DEV)
        h = ex.serve_int8(b, q, r)
        exact, _ = ex.forward(b, r, None)
        # 8-bit rows and weights: each product's terms off by 1/254 of the row's and the
        # channel's largest, independently; three products in a chain stay far below a tenth
        assert float((h - exact).norm() / (exact - r).norm()) < 0.1


def test_example_gradients_with_the_grouped_router(ex):
    """Against autograd in 64 bits, the routing held."""
    b = ex.Block(H=64, N=32, E=8, k=2, router="sigmoid", groups=4, topk_groups=2, balance_coef=0.5,
                 z_coef=0.1, route_scale=2.0)
    T, cuts = 60, [0, 17, 18, 60]
    r = torch.randn(T, b.H, generator=gen(3)).to(DEV)
    h, s = ex.forward(b, r, torch.tensor(cuts, dtype=I32, device=DEV))
    grad_h = torch.randn(T, b.H, generator=gen(5)).to(DEV) / T
    _, grads = ex.backward(b, s, grad_h)
    idx = s["idx"].cpu().long()
    p = {k: v.cpu().double().requires_grad_() for k, v in b.p.items()}
    r64, eps = r.cpu().double(), 1e-6
    n = r64 * torch.rsqrt(r64.square().mean(1, keepdim=True) + eps) * p["pre"]
    scores = n @ p["router"]
    sg = torch.sigmoid(scores)
    sel = sg.gather(1, idx)
    w = b.route_scale * sel / sel.sum(1, keepdim=True)
    y = torch.zeros_like(r64)
    for j in range(b.k):
        for e in range(b.E):
            t = (idx[:, j] == e).nonzero()[:, 0]
            gate, up = (n[t] @ p["up"][e].T).chunk(2, -1)
            y = y.index_add(0, t, w[t, j, None]
                            * ((gate * torch.sigmoid(gate) * up) @ p["down"][e].T))
    z = y * torch.rsqrt(y.square().mean(1, keepdim=True) + eps) * p["post"]
    total = (grad_h.cpu().double() * (r64 + b.scale * torch.sigmoid(p["gate"]) * z)).sum()
    pn, S = sg / sg.sum(1, keepdim=True), len(cuts) - 1
    for i in range(S):
        q = slice(cuts[i], cuts[i + 1])
        m = cuts[i + 1] - cuts[i]
        f = torch.bincount(idx[q].flatten(), minlength=b.E).double() * b.E / (b.k * m)
        total = total + b.balance_coef / S * (f * pn[q].mean(0)).sum()
        total = total + b.z_coef / S * torch.logsumexp(scores[q], 1).square().mean()
    total.backward()
    for name, g in grads.items():
        # the block rounds n, the expert rows and their gradients to bf16 (2^-8 each, about
        # six roundings in a chain): normwise
        want = p[name].grad
        assert float((g.cpu().double() - want).norm()) <= 6 * 2.0 ** -8 * float(want.norm()), name


def calls():
    """Closures over a stream whose every input is at hand before the call."""
    r = gen(9)
    scores = torch.randn(3000, 64, generator=r).to(DEV)
    bias = (torch.randn(64, generator=r) * 0.1).to(DEV)
    idx, w = ops.router_gate(scores, 8, bias=bias, score_func="sigmoid", num_groups=8, topk_groups=3)
    add = torch.randn(3000, 64, generator=r).to(DEV)
    x = torch.randn(900, 2048, generator=r).to(DEV)
    few, few_sf = ops.cast_int8(x[:5].contiguous())
    many, many_sf = ops.cast_int8(x)
    wq, ws = ops.cast_int8((torch.randn(4 * 384, 2048, generator=r) * 0.02).to(DEV))
    wq, ws = wq.view(4, 384, 2048), ws.view(4, 384)
    off = torch.tensor([0, 220, 220, 470, 900], dtype=I32, device=DEV)
    some = torch.tensor([0, 2, 2, 4, 5], dtype=I32, device=DEV)
    mid = torch.tensor([0, 50, 90, 180, 260], dtype=I32, device=DEV)
    mid_x, mid_sf = many[:260].contiguous(), many_sf[:260].contiguous()
    return {
        "router_gate": lambda s: ops.router_gate(scores, 8, bias=bias, score_func="sigmoid",
                                                 num_groups=8, topk_groups=3, stream=s),
        "router_gate_backward": lambda s: (ops.router_gate_backward(
            scores, idx, w, score_func="sigmoid", add=add, stream=s),),
        "cast_int8": lambda s: ops.cast_int8(x, stream=s),
        # a cluster per tile, a CTA per tile, a pair of CTAs per tile
        "matmul_few": lambda s: (ops.expert_matmul_int8(few, few_sf, wq, ws, some, stream=s),),
        "matmul_mid": lambda s: (ops.expert_matmul_int8(mid_x, mid_sf, wq, ws, mid, swiglu=True,
                                                        stream=s),),
        "matmul_many": lambda s: (ops.expert_matmul_int8(many, many_sf, wq, ws, off, stream=s),),
    }


NAMES = ["router_gate", "router_gate_backward", "cast_int8", "matmul_few", "matmul_mid",
         "matmul_many"]


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(None)
        got = call(None)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_beside_other_work_of_the_current_stream(name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
    got = call(s)
    sizes = [1 << i for i in range(9, 23)] + [t.numel() * t.element_size() for t in got]
    for _ in range(3):
        held = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del held


def test_products_on_several_streams_at_once():
    """The three forms beside one another, each many times."""
    c = calls()
    names = ["matmul_few", "matmul_mid", "matmul_many", "matmul_many"]
    want = {n: c[n](None)[0].clone() for n in names}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in names]
    got = [[c[n](s)[0] for _ in range(10)] for n, s in zip(names, streams)]
    torch.cuda.synchronize()
    for n, outs in zip(names, got):
        for o in outs:
            assert torch.equal(o, want[n])


def test_weights_cold_from_memory_are_exact():
    """More weights than the cache holds, runs of rows of many lengths, twice on fresh
    weights: integer sums below 2^24 are exact in f32, and the scales are powers of two."""
    E, k, K, N, T = 256, 8, 2048, 1024, 6000
    for seed in (1, 2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        w = torch.randint(-40, 41, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
        x = torch.randint(-40, 41, (T, K), generator=g, device=DEV, dtype=torch.int8)
        scores = torch.randn(T, E, generator=g, device=DEV) + torch.randn(E, generator=g,
                                                                         device=DEV)
        idx, _ = ops.topk_gate(scores, k)
        _, offsets, _, src = ops.route_map(idx, E)
        xs = torch.full((T,), 0.5, device=DEV)
        ws = torch.full((E, N), 0.25, device=DEV)
        # 40 * 40 * 2048 < 2^24
        first = ops.expert_matmul_int8(x, xs, w, ws, offsets, sorted_src=src, k=k, out_dtype=F32)
        for _ in range(3):
            again = ops.expert_matmul_int8(x, xs, w, ws, offsets, sorted_src=src, k=k,
                                           out_dtype=F32)
            assert torch.equal(first, again)
        ends = offsets.tolist()
        for e in range(E):
            rows = slice(ends[e], ends[e + 1])
            want = x[(src[rows] // k).long()].float() @ w[e].float().T * 0.125
            assert torch.equal(first[rows], want), e


@pytest.mark.parametrize("rows", [5, 130, 700])
def test_products_write_their_rows_only(rows):
    r = gen(rows)
    x, xs = ops.cast_int8(torch.randn(rows, 1024, generator=r).to(DEV))
    w, ws = ops.cast_int8(torch.randn(3 * 200, 1024, generator=r).to(DEV))
    w, ws = w.view(3, 200, 1024), ws.view(3, 200)
    off = torch.tensor([0, rows // 2, rows // 2, rows - 2], dtype=I32, device=DEV)
    for n, sw in ((200, False), (100, True)):
        for dt in (BF, F32):
            buf = torch.full((rows * n + 512,), 7.0, dtype=dt, device=DEV)
            out = buf[256:256 + rows * n].view(rows, n)
            ops.expert_matmul_int8(x, xs, w, ws, off, swiglu=sw, out_dtype=dt, out=out)
            assert (buf[:256] == 7).all() and (buf[256 + rows * n:] == 7).all()
            assert (out[rows - 2:] == 7).all()
            want, mag, largest = ref.matmul(x, xs, w, ws, off, None, 1, sw)
            assert largest < 2 ** 24
            check(out[:rows - 2], want[:rows - 2], mag[:rows - 2] / 8, "products")


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("shape", [(1, 8, 8), (6, 256, 8), (9, 40, 7), (5, 33, 16), (7, 512, 12),
                                   (3, 200, 16), (6, 1024, 32), (2, 1024, 3)])
def test_router_gradient_of_an_expert_named_twice(shape, func, renorm):
    """Both gradients reach the entry, in place too; entries named not at all between
    others and tokens that share no warp evenly."""
    T, E, k = shape
    r = gen(T * E + k)
    x = torch.randn(T, E, generator=r) * 3
    idx = torch.randint(0, max(1, min(E, k // 2)), (T, k), generator=r, dtype=I32)
    idx[-1, 0] = -1
    gw = torch.randn(T, k, generator=r)
    add = torch.randn(T, E, generator=r) * 0.1
    args = dict(score_func=func, renormalize=renorm, scale=2.5)
    for a in (None, add):
        want, mag = ref.gate_grad(x, idx, gw, func, renorm, 2.5, a)
        got = ops.router_gate_backward(x.to(DEV), idx.to(DEV), gw.to(DEV),
                                       add=None if a is None else a.to(DEV), **args)
        assert ops.device_status() == ops.MOE_DEVERR_EXPERT_RANGE
        check(got, want, mag, "grad_scores")
    same = add.to(DEV)
    ops.router_gate_backward(x.to(DEV), idx.to(DEV), gw.to(DEV), add=same, out=same, **args)
    assert ops.device_status() == ops.MOE_DEVERR_EXPERT_RANGE
    check(same, want, mag, "in place")


def many_scores(kind, T, E, r):
    x = torch.randn(T, E, generator=r) * 2
    if kind == "few digits":  # equal values, with the bias of an untrained router
        return x.bfloat16().float(), torch.zeros(E)
    if kind == "closed":
        x[torch.rand(T, E, generator=r) < 0.4] = -float("inf")
        x[::5, 3:] = -float("inf")
        x[7] = -float("inf")
    elif kind == "one value":  # nearly: borders that f32 cannot tell
        x[::2] = 0.75
        x[1::4] = 0.75 + 1e-7 * torch.randn(E, generator=r)
        return x, torch.zeros(E)
    elif kind == "in one place":  # all large values in an eighth of the row
        x[:, E // 8:E // 4] += 9
    elif kind == "saturated":
        x *= 20
    return x, torch.randn(E, generator=r) * 0.05


@pytest.mark.parametrize("kind", ["plain", "few digits", "closed", "one value", "in one place",
                                  "saturated"])
@pytest.mark.parametrize("case", [(64, 8, 8, 4), (128, 3, 4, 1), (160, 6, 8, 3), (192, 8, 1, 1),
                                  (256, 8, 8, 4), (256, 8, 2, 1), (256, 1, 1, 1), (384, 16, 16, 8),
                                  (512, 9, 8, 3), (512, 8, 1, 1), (16, 2, 1, 1), (16, 4, 4, 2),
                                  (32, 8, 8, 4), (32, 3, 2, 1), (16, 5, 2, 2)])
def test_router_of_many_tokens(case, kind):
    """More tokens than SMs many times over, not a multiple of any warp's: the 64-bit
    selection for every token, with each score and group rule."""
    E, k, G, g = case
    T = 13 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    x, bias = many_scores(kind, T, E, gen(E + k))
    for i, (func, gs) in enumerate([("sigmoid", "top2"), ("softmax", "max"), ("sigmoid", "max"),
                                    ("softmax", "top2")]):
        b = None if i == 3 or (i == 0 and kind == "saturated") else bias
        some = torch.arange(i % 2, T, 2)  # the oracle takes its time: every other token
        want, w = ref.gate(x[some], k, func, b, G, g, gs, i % 2 == 0, 2.5)
        idx, got = ops.router_gate(x.to(DEV), k, score_func=func, num_groups=G, topk_groups=g,
                                   bias=None if b is None else b.to(DEV), group_score=gs,
                                   renormalize=i % 2 == 0, scale=2.5)
        assert torch.equal(idx.cpu()[some].long(), want), (func, gs)
        check(got.cpu()[some], w, w, "weights")


def test_router_of_many_tokens_as_of_few():
    """A token's result does not depend on how many tokens come with it."""
    r = gen(5)
    x = (torch.randn(5000, 256, generator=r) * 2).to(DEV)
    b = (torch.randn(256, generator=r) * 0.1).to(DEV)
    args = dict(score_func="sigmoid", bias=b, num_groups=8, topk_groups=4)
    idx, w = ops.router_gate(x, 8, **args)
    for at in (0, 1, 2047, 4999):
        one, ow = ops.router_gate(x[at:at + 1].contiguous(), 8, **args)
        assert torch.equal(one[0], idx[at])
        check(ow[0], cpu64(w[at]), cpu64(w[at]), "weights")


def test_under_the_debug_bounds_library():
    """The same kernels with their internal checks compiled in report nothing."""
    env = dict(os.environ, MOE_DEBUG_BOUNDS="1")
    code = ("import sys; sys.path.insert(0, %r); import torch; "
            "from moe_routing_precision_gb300 import _build, ops; _build.build(); "
            "from tests import test_gpu_router_int8_use as t; c = t.calls(); "
            "[c[n](None) for n in t.NAMES]; torch.cuda.synchronize(); "
            "assert ops.lib().moe_debug_bounds_enabled() == 1; "
            "assert ops.device_status() == 0; print('clean')" % ROOT)
    out = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True,
                         text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.strip().endswith("clean"), out.stderr[-2000:]
