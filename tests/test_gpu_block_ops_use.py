"""The operators around the routed experts as a program uses them: together in
the example block (its gradients against autograd in 64 bits, its 4-bit decoding
against the dequantised weights), captured in a CUDA graph, on other streams,
with guarded output buffers, and with the debug-bounds library."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

from moe_routing_precision_gb300 import _build, ops
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


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


def _plain_total(b, p, r, grad_h, idx, cuts):
    """<grad_h, h> + coefficients * losses in 64 bits, routing given."""
    eps = 1e-6
    n = r * torch.rsqrt(r.square().mean(1, keepdim=True) + eps) * p["pre"]
    scores = n @ p["router"]
    w = torch.softmax(scores.gather(1, idx), 1)
    y = torch.zeros_like(r)
    for j in range(b.k):
        for e in range(b.E):
            t = (idx[:, j] == e).nonzero()[:, 0]
            gate, up = (n[t] @ p["up"][e].T).chunk(2, -1)
            y = y.index_add(0, t, w[t, j, None]
                            * ((gate * torch.sigmoid(gate) * up) @ p["down"][e].T))
    z = y * torch.rsqrt(y.square().mean(1, keepdim=True) + eps) * p["post"]
    h = r + b.scale * torch.sigmoid(p["gate"]) * z
    total = (grad_h * h).sum()
    prob, S = torch.softmax(scores, 1), len(cuts) - 1
    for i in range(S):
        s = slice(cuts[i], cuts[i + 1])
        m = cuts[i + 1] - cuts[i]
        f = torch.bincount(idx[s].flatten(), minlength=b.E).double() * b.E / (b.k * m)
        total = total + b.balance_coef / S * (f * prob[s].mean(0)).sum()
        total = total + b.z_coef / S * torch.logsumexp(scores[s], 1).square().mean()
    return total


def test_example_gradients_match_autograd(ex):
    b = ex.Block(H=64, N=32, E=4, k=2, balance_coef=0.5, z_coef=0.1)
    g = torch.Generator().manual_seed(3)
    T = 60
    r = torch.randn(T, b.H, generator=g).to(DEV)
    cuts = [0, 17, 18, 60]
    h, s = ex.forward(b, r, torch.tensor(cuts, dtype=torch.int32, device=DEV))
    grad_h = torch.randn(T, b.H, generator=g).to(DEV) / T
    grad_r, grads = ex.backward(b, s, grad_h)
    p = {k: v.cpu().double().requires_grad_() for k, v in b.p.items()}
    r64 = r.cpu().double().requires_grad_()
    _plain_total(b, p, r64, grad_h.cpu().double(), s["idx"].cpu().long(), cuts).backward()
    # the block rounds n, the expert rows and their gradients to bf16 (2^-8 each,
    # about six roundings in a chain): normwise
    for name, got, want in [("r", grad_r, r64.grad)] + [(k, grads[k], p[k].grad) for k in grads]:
        err = float((got.cpu().double() - want).norm() / want.norm())
        assert err <= 6 * 2.0 ** -8, (name, err)


def test_example_trains(ex):
    hist = ex.train(ex.Block(), steps=6, say=lambda *_: None)
    assert hist[-1] < hist[0] and all(b <= a * 1.01 for a, b in zip(hist, hist[1:])), hist


@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_example_decodes(ex, T, ue8m0):
    b = ex.Block(H=256, N=96, E=8, k=2, group=32)
    q = ex.quantise(b, ue8m0)
    r = torch.randn(T, b.H, generator=torch.Generator().manual_seed(T)).to(DEV)
    h = ex.decode(b, q, r).cpu().double()
    deq = {k: ref.dequant(v[0], v[1], b.group) for k, v in q.items()}
    p = {k: v.cpu().double() for k, v in b.p.items()}
    r64 = r.cpu().double()
    n = (r64 * torch.rsqrt(r64.square().mean(1, keepdim=True) + 1e-6) * p["pre"])
    n = n.to(BF).double()
    scores = n @ p["router"]
    w, idx = scores.topk(b.k, 1)
    w = torch.softmax(w, 1)
    y = torch.zeros_like(r64)
    for t in range(T):
        for j in range(b.k):
            e = int(idx[t, j])
            gate, up = (deq["up"][e] @ n[t]).chunk(2)
            act = (gate * torch.sigmoid(gate) * up).to(BF).double()
            y[t] += w[t, j] * (deq["down"][e] @ act).to(BF).double()
    z = y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6) * p["post"]
    want = b.scale * torch.sigmoid(p["gate"]) * z
    # three bf16 roundings in a chain
    assert float((h - r64 - want).norm() / want.norm()) <= 3 * 2.0 ** -8


def test_example_runs_as_a_program():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_block.py"), "--steps",
                          "2", "--tokens", "64"], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "decoded 4 tokens" in out.stdout, out.stdout + out.stderr


def _calls(T=130, H=264, E=24, k=3, seed=0):
    """One call of every entry point on fixed inputs: name -> closure over a stream."""
    g = torch.Generator().manual_seed(seed)

    def randn(*s, dtype=F32):
        return torch.randn(*s, generator=g).to(dtype).to(DEV)

    r, y, gate = randn(T, H), randn(T, H, dtype=BF), randn(H)
    pw, nw = randn(H), randn(H)
    big = {n: randn(700, H, dtype=BF) for n in ("r", "y")}
    h, n, rp, rn = ops.block_norm(r, y, post_weight=pw, gate=gate, gate_act="sigmoid",
                                  pre_weight=nw)
    gh, gn = randn(T, H), randn(T, H, dtype=BF)
    scores = randn(T, E)
    idx, w = ops.topk_gate(scores, k)
    counts, offsets, pos, src = ops.route_map(idx, E)
    seq = torch.tensor([0, 50, 130], dtype=torch.int32, device=DEV)
    long_scores = randn(4000, E)
    long_idx, _ = ops.topk_gate(long_scores, k)
    _, _, lc, _, lt = ops.balance_loss(long_scores, long_idx)
    gb, gz, gw = randn(1), randn(1), randn(T, k)
    _, _, c2, _, t2 = ops.balance_loss(scores, idx, seq_offsets=seq)
    ye = randn(T * k, H, dtype=BF)
    few = idx[:9].contiguous()
    _, off9, _, src9 = ops.route_map(few, E)
    x9 = randn(9, 256, dtype=BF)
    w4 = torch.randint(0, 256, (E, 40, 128), generator=g).to(torch.uint8).to(DEV)
    sf = (torch.rand(E, 40, 8, generator=g) + 0.5).to(DEV)
    return {
        "norm": lambda s: ops.block_norm(r, y, post_weight=pw, gate=gate, gate_act="sigmoid",
                                         pre_weight=nw, stream=s),
        "norm_many": lambda s: ops.block_norm(big["r"], big["y"], post_weight=pw, pre_weight=nw,
                                              stream=s),
        "norm_backward": lambda s: ops.block_norm_backward(
            gh, gn, h, y=y, post_weight=pw, gate=gate, gate_act="sigmoid", pre_weight=nw,
            rstd_post=rp, rstd_pre=rn, stream=s),
        "balance_one": lambda s: ops.balance_loss(scores, idx, seq_offsets=seq, stream=s),
        "balance": lambda s: ops.balance_loss(long_scores, long_idx, stream=s),
        "balance_backward": lambda s: (ops.balance_loss_backward(
            scores, c2, t2, gb.expand(2).contiguous(), gz.expand(2).contiguous(), seq_offsets=seq,
            topk_idx=idx, topk_weights=w, grad_topk_weights=gw, stream=s),
            ops.balance_loss_backward(long_scores, lc, lt, gb, gz, k=k, stream=s)),
        "combine_backward": lambda s: ops.combine_backward(gh, ye, w, pos, stream=s),
        "matvec": lambda s: (ops.expert_matvec_fp4(x9, w4, sf, off9, sorted_src=src9, k=k,
                                                   swiglu=True, stream=s),),
    }


def _flat(out):
    if torch.is_tensor(out):
        return [out]
    return [t for o in out if o is not None for t in _flat(o)]


@pytest.mark.parametrize("name", ["norm", "norm_many", "norm_backward", "balance_one", "balance",
                                  "balance_backward", "combine_backward", "matvec"])
def test_other_stream_and_graph(name):
    """The same bits on the default stream, on another one named by `stream`,
    on another one made current, and from a captured graph replayed twice."""
    call = _calls()[name]
    want = [t.clone() for t in _flat(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = _flat(call(s))
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with torch.cuda.stream(s):
        got = _flat(call(None))
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _flat(call(None))
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


class Guarded:
    """A buffer with 64 sentinel elements before and behind it."""

    def __init__(self, shape, dtype, pad=64):
        n = 1
        for d in shape:
            n *= d
        self.raw = torch.full((n + 2 * pad,), 77, dtype=dtype, device=DEV)
        self.pad, self.view = pad, self.raw[pad:pad + n].view(shape)

    def intact(self):
        return bool((self.raw[:self.pad] == 77).all() and (self.raw[-self.pad:] == 77).all())


@pytest.mark.parametrize("T,H", [(3, 40), (3, 41), (700, 256), (701, 249), (515, 1155)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_writes_stay_inside(T, H, dtype):
    g = torch.Generator().manual_seed(T + H)
    r = torch.randn(T, H, generator=g).to(dtype).to(DEV)
    y = torch.randn(T, H, generator=g).to(BF).to(DEV)
    w = torch.ones(H, device=DEV)
    h, n = Guarded((T, H), dtype), Guarded((T, H), BF)
    ops.block_norm(r, y, post_weight=w, pre_weight=w, out=(h.view, n.view))
    torch.cuda.synchronize()
    assert h.intact() and n.intact()
    want = ref.norm_forward(r, y, w, None, "none", 1.0, w, 1e-6)
    ref.check(h.view, *want["h"], "h")
    ref.check(n.view, *want["n"], "n")


def test_other_writes_stay_inside():
    g = torch.Generator().manual_seed(5)
    T, H, k, E = 37, 72, 3, 30
    idx = torch.randn(T, E, generator=g).topk(k, 1).indices.to(torch.int32).to(DEV)
    scores = torch.randn(T, E, generator=g).to(DEV)
    _, _, counts, _, tokens = ops.balance_loss(scores, idx)
    out = Guarded((T, E), F32)
    ops.balance_loss_backward(scores, counts, tokens, torch.ones(1, device=DEV), k=k, out=out.view)
    assert out.intact()
    _, offsets, pos, src = ops.route_map(idx, E)
    gy, gw = Guarded((T * k, H), BF), Guarded((T, k), F32)
    ops.combine_backward(torch.randn(T, H, generator=g).to(DEV),
                         torch.randn(T * k, H, generator=g).to(BF).to(DEV),
                         torch.rand(T, k, generator=g).to(DEV), pos, out=(gy.view, gw.view))
    assert gy.intact() and gw.intact()
    for K, N, dtype in ((32, 3, BF), (64, 17, F32), (288, 33, BF)):
        o = Guarded((T * k, N), dtype)
        w4 = torch.randint(0, 256, (E, N, K // 2), generator=g).to(torch.uint8).to(DEV)
        sf = torch.rand(E, N, K // 32, generator=g).to(DEV)
        x = torch.randn(T, K, generator=g).to(BF).to(DEV)
        ops.expert_matvec_fp4(x, w4, sf, offsets, sorted_src=src, k=k, out_dtype=dtype, out=o.view)
        assert o.intact()
        want, mag, _ = ref.expert_matvec(x, w4, sf, 32, offsets, src, k, False, T * k)
        ref.check(o.view, want, mag, f"K = {K}")


def test_all_of_it_with_the_debug_checks():
    env = dict(os.environ, MOE_DEBUG_BOUNDS="1")
    _build.build(debug_bounds=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-p",
                        "no:cacheprovider", "tests/test_gpu_block_ops.py"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
