"""The experts' 8-bit products in each form of their kernel (matmul_forms.py), against
64 bits (router_int8_ref.py, where the tolerances are derived)."""
import os
import subprocess
import sys

import pytest
import torch

from moe_routing_precision_gb300 import ops
from tests import matmul_forms as forms
from tests import router_int8_ref as ref
from tests.block_ref import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_routing_precision_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    assert ops.device_status() == 0
    yield
    assert ops.device_status() == 0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def took(form, w, rows, swiglu):
    """Whether a call with these weights and rows takes the form that it is meant for."""
    E, M, K = w.shape
    return ops.debug_matmul_int8_form(E, rows, K, M // 2 if swiglu else M, swiglu) == form


def run(p, swiglu, out_dtype, src=None, k=1, out=None):
    x, xs, w, ws, off = (t.to(DEV) for t in p)
    return ops.expert_matmul_int8(x, xs, w, ws, off, swiglu=swiglu, out_dtype=out_dtype, k=k,
                                  sorted_src=None if src is None else src.to(DEV), out=out)


def gathered(p, k, seed):
    """The same rows out of a shuffled x with k copies of each token, some of them absent:
    (x, x_sf, w, w_sf, offsets), sorted_src."""
    x, xs, w, ws, off = p
    R = x.shape[0]
    r = torch.Generator().manual_seed(seed)
    token = torch.randperm(R, generator=r)
    src = (token * k + torch.randint(0, k, (R,), generator=r)).to(I32)
    src[torch.rand(R, generator=r) < 0.1] = -1
    src[R // 2] = -7
    return p, src


def expected(p, swiglu, src=None, k=1):
    want, mag, largest = ref.matmul(*p, src, k, swiglu)
    assert largest < 2 ** 24      # the sums are exact: see the reference's tolerances
    return want, mag


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("form", forms.FORMS)
def test_against_64_bits(form, swiglu):
    """Many tiles for each CTA, more blocks of channels than stages, experts without rows, a
    last tile and a last block that are part empty; rows behind the last expert's and what
    lies around the output are left as they were."""
    for extra, K in ((0, None), (3, 640 if form == "pair" else 1024)):
        p = forms.inputs(form, swiglu, sms(), 5 + extra, extra=extra, K=K)
        R, M = p[0].shape[0], p[3].shape[1]
        N, rows = M // 2 if swiglu else M, R - extra
        assert took(form, p[2], R, swiglu)
        want, mag = expected(p, swiglu)
        for dt in (BF, F32):
            buf = torch.full((R * N + 512,), 7.0, dtype=dt, device=DEV)
            out = buf[256:256 + R * N].view(R, N)
            run(p, swiglu, dt, out=out)
            assert (buf[:256] == 7).all() and (buf[256 + rows * N:] == 7).all()
            check(out[:rows], want[:rows], mag[:rows] / 8, "products")


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("form", forms.FORMS)
def test_gathered_absent_and_bad_rows(form, swiglu):
    p, src = gathered(forms.inputs(form, swiglu, sms(), 8), 3, 9)
    assert took(form, p[2], src.numel(), swiglu)
    want, mag = expected(p, swiglu, src, 3)
    for dt in (BF, F32):
        got = run(p, swiglu, dt, src, 3)
        check(got, want, mag / 8, "products")
        assert (got[(src < 0).to(DEV)] == 0).all()
    assert ops.device_status() == 0
    bad = src.clone()
    bad[::11] = 3 * p[0].shape[0] + 1     # a token behind the last one
    got = run(p, swiglu, F32, bad, 3)
    assert ops.device_status() == ops.MOE_DEVERR_POS_RANGE
    want, mag = expected(p, swiglu, bad, 3)
    check(got, want, mag / 8, "products")
    assert (got[::11] == 0).all()


@pytest.mark.parametrize("form", forms.FORMS)
def test_extreme_integers(form):
    """-128 and 127 everywhere, 1024 channels: partial sums reach 2^24, exactly."""
    x, xs, w, ws, off = forms.inputs(form, False, sms(), 1, K=1024)
    x.fill_(-128), w.fill_(-128)
    x[1::2], x[3, ::2] = 127, -128
    w[:, 1::3], w[:, 5, ::2] = 127, 1
    assert took(form, w, x.shape[0], False)
    got = run((x, torch.ones_like(xs), w, torch.ones_like(ws), off), False, F32)
    want = ref.matmul(x, torch.ones_like(xs), w, torch.ones_like(ws), off, None, 1, False)[0]
    assert torch.equal(got.cpu().double(), want)


@pytest.mark.parametrize("form", forms.FORMS)
def test_sums_past_24_bits(form):
    """Sums of one sign, far past 2^24: a sum of f32 in K / 16 steps, each off by an ulp at
    most, and as many more where a cluster adds up."""
    K = 2560
    x, xs, w, ws, off = forms.inputs(form, False, sms(), 2, K=K)
    x, w = x.abs() + 80, w.abs() + 80
    assert took(form, w, x.shape[0], False)
    got = run((x, torch.ones_like(xs), w, torch.ones_like(ws), off), False, F32)
    want = ref.matmul(x, torch.ones_like(xs), w, torch.ones_like(ws), off, None, 1, False)[0]
    assert ((got.cpu().double() - want).abs() <= want * (K / 16 + 8) * 2.0 ** -23).all()


def test_a_decoding_batch_with_cold_weights_is_exact():
    """A CTA per tile over more weights than the cache holds (a decoding batch): integer sums
    below 2^24 are exact in f32, and the scales are powers of two."""
    E, k, K, N, T = 256, 8, 2048, 1024, 64
    for seed, swiglu in ((1, False), (2, True)):
        g = torch.Generator(device=DEV).manual_seed(seed)
        w = torch.randint(-40, 41, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
        x = torch.randint(-40, 41, (T, K), generator=g, device=DEV, dtype=torch.int8)
        scores = torch.randn(T, E, generator=g, device=DEV) + torch.randn(E, generator=g,
                                                                         device=DEV)
        idx, _ = ops.topk_gate(scores, k)
        _, offsets, _, src = ops.route_map(idx, E)
        assert took("cta", w, T * k, swiglu)
        xs, ws = torch.full((T,), 2.0 ** -9, device=DEV), torch.full((E, N), 0.25, device=DEV)
        # 40 * 40 * 2048 < 2^24
        runs = [ops.expert_matmul_int8(x, xs, w, ws, offsets, sorted_src=src, k=k, swiglu=swiglu,
                                       out_dtype=F32) for _ in range(4)]
        assert all(torch.equal(runs[0], r) for r in runs[1:])
        ends = offsets.tolist()
        for e in range(E):
            rows = slice(ends[e], ends[e + 1])
            want = x[(src[rows] // k).long()].double() @ w[e].double().T * 2.0 ** -11
            if swiglu:
                gate, up = want.chunk(2, 1)
                want = gate * torch.sigmoid(gate) * up
                check(runs[0][rows], want.cpu(), (want.abs() * (1 + gate.abs())).cpu() / 8, e)
            else:
                assert torch.equal(runs[0][rows].double(), want), e


def calls():
    """Closures over a stream, a form each, with their inputs at hand."""
    out = {}
    for form in forms.FORMS:
        for swiglu in (False, True):
            p, src = gathered(forms.inputs(form, swiglu, sms(), 4), 2, 4)
            x, xs, w, ws, off = (t.to(DEV) for t in p)
            assert took(form, w, src.numel(), swiglu)
            kw = dict(sorted_src=src.to(DEV), k=2, swiglu=swiglu)
            out[f"{form} {swiglu}"] = (lambda s, a=(x, xs, w, ws, off), kw=kw:
                                       ops.expert_matmul_int8(*a, stream=s, **kw))
    return out


def test_forms_captured_and_replayed():
    c = calls()
    want = {n: f(None).clone() for n, f in c.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = {n: f(None) for n, f in c.items()}
    for _ in range(3):
        for t in got.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n in c:
            assert torch.equal(got[n], want[n]), n


def test_forms_on_several_streams_at_once():
    """Every form beside the others, each many times."""
    c = calls()
    want = {n: f(None).clone() for n, f in c.items()}
    torch.cuda.synchronize()
    streams = {n: torch.cuda.Stream() for n in c}
    got = {n: [] for n in c}
    for _ in range(10):
        for n, f in c.items():
            got[n].append(f(streams[n]))
    torch.cuda.synchronize()
    for n in c:
        assert all(torch.equal(o, want[n]) for o in got[n]), n


def test_forms_under_the_debug_bounds_library():
    env = dict(os.environ, MOE_DEBUG_BOUNDS="1")
    code = ("import sys; sys.path.insert(0, %r); import torch; "
            "from moe_routing_precision_gb300 import _build, ops; _build.build(); "
            "from tests import test_gpu_matmul_int8_forms as t; c = t.calls(); "
            "[f(None) for f in c.values()]; torch.cuda.synchronize(); "
            "assert ops.lib().moe_debug_bounds_enabled() == 1; "
            "assert ops.device_status() == 0; print('clean')" % ROOT)
    out = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True,
                         text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.strip().endswith("clean"), out.stderr[-2000:]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("form", forms.FORMS)
def test_scales_one_after_the_other(form, swiglu):
    """(sum * x_sf) * w_sf: the product of the two scales may leave f32's range where the
    result does not."""
    x, xs, w, ws, off = forms.inputs(form, swiglu, sms(), 1)
    assert took(form, w, x.shape[0], swiglu)
    N = ws.shape[1] // 2
    # scales of about 2^-70 and 2^-66, whose product is subnormal, below sums of about 2^14
    xs, ws = (1 + xs) * 2.0 ** -70, (1 + ws) * 2.0 ** -66
    if swiglu:
        ws[:, N:] *= 2.0 ** 126
    else:
        ws[:, ::2] *= 2.0 ** 126
    # rows of zeros under scales of 2^70, beside weights' scales of 2^60
    x[::3] = 0
    xs[::3] = 2.0 ** 70
    got = run((x, xs, w, ws, off), swiglu, F32).cpu().double()
    want, mag, largest = ref.matmul(x, xs, w, ws, off, None, 1, swiglu)
    assert largest < 2 ** 24
    # and up to two roundings to the subnormals' spacing of 2^-149, times what the SwiGLU
    # then multiplies them by
    up = 0.0
    if swiglu:
        up = ref.matmul(x, xs, w[:, N:].contiguous(), ws[:, N:].contiguous(), off, None, 1,
                        False)[0].abs()
    tol = 16 * 2.0 ** -24 * mag + 2.0 ** -148 * (1 + up)
    assert (got[::3] == 0).all()
    assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max()


@pytest.fixture
def hooks():
    yield ops.debug_set
    ops.debug_set(ops.DEBUG_WEIGHT_STAGES, -1)
    ops.debug_set(ops.DEBUG_WAIT_TIMEOUT_NS, 1_000_000_000)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("form", forms.FORMS)
def test_waits_that_run_out_end_in_an_error(form, swiglu, hooks):
    """Weights that no CTA asks for past its first stages: every warp's waits run out, the
    copies and products in flight end, and the next call is right."""
    p = forms.inputs(form, swiglu, sms(), 3)
    assert took(form, p[2], p[0].shape[0], swiglu)
    want = run(p, swiglu, F32)
    assert ops.device_status() == 0
    hooks(ops.DEBUG_WAIT_TIMEOUT_NS, 2_000_000)
    # none at all; fewer than a ring; fewer than, and more than, a tile's
    for stages in (0, 1, 3, 4, 6, 11):
        hooks(ops.DEBUG_WEIGHT_STAGES, stages)
        if form == "cluster" and stages > 1:
            continue                     # a CTA has one tile's share: two or five blocks
        run(p, swiglu, F32)
        assert ops.device_status() == ops.MOE_DEVERR_TIMEOUT, stages
        hooks(ops.DEBUG_WEIGHT_STAGES, -1)
        got = run(p, swiglu, F32)
        assert ops.device_status() == 0 and torch.equal(got, want), stages
