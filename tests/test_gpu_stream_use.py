"""Calls whose kernels run on a stream that is not the current one, while the current
one keeps allocating: nothing a call made for itself is reused too early, and
nothing it was given is still in use."""
import pytest
import torch

from moe_routing_precision_gb300 import _build, ops
from tests.test_gpu_block_ops_use import _calls, _flat

pytestmark = pytest.mark.gpu
NAMES = ["norm", "norm_many", "norm_backward", "balance_one", "balance", "combine_backward",
         "matvec"]
SPIN = 20_000_000                 # clock cycles: about 10 ms, far above any call's time


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    torch.cuda.set_device(0)
    assert ops.device_status() == 0
    yield
    assert ops.device_status() == 0


def _more_calls():
    """Closures over a stream whose every input is at hand before the call."""
    g = torch.Generator().manual_seed(2)
    T, E, k, H = 700, 64, 4, 256
    scores = torch.randn(T, E, generator=g).cuda()
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    idx, w = ops.topk_gate(scores, k)
    _, _, pos, src = ops.route_map(idx, E)
    rows = x.repeat(k, 1)
    _, _, counts, _, tokens = ops.balance_loss(scores, idx)
    gb, gz = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
    return {
        "balance_backward": lambda s: ops.balance_loss_backward(
            scores, counts, tokens, gb, gz, topk_idx=idx, topk_weights=w, grad_topk_weights=w,
            stream=s),
        "topk_gate": lambda s: ops.topk_gate(scores, k, stream=s),
        "route_map": lambda s: ops.route_map(idx, E, stream=s),
        "route_expand_cast_fp8": lambda s: ops.route_expand_cast_fp8(scores, x, k, stream=s),
        "expand_cast_fp8_ex": lambda s: ops.expand_cast_fp8_ex(
            x, pos, sorted_src=src, sf_flags=ops.SF_COLMAJOR, workspace=True, stream=s),
        "combine": lambda s: ops.combine(rows, w, pos, stream=s),
    }


@pytest.mark.parametrize("name", NAMES + ["balance_backward", "topk_gate", "route_map",
                                          "route_expand_cast_fp8", "expand_cast_fp8_ex",
                                          "combine"])
def test_calls_beside_other_work_of_the_current_stream(name):
    call = (_calls() if name in NAMES else _more_calls())[name]
    want = [t.clone() for t in _flat(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    # what the call drops or returns is not handed to the current stream meanwhile
    with torch.cuda.stream(s):
        torch.cuda._sleep(SPIN)
    got = _flat(call(s))
    sizes = [1 << i for i in range(9, 23)] + [t.numel() * t.element_size() for t in got]
    for _ in range(3):
        held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
        held = [h.fill_(254) for h in held]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del held, got
    torch.cuda.synchronize()
    # and memory that the current stream is yet to write is not taken for it
    freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda._sleep(SPIN)
    freed = [f.fill_(255) for f in freed]
    del freed
    got = _flat(call(s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["norm_many", "norm_backward", "balance", "matvec"])
def test_calls_on_a_forked_stream_of_a_captured_graph(name):
    """The capture forks to another stream for the call and joins again; the call's own
    tensors are dropped during the capture."""
    call = _calls()[name]
    want = [t.clone() for t in _flat(call(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        s.wait_stream(here)
        call(s)
        got = _flat(call(s))
        here.wait_stream(s)
        got = [t.clone() for t in got]
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    del graph
    torch.cuda.synchronize()
    again = _flat(call(s))
    torch.cuda.synchronize()
    for a, b in zip(again, want):
        assert torch.equal(a, b)
