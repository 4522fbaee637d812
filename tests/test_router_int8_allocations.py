"""Tensors that the router's, the row cast's and the 8-bit products' calls allocate for
themselves belong to the stream their kernels run on (no GPU needed; the stand-ins are
test_stream_allocations.py's)."""
import pytest

from moe_routing_precision_gb300 import ops
from tests.test_stream_allocations import BF, F32, I32, FakeStream, _t, rec  # noqa: F401
import torch

I8 = torch.int8
T, H, E, K = 6, 256, 8, 2

CALLS = {
    "router_gate": lambda s: ops.router_gate(_t(T, E), K, bias=_t(E), stream=s),
    "router_gate_backward": lambda s: ops.router_gate_backward(
        _t(T, E), _t(T, K, dtype=I32), _t(T, K), add=_t(T, E), stream=s),
    "cast_int8": lambda s: ops.cast_int8(_t(T, H, dtype=BF), stream=s),
    "expert_matmul_int8": lambda s: ops.expert_matmul_int8(
        _t(T, H, dtype=I8), _t(T), _t(1, 16, H, dtype=I8), _t(1, 16), stream=s),
}


@pytest.fixture
def calls(rec, monkeypatch):  # noqa: F811
    monkeypatch.setattr(ops, "_one_device", lambda *a: None)
    return rec


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("form", ["stream", "handle", "default"])
def test_belong_to_the_named_stream(calls, name, form):
    named = {"stream": FakeStream(0x20), "handle": 0x20, "default": 0}[form]
    CALLS[name](named)
    handle = 0 if form == "default" else 0x20
    assert len(calls.calls) == 1 and calls.calls[0][1][-1] == (handle or None)
    assert calls.made
    for t, s in calls.made:
        assert s == handle
        assert any(u is t and r == 0x10 for u, r in calls.recorded)


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("named", [None, 0x10])
def test_are_plain_on_the_current_stream(calls, name, named):
    CALLS[name](named)
    assert calls.made and all(s == 0x10 for _, s in calls.made) and not calls.recorded
    assert calls.calls[0][1][-1] == 0x10
