"""Host-side refusals of the router with groups, the row cast to 8-bit integers and the
experts' products in them (no GPU): the C entry points reject bad arguments before any
CUDA call, and the binding refuses tensors of the wrong type, shape or place."""
import pytest
import torch

from moe_routing_precision_gb300 import _build

FAKE = 0x10000  # never dereferenced: every call below is rejected on the host
INVALID, UNSUPPORTED = 1, 2
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    _build.build()
    from moe_routing_precision_gb300 import ops
    lib = ops.lib()
    before = lib.moe_kernel_launch_count()
    yield lib
    assert lib.moe_kernel_launch_count() == before


def test_router_gate_refusals(L):
    def f(s=FAKE, T=4, E=64, k=4, func=1, b=FAKE, G=8, g=4, gs=1, rn=1, scale=1.0, i=FAKE, w=FAKE):
        return L.moe_router_gate(s, T, E, k, func, b, G, g, gs, rn, scale, i, w, None)
    assert f(T=0) == 0 and f(T=0, s=None, i=None, w=None) == 0
    assert f(T=-1) == INVALID and f(T=1 << 31) == INVALID
    assert f(E=0) == INVALID and f(E=1032) == INVALID and f(k=0) == INVALID and f(k=33) == INVALID
    assert f(func=2) == INVALID and f(func=-1) == INVALID and f(gs=2) == INVALID
    assert f(G=0) == INVALID and f(G=7) == INVALID and f(G=64) == INVALID    # 64 > 32 groups
    assert f(g=0) == INVALID and f(g=9) == INVALID
    assert f(k=9, g=1) == INVALID            # more than the open groups hold
    assert f(scale=NAN) == INVALID and f(scale=INF) == INVALID
    assert f(s=None) == INVALID and f(i=None) == INVALID and f(w=None) == INVALID
    for name in ("s", "b", "i", "w"):
        assert f(**{name: FAKE + 2}) == INVALID


def test_router_gate_backward_refusals(L):
    def f(s=FAKE, T=4, E=64, k=4, func=1, rn=1, scale=1.0, i=FAKE, gw=FAKE, add=FAKE, o=FAKE):
        return L.moe_router_gate_backward(s, T, E, k, func, rn, scale, i, gw, add, o, None)
    assert f(T=0) == 0 and f(T=-1) == INVALID and f(T=1 << 31) == INVALID
    assert f(E=0) == INVALID and f(E=1025) == INVALID and f(k=65) == INVALID
    assert f(func=2) == INVALID and f(scale=NAN) == INVALID
    assert f(s=None) == INVALID and f(i=None) == INVALID and f(gw=None) == INVALID
    assert f(o=None) == INVALID
    for name in ("s", "i", "gw", "add", "o"):
        assert f(**{name: FAKE + 2}) == INVALID


def test_cast_int8_refusals(L):
    def f(x=FAKE, dt=0, T=4, H=64, q=FAKE, sf=FAKE):
        return L.moe_cast_int8(x, dt, T, H, q, sf, None)
    assert f(T=0) == 0 and f(T=-1) == INVALID and f(H=0) == INVALID and f(dt=2) == INVALID
    assert f(T=1 << 31, H=1) == UNSUPPORTED and f(T=1 << 24, H=1 << 17) == UNSUPPORTED
    assert f(x=None) == INVALID and f(q=None) == INVALID and f(sf=None) == INVALID
    assert f(x=FAKE + 1) == INVALID and f(dt=1, x=FAKE + 2) == INVALID and f(sf=FAKE + 2) == INVALID


def test_expert_matmul_int8_refusals(L):
    def f(x=FAKE, xs=FAKE, X=4, w=FAKE, ws=FAKE, off=FAKE, src=FAKE, E=8, k=2, R=8, K=64, N=32,
          sw=0, o=FAKE, od=0):
        return L.moe_expert_matmul_int8(x, xs, X, w, ws, off, src, E, k, R, K, N, sw, o, od, None)
    assert f(R=0) == 0
    assert f(R=-1) == INVALID and f(X=-1) == INVALID and f(N=0) == INVALID
    assert f(K=0) == INVALID and f(K=24) == INVALID and f(K=8) == INVALID
    assert f(K=65552) == UNSUPPORTED and f(R=1 << 31) == UNSUPPORTED
    assert f(N=1 << 28, E=8) == UNSUPPORTED and f(N=1 << 27, E=8, sw=1) == UNSUPPORTED
    assert f(E=0) == INVALID and f(E=1025) == INVALID and f(k=0) == INVALID and f(k=33) == INVALID
    assert f(off=None) == INVALID                       # several experts, no offsets
    assert f(src=None, X=7) == INVALID                  # fewer rows of x than of out
    assert f(od=2) == INVALID
    for name in ("x", "xs", "w", "ws", "o"):
        assert f(**{name: None}) == INVALID
    assert f(x=FAKE + 8) == INVALID and f(w=FAKE + 8) == INVALID
    assert f(xs=FAKE + 2) == INVALID and f(ws=FAKE + 2) == INVALID
    assert f(off=FAKE + 2) == INVALID and f(src=FAKE + 2) == INVALID
    assert f(o=FAKE + 1) == INVALID and f(od=1, o=FAKE + 2) == INVALID


def test_binding_refuses_tensors_off_the_device():
    from moe_routing_precision_gb300 import ops
    s = torch.zeros(2, 8)
    i8 = torch.zeros(2, 16, dtype=torch.int8)
    with pytest.raises(ValueError):
        ops.router_gate(s, 2)
    with pytest.raises(ValueError):
        ops.router_gate_backward(s, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
    with pytest.raises(ValueError):
        ops.cast_int8(s)
    with pytest.raises(TypeError):
        ops.cast_int8(s.double())
    with pytest.raises(ValueError):
        ops.expert_matmul_int8(i8, torch.zeros(2), i8[None], torch.zeros(1, 2))
