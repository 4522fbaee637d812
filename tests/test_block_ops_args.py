"""Host-side refusals of the operators around the routed experts (no GPU):
the C entry points reject bad arguments before any CUDA call, and the binding
refuses tensors of the wrong type, shape or place."""
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


def test_block_norm_refusals(L):
    def f(res=FAKE, sd=0, y=FAKE, bd=0, T=4, H=64, pw=FAKE, gate=None, kind=0, act=0, scale=1.0,
          nw=FAKE, eps=1e-6, h=FAKE, n=FAKE, rp=FAKE, rn=FAKE):
        return L.moe_block_norm(res, sd, y, bd, T, H, pw, gate, kind, act, scale, nw, eps, h, n,
                                rp, rn, None)
    assert f(T=0) == 0
    assert f(T=-1) == INVALID and f(H=0) == INVALID
    assert f(H=16385) == UNSUPPORTED and f(T=1 << 40) == UNSUPPORTED
    assert f(sd=2) == INVALID and f(bd=-1) == INVALID
    assert f(kind=4, gate=FAKE) == INVALID and f(act=2) == INVALID
    assert f(kind=1) == INVALID                       # a gate kind without a gate
    assert f(gate=FAKE) == INVALID                    # and a gate without a kind
    assert f(eps=0.0) == INVALID and f(eps=NAN) == INVALID and f(eps=INF) == INVALID
    assert f(scale=NAN) == INVALID and f(scale=INF) == INVALID
    assert f(res=None) == INVALID and f(h=None) == INVALID and f(n=None) == INVALID
    assert f(nw=None) == INVALID                      # n without its weight
    assert f(y=None) == INVALID                       # post_weight without y
    assert f(y=None, pw=None, nw=None, n=None) == INVALID   # nothing to do
    assert f(res=FAKE + 1) == INVALID and f(sd=1, res=FAKE + 2) == INVALID
    assert f(pw=FAKE + 2) == INVALID and f(rn=FAKE + 2) == INVALID
    assert f(kind=3, gate=FAKE + 1) == INVALID and f(kind=2, gate=FAKE + 2) == INVALID


def test_block_norm_backward_refusals(L):
    need = L.moe_block_norm_backward_workspace_bytes(4, 64)
    assert need >= 4 * 2 * 64 * 4 and L.moe_block_norm_backward_workspace_bytes(0, 64) == 0
    assert L.moe_block_norm_backward_workspace_bytes(1 << 20, 7168) <= 320 * 3 * 7168 * 4

    def f(gh=FAKE, gn=FAKE, h=FAKE, sd=0, y=FAKE, bd=0, T=4, H=64, pw=FAKE, gate=None, kind=0,
          act=0, scale=1.0, nw=FAKE, rp=FAKE, rn=FAKE, gr=FAKE, gy=FAKE, gpw=FAKE, gg=None,
          gnw=FAKE, ws=FAKE, wsb=need):
        return L.moe_block_norm_backward(gh, gn, h, sd, y, bd, T, H, pw, gate, kind, act, scale,
                                         nw, rp, rn, gr, gy, gpw, gg, gnw, ws, wsb, None)
    assert f(T=-1) == INVALID and f(H=0) == INVALID and f(H=20000) == UNSUPPORTED
    assert f(wsb=need - 1) == INVALID and f(ws=None) == INVALID and f(ws=FAKE + 8) == INVALID
    assert f(gn=None) == INVALID and f(h=None) == INVALID and f(rn=None) == INVALID
    assert f(rp=None) == INVALID and f(gpw=None) == INVALID and f(gnw=None) == INVALID
    assert f(gr=None) == INVALID and f(gy=None) == INVALID
    assert f(kind=1, gate=FAKE) == INVALID            # a gate without its gradient
    assert f(gg=FAKE) == INVALID                      # and the reverse
    assert f(y=None) == INVALID
    assert f(gh=FAKE + 1) == INVALID and f(gy=FAKE + 1) == INVALID


def test_balance_loss_refusals(L):
    need = L.moe_balance_loss_workspace_bytes(10000, 16, 3)
    assert need > 0 and L.moe_balance_loss_workspace_bytes(100, 16, 3) == 0
    assert L.moe_balance_loss_workspace_bytes(0, 16, 1) == 0
    assert L.moe_balance_loss_workspace_bytes(100, 2000, 1) == 0

    def f(s=FAKE, i=FAKE, T=10000, E=16, k=2, func=0, seq=FAKE, S=3, mask=None, b=FAKE, z=FAKE,
          c=FAKE, p=FAKE, t=FAKE, ws=FAKE, wsb=need):
        return L.moe_balance_loss(s, i, T, E, k, func, seq, S, mask, b, z, c, p, t, ws, wsb, None)
    assert f(T=-1) == INVALID and f(T=1 << 31) == INVALID
    assert f(E=0) == INVALID and f(E=1025) == INVALID and f(k=17) == INVALID and f(k=0) == INVALID
    assert f(func=2) == INVALID
    assert f(S=0) == INVALID and f(S=65536) == INVALID and f(seq=None) == INVALID
    for name in "s i b z c p t ws".split():
        assert f(**{name: None}) == INVALID, name
    assert f(ws=FAKE + 8) == INVALID and f(wsb=need - 1) == INVALID and f(s=FAKE + 2) == INVALID

    def g(s=FAKE, T=100, E=16, k=2, func=0, seq=None, S=1, mask=None, c=FAKE, t=FAKE, gb=FAKE,
          gz=FAKE, i=FAKE, w=FAKE, gw=FAKE, out=FAKE):
        return L.moe_balance_loss_backward(s, T, E, k, func, seq, S, mask, c, t, gb, gz, i, w, gw,
                                           out, None)
    assert g(T=0) == 0
    assert g(T=-1) == INVALID and g(E=2000) == INVALID and g(k=33, E=64) == INVALID
    assert g(func=-1) == INVALID and g(S=2) == INVALID
    for name in "s c t out i w".split():
        assert g(**{name: None}) == INVALID, name
    assert g(gw=FAKE + 2) == INVALID and g(out=FAKE + 1) == INVALID


def test_combine_backward_refusals(L):
    def f(go=FAKE, gd=0, y=FAKE, w=FAKE, pos=FAKE, src=None, T=4, H=64, k=2, R=8, gy=FAKE,
          gw=FAKE):
        return L.moe_combine_backward(go, gd, y, w, pos, src, T, H, k, R, gy, gw, None)
    assert f(T=0) == 0
    assert f(gd=2) == INVALID and f(T=-1) == INVALID and f(H=60) == INVALID
    assert f(k=0) == INVALID and f(k=33) == INVALID and f(R=-1) == INVALID
    assert f(R=1 << 31) == INVALID and f(T=1 << 31) == UNSUPPORTED
    for name in "go y w pos gy gw".split():
        assert f(**{name: None}) == INVALID, name
    assert f(go=FAKE + 8) == INVALID and f(y=FAKE + 8) == INVALID and f(gy=FAKE + 8) == INVALID
    assert f(src=FAKE + 2) == INVALID


def test_expert_matvec_refusals(L):
    def f(x=FAKE, nx=8, w=FAKE, sf=FAKE, st=0, group=32, off=FAKE, src=FAKE, E=4, k=2, R=8, K=64,
          N=16, sw=0, out=FAKE, od=0):
        return L.moe_expert_matvec_fp4(x, nx, w, sf, st, group, off, src, E, k, R, K, N, sw, out,
                                       od, None)
    assert f(R=0) == 0
    assert f(group=48) == UNSUPPORTED and f(K=16416) == UNSUPPORTED
    assert f(R=(1 << 18) + 1) == UNSUPPORTED and f(N=1 << 26) == UNSUPPORTED
    assert f(st=2) == INVALID and f(od=2) == INVALID
    assert f(E=0) == INVALID and f(E=1025) == INVALID and f(k=0) == INVALID and f(k=33) == INVALID
    assert f(K=48) == INVALID and f(K=96, group=64) == INVALID and f(K=0) == INVALID
    assert f(N=0) == INVALID and f(R=-1) == INVALID and f(nx=-1) == INVALID
    assert f(off=None) == INVALID                     # several experts without offsets
    assert f(src=None, nx=7) == INVALID               # fewer rows of x than of out
    for name in "x w sf out".split():
        assert f(**{name: None}) == INVALID, name
    assert f(x=FAKE + 8) == INVALID and f(w=FAKE + 8) == INVALID and f(sf=FAKE + 2) == INVALID
    assert f(st=1, sf=FAKE + 2) == INVALID
    assert f(out=FAKE + 1) == INVALID and f(od=1, out=FAKE + 2) == INVALID


def test_binding_refuses_what_it_cannot_take():
    from moe_routing_precision_gb300 import ops
    _build.build()
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.block_norm(bf, bf, pre_weight=torch.ones(64))
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        ops.block_norm(bf.half(), bf)
    with pytest.raises(ValueError, match="CUDA"):
        ops.block_norm_backward(bf, bf, bf, pre_weight=torch.ones(64), rstd_pre=torch.ones(4))
    with pytest.raises(ValueError, match="CUDA"):
        ops.balance_loss(torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        ops.balance_loss_backward(torch.zeros(4, 16), None, None)
    with pytest.raises(ValueError, match="CUDA"):
        ops.combine_backward(bf, bf, torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        ops.expert_matvec_fp4(bf, torch.zeros(1, 8, 32, dtype=torch.uint8), torch.zeros(1, 8, 2))
