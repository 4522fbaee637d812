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
