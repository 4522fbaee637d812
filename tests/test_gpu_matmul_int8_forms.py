"""The experts' 8-bit products in each form of their kernel (matmul_forms.py), against
64 bits (router_int8_ref.py, where the tolerances are derived)."""
import pytest
import torch

from moe_routing_precision_gb300 import ops
from tests import matmul_forms as forms
from tests import router_int8_ref as ref
from tests.block_ref import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
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


def run(p, swiglu, out_dtype, src=None, k=1, out=None):
    x, xs, w, ws, off = (t.to(DEV) for t in p)
    return ops.expert_matmul_int8(x, xs, w, ws, off, swiglu=swiglu, out_dtype=out_dtype, k=k,
                                  sorted_src=None if src is None else src.to(DEV), out=out)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("form", forms.FORMS)
def test_scales_one_after_the_other(form, swiglu):
    """(sum * x_sf) * w_sf: the product of the two scales may leave f32's range where the
    result does not."""
    x, xs, w, ws, off = forms.inputs(form, swiglu, sms(), 1)
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
