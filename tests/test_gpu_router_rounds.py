"""The router with more tokens than its warps take at once: second and later rounds of every
form, tokens that are done again at the end of a warp's rounds among them, and more tokens
than 32 for each warp of a full device.

A few hundred different rows are checked against 64 bits; the many tokens are drawn from
them, and each has to get its row's result."""
import pytest
import torch

from moe_routing_precision_gb300 import ops
from tests import router_int8_ref as ref
from tests.block_ref import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from moe_routing_precision_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    assert ops.device_status() == 0
    yield
    assert ops.device_status() == 0


def rows(E, r):
    """Plain rows, and such as f32 does not settle: near one value, of few values, closed
    experts, all large values in one place, saturated."""
    x = torch.randn(300, E, generator=r) * 2
    x[:20] = 0.75
    x[20:40] = 0.75 + 1e-7 * torch.randn(20, E, generator=r)
    x[40:80] = x[40:80].bfloat16().float().round()
    x[80:120][torch.rand(40, E, generator=r) < 0.4] = -float("inf")
    x[120:130, 2:] = -float("inf")
    x[130] = -float("inf")
    x[140:160, E // 8:E // 4] += 9
    x[160:180] *= 20
    return x


# E, k, G, g, tokens of a warp at once (1: a warp per token), bias
CASES = [(16, 2, 4, 2, 8, True), (64, 8, 8, 3, 4, True), (256, 8, 8, 4, 4, True),
         (256, 8, 1, 1, 4, True), (512, 9, 8, 3, 2, True),
         (40, 4, 5, 2, 1, True), (64, 16, 8, 4, 1, True), (96, 6, 1, 1, 1, False),
         (256, 8, 1, 1, 1, False), (48, 5, 6, 2, 1, False)]


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("case", CASES)
def test_every_round(case, func):
    E, k, G, g, Q, biased = case
    r = torch.Generator().manual_seed(E + k + G)
    base = rows(E, r)
    bias = torch.randn(E, generator=r) * 0.05 if biased else None
    renorm = func == "sigmoid"
    kw = dict(score_func=func, bias=None if bias is None else bias.to(DEV), num_groups=G,
              topk_groups=g, renormalize=renorm, scale=1.5)
    want, w = ref.gate(base, k, func, bias, G, g, "top2", renorm, 1.5)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # tokens of a round: 4 blocks of 4 warps per SM, or 8 of 8
    at_once = sms * (16 * Q if Q > 1 else 64)
    most = at_once * 32 // Q        # 32 tokens for each warp
    for T in (at_once + 1, 2 * at_once + 5, most - 3, most + 3, most + at_once // 3 + 7):
        pick = torch.randint(0, len(base), (T,), generator=r)
        pick[-3:] = torch.tensor([0, 30, 130])     # the last ones are done again
        pick[at_once:at_once + 1] = 25
        idx, got = ops.router_gate(base.to(DEV)[pick.to(DEV)], k, **kw)
        bad = (idx.cpu().long() != want[pick]).any(1).nonzero().flatten()
        assert bad.numel() == 0, (T, bad.numel(), bad[:5].tolist(), pick[bad[:5]].tolist())
        check(got.cpu(), w[pick], w[pick], "weights")


@pytest.mark.parametrize("E,k", [(256, 8), (64, 6), (40, 20)])
def test_gradient_of_many_tokens(E, k):
    r = torch.Generator().manual_seed(E)
    n, T = 400, 100003
    x = torch.randn(n, E, generator=r) * 2
    idx = torch.rand(n, E, generator=r).argsort(1)[:, :k].int().contiguous()
    gw, add = torch.randn(n, k, generator=r), torch.randn(n, E, generator=r)
    pick = torch.randint(0, n, (T,), generator=r)
    at = pick.to(DEV)
    for func, renorm in (("sigmoid", True), ("softmax", False)):
        want, mag = ref.gate_grad(x, idx, gw, func, renorm, 2.5, add)
        got = ops.router_gate_backward(x.to(DEV)[at], idx.to(DEV)[at], gw.to(DEV)[at],
                                       score_func=func, renormalize=renorm, scale=2.5,
                                       add=add.to(DEV)[at])
        check(got.cpu(), want[pick], mag[pick], "grad_scores")
