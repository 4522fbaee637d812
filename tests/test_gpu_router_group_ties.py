"""The router's groups where more of them tie above the border than may stay: equal scores
in several groups, or sigmoids that 64 bits round to 1.  The lower groups stay."""
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


CASES = [(64, 8, 8, 2), (256, 8, 8, 3), (72, 4, 6, 2), (96, 8, 12, 5), (16, 2, 8, 3),
         (512, 8, 16, 4), (1000, 5, 25, 7), (60, 5, 12, 4)]


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("case", CASES)
def test_groups_that_tie_above_the_border(case, func):
    E, k, G, g = case
    n = E // G
    r = torch.Generator().manual_seed(E + k)
    many = 13 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    for T in (40, many):
        x = torch.randn(T, E, generator=r) - 3
        for t in range(T):
            # from one to all groups with the same two largest, the rest well below or near
            tied = torch.randperm(G, generator=r)[:t % G + 1]
            x[t].view(G, n)[tied, 0] = 2.0
            if n > 1:
                x[t].view(G, n)[tied, n - 1] = 40.0 if t % 3 == 0 else 1.5
        some = torch.arange(0, T, 1 if T == 40 else 7)
        for gs in ("top2", "max"):
            for bias in (None, torch.full((E,), 0.125), torch.zeros(E)):
                want, w = ref.gate(x[some], k, func, bias, G, g, gs, True, 1.0)
                idx, got = ops.router_gate(x.to(DEV), k, score_func=func, num_groups=G,
                                           topk_groups=g, group_score=gs,
                                           bias=None if bias is None else bias.to(DEV))
                assert torch.equal(idx.cpu()[some].long(), want), (T, gs)
                check(got.cpu()[some], w, w, "weights")
