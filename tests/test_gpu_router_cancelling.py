"""The router's groups where a group's two largest cancel: a large bias of one sign beside
one of the other, so that the sum is as small as the roundings of its two terms.  The
selection is still that of 64 bits, in every form of the kernel."""
import itertools
import math

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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def selections(x, bias, k, func, G, g):
    """Every selection that 64 bits admit for one token.  Groups whose sums are closer than
    the roundings of 64 bits are not told apart: a score is off by two units of 2^-53, and
    both s + bias and the sum of two of them round, by 2^-53 of at most |a| + |b|, for each
    of the two groups compared.  That is less than 2^-50 of the largest |a| + |b|.  (Rows of
    one value have groups that tie as real numbers, whose 64-bit sums do not.)"""
    E = x.numel()
    n = E // G
    s = ref.scores(x[None], func)[0].tolist()
    b = bias.double().tolist()
    c = [u + v for u, v in zip(s, b)]
    sums, size = [], 0.0
    for i in range(G):
        two = sorted(range(i * n, (i + 1) * n), key=lambda e: -c[e])[:2]
        sums.append(math.fsum(v for e in two for v in (s[e], b[e])))
        size = max(size, sum(abs(c[e]) for e in two))
    by = sorted(sums, reverse=True)
    low, high, off = by[g - 1], by[g], 2.0 ** -50 * size
    if low - high > off:
        near = []
        sure = [i for i in range(G) if sums[i] >= low]
    else:
        near = [i for i in range(G) if high - off <= sums[i] <= low + off]
        sure = [i for i in range(G) if sums[i] > low + off]
    for some in itertools.combinations(near, g - len(sure)):
        open_ = [e for i in sorted(sure + list(some)) for e in range(i * n, (i + 1) * n)]
        yield sorted(open_, key=lambda e: (-c[e], e))[:k]


def compare(x, bias, k, func, G, g, some=None):
    """The kernel's selection and weights of x's tokens (`some`: those looked at)."""
    idx, w = ops.router_gate(x.to(DEV), k, score_func=func, bias=bias.to(DEV), num_groups=G,
                             topk_groups=g)
    some = torch.arange(x.shape[0]) if some is None else some
    x, idx, w = x[some], idx.cpu()[some].long(), w.cpu()[some]
    want, _ = ref.gate(x, k, func, bias, G, g, "top2", True, 1.0)
    for t in (idx != want).any(1).nonzero().flatten().tolist():
        assert idx[t].tolist() in selections(x[t], bias, k, func, G, g), (
            t, idx[t].tolist(), want[t].tolist())
    ww = ref.weights(x, idx, func, True, 1.0)
    check(w, ww, ww, "weights")


@pytest.mark.parametrize("x,bias", [
    # sums of two: 1.000070 and 1.000079; f32 rounds to 1.000122 and 1.0
    ([2.8e-4, 0.0, 2.0e-4, 1.16e-4], [1024.0, -1024.0, 1024.0, -1024.0]),
    # 1.44360298 and 1.44360271
    ([1.42690682, 0.56316298, 1.10719311, 0.80947334], [256.0, -256.0, 256.0, -256.0]),
])
def test_two_groups_of_two(x, bias):
    x, bias = torch.tensor([x, x[2:] + x[:2]]), torch.tensor(bias)
    compare(x, bias, 2, "sigmoid", 2, 1)
    compare(x[:, [1, 0, 3, 2]].contiguous(), bias[[1, 0, 3, 2]], 2, "sigmoid", 2, 1)


def cancelling(T, E, G, B, func, r):
    """One expert of each group far up, the others as far down; the scores' spread is that of
    the roundings of B (the softmax's scores are about 1 / E)."""
    n = E // G
    bias = torch.empty(G, n)
    for i in range(G):
        bias[i] = -B * (1 + i / 8)
        bias[i, i % n] = B * (1 + i / 8)
    spread = min(1.0, B * 2.0 ** -21 * (E if func == "softmax" else 1))
    return torch.randn(T, E, generator=r) * spread, bias.flatten()


CASES = [  # E, k, G, g: a warp per token and several tokens per warp
    (256, 8, 8, 4), (256, 8, 4, 1), (64, 4, 8, 2), (160, 6, 8, 3), (512, 8, 16, 4), (16, 2, 4, 1),
    (96, 6, 12, 5), (72, 4, 6, 2), (256, 32, 8, 4), (480, 30, 15, 2),
]


@pytest.mark.parametrize("func", ["sigmoid", "softmax"])
@pytest.mark.parametrize("B", [64.0, 1000.0, 2.0 ** 20])
@pytest.mark.parametrize("case", CASES)
def test_biases_of_both_signs(case, B, func):
    E, k, G, g = case
    r = gen(E + k)
    x, bias = cancelling(60, E, G, B, func, r)
    compare(x, bias, k, func, G, g)
    # as many tokens as the form with several tokens per warp takes
    T = 13 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    x, bias = cancelling(T, E, G, B, func, r)
    x[::3, 1:] = x[::3, 1:2]      # one value but for the first: more equal experts than lanes
    compare(x, bias, k, func, G, g, torch.arange(0, T, 4))


@pytest.mark.parametrize("B", [1000.0, 2.0 ** 40, 2.0 ** 99])
def test_groups_closed_by_a_bias(B):
    """A bias far down closes experts, whole groups, or all but one of a group; the others
    are selected as without it."""
    E, k, G, g = 256, 8, 8, 4
    T = 13 * torch.cuda.get_device_properties(0).multi_processor_count + 3
    r = gen(3)
    x = torch.randn(T, E, generator=r)
    bias = torch.randn(E, generator=r) * 0.05
    bias[:40] = -B               # a group and a quarter
    bias[65:96] = -B             # all but one
    bias[200:210] = -B
    for func in ("sigmoid", "softmax"):
        compare(x[:40], bias, k, func, G, g)
        compare(x, bias, k, func, G, g, torch.arange(0, T, 4))
