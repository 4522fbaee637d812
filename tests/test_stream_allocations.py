"""Tensors that a call allocates for itself while its kernels run on a stream named by
`stream` that is not the current one (no GPU needed: the allocations, the streams
and the library are stand-ins that record).

Each such tensor belongs to the stream its kernels run on, so that neither an
earlier user of its memory nor a later one can meet them, and the caller's
stream is recorded on it, so that it is not reused before that stream is done
with it."""
import contextlib

import pytest
import torch

from moe_routing_precision_gb300 import ops

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Recorder:
    def __init__(self):
        self.current = FakeStream(0x10)
        self.made, self.recorded, self.calls = [], [], []

    def allocator(self, real):
        def f(*a, **kw):
            t = real(*a, **kw)
            self.made.append((t, self.current.cuda_stream))
            return t
        return f

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def __getattr__(self, name):                 # the library
        def f(*a):
            if name.endswith("_bytes"):
                return 512
            self.calls.append((name, a))
            return 0
        return f


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(ops, "lib", lambda: r)
    monkeypatch.setattr(ops, "_dev", lambda t, *a: t)
    monkeypatch.setattr(ops, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: r.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "stream", r.stream)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: r.recorded.append((t, s.cuda_stream)), raising=False)
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, r.allocator(getattr(torch, name)))
    for f in (ops.block_norm_backward_workspace_bytes, ops.balance_loss_workspace_bytes):
        f.cache_clear()
    yield r
    for f in (ops.block_norm_backward_workspace_bytes, ops.balance_loss_workspace_bytes):
        f.cache_clear()


T, H, E, K = 6, 256, 8, 2


def _t(*shape, dtype=F32):
    return torch.ones(shape, dtype=dtype)


CALLS = {
    "topk_gate": lambda s: ops.topk_gate(_t(T, E), K, stream=s),
    "route_map": lambda s: ops.route_map(_t(T, K, dtype=I32), E, stream=s),
    "route_map_aligned": lambda s: ops.route_map_aligned(_t(T, K, dtype=I32), E, 8, stream=s),
    "expand_cast_fp8": lambda s: ops.expand_cast_fp8(_t(T, H, dtype=BF), _t(T, K, dtype=I32),
                                                     stream=s),
    "expand_cast_fp8_padded": lambda s: ops.expand_cast_fp8_padded(
        _t(T, H, dtype=BF), _t(T, K, dtype=I32), _t(20, dtype=I32), stream=s),
    "expand_cast_fp8_ex": lambda s: ops.expand_cast_fp8_ex(
        _t(T, H, dtype=BF), _t(T, K, dtype=I32), sorted_src=_t(T * K, dtype=I32),
        sf_flags=ops.SF_COLMAJOR, workspace=True, stream=s),
    "expand_cast_fp4": lambda s: ops.expand_cast_fp4(
        _t(T, H, dtype=BF), _t(T, K, dtype=I32), sorted_src=_t(T * K, dtype=I32),
        sf_flags=ops.SF_COLMAJOR, workspace=True, stream=s),
    "swiglu_cast_fp8": lambda s: ops.swiglu_cast_fp8(_t(T, 2 * H, dtype=BF), stream=s),
    "swiglu_cast_fp8_ex": lambda s: ops.swiglu_cast_fp8_ex(_t(T, 2 * H, dtype=BF), stream=s),
    "swiglu_cast_fp4": lambda s: ops.swiglu_cast_fp4(_t(T, 2 * H, dtype=BF), stream=s),
    "route_expand_cast_fp8": lambda s: ops.route_expand_cast_fp8(_t(T, E), _t(T, H, dtype=BF), K,
                                                                 stream=s),
    "combine": lambda s: ops.combine(_t(T * K, H, dtype=BF), _t(T, K), _t(T, K, dtype=I32),
                                     stream=s),
    "debug_cvt": lambda s: ops.debug_cvt(_t(40), ops.CVT_E4M3, stream=s),
    "block_norm": lambda s: ops.block_norm(_t(T, H), _t(T, H, dtype=BF), post_weight=_t(H),
                                           pre_weight=_t(H), stream=s),
    "block_norm_alone": lambda s: ops.block_norm(_t(T, H), pre_weight=_t(H), stream=s),
    "block_norm_backward": lambda s: ops.block_norm_backward(
        _t(T, H), _t(T, H, dtype=BF), _t(T, H), y=_t(T, H, dtype=BF), post_weight=_t(H), gate=_t(H),
        pre_weight=_t(H), rstd_post=_t(T), rstd_pre=_t(T), stream=s),
    "balance_loss": lambda s: ops.balance_loss(_t(T, E), _t(T, K, dtype=I32), stream=s),
    "balance_loss_backward": lambda s: ops.balance_loss_backward(
        _t(T, E), _t(1, E, dtype=I32), _t(1, dtype=I32), _t(1), k=K, stream=s),
    "combine_backward": lambda s: ops.combine_backward(
        _t(T, H), _t(T * K, H, dtype=BF), _t(T, K), _t(T, K, dtype=I32), stream=s),
    "expert_matvec_fp4": lambda s: ops.expert_matvec_fp4(
        _t(T, H, dtype=BF), _t(1, 16, H // 2, dtype=U8), _t(1, 16, H // 32), stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("form", ["stream", "handle", "default"])
def test_belong_to_the_named_stream(rec, name, form):
    named = {"stream": FakeStream(0x20), "handle": 0x20, "default": 0}[form]
    CALLS[name](named)
    handle = 0 if form == "default" else 0x20
    assert len(rec.calls) == 1 and rec.calls[0][1][-1] == (handle or None)
    assert rec.made
    for t, s in rec.made:
        assert s == handle, "allocated on the caller's stream, used on the named one"
        assert any(u is t and r == 0x10 for u, r in rec.recorded)
    assert rec.current.cuda_stream == 0x10


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("named", [None, 0x10])
def test_are_plain_on_the_current_stream(rec, name, named):
    CALLS[name](named)
    assert rec.made and all(s == 0x10 for _, s in rec.made) and not rec.recorded
    assert rec.calls[0][1][-1] == 0x10
