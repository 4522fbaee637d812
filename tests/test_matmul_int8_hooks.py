"""The test hooks of the experts' 8-bit products (no GPU)."""
from moe_routing_precision_gb300 import _build


def test_hooks_take_and_refuse():
    _build.build()
    from moe_routing_precision_gb300 import ops
    L = ops.lib()
    for n in (0, 5, 1 << 40, -1):
        assert L.moe_debug_set(ops.DEBUG_WEIGHT_STAGES, n) == ops.MOE_OK
    assert L.moe_debug_set(ops.DEBUG_WEIGHT_STAGES, -2) == ops.MOE_ERR_INVALID_ARG
