"""The test hooks of the experts' 8-bit products (no GPU)."""
from moe_routing_precision_gb300 import _build


def test_hooks_take_and_refuse():
    _build.build()
    from moe_routing_precision_gb300 import ops
    L = ops.lib()
    for n in (0, 5, 1 << 40, -1):
        assert L.moe_debug_set(ops.DEBUG_WEIGHT_STAGES, n) == ops.MOE_OK
    assert L.moe_debug_set(ops.DEBUG_WEIGHT_STAGES, -2) == ops.MOE_ERR_INVALID_ARG


def test_form_refuses_bad_sizes():
    _build.build()
    import ctypes

    from moe_routing_precision_gb300 import ops
    f, out = ops.lib().moe_debug_matmul_int8_form, ctypes.c_int32()
    good = (8, 64, 1024, 256, 0, ctypes.byref(out))
    for i, bad in ((0, 0), (0, 1025), (1, 0), (1, 1 << 31), (2, 8), (2, 65552), (3, 0), (5, None)):
        args = list(good)
        args[i] = bad
        assert f(*args) == ops.MOE_ERR_INVALID_ARG, (i, bad)
