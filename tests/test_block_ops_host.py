"""Host-side rules of the operators around the routed experts (no GPU)."""
import pytest

from moe_routing_precision_gb300 import _build


@pytest.fixture(scope="module")
def L():
    _build.build()
    from moe_routing_precision_gb300 import ops
    return ops.lib()


@pytest.mark.parametrize("T,E,S,table", [
    (16384, 1, 1, True), (5461, 3, 1, True), (963, 17, 1, True), (496, 33, 1, True),
    (16384, 1, 4, True), (963, 17, 100, True),       # too long for any one block
    (64, 16, 1, False), (64, 256, 1, False), (128, 17, 1, False), (129, 17, 1, True),
    (496, 33, 4, False), (513, 17, 4, True), (16, 1024, 1, False), (17, 1024, 1, True),
    # eight passes with 16-byte aligned rows, 64 without: the table's size is named
    (1024, 16, 1, True), (128, 16, 1, False)])
def test_balance_loss_workspace_follows_the_passes_of_a_block(L, T, E, S, table):
    """One block walks a sequence's tokens 16 warps at a time (4 to 32 lanes a token):
    beyond eight passes for each of up to four sequences the table is faster."""
    assert (L.moe_balance_loss_workspace_bytes(T, E, S) > 0) == table
