"""What the C ABI of the products grouped by expert refuses, each limit by itself: every other argument is one that it
takes, so that only the check in question can refuse (fake addresses, never read: every call returns before a launch)."""
import pytest

from quantized_routed_moe_router_amd import binding as B
from test_grouped_cpu import dims, dx


@pytest.mark.parametrize("T,k", [(1000, 2), (1, 1), (70000, 8)])
def test_workspace_of_no_positions(T, k):
    """Tokens without positions: their places have to be told apart from others' all the same."""
    d = dims(rows=0, tokens=T, top_k=k)
    need = B.lib().ds4moe_grouped_workspace_bytes(d)
    assert need >= 4 * T * k
    assert dx(d, n=need - 1) == B.DS4MOE_ERR_WORKSPACE
    assert B.lib().ds4moe_grouped_workspace_bytes(dims(rows=0, tokens=0)) > 0
