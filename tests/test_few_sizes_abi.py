"""The workspace of ep_moe_few, to the byte (no GPU needed: calls that are refused launch nothing)."""
import pytest

from combine_get_dispatch_gb300 import ep
from test_few_newton_abi import few


@pytest.mark.parametrize("R,T_r,k,I", [(2, 4, 2, 128), (1, 1, 1, 8), (1, 32, 4, 72), (1, 33, 4, 72), (1, 64, 2, 2048), (4, 16, 2, 1416)])
def test_workspace_to_the_byte(R, T_r, k, I):
    size = ep.ep_moe_few_workspace_size(R, T_r, k, 4, I)
    assert size == R * T_r * k * I * 4   # h: two words of 16 bits, or one of 32
    before = ep.ep_launch_count()
    assert few(R=R, T_r=T_r, k=k, I=I, size=size - 1) == ep.EP_ERR_INVALID_ARG
    assert ep.ep_launch_count() == before
