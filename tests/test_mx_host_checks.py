"""More of the host's refusals of the MXFP4 and balance entry points (CPU only: no call here reaches a
kernel)."""
from quantized_expert_grouped_amd import abi


def test_balance_workspace_of_more_tokens_than_the_call_takes():
    """T * K above 2^30 is refused whatever K is once T alone is above it: no workspace either."""
    assert abi.balance_workspace_size(1 << 30, 8) > 0
    for T in ((1 << 30) + 1, (1 << 31) - 1):
        assert abi.balance_workspace_size(T, 8) == 0
        p = 1 << 20
        assert abi.lib().moe_balance_loss(p, 0, 8, T, 8, p, 1, None, p, p, p, p, 1 << 30, None) == -2
