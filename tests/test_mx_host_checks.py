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


def test_balance_gradient_over_its_logits_with_other_strides():
    p = 1 << 20
    bwd = abi.lib().moe_balance_loss_backward
    for ld, ld_grad in ((64, 72), (72, 64)):
        assert bwd(p, 0, ld, 100, 64, p, 4, None, None, p, ld_grad, None) == -1
