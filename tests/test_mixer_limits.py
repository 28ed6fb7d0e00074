"""Host side: how many sequences a call of the state-space layer's operators may have."""
import gated_delta_rule_52_amd as gdn
from test_block_abi import P
from test_mixer_abi import conv, conv_backward, conv_forward


def test_convolution_sequences_at_the_limit():
    """Every strip of a packed call looks for its sequence along the bounds; single
    tokens have none (refused below for the state that is not given, not for their number)."""
    size = gdn.lib().gdn_conv_workspace_bytes
    assert size(conv(B=65536)) > 0 and size(conv(B=65537)) == 0
    assert conv_forward(conv(B=65537)) == conv_backward(conv(B=65537)) == 2
    assert gdn.lib().gdn_conv_step(conv(B=65537, T=65537), P, P, None, None, P, None) == 1
    assert gdn.lib().gdn_conv_step(conv(B=(1 << 25) + 1, T=(1 << 25) + 1), P, P, None, None, P, None) == 2
