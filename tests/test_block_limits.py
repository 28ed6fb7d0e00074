"""Sizes at and past the limits of the operators around the layer: refused before
any launch (no pointer below is ever followed, and no call below is accepted)."""
import ctypes

import pytest
import torch

import gated_delta_rule_52_amd as gdn
from test_block_abi import BIG, P, attn


@pytest.mark.parametrize("T", [(1 << 25) - 1, 1 << 25, (1 << 26) - 1])
def test_append_tokens_of_one_launch(T):
    """Two tokens a workgroup of 256: from 2^25 - 1 tokens on that is 2^32 work-items,
    more than a launch can have."""
    sh = attn(T=T, Hq=1, Hkv=1)
    assert gdn.lib().gdn_attn_append(sh, P, P, P, P, P, P, P, P, P, P, P, None) == 2
