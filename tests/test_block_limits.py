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


@pytest.mark.parametrize("B", [0x7fffffff, 0x7fffffff - 1000])
def test_sequences_near_the_last_int(B):
    """The blocks of a call are more than an int holds: too many, not fewer than none."""
    L = gdn.lib()
    sh = attn(B=B, T=1 << 20)
    assert L.gdn_attn_workspace_bytes(sh, gdn.GDN_ATTN_PAGED) == 0
    assert L.gdn_attn_workspace_bytes(sh, gdn.GDN_ATTN_BACKWARD) == 0
    assert L.gdn_attn_forward(sh, P, P, P, P, P, P, None) == 2
    assert L.gdn_attn_paged(sh, P, P, P, P, P, P, P, P, BIG, None) == 2
    assert L.gdn_attn_backward(sh, P, P, P, P, P, P, P, P, P, P, P, BIG, None) == 2


@pytest.mark.parametrize("shape", [
    dict(T=(1 << 27) - 1, Hq=1, Hkv=1, D=128),        # a row by 32 lanes, to the last of 2^32 work-items
    dict(T=((1 << 27) - 1) // 7, Hq=7, Hkv=1, D=128),
    dict(B=1 << 23, T=1 << 20, Hq=1, Hkv=1),          # blocks of keys and of queries in one launch
    dict(B=1 << 22, T=1 << 20, Hq=2, Hkv=2),
])
def test_fp32_gradients_of_one_launch(shape):
    """The fp32 backward's two launches (a row's delta, and both gradient passes in
    one) stay below 2^32 work-items or the call is refused."""
    L = gdn.lib()
    sh = attn(dtype=0, **shape)
    assert L.gdn_attn_workspace_bytes(sh, gdn.GDN_ATTN_BACKWARD) == 0
    assert L.gdn_attn_backward(sh, P, P, P, P, P, P, P, P, P, P, P, BIG, None) == 2


@pytest.mark.parametrize("shape", [
    dict(dtype=0, T=(1 << 27) - 8, Hq=1, Hkv=1, D=128), dict(dtype=0, T=(1 << 27) - 1, Hq=1, Hkv=1, D=64),
    dict(dtype=1, T=(1 << 27) - 1, Hq=1, Hkv=1, D=128), dict(dtype=1, B=1 << 23, T=1 << 20, Hq=1, Hkv=1),
    dict(dtype=0, B=1 << 22, T=1 << 20, Hq=1, Hkv=1),
])
def test_gradients_below_the_limit(shape):
    assert gdn.lib().gdn_attn_workspace_bytes(attn(**shape), gdn.GDN_ATTN_BACKWARD) > 0
