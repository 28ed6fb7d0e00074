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


class Claimed:
    """What the binding asks of a device tensor, for sizes that no test allocates."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 256


F, I = torch.float32, torch.int32
W = 1 << 32  # a 32-bit count of it is 0


@pytest.mark.parametrize("call", [
    lambda t: gdn.gdn_norm_block(t(W, 8), t(8, dtype=F), out=(None, t(W, 8), None)),
    lambda t: gdn.gdn_norm_block(t(1 << 16, 1 << 16, 8), t(8, dtype=F), out=(None, t(1 << 16, 1 << 16, 8), None)),
    lambda t: gdn.gdn_norm_block(t(1, W + 8), t(W + 8, dtype=F), out=(None, t(1, W + 8), None)),
    lambda t: gdn.gdn_norm_block_backward(t(W, 8), t(W, 8), t(8, dtype=F), t(W, dtype=F),
                                          out=(t(W, 8), None, t(8, dtype=F), None)),
    lambda t: gdn.gdn_norm_gate(t(W, 1, 16), t(W, 1, 16), t(16, dtype=F), out=(t(W, 1, 16), None)),
    lambda t: gdn.gdn_norm_gate(t(1, W + 1, 16), t(1, W + 1, 16), t(16, dtype=F), out=(t(1, W + 1, 16), None)),
    lambda t: gdn.gdn_norm_gate_backward(t(W, 1, 16), t(W, 1, 16), t(W, 1, 16), t(16, dtype=F), t(W, 1, dtype=F),
                                         out=(t(W, 1, 16), t(W, 1, 16), t(16, dtype=F))),
    lambda t: gdn.gdn_attn_forward(t(W, 1, 64), t(W, 1, 64), t(W, 1, 64), t(2, dtype=I), o=t(W, 1, 64), lse=t(W, 1, dtype=F)),
    lambda t: gdn.gdn_attn_forward(t(1, 1, W + 64), t(1, 1, W + 64), t(1, 1, W + 64), t(2, dtype=I), o=t(1, 1, W + 64),
                                   lse=t(1, 1, dtype=F)),
    lambda t: gdn.gdn_attn_forward(t(1, 1, 64), t(1, 1, 64), t(1, 1, 64), t(W + 2, dtype=I), o=t(1, 1, 64), lse=t(1, 1, dtype=F)),
    lambda t: gdn.gdn_attn_backward(t(W, 1, 64), t(W, 1, 64), t(W, 1, 64), t(2, dtype=I), t(W, 1, 64), t(W, 1, dtype=F), t(W, 1, 64),
                                    out=(t(W, 1, 64), t(W, 1, 64), t(W, 1, 64))),
    lambda t: gdn.gdn_attn_append(None, t(W, 1, 64), t(W, 1, 64), None, None, t(2, dtype=I), t(1, dtype=I), t(1, 4, dtype=I),
                                  t(4, 16, 1, 64), t(4, 16, 1, 64)),
    lambda t: gdn.gdn_attn_append(None, t(1, 1, 64), t(1, 1, 64), t(W + 4, 32, dtype=F), t(W + 4, 32, dtype=F), t(2, dtype=I),
                                  t(1, dtype=I), t(1, 4, dtype=I), t(4, 16, 1, 64), t(4, 16, 1, 64)),
    lambda t: gdn.gdn_attn_append(None, t(1, 1, 64), t(1, 1, 64), None, None, t(2, dtype=I), t(1, dtype=I), t(1, W + 4, dtype=I),
                                  t(4, 16, 1, 64), t(4, 16, 1, 64)),
    lambda t: gdn.gdn_attn_append(None, t(1, 1, 64), t(1, 1, 64), None, None, t(2, dtype=I), t(1, dtype=I), t(1, 4, dtype=I),
                                  t(W + 4, 16, 1, 64), t(W + 4, 16, 1, 64)),
    lambda t: gdn.gdn_attn_paged(t(W, 1, 64), t(4, 16, 1, 64), t(4, 16, 1, 64), t(1, 4, dtype=I), t(2, dtype=I), t(1, dtype=I),
                                 o=t(W, 1, 64)),
    lambda t: gdn.gdn_attn_paged(t(1, 1, 64), t(4, W + 16, 1, 64), t(4, W + 16, 1, 64), t(1, 4, dtype=I), t(2, dtype=I),
                                 t(1, dtype=I), o=t(1, 1, 64)),
])
def test_binding_refuses_counts_past_an_int(call):
    """The shapes of the C ABI hold 32-bit counts; one that does not fit is refused
    instead of losing its high bits."""
    with pytest.raises(ValueError, match="at most 2147483647"):
        call(Claimed)
