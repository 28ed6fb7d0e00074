"""Sequence bounds outside the rows mean the same to every call: they are clamped
to 0 <= start <= end <= T."""
import pytest
import torch

from test_gpu_attention import DT, ints, make_cache, qkv, rand

pytestmark = pytest.mark.gpu

OUTSIDE = [  # bounds as given, and what they are clamped to, for 50 rows
    ([-5, 20, 9999], [0, 20, 50]), ([0, 9999], [0, 50]), ([-9, -3, 50], [0, 0, 50]), ([0, 30, 60, 90], [0, 30, 50, 50]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("given,inside", OUTSIDE, ids=str)
def test_append_clamps(dtype, given, inside):
    """A sequence's new tokens are the rows between its clamped bounds, so their
    positions count back from kv_len by that number, as in the attention."""
    import gated_delta_rule_52_amd as gdn
    dt, T, B = DT[dtype], 50, len(given) - 1
    q, k, v = qkv(T, 4, 2, 64, dt, True)
    whole = [b - a + 7 for a, b in zip(inside[:-1], inside[1:])]
    kc, vc, table = make_cache(whole, 16, 2, 64, dt, poison=3.0)
    ang = torch.rand(128, 32, generator=torch.Generator().manual_seed(3))
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    got = []
    for cu in (given, inside):
        k1, v1 = kc.clone(), vc.clone()
        qo = torch.full((T, 4, 64), 5.0, dtype=dt, device="cuda")
        gdn.gdn_attn_append(q, k, v, cos, sin, ints(cu), ints(whole), table, k1, v1, q_out=qo)
        got.append((qo, k1, v1, gdn.gdn_attn_paged(qo, k1, v1, table, ints(cu), ints(whole))))
    torch.cuda.synchronize()
    assert len(whole) == B and not torch.equal(got[1][1], kc)
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("given,inside", OUTSIDE, ids=str)
def test_prompt_and_gradients_clamp(dtype, given, inside):
    import gated_delta_rule_52_amd as gdn
    q, k, v = qkv(50, 4, 2, 64, DT[dtype], False)
    dO = rand(50, 4, 64, dtype=DT[dtype], seed=4)
    got = []
    for cu in (given, inside):
        o, lse = gdn.gdn_attn_forward(q, k, v, ints(cu))
        got.append((o, lse) + gdn.gdn_attn_backward(q, k, v, ints(cu), o, lse, dO))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)
