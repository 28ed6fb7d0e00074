"""Host side of the operators around the layer: refusals before any launch (no
pointer below is ever followed), workspace sizes, and the plain forms' gradients
against differences."""
import ctypes

import pytest
import torch

import block_reference as ref
import gated_delta_rule_52_amd as gdn

P, MIS = ctypes.c_void_p(256), ctypes.c_void_p(264)
BIG = 1 << 40


def norm(**kw):
    d = dict(tokens=4, heads=1, width=64, dtype=0, eps=1e-6, gate_stride=0)
    d.update(kw)
    return ctypes.byref(gdn.GdnNormShape(*d.values()))


def attn(**kw):
    d = dict(B=2, T=8, Hq=4, Hkv=2, D=64, dtype=1, scale=0.0, q_stride=0, k_stride=0, v_stride=0, num_pages=4,
             page_size=16, max_pages=2, rot_dim=64, max_pos=32)
    d.update(kw)
    return ctypes.byref(gdn.GdnAttnShape(*d.values()))


def block(sh, x=P, y=None, a=None, w=P, h=None, n=P, r=None):
    return gdn.lib().gdn_norm_block(sh, x, y, a, w, h, n, r, None)


def test_structs_match_the_header():
    # natural alignment of the declared fields
    assert ctypes.sizeof(gdn.GdnNormShape) == 32
    assert ctypes.sizeof(gdn.GdnAttnShape) == 80


@pytest.mark.parametrize("bad,code", [
    (dict(tokens=-1), 1), (dict(heads=2), 1), (dict(width=0), 1), (dict(dtype=2), 1), (dict(eps=0.0), 1),
    (dict(eps=float("nan")), 1), (dict(gate_stride=64), 1), (dict(width=66), 2), (dict(width=8200), 2),
    (dict(width=4, dtype=1), 2), (dict(tokens=1 << 30), 2),
])
def test_norm_block_refusals(bad, code):
    assert block(norm(**bad)) == code
    assert gdn.lib().gdn_norm_workspace_bytes(norm(**bad), 0) == 0


def test_norm_block_pointers():
    L = gdn.lib()
    assert block(norm(), x=None) == 1 and block(norm(), w=None) == 1 and block(norm(), n=None) == 1
    assert block(norm(), a=P) == 1  # a scale and nothing to scale
    assert block(norm(), x=MIS) == 3 and block(norm(), y=P, h=MIS) == 3
    assert block(norm(tokens=0)) == 0
    sh = norm()
    back = lambda dy, da, ws, n: L.gdn_norm_block_backward(sh, P, None, P, P, P, P, P, P, dy, P, da, ws, n, None)
    assert back(None, P, P, BIG) == 1 and back(P, None, P, BIG) == 1
    assert back(P, P, None, BIG) == 4 and back(P, P, P, 16) == 4
    assert back(P, P, MIS, BIG) == 3


@pytest.mark.parametrize("bad,code", [
    (dict(width=48), 2), (dict(width=256), 2), (dict(heads=0), 1), (dict(gate_stride=-4), 1),
    (dict(heads=2, gate_stride=64), 1), (dict(gate_stride=66), 3), (dict(tokens=1 << 24, heads=64), 2),
])
def test_norm_gate_refusals(bad, code):
    assert gdn.lib().gdn_norm_gate(norm(**bad), P, P, P, P, None, None) == code
    assert gdn.lib().gdn_norm_workspace_bytes(norm(**bad), 1) == 0


def test_norm_gate_pointers():
    L = gdn.lib()
    assert L.gdn_norm_gate(norm(), P, None, P, P, None, None) == 1
    assert L.gdn_norm_gate(norm(), P, MIS, P, P, None, None) == 3
    assert L.gdn_norm_gate(norm(tokens=0), None, None, None, None, None, None) == 0
    assert L.gdn_norm_gate_backward(norm(), P, P, P, P, P, P, P, None, P, BIG, None) == 1
    assert L.gdn_norm_gate_backward(norm(), P, P, P, P, P, P, P, P, P, 16, None) == 4


SHAPES = [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(dtype=3), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(D=80), 2), (dict(D=256), 2), (dict(q_stride=128), 1), (dict(k_stride=-8), 1),
    (dict(q_stride=260), 3), (dict(v_stride=1 << 25), 2), (dict(Hq=2048), 2), (dict(T=1 << 26), 2),
]
PAGES = [
    (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(page_size=0), 1), (dict(page_size=8), 2),
    (dict(page_size=48), 2), (dict(page_size=2048), 2), (dict(max_pages=1 << 27), 2),
]


@pytest.mark.parametrize("bad,code", SHAPES)
def test_prompt_refusals(bad, code):
    L = gdn.lib()
    assert L.gdn_attn_forward(attn(**bad), P, P, P, P, P, P, None) == code
    assert L.gdn_attn_backward(attn(**bad), P, P, P, P, P, P, P, P, P, P, P, BIG, None) == code
    assert L.gdn_attn_workspace_bytes(attn(**bad), gdn.GDN_ATTN_BACKWARD) == 0


@pytest.mark.parametrize("bad,code", SHAPES + PAGES)
def test_paged_refusals(bad, code):
    L = gdn.lib()
    assert L.gdn_attn_paged(attn(**bad), P, P, P, P, P, P, P, P, BIG, None) == code
    assert L.gdn_attn_workspace_bytes(attn(**bad), gdn.GDN_ATTN_PAGED) == 0


@pytest.mark.parametrize("bad,code", SHAPES + PAGES + [(dict(rot_dim=24), 1), (dict(rot_dim=128), 1),
                                                        (dict(rot_dim=-16), 1), (dict(max_pos=0), 1)])
def test_append_refusals(bad, code):
    assert gdn.lib().gdn_attn_append(attn(**bad), P, P, P, P, P, P, P, P, P, P, P, None) == code


def test_attention_pointers():
    L = gdn.lib()
    sh = attn()
    assert L.gdn_attn_forward(sh, None, P, P, P, P, P, None) == 1
    assert L.gdn_attn_forward(sh, P, P, P, None, P, P, None) == 1
    assert L.gdn_attn_forward(sh, P, MIS, P, P, P, P, None) == 3
    assert L.gdn_attn_forward(sh, P, P, P, ctypes.c_void_p(258), P, P, None) == 3
    assert L.gdn_attn_forward(attn(T=0), None, None, None, None, None, None, None) == 0
    assert L.gdn_attn_backward(sh, P, P, P, P, P, None, P, P, P, P, P, BIG, None) == 1
    assert L.gdn_attn_backward(sh, P, P, P, P, P, P, P, P, P, P, P, 16, None) == 4
    assert L.gdn_attn_append(sh, P, P, P, P, P, P, P, P, P, P, None, None) == 1  # q without q_out
    assert L.gdn_attn_append(sh, P, P, P, None, P, P, P, P, P, P, P, None) == 1
    assert L.gdn_attn_append(sh, P, P, P, P, P, P, P, P, MIS, P, P, None) == 3
    assert L.gdn_attn_paged(sh, P, P, P, None, P, P, P, P, BIG, None) == 1
    # two sequences of up to 65536 positions: the key axis is split, which takes a workspace
    long = attn(T=2, max_pages=4096)
    assert L.gdn_attn_workspace_bytes(long, gdn.GDN_ATTN_PAGED) > 256
    assert L.gdn_attn_paged(long, P, P, P, P, P, P, P, P, 256, None) == 4
    assert L.gdn_attn_workspace_bytes(sh, 7) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        gdn.gdn_norm_block(x, torch.ones(64))
    with pytest.raises(TypeError):
        gdn.gdn_norm_block(x.half(), torch.ones(64))
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(torch.zeros(2, 2, 64), torch.zeros(2, 2, 64), torch.zeros(2, 2, 64),
                             torch.tensor([0, 2], dtype=torch.int32))


def differences(f, args, grads, eps=1e-6):
    """Central differences of f along one direction per argument, in 64 bits."""
    g = torch.Generator().manual_seed(5)
    for i, (x, dx) in enumerate(zip(args, grads)):
        u = torch.randn(x.shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = x + eps * u, x - eps * u
        d = (f(*up) - f(*down)) / (2 * eps)
        want = (dx * u).sum()
        # truncation eps^2, cancellation 2^-52 / eps
        assert abs(d - want) <= 1e-7 * (1 + abs(want) + dx.abs().sum()), i


def test_plain_gradients_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    x, y, w, a, dn, dh = r(5, 16), r(5, 16), r(16), r(16), r(5, 16), r(5, 16)

    def loss(x, y, w, a):
        h, n, _ = ref.norm_block(x, w, y, a)
        return (n * dn).sum() + (h * dh).sum()

    dx, dy, dw, da = ref.norm_block_backward(dn, dh, x, w, y, a)
    differences(loss, (x, y, w, a), (dx, dy, dw, da))
    o, z, w = r(3, 2, 16), r(3, 2, 16), r(16)
    dy = r(3, 2, 16)
    differences(lambda o, z, w: (ref.norm_gate(o, z, w)[0] * dy).sum(), (o, z, w), ref.norm_gate_backward(dy, o, z, w))
    q, k, v, do = r(7, 8), r(7, 8), r(7, 8), r(7, 8)
    see = torch.ones(7, 7, dtype=torch.bool).tril()
    f = lambda q, k, v: (ref.attention_head(q, k, v, see, 0.3)[0] * do).sum()
    o, lse = ref.attention_head(q, k, v, see, 0.3)[:2]
    back = ref.attention_head_backward(q, k, v, see, 0.3, o, lse, do)
    differences(f, (q, k, v), [back[n][0] for n in ("dq", "dk", "dv")])
