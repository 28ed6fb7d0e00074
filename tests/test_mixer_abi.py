"""Host side of the state-space layer's operators and of the page step: refusals
before any launch (no pointer below is ever followed), workspace sizes, and the
plain forms against one another and against differences."""
import ctypes

import pytest
import torch

import gated_delta_rule_52_amd as gdn
import mixer_reference as ref
from test_block_abi import BIG, MIS, P, differences

Q = ctypes.c_void_p(512)
ODD = ctypes.c_void_p(258)


def conv(**kw):
    d = dict(B=2, T=8, C=64, W=4, dtype=1, silu=1, x_stride=0)
    d.update(kw)
    return ctypes.byref(gdn.GdnConvShape(*d.values()))


def ssm(**kw):
    d = dict(B=2, T=8, H=4, G=2, N=64, P=64, dtype=1, softplus=1, x_stride=0, b_stride=0, c_stride=0)
    d.update(kw)
    return ctypes.byref(gdn.GdnSsmShape(*d.values()))


def pages(**kw):
    d = dict(B=2, num_pages=8, page_size=16, max_pages=4, rows=32)
    d.update(kw)
    return ctypes.byref(gdn.GdnPagesShape(*d.values()))


def test_structs_match_the_header():
    assert ctypes.sizeof(gdn.GdnConvShape) == 32
    assert ctypes.sizeof(gdn.GdnSsmShape) == 56
    assert ctypes.sizeof(gdn.GdnPagesShape) == 20


def conv_forward(sh, x=P, w=P, b=None, cu=P, s=None, y=Q, o=None):
    return gdn.lib().gdn_conv_forward(sh, x, w, b, cu, s, y, o, None)


def conv_backward(sh, x=P, w=P, cu=P, dy=P, dx=Q, dw=P, ws=P, n=BIG):
    return gdn.lib().gdn_conv_backward(sh, x, w, None, cu, None, dy, None, dx, dw, None, None, ws, n, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(C=0), 1), (dict(dtype=2), 1), (dict(silu=2), 1), (dict(x_stride=-8), 1),
    (dict(x_stride=56), 1), (dict(W=1), 2), (dict(W=5), 2), (dict(C=60), 2), (dict(C=6, dtype=0), 2), (dict(x_stride=68), 3),
    (dict(C=(1 << 20) + 8), 2), (dict(T=(1 << 28) + 1), 2), (dict(B=(1 << 25) + 1), 2),
])
def test_conv_refusals(bad, code):
    assert conv_forward(conv(**bad)) == code
    assert conv_backward(conv(**bad)) == code
    assert gdn.lib().gdn_conv_workspace_bytes(conv(**bad)) == 0


def test_conv_pointers():
    sh, L = conv(), gdn.lib()
    for k in ("x", "w", "cu", "y"):
        assert conv_forward(sh, **{k: None}) == 1, k
    for k in ("x", "w", "b", "s", "y", "o"):
        assert conv_forward(sh, **{k: MIS}) == 3, k
    assert conv_forward(sh, cu=ODD) == 3
    assert conv_forward(sh, y=P) == 1  # y is x
    for k in ("x", "w", "cu", "dy", "dx", "dw"):
        assert conv_backward(sh, **{k: None}) == 1, k
    assert conv_backward(sh, dx=P) == 1  # dx is x and dy
    assert conv_backward(sh, ws=None) == 4 and conv_backward(sh, n=16) == 4 and conv_backward(sh, ws=MIS) == 3
    assert L.gdn_conv_step(sh, P, P, None, P, Q, None) == 1  # T is not B
    one = conv(T=2)
    assert L.gdn_conv_step(one, P, P, None, None, Q, None) == 1
    assert L.gdn_conv_step(one, P, P, None, MIS, Q, None) == 3
    assert L.gdn_conv_step(one, P, P, None, P, P, None) == 1


SCANS = [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(H=3), 1), (dict(G=0), 1), (dict(dtype=3), 1), (dict(softplus=2), 1),
    (dict(N=32), 2), (dict(N=256), 2), (dict(P=32), 2), (dict(P=192), 2), (dict(x_stride=128), 1), (dict(b_stride=-8), 1),
    (dict(x_stride=260), 3), (dict(c_stride=1 << 25), 2), (dict(H=2048), 2), (dict(T=1 << 26), 2), (dict(B=1 << 22), 2),
]


def ssm_forward(sh, x=P, dt=P, A=P, B=P, C=P, cu=P, h0=None, y=P, hT=None, ws=P, n=BIG):
    return gdn.lib().gdn_ssm_forward(sh, x, dt, A, B, C, None, None, cu, h0, y, hT, ws, n, None)


def ssm_backward(sh, x=P, dt=P, A=P, B=P, C=P, cu=P, dy=P, dhT=None, dx=P, ddt=P, dA=P, dB=P, dC=P, dh0=None, ws=P, n=BIG):
    return gdn.lib().gdn_ssm_backward(sh, x, dt, A, B, C, None, None, cu, None, dy, dhT, dx, ddt, dA, dB, dC, None, None, dh0, ws,
                                      n, None)


@pytest.mark.parametrize("bad,code", SCANS)
def test_scan_refusals(bad, code):
    L = gdn.lib()
    assert ssm_forward(ssm(**bad)) == code
    assert ssm_backward(ssm(**bad)) == code
    for call in (gdn.GDN_SSM_FORWARD, gdn.GDN_SSM_BACKWARD):
        assert L.gdn_ssm_workspace_bytes(ssm(**bad), call) == 0
    if "T" not in bad and "B" not in bad:
        assert L.gdn_ssm_step(ssm(T=2, **bad), P, P, P, P, P, None, None, P, P, None) == code


def test_scan_pointers():
    sh, L = ssm(), gdn.lib()
    for k in ("x", "dt", "A", "B", "C", "cu", "y"):
        assert ssm_forward(sh, **{k: None}) == 1, k
    for k in ("x", "B", "C", "h0", "y", "hT", "ws"):
        assert ssm_forward(sh, **{k: MIS}) == 3, k
    for k in ("dt", "A", "cu"):
        assert ssm_forward(sh, **{k: ODD}) == 3, k
    assert ssm_forward(sh, ws=None) == 4 and ssm_forward(sh, n=16) == 4
    for k in ("x", "dt", "A", "B", "C", "cu", "dy", "dx", "ddt", "dA", "dB", "dC"):
        assert ssm_backward(sh, **{k: None}) == 1, k
    for k in ("x", "dy", "dhT", "dx", "dB", "dC", "dh0"):
        assert ssm_backward(sh, **{k: MIS}) == 3, k
    assert ssm_backward(sh, n=16) == 4
    assert ssm_backward(sh, dhT=P, dh0=P) == 1  # the gradients read dhT after dh0 is written
    assert L.gdn_ssm_step(sh, P, P, P, P, P, None, None, P, P, None) == 1  # T is not B
    assert L.gdn_ssm_step(ssm(T=2), P, P, P, P, P, None, None, None, P, None) == 1
    assert L.gdn_ssm_step(ssm(T=2), P, P, P, P, P, None, None, MIS, P, None) == 3
    assert L.gdn_ssm_workspace_bytes(sh, 2) == 0
    few, many = ssm(T=1000), ssm(T=100000)
    size = L.gdn_ssm_workspace_bytes
    assert 0 < size(few, 0) < size(many, 0) < size(many, 1)


def test_scan_refuses_outputs_that_are_inputs():
    """A workgroup's results would be another's operands."""
    L, sh = gdn.lib(), ssm()
    at = [ctypes.c_void_p(4096 * (i + 1)) for i in range(20)]
    names = ("x", "dt", "A", "B", "C", "cu", "h0", "dy", "dhT", "dx", "ddt", "dA", "dB", "dC", "dh0", "ws")
    p = dict(zip(names, at))

    def back(**kw):
        q = dict(p, **kw)
        return L.gdn_ssm_backward(sh, q["x"], q["dt"], q["A"], q["B"], q["C"], None, None, q["cu"], q["h0"], q["dy"], q["dhT"], q["dx"],
                                  q["ddt"], q["dA"], q["dB"], q["dC"], None, None, q["dh0"], q["ws"], BIG, None)

    for out, of in (("dx", "x"), ("dx", "dy"), ("dB", "B"), ("dB", "C"), ("dC", "B"), ("dC", "C"), ("dC", "dB"), ("dh0", "h0"),
                    ("dh0", "dhT")):
        assert back(**{out: p[of]}) == 1, (out, of)
    assert ssm_forward(sh, x=at[0], y=at[0]) == 1
    assert L.gdn_ssm_step(ssm(T=2), at[0], at[1], at[2], at[3], at[4], None, None, at[5], at[0], None) == 1


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), 1), (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(page_size=0), 1), (dict(rows=-1), 1),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=2048), 2), (dict(max_pages=1 << 27), 2), (dict(B=8193), 2),
])
def test_pages_refusals(bad, code):
    L = gdn.lib()
    assert L.gdn_pages_release(pages(**bad), P, P, P, P, P, P, P, None) == code
    assert L.gdn_pages_take(pages(**bad), P, P, P, P, P, P, P, P, None, None, None) == code


def test_pages_pointers():
    L, sh = gdn.lib(), pages()
    for i in range(7):
        p = [P] * 7
        p[i] = None
        assert L.gdn_pages_release(sh, *p, None) == 1, i
        p[i] = ODD
        assert L.gdn_pages_release(sh, *p, None) == 3, i
    for i in range(8):
        p = [P] * 8
        p[i] = None
        assert L.gdn_pages_take(sh, *p, None, None, None) == 1, i
        p[i] = ODD
        assert L.gdn_pages_take(sh, *p, None, None, None) == 3, i
    assert L.gdn_pages_take(sh, *[P] * 8, None, ctypes.c_void_p(260), None) == 3


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        gdn.gdn_conv_forward(x, torch.zeros(64, 4), cu)
    with pytest.raises(ValueError):
        gdn.gdn_ssm_forward(x.view(4, 1, 64), torch.zeros(4, 1), torch.zeros(1), x.view(4, 1, 64), x.view(4, 1, 64), cu)
    with pytest.raises(ValueError):
        gdn.gdn_pages_release(cu, cu, cu.view(1, 2), cu, cu, 16)


def r(*s, seed=0):
    g = torch.Generator().manual_seed(seed + 17 * sum(s))
    return torch.randn(s, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_plain_convolution_against_differences(W, silu):
    cu, C = [0, 1, 6, 6, 9], 3
    x, w, b, s, dy, dso = r(9, C), r(C, W), r(C), r(4, W - 1, C), r(9, C, seed=1), r(4, W - 1, C, seed=2)

    def loss(x, w, b, s):
        y, _, out = ref.conv(x, w, cu, b, s, silu)
        return (y * dy).sum() + (out * dso).sum()

    ref.HALF[torch.float64] = 2.0 ** -53
    g = ref.conv_backward(x, w, cu, dy, b, s, dso, silu)
    differences(loss, (x, w, b, s), [g[n][0] for n in ("dx", "dweight", "dbias", "dstate")])


@pytest.mark.parametrize("softplus", [True, False])
def test_plain_scans_agree(softplus):
    """Pair by pair and token by token; the gradients by formula and by autograd."""
    cu, H, G, N, Pn = [0, 1, 1, 8, 14], 4, 2, 5, 3
    x, dt, Bm, Cm = r(14, H, Pn), r(14, H, seed=1), r(14, G, N), r(14, G, N, seed=1)
    A, D, bias, h0 = -r(H).abs(), r(H, seed=2), r(H, seed=3), r(4, H, N, Pn)
    if not softplus:
        dt, bias = dt.abs(), bias.abs()
    dy, dhT = r(14, H, Pn, seed=4), r(4, H, N, Pn, seed=4)
    ref.HALF[torch.float64] = 2.0 ** -53
    out = ref.ssm(x, dt, A, Bm, Cm, cu, D, bias, softplus, h0, dy, dhT)
    leaves = [t.clone().requires_grad_() for t in (x, dt, A, Bm, Cm, D, bias, h0)]
    X, DT, AA, BB, CC, DD, BI, H0 = leaves
    y, hT = ref.ssm_serial(X, DT, AA, BB, CC, cu, DD, BI, softplus, H0)
    ((y * dy).sum() + (hT * dhT).sum()).backward()
    close = lambda a, b: float((a - b).abs().max()) <= 1e-11 * (1 + float(b.abs().max()))  # noqa: E731
    assert close(out["y"][0], y.detach()) and close(out["hT"][0], hT.detach())
    for name, t in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"), leaves):
        assert close(out[name][0], t.grad), name

    def loss(*a):
        y, hT = ref.ssm_serial(a[0], a[1], a[2], a[3], a[4], cu, a[5], a[6], softplus, a[7])
        return (y * dy).sum() + (hT * dhT).sum()

    differences(loss, (x, dt, A, Bm, Cm, D, bias, h0),
                [out[k][0] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")])


def test_plain_pages():
    free, table = [5, 6, 7, 8, -1, -1], [[0, 1, -1], [2, -1, -1], [3, 4, -1]]
    kv, count, free = ref.pages_release([0, 0, 1], [20, 16, 17], table, free, 4, 16)
    assert (kv, count, free) == ([20, 16, 0], 6, [5, 6, 7, 8, 3, 4])
    kv, count, table, cu, pos, slots = ref.pages_take([1, 2, 40], kv, table, free, count, 16, 64)
    assert kv == [21, 18, 40] and count == 2 and cu == [0, 1, 3, 43]
    assert table == [[0, 1, -1], [2, 4, -1], [3, 8, 7]]
    assert pos[:4] == [20, 16, 17, 0] and slots[:4] == [20, 64, 65, 48] and slots[-1] == 7 * 16 + 7


def test_scan_sequences_at_the_limit():
    """Every workgroup of the packed calls looks for its chunk along the bounds."""
    size = gdn.lib().gdn_ssm_workspace_bytes
    assert size(ssm(B=65537, H=1, G=1), 0) == size(ssm(B=65537, H=1, G=1), 1) == 0
    assert size(ssm(B=65536, H=1, G=1), 0) > 0 and size(ssm(B=65536, H=1, G=1), 1) > 0
    assert ssm_forward(ssm(B=65537, H=1, G=1)) == ssm_backward(ssm(B=65537, H=1, G=1)) == 2
