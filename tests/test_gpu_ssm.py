"""The selective state space scan against the plain 64-bit form, within the bounds
that mixer_reference.py derives."""
import pytest
import torch

import mixer_reference as ref
from gpu_util import log
from mixer_reference import worst
from test_gpu_attention import DT, NAN, cumulate, ints, rand

pytestmark = pytest.mark.gpu

GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")


def make(T, B, H, G, N, P, dt, fused=True, decay=1.0):
    """Inputs as a convolution and a projection give them; A down to -16 decay."""
    if fused:  # slices of one tensor
        xbc = rand(T, H * P + 2 * G * N, dtype=dt)
        x = xbc[:, :H * P].unflatten(1, (H, P))
        Bm, Cm = (xbc[:, H * P + i * G * N:H * P + (i + 1) * G * N].unflatten(1, (G, N)) for i in (0, 1))
    else:
        x, Bm, Cm = rand(T, H, P, dtype=dt), rand(T, G, N, dtype=dt, seed=1), rand(T, G, N, dtype=dt, seed=2)
    return dict(x=x, dt=rand(T, H, std=0.5, seed=3), A=-torch.linspace(1, 16, H, device="cuda") * decay, B=Bm, C=Cm,
                D=rand(H, seed=4), dt_bias=torch.linspace(-5, -2, H, device="cuda"), h0=rand(B, H, N, P, seed=5),
                dy=rand(T, H, P, dtype=dt, seed=6), dhT=rand(B, H, N, P, std=0.3, seed=7))


def forward(s, cu, **kw):
    import gated_delta_rule_52_amd as gdn
    return gdn.gdn_ssm_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], ints(cu), D=s["D"], dt_bias=s["dt_bias"], h0=s["h0"], **kw)


def backward(s, cu, **kw):
    import gated_delta_rule_52_amd as gdn
    return gdn.gdn_ssm_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], ints(cu), s["dy"], D=s["D"], dt_bias=s["dt_bias"],
                                h0=s["h0"], dhT=s["dhT"], **kw)


def blank(s, dt):
    like = dict(zip(GRADS, (s[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0"))))
    return tuple(None if t is None else torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in like.values())


LENS = [[1], [2, 1, 3], [0, 63, 64, 65, 0], [127, 128, 129, 1], [300, 31, 33], [0, 0]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,N,P,state", [(2, 1, 64, 64, True), (2, 2, 128, 64, False), (3, 1, 64, 128, False), (4, 2, 128, 128, True)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_scan(dtype, H, G, N, P, state, lens):
    dt, cu, B = DT[dtype], cumulate(lens), len(lens)
    n, T = cu[-1], cu[-1] + 3  # rows behind the last sequence
    log(f"scan {dtype} H={H} G={G} N={N} P={P} state={state} {lens}")
    s = make(T, B, H, G, N, P, dt, fused=H != 3)
    if not state:
        s["h0"] = s["dhT"] = None
    for k in ("x", "B", "C", "dy", "dt"):
        s[k][n:] = NAN
    y = torch.full((T, H, P), 7.0, dtype=dt, device="cuda")
    hT = torch.full((B, H, N, P), 7.0, device="cuda")
    forward(s, cu, y=y, hT=hT)
    out = blank(s, dt)
    backward(s, cu, out=out)
    first = [None if t is None else t.clone() for t in out]
    backward(s, cu, out=out)
    torch.cuda.synchronize()
    assert all(a is None or torch.equal(a, b) for a, b in zip(first, out))
    got = dict(zip(GRADS, out), y=y, hT=hT)
    for k in ("y", "dx", "ddt", "dB", "dC"):
        assert (got[k][n:] == 7.0).all(), f"{k}: a row of no sequence was written"
        got[k] = got[k][:n]
    want = ref.ssm(s["x"][:n], s["dt"][:n], s["A"], s["B"][:n], s["C"][:n], cu, s["D"], s["dt_bias"], True, s["h0"],
                   s["dy"][:n], s["dhT"])
    errs = {k: worst(v, *want[k]) for k, v in got.items() if v is not None}
    log("  " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,H,G,N,P", [([2500, 40, 700], 4, 1, 128, 64), ([1700], 8, 2, 64, 64), ([513, 1025, 129], 2, 1, 128, 128)])
def test_scan_long(dtype, lens, H, G, N, P):
    """Several segments a sequence, and a group's heads in one part or more."""
    dt, cu, B = DT[dtype], cumulate(lens), len(lens)
    log(f"long scan {dtype} {lens} H={H} G={G} N={N} P={P}")
    s = make(cu[-1], B, H, G, N, P, dt)
    got = dict(zip(GRADS, backward(s, cu)))
    got["y"], got["hT"] = forward(s, cu)
    torch.cuda.synchronize()
    want = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["D"], s["dt_bias"], True, s["h0"], s["dy"], s["dhT"])
    errs = {k: worst(v, *want[k]) for k, v in got.items()}
    log("  " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs
    # Float32 results of bf16 inputs are as exact as those of float32 ones: 2^-18 (64
    # roundings of fp32) in the 2-norm, where one rounding of an operand to bf16 would
    # leave 2^-9.  A sum over the tokens is off by its terms' errors, so by that share
    # of the sum of their magnitudes, not of itself: its terms may cancel.
    far = lambda k: float((got[k].cpu().double() - want[k][0]).norm())  # noqa: E731
    rel = {k: far(k) / float(want[k][0].norm()) for k in ("hT", "ddt", "dh0")}
    rel["ddt_bias"] = far("ddt_bias") / float(want["ddt"][0].abs().sum(0).norm())
    log("  " + " ".join(f"{k}={v:.1e}" for k, v in rel.items()))
    assert max(rel.values()) <= 2.0 ** -18, rel


def test_scan_strong_decay_and_no_softplus():
    """Steps that leave nothing of the state (decays of e^-100 a token), and steps
    taken as they are, zeros among them."""
    import gated_delta_rule_52_amd as gdn
    cu = [0, 150, 170]
    for decay, softplus in ((1.0, False), (400.0, True), (0.0, True)):
        s = make(170, 2, 2, 1, 64, 64, torch.float32, decay=decay)
        if not softplus:
            s["dt"], s["dt_bias"] = s["dt"].abs(), None
            s["dt"][30:50] = 0
        a = (s["x"], s["dt"], s["A"], s["B"], s["C"], ints(cu))
        kw = dict(D=s["D"], dt_bias=s["dt_bias"], softplus=softplus, h0=s["h0"])
        y, hT = gdn.gdn_ssm_forward(*a, **kw)
        got = dict(zip(GRADS, gdn.gdn_ssm_backward(*a, s["dy"], dhT=s["dhT"], **kw)), y=y, hT=hT)
        torch.cuda.synchronize()
        want = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["D"], s["dt_bias"], softplus, s["h0"], s["dy"], s["dhT"])
        errs = {k: worst(v, *want[k]) for k, v in got.items() if v is not None}
        log(f"decay {decay} softplus {softplus}: " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
        assert max(errs.values()) <= 1, errs


def test_scan_gradient_against_differences():
    """The kernels' own loss along each gradient: central differences of fp32
    outputs, summed in 64 bits.  A step that moves the loss by 1/16 of the argument's
    size leaves third derivatives of the order of its cube, below 1 % here, and
    2^-24 / h of rounding a summed output."""
    import gated_delta_rule_52_amd as gdn
    cu = ints([0, 40, 75])
    s = make(75, 2, 2, 1, 64, 64, torch.float32)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    args = [s[k].contiguous() * (0.5 if k in "BC" else 1) for k in names]
    split = lambda a: (a[:5] + [cu], dict(D=a[5], dt_bias=a[6], h0=a[7]))  # noqa: E731

    def loss(a):
        p, kw = split(a)
        y, hT = gdn.gdn_ssm_forward(*p, **kw)
        return float((y.double() * s["dy"].double()).sum() + (hT.double() * s["dhT"].double()).sum())

    p, kw = split(args)
    grads = gdn.gdn_ssm_backward(*p, s["dy"], dhT=s["dhT"], **kw)
    for i, g in enumerate(grads):
        u = g / g.norm()
        h = 2.0 ** -6
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * u, args[i] - h * u
        d, want = (loss(up) - loss(down)) / (2 * h), float((g.double() * u.double()).sum())
        log(f"  {names[i]}: {d:.6f} against {want:.6f}")
        assert abs(d - want) <= 0.01 * abs(want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,N,P", [(2, 1, 64, 64), (4, 2, 128, 64), (3, 3, 64, 128), (6, 1, 128, 128)])
def test_step(dtype, H, G, N, P):
    """Token by token against the serial recurrence in 64 bits.  A state takes four
    roundings a token of its terms' sizes, y the sum over N of them and its storage."""
    import gated_delta_rule_52_amd as gdn
    dt, B, n = DT[dtype], 5, 6
    s = make(B * n, B, H, G, N, P, dt)
    st = s["h0"].clone()
    ys = []
    for t in range(n):
        rows = slice(t * B, t * B + B)  # rows of a wider tensor: strided
        ys.append(gdn.gdn_ssm_step(s["x"][rows], s["dt"][rows], s["A"], s["B"][rows], s["C"][rows], st, D=s["D"], dt_bias=s["dt_bias"]))
    torch.cuda.synchronize()
    order = torch.arange(B * n).view(n, B).T.reshape(-1)  # sequence after sequence
    g = {k: s[k].cpu().double()[order] for k in ("x", "dt", "B", "C")}
    rest = [s[k].cpu().double() for k in ("A", "D", "dt_bias", "h0")]
    cu = [n * b for b in range(B + 1)]
    y, hT = ref.ssm_serial(g["x"], g["dt"], rest[0], g["B"], g["C"], cu, rest[1], rest[2], True, rest[3])
    ya, ha = ref.ssm_serial(g["x"].abs(), g["dt"], rest[0], g["B"].abs(), g["C"].abs(), cu, rest[1].abs(), rest[2], True, rest[3].abs())
    # the exponent of a decay is at most 8: as many more roundings
    u = ref.U32 * (14 * n + N + 8)
    errs = (worst(torch.stack(ys, 1).flatten(0, 1), y, ref.HALF[dt] * y.abs() + u * ya), worst(st, hT, u * ha))
    log(f"step {dtype} H={H} G={G} N={N} P={P}: y={errs[0]:.2f} state={errs[1]:.2f}")
    assert max(errs) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pieces(dtype):
    """A sequence at once and in pieces that carry the state in place: float32 states,
    equal up to the roundings that both are allowed."""
    dt, H, G, N, P, n = DT[dtype], 2, 1, 128, 64, 700
    s = make(n, 1, H, G, N, P, dt)
    want = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], [0, n], s["D"], s["dt_bias"], True, s["h0"])
    st, at, ys = s["h0"].clone(), 0, []
    for m in (1, 130, 64, 0, 500, 5):
        p = {k: v[at:at + m] if k in ("x", "dt", "B", "C", "dy") else v for k, v in s.items()}
        p["h0"] = st
        y, out = forward(p, [0, m], hT=st)
        assert out is st
        ys.append(y)
        at += m
    errs = worst(torch.cat(ys), *want["y"]), worst(st, *want["hT"])
    log(f"pieces {dtype}: y={errs[0]:.3f} hT={errs[1]:.3f}")
    assert max(errs) <= 1


def test_states_in_place_over_segments():
    """hT may be h0 also where a sequence is several segments."""
    s = make(3000, 2, 2, 1, 64, 64, torch.bfloat16)
    cu = [0, 2800, 3000]
    y, hT = forward(s, cu)
    st = s["h0"].clone()
    y2, _ = forward(dict(s, h0=st), cu, hT=st)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(hT, st)


def test_many_sequences():
    """More sequences than a wave has lanes, empty ones among them."""
    lens = [(7 * i) % 5 * ((i % 3) + 1) for i in range(150)]
    cu, dt = cumulate(lens), torch.bfloat16
    s = make(cu[-1], 150, 2, 1, 64, 64, dt)
    got = dict(zip(GRADS, backward(s, cu)))
    got["y"], got["hT"] = forward(s, cu)
    torch.cuda.synchronize()
    want = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["D"], s["dt_bias"], True, s["h0"], s["dy"], s["dhT"])
    errs = {k: worst(v, *want[k]) for k, v in got.items()}
    log("many: " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


def test_bounds_of_cu_are_clamped():
    s = make(200, 2, 2, 1, 64, 64, torch.bfloat16)
    for a, c in zip(forward(s, [-5, 120, 9999]) + backward(s, [-5, 120, 9999]), forward(s, [0, 120, 200]) + backward(s, [0, 120, 200])):
        assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_sequence_among_short_ones(dtype):
    """Cut into segments although the mean sequence is short."""
    lens = [1, 0, 2] * 20 + [8700 if dtype == "bf16" else 4400] + [1] * 30 + [130, 0, 3]
    cu, B = cumulate(lens), len(lens)
    s = make(cu[-1], B, 2, 1, 64, 64, DT[dtype], decay=0.1)
    got = dict(zip(GRADS, backward(s, cu)))
    got["y"], got["hT"] = forward(s, cu)
    torch.cuda.synchronize()
    want = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["D"], s["dt_bias"], True, s["h0"], s["dy"], s["dhT"])
    errs = {k: worst(v, *want[k]) for k, v in got.items()}
    log(f"one long {dtype}: " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs
    st = s["h0"].clone()
    y2, _ = forward(dict(s, h0=st), cu, hT=st)
    torch.cuda.synchronize()
    assert torch.equal(got["y"], y2) and torch.equal(got["hT"], st)


def test_step_gradients_are_not_biased():
    """The steps' gradients of bf16 inputs against those of the same values in float32.
    Their differences are roundings of either, as often up as down and of each token's
    own sums, so the sum over n tokens is normal with the deviation sqrt(sum of squares):
    within 4.5 of it for each of 8 heads (7e-6 a head).  A rounding that goes one way
    shows here, and in dA and ddt_bias, long before it does in a token's gradient."""
    T, H = 32768, 8
    s = make(T, 8, H, 1, 64, 64, torch.bfloat16)
    s["A"] = torch.linspace(-14, -7, H).cuda()
    wide = {k: v.float() if v.dtype == torch.bfloat16 else v for k, v in s.items()}
    cu = [4096 * b for b in range(9)]
    d = (backward(s, cu)[1].double() - backward(wide, cu)[1].double()) * (1 + torch.exp(-(s["dt"].double() + s["dt_bias"].double())))
    z = d.sum(0) / d.square().sum(0).sqrt()
    log("bias of ddelta: " + " ".join(f"{v:.2f}" for v in z.tolist()))
    assert z.abs().max() <= 4.5, z


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_of_cu_that_decrease(dtype):
    """A bound below an earlier one counts as that one: no row is two sequences', and
    the workspace's chunks suffice however often the bounds go up and down."""
    from itertools import accumulate
    T, B = 300, 140
    for given in ([0, 150, 40, T], [T, 0] * 2 + [T], [0] + [T, 0] * 69 + [T], [(i * 7) % 50 for i in range(140)] + [T]):
        nb = len(given) - 1
        s = make(T, nb, 2, 1, 64, 64, DT[dtype])
        inside = list(accumulate(given, max))
        assert nb <= B and inside[-1] == given[-1]
        for a, c in zip(forward(s, given) + backward(s, given), forward(s, inside) + backward(s, inside)):
            assert torch.equal(a, c)


def test_nonfinite_values_stay_in_their_sequence_and_head():
    s = make(400, 3, 2, 1, 64, 64, torch.bfloat16)
    cu = [0, 130, 290, 400]
    a = forward(s, cu) + backward(s, cu)
    s2 = dict(s, x=s["x"].clone(), dy=s["dy"].clone())
    s2["x"][200, 1, 3], s2["dy"][150, 0, 5] = NAN, float("inf")
    b = forward(s2, cu) + backward(s2, cu)
    other = torch.ones(400, dtype=torch.bool)
    other[130:290] = False
    torch.cuda.synchronize()
    for i, (p, q) in enumerate(zip(a, b)):
        if p.shape[0] == 400:
            assert torch.equal(p[other], q[other]), i
        elif p.shape[0] == 3:
            assert torch.equal(p[[0, 2]], q[[0, 2]]), i
    assert torch.equal(a[0][:, 0], b[0][:, 0]) and torch.isnan(b[0][200:290, 1, 3]).all()


def test_empty_calls():
    import gated_delta_rule_52_amd as gdn
    s = make(0, 2, 2, 1, 64, 64, torch.bfloat16)
    y, hT = forward(s, [0, 0, 0])
    g = backward(s, [0, 0, 0])
    torch.cuda.synchronize()
    assert y.shape == (0, 2, 64) and torch.equal(hT, s["h0"]) and torch.equal(g[-1], s["dhT"])
    assert all((g[i] == 0).all() for i in (2, 5, 6))
    assert gdn.gdn_ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h0"][:0]).shape == (0, 2, 64)


def test_scan_binding_refusals():
    import gated_delta_rule_52_amd as gdn
    s = make(20, 1, 2, 1, 64, 64, torch.float32, fused=False)
    cu = ints([0, 20])
    a = [s[k] for k in ("x", "dt", "A", "B", "C")]
    f = gdn.gdn_ssm_forward
    for bad in (lambda: f(*a[:3], a[3][:5], a[4], cu), lambda: f(a[0], a[1].t(), *a[2:], cu), lambda: f(*a, cu, D=s["D"][:1]),
                lambda: f(*a, cu, h0=s["h0"][:, :1]), lambda: f(*a, cu, y=s["x"][:5]), lambda: f(*a, cu, hT=s["h0"].mT),
                lambda: f(a[0].expand(20, 2, 64)[:1].expand(20, 2, 64), *a[1:], cu), lambda: gdn.gdn_ssm_step(*a, None),
                lambda: gdn.gdn_ssm_backward(*a, cu, s["dy"][:5]), lambda: gdn.gdn_ssm_backward(*a, cu, s["dy"], out=(None,) * 8)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(*a, cu.long()), lambda: f(a[0].bfloat16(), *a[1:], cu), lambda: f(a[0], a[1].bfloat16(), *a[2:], cu)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(gdn.GdnError):
        gdn.gdn_ssm_backward(*a, cu, s["dy"], dhT=s["dhT"], h0=s["h0"],
                             out=(a[0].clone(), a[1].clone(), a[2].clone(), a[3].clone(), a[4].clone(), None, None, s["dhT"]))
