"""Infinities and NaN in the scan: they reach the results that depend on them and no
others.  The results that may change follow from the formulas alone; all others keep
their bits, the earlier tokens of the same chunk among them."""
import pytest
import torch

from gpu_util import log
from test_gpu_attention import DT, NAN
from test_gpu_ssm import GRADS, backward, forward, make

pytestmark = pytest.mark.gpu

INF = float("inf")
CU = [0, 70, 370, 400]  # the second sequence: three chunks of bf16, five of float32
HEADS = [(4, 2, 64, 64), (2, 1, 128, 128), (3, 1, 64, 64)]
# place in its sequence: a chunk's first and last token, inside a block, a block's edges, the sequence's end
PLACES = [0, 13, 31, 32, 100, 127, 128, 250, 299]


def spoiled(s, name, at, value):
    t = s[name].clone()
    t[at] = value
    return dict(s, **{name: t})


def check(clean, got, may):
    """Results outside `may` have their bits, those inside are not finite."""
    for k, m in may.items():
        a, b = clean[k], got[k]
        assert torch.equal(a[~m], b[~m]), f"{k}: a result that does not depend on it"
        assert not torch.isfinite(b[m]).any(), f"{k}: a result that depends on it"


def nothing(results):
    return {k: torch.zeros(v.shape, dtype=torch.bool, device="cuda") for k, v in results.items()}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_outputs(dtype, heads, value):
    H, G, N, P = heads
    s = make(CU[-1], 3, *heads, DT[dtype])
    run = lambda s: dict(zip(("y", "hT"), forward(s, CU)))  # noqa: E731
    clean = run(s)
    lo, hi = CU[1], CU[2]
    h, g, n, p = 1, 1 // (H // G), N - 5, P - 3
    of = slice(g * (H // G), (g + 1) * (H // G))
    for place in PLACES:
        t = lo + place
        for name in ("x", "B", "C", "dt"):
            may = nothing(clean)
            if name == "x":
                got = run(spoiled(s, name, (t, h, p), value))
                may["y"][t:hi, h, p] = may["hT"][1, h, :, p] = True
            elif name == "B":
                got = run(spoiled(s, name, (t, g, n), value))
                may["y"][t:hi, of] = may["hT"][1, of, n] = True
            elif name == "C":
                got = run(spoiled(s, name, (t, g, n), value))
                may["y"][t, of] = True
            else:
                if value == -INF:
                    continue  # a step of log(1 + 0): the token is passed over
                got = run(spoiled(s, name, (t, h), value))
                may["y"][t:hi, h] = may["hT"][1, h] = True
            torch.cuda.synchronize()
            log(f"outputs {dtype} {heads} {value} in {name} at {place}")
            check(clean, got, may)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_outputs_of_infinite_values(dtype):
    """The sign of an infinity is that of its products, where they are not 0."""
    s = make(40, 1, 2, 1, 64, 64, DT[dtype])
    s["h0"], s["B"], s["C"] = s["h0"] * 0, s["B"].abs() + 0.5, -s["C"].abs() - 0.5
    y, _ = forward(spoiled(s, "x", (9, 1, 7), INF), [0, 40])
    torch.cuda.synchronize()
    assert (y[10:, 1, 7] == -INF).all() and torch.isfinite(y[:9]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_several_values_in_a_block(dtype):
    """Each reaches its own tokens and values."""
    s = make(CU[-1], 3, 2, 1, 64, 64, DT[dtype])
    clean = forward(s, CU)[0]
    t = s["x"].clone()
    may = torch.zeros(clean.shape, dtype=torch.bool, device="cuda")
    for i, (at, h, p) in enumerate([(70, 0, 0), (99, 0, 0), (75, 1, 63), (101, 1, 62), (80, 0, 31), (90, 0, 32), (369, 1, 5), (399, 0, 9)]):
        t[at, h, p] = (NAN, INF, -INF)[i % 3]
        may[at:370 if at < 370 else 400, h, p] = True
    y = forward(dict(s, x=t), CU)[0]
    torch.cuda.synchronize()
    check({"y": clean}, {"y": y}, {"y": may})


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("value", [NAN, INF])
def test_gradients(dtype, heads, value):
    """dy and C reach what lies before their token, x and B what lies behind: dx and dB of
    the tokens up to it, dC of those from it on, and the steps on the way."""
    H, G, N, P = heads
    s = make(CU[-1], 3, *heads, DT[dtype])
    run = lambda s: dict(zip(GRADS, backward(s, CU)))  # noqa: E731
    clean = run(s)
    lo, hi = CU[1], CU[2]
    h, g, n, p = 1, 1 // (H // G), N - 5, P - 3
    of = slice(g * (H // G), (g + 1) * (H // G))
    for place in PLACES:
        t = lo + place
        for name in ("x", "dy", "B", "C"):
            may, own = nothing(clean), slice(h, h + 1) if name in ("x", "dy") else of
            got = run(spoiled(s, name, (t, h, p) if name in ("x", "dy") else (t, g, n), value))
            may["ddt_bias"][own] = True
            # nothing decays what the last token puts in: dg is of the tokens behind it
            may["dA"][own] = name in ("dy", "C") or t < hi - 1
            if name == "x":
                may["dB"][t, g] = may["dC"][t:hi, g] = may["ddt"][t:hi, h] = may["dD"][h] = True
            elif name == "dy":
                may["dx"][lo:t + 1, h, p] = may["dB"][lo:t + 1, g] = may["dC"][t, g] = may["ddt"][lo:t + 1, h] = True
                may["dh0"][1, h, :, p] = may["dD"][h] = True
            elif name == "B":
                may["dx"][t, of] = may["dC"][t:hi, g, n] = may["ddt"][t:hi, of] = True
            else:
                may["dx"][lo:t + 1, of] = may["dB"][lo:t + 1, g, n] = may["ddt"][lo:t + 1, of] = may["dh0"][1, of, n] = True
            torch.cuda.synchronize()
            log(f"gradients {dtype} {heads} {value} in {name} at {place}")
            check(clean, got, may)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_states_that_are_not_finite(dtype):
    """h0 reaches dC and the steps of all its sequence, dhT dx, dB, dh0 and the steps."""
    s = make(CU[-1], 3, 4, 2, 64, 64, DT[dtype])
    run = lambda s: dict(zip(GRADS, backward(s, CU)))  # noqa: E731
    clean = run(s)
    at = slice(CU[1], CU[2])
    for name in ("h0", "dhT"):
        may = nothing(clean)
        may["ddt"][at, 3] = may["dA"][3] = may["ddt_bias"][3] = True
        if name == "h0":
            may["dC"][at, 1, 9] = True
        else:
            may["dx"][at, 3, 7] = may["dB"][at, 1, 9] = may["dh0"][1, 3, 9, 7] = True
        got = run(spoiled(s, name, (1, 3, 9, 7), NAN))
        torch.cuda.synchronize()
        check(clean, got, may)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("place", [0, 100, 299])
def test_steps_that_are_not_finite_stay_in_their_sequence_and_head(dtype, place):
    """In the gradients: of the head in its sequence, and of its group there."""
    H, G = 4, 2
    s = make(CU[-1], 3, H, G, 64, 64, DT[dtype])
    clean = backward(s, CU)
    got = backward(spoiled(s, "dt", (CU[1] + place, 1), NAN), CU)
    torch.cuda.synchronize()
    at = slice(CU[1], CU[2])
    for k, a, b in zip(GRADS, clean, got):
        same = torch.ones(a.shape, dtype=torch.bool, device="cuda")
        if k in ("dx", "ddt"):
            same[at, 1] = False
        elif k in ("dB", "dC"):
            same[at, 0] = False
        elif k == "dh0":
            same[1, 1] = False
        else:
            same[1] = False
        assert torch.equal(a[same], b[same]), k
        assert k in ("dB", "dC", "dD") or not torch.isfinite(b[~same]).all(), k
