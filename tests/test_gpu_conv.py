"""The short causal convolution against the plain 64-bit form, within the bounds that
mixer_reference.py derives."""
import pytest
import torch

import mixer_reference as ref
from gpu_util import log
from mixer_reference import worst
from test_gpu_attention import DT, NAN, cumulate, ints, rand

pytestmark = pytest.mark.gpu

LENS = [[1], [2, 1, 3], [0, 5, 0, 0, 4], [7, 8, 9, 31, 33], [150], [0, 0]]


def inputs(T, C, W, B, dt, wide, state=True):
    x = rand(T, C + (72 if wide else 0), dtype=dt)[:, :C]
    w, b = rand(C, W, seed=1) * 0.5, rand(C, seed=2)
    return x, w, b, rand(B, W - 1, C, dtype=dt, seed=3) if state else None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W,C,state,silu", [(4, 64, True, True), (4, 264, False, True), (3, 8, True, False), (2, 136, True, True),
                                            (3, 128, False, True), (2, 16, False, False)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_conv(dtype, W, C, state, silu, lens):
    import gated_delta_rule_52_amd as gdn
    dt, cu, B = DT[dtype], cumulate(lens), len(lens)
    n, T = cu[-1], cu[-1] + 3  # rows behind the last sequence
    log(f"conv {dtype} W={W} C={C} state={state} silu={silu} {lens}")
    x, w, b, s = inputs(T, C, W, B, dt, wide=C != 64, state=state)
    x[n:] = NAN
    bias = b if C != 16 else None
    y = torch.full((T, C), 7.0, dtype=dt, device="cuda")
    so = torch.full((B, W - 1, C), 7.0, dtype=dt, device="cuda")
    gdn.gdn_conv_forward(x, w, ints(cu), bias, s, silu=silu, y=y, state_out=so)
    dy, dso = rand(T, C, dtype=dt, seed=5), rand(B, W - 1, C, dtype=dt, seed=6) if state else None
    out = (torch.full((T, C), 7.0, dtype=dt, device="cuda"), torch.full((C, W), 7.0, device="cuda"),
           torch.full((C,), 7.0, device="cuda"), torch.full((B, W - 1, C), 7.0, dtype=dt, device="cuda"))
    gdn.gdn_conv_backward(x, w, ints(cu), dy, bias, s, silu=silu, dstate_out=dso, out=out)
    torch.cuda.synchronize()
    assert (y[n:] == 7.0).all() and (out[0][n:] == 7.0).all(), "a row of no sequence was written"
    wy, by, ws = ref.conv(x[:n], w, cu, bias, s, silu)
    assert torch.equal(so.cpu().double(), ws)
    errs = {"y": worst(y[:n], wy, by)}
    want = ref.conv_backward(x[:n], w, cu, dy[:n], bias, s, dso, silu)
    for got, name in zip((out[0][:n],) + out[1:], ("dx", "dweight", "dbias", "dstate")):
        errs[name] = worst(got, *want[name])
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,C", [([700, 900, 1, 2, 3, 500], 1024), ([5000], 512)])
def test_conv_long_strips(dtype, lens, C):
    """Strips of 16 and 32 rows, sequences that begin inside of them."""
    import gated_delta_rule_52_amd as gdn
    dt, cu, B = DT[dtype], cumulate(lens), len(lens)
    T = cu[-1]
    log(f"conv {dtype} {lens} C={C}")
    x, w, b, s = inputs(T, C, 4, B, dt, True)
    y, so = gdn.gdn_conv_forward(x, w, ints(cu), b, s)
    dy, dso = rand(T, C, dtype=dt, seed=5), rand(B, 3, C, dtype=dt, seed=6)
    out = gdn.gdn_conv_backward(x, w, ints(cu), dy, b, s, dstate_out=dso)
    again = gdn.gdn_conv_backward(x, w, ints(cu), dy, b, s, dstate_out=dso)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    few = [0, 1, 8, C // 2 + 3, C - 1]  # channels are independent: these are checked
    pick = lambda t, d=-1: t.index_select(t.dim() + d, torch.tensor(few, device="cuda"))  # noqa: E731
    xs, ws, bs, ss = pick(x), pick(w, -2), pick(b), pick(s)
    wy, by, wso = ref.conv(xs, ws, cu, bs, ss)
    errs = {"y": worst(pick(y), wy, by)}
    assert torch.equal(pick(so).cpu().double(), wso)
    want = ref.conv_backward(xs, ws, cu, pick(dy), bs, ss, pick(dso))
    for got, name in zip((pick(out[0]), pick(out[1], -2), pick(out[2]), pick(out[3])), ("dx", "dweight", "dbias", "dstate")):
        errs[name] = worst(got, *want[name])
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_pieces_and_steps(dtype, W):
    """A sequence at once, in pieces with the state updated in place, and token by
    token: the same bits, since every output is the same sum."""
    import gated_delta_rule_52_amd as gdn
    dt, C, B, n = DT[dtype], 72, 3, 21
    x, w, b, s0 = inputs(B * n, C, W, B, dt, False)
    whole, last = gdn.gdn_conv_forward(x, w, ints([0, n, 2 * n, 3 * n]), b, s0)
    x3, want = x.view(B, n, C), whole.view(B, n, C)
    s, at = s0.clone(), 0
    for m in (1, 0, 2, 5, 13):  # equal pieces of the three sequences
        y, out = gdn.gdn_conv_forward(x3[:, at:at + m].reshape(B * m, C).contiguous(), w, ints([0, m, 2 * m, 3 * m]), b, s, state_out=s)
        assert out is s and torch.equal(y.view(B, m, C), want[:, at:at + m]), m
        at += m
    assert torch.equal(s, last)
    s = s0.clone()
    for t in range(n):
        y = gdn.gdn_conv_step(rand(B, C + 8, dtype=dt)[:, :C].copy_(x3[:, t]), w, s, b)
        assert torch.equal(y, want[:, t]), t
    assert torch.equal(s, last)


def test_conv_bounds_of_cu_are_clamped():
    import gated_delta_rule_52_amd as gdn
    x, w, b, s = inputs(50, 64, 4, 2, torch.bfloat16, False)
    dy = rand(50, 64, dtype=torch.bfloat16, seed=4)
    for a, c in zip((gdn.gdn_conv_forward(x, w, ints([-5, 20, 9999]), b, s) + gdn.gdn_conv_backward(x, w, ints([-5, 20, 9999]), dy, b, s)),
                    (gdn.gdn_conv_forward(x, w, ints([0, 20, 50]), b, s) + gdn.gdn_conv_backward(x, w, ints([0, 20, 50]), dy, b, s))):
        assert torch.equal(a, c)


def test_conv_nonfinite_rows_reach_their_windows_only():
    import gated_delta_rule_52_amd as gdn
    x, w, b, s = inputs(60, 64, 4, 2, torch.float32, False)
    cu = ints([0, 25, 60])
    y, _ = gdn.gdn_conv_forward(x, w, cu, b, s)
    x2 = x.clone()
    x2[10], x2[24], x2[40] = NAN, float("inf"), NAN
    y2, _ = gdn.gdn_conv_forward(x2, w, cu, b, s)
    bad = torch.zeros(60, dtype=torch.bool)
    bad[[10, 11, 12, 13, 24, 40, 41, 42, 43]] = True
    assert torch.equal(y[~bad], y2[~bad]) and not torch.isfinite(y2[[10, 13, 40, 43]]).any()
    dy = rand(60, 64, seed=9)
    g = gdn.gdn_conv_backward(x, w, cu, dy, b, s)[0]
    dy[30] = NAN
    g2 = gdn.gdn_conv_backward(x, w, cu, dy, b, s)[0]
    bad = torch.zeros(60, dtype=torch.bool)
    bad[27:31] = True
    assert torch.equal(g[~bad], g2[~bad]) and torch.isnan(g2[bad]).all()


def test_conv_binding_refusals():
    import gated_delta_rule_52_amd as gdn
    x, w, b, s = inputs(10, 64, 4, 2, torch.float32, False)
    cu = ints([0, 5, 10])
    for bad in (lambda: gdn.gdn_conv_forward(x, w.t(), cu), lambda: gdn.gdn_conv_forward(x, w, cu, b[:5]),
                lambda: gdn.gdn_conv_forward(x, w, cu, b, s[:1]), lambda: gdn.gdn_conv_forward(x.t(), w[:10], cu),
                lambda: gdn.gdn_conv_forward(x.expand(10, 64)[:1].expand(10, 64), w, cu),
                lambda: gdn.gdn_conv_forward(x, w, cu, y=x[:5]), lambda: gdn.gdn_conv_backward(x, w, cu, x[:5]),
                lambda: gdn.gdn_conv_backward(x, w, cu, x, out=(None, None, None, None)), lambda: gdn.gdn_conv_step(x, w, None)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gdn.gdn_conv_forward(x, w.double(), cu), lambda: gdn.gdn_conv_forward(x, w, cu.long()),
                lambda: gdn.gdn_conv_forward(x.half(), w, cu), lambda: gdn.gdn_conv_forward(x, w, cu, b, s.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(gdn.GdnError):
        gdn.gdn_conv_forward(x, w, cu, y=x)
