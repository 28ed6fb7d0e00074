"""Sequence bounds that decrease, in the state-space layer's operators: a bound below
an earlier one counts as that one, whatever the size of the call, so that the given
bounds and their running maximum have the same results, bit for bit."""
from itertools import accumulate

import pytest
import torch

import mixer_reference as ref
from gpu_util import log
from mixer_reference import worst
from test_gpu_attention import DT, ints, rand
from test_gpu_ssm import backward, blank, forward, make

pytestmark = pytest.mark.gpu

T = 300
GIVEN = [[0, T, 100], [0, T, 0], [0, 200, 90, 150], [5, 260, 4, 270, 269], [T, 0], [0, 40] * 40 + [7], [10, -3, 120, 9999, 31]]


def ordered(given, rows=T):
    return list(accumulate((min(max(v, 0), rows) for v in given), max))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G", [(4, 1), (4, 4), (6, 2)])
@pytest.mark.parametrize("given", GIVEN, ids=lambda g: "-".join(map(str, g[:5])))
def test_scan_whose_last_bound_is_not_the_greatest(dtype, H, G, given):
    """A group's heads dealt to several workgroups (H / G > 1), and to one."""
    log(f"scan bounds {dtype} H={H} G={G} {given[:6]}")
    dt, B = DT[dtype], len(given) - 1
    s = make(T, B, H, G, 64, 64, dt)
    results = []
    for cu in (given, ordered(given)):
        y = torch.full((T, H, 64), 7.0, dtype=dt, device="cuda")
        hT, out = torch.full((B, H, 64, 64), 7.0, device="cuda"), blank(s, dt)
        forward(s, cu, y=y, hT=hT)
        backward(s, cu, out=out)
        torch.cuda.synchronize()
        results.append((y, hT) + out)
    names = ("y", "hT", "dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")
    assert not [n for n, a, b in zip(names, *results) if not torch.equal(a, b)]


def conv_run(cu, x, w, b, state, dy, dso):
    import gated_delta_rule_52_amd as gdn
    like = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")  # noqa: E731
    y, so = torch.full(dy.shape, 7.0, dtype=dy.dtype, device="cuda"), like(state)
    out = (like(dy), like(w), like(b), like(state))
    gdn.gdn_conv_forward(x, w, ints(cu), b, state, y=y, state_out=so)
    gdn.gdn_conv_backward(x, w, ints(cu), dy, b, state, dstate_out=dso, out=out)
    torch.cuda.synchronize()
    return dict(zip(("y", "state", "dx", "dweight", "dbias", "dstate"), (y, so) + out))


def conv_inputs(rows, B, C, W, dt):
    return (rand(rows, C + 8, dtype=dt)[:, :C], rand(C, W, std=0.5, seed=1), rand(C, seed=2), rand(B, W - 1, C, dtype=dt, seed=3),
            rand(rows, C, dtype=dt, seed=4), rand(B, W - 1, C, dtype=dt, seed=5))


MANY = [(7 * i) % 300 for i in range(9000)] + [250]  # more than 8192 sequences, most of them empty


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W,C", [(4, 512), (2, 64), (3, 200)])
@pytest.mark.parametrize("given", GIVEN + [MANY], ids=lambda g: "-".join(map(str, g[:5])))
def test_conv_whose_bounds_decrease(dtype, W, C, given):
    """A wave a strip, and several strips a wave."""
    log(f"conv bounds {dtype} W={W} C={C} {given[:6]}")
    args = conv_inputs(T, len(given) - 1, C, W, DT[dtype])
    a, b = conv_run(given, *args), conv_run(ordered(given), *args)
    assert not [k for k in a if not torch.equal(a[k], b[k])]
    inside = ordered(given)
    none = torch.ones(T, dtype=torch.bool)
    none[inside[0]:inside[-1]] = False
    assert (a["y"][none] == 7.0).all() and (a["dx"][none] == 7.0).all(), "a row of no sequence was written"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,C", [(63, 512), (64, 24), (65, 512), (255, 24), (256, 512), (257, 24), (511, 24), (512, 512), (513, 24), (1300, 512), (2600, 24), (9000, 256)])
def test_conv_of_many_sequences(dtype, B, C):
    """About the numbers of sequences that are looked through at a time; empty ones among
    them, and rows before the first."""
    dt = DT[dtype]
    cu = [9]
    for i in range(B):
        few = B < 5000 or i % 8 == 0  # the plain form goes row by row
        cu.append(cu[-1] + (5 * i) % 7 // 2 * few + (40 if i % 200 == 150 else 0))
    n = cu[-1]
    log(f"conv {dtype} B={B} C={C}: {n} rows")
    x, w, b, state, dy, dso = conv_inputs(n + 2, B, C, 4, dt)
    got = conv_run(cu, x, w, b, state, dy, dso)
    few = torch.tensor([0, 1, C // 2 + 3, C - 1], device="cuda")  # channels are independent
    pick = lambda t, d=-1: t.index_select(t.dim() + d, few)  # noqa: E731
    xs, ws, bs, ss, ys, os = pick(x), pick(w, -2), pick(b), pick(state), pick(dy), pick(dso)
    wy, by, wst = ref.conv(xs, ws, cu, bs, ss)
    rows = slice(cu[0], n)
    errs = {"y": worst(pick(got["y"])[rows], wy[rows], by[rows])}
    assert torch.equal(pick(got["state"]).cpu().double(), wst)
    for k, (want, bound) in ref.conv_backward(xs, ws, cu, ys, bs, ss, os).items():
        g = pick(got[k], -2 if k == "dweight" else -1)
        errs[k] = worst(g[rows], want[rows], bound[rows]) if k == "dx" else worst(g, want, bound)
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs
    assert all((got[k][[0, 8, n, n + 1]] == 7.0).all() for k in ("y", "dx"))
