"""Calls of the state-space layer's operators at the ends of what they take: no rows at
all, tensors of more than 2^31 elements, steps that grow, single tokens as packed calls."""
import pytest
import torch

import mixer_reference as ref
from gpu_util import log
from mixer_reference import worst
from test_gpu_attention import DT, ints, rand
from test_gpu_ssm import GRADS, backward, forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_convolution_without_rows(dtype):
    """States and their gradients pass through, and the weights have none."""
    import gated_delta_rule_52_amd as gdn
    dt, C, B = DT[dtype], 72, 3
    x, w, b = torch.empty(0, C, dtype=dt, device="cuda"), rand(C, 4), rand(C, seed=1)
    st, dso = rand(B, 3, C, dtype=dt, seed=2), rand(B, 3, C, dtype=dt, seed=3)
    y, out = gdn.gdn_conv_forward(x, w, ints([0] * (B + 1)), b, st)
    dx, dw, db, ds = gdn.gdn_conv_backward(x, w, ints([0] * (B + 1)), x, b, st, dstate_out=dso)
    torch.cuda.synchronize()
    assert y.shape == dx.shape == (0, C) and torch.equal(out, st) and torch.equal(ds, dso)
    assert not dw.any() and not db.any()


def tiled(rows, *shape, dtype, seed):
    """rows of `shape`, 4096 random ones over and over"""
    base = rand(4096, *shape, dtype=dtype, seed=seed)
    out = torch.empty(rows, *shape, dtype=dtype, device="cuda")
    for i in range(0, rows, 4096):
        out[i:i + 4096] = base[:min(4096, rows - i)]
    return out


def test_convolution_past_32_bits():
    """More than 2^31 elements: the last sequence as it is by itself."""
    import gated_delta_rule_52_amd as gdn
    C, n, dt = 1024, 77, torch.bfloat16
    T = (1 << 21) + 5 * 4096 + n
    x, dy = tiled(T, C, dtype=dt, seed=1), tiled(T, C, dtype=dt, seed=2)
    w, b, st = rand(C, 4, std=0.5), rand(C, seed=1), rand(2, 3, C, dtype=dt, seed=3)
    assert x.numel() > 1 << 31
    y, out = gdn.gdn_conv_forward(x, w, ints([0, T - n, T]), b, st)
    dx = gdn.gdn_conv_backward(x, w, ints([0, T - n, T]), dy, b, st, dstate_out=st)[0]
    xs, ys = x[-n:].clone(), dy[-n:].clone()
    y1, out1 = gdn.gdn_conv_forward(xs, w, ints([0, n]), b, st[1:].clone())
    g1 = gdn.gdn_conv_backward(xs, w, ints([0, n]), ys, b, st[1:].clone(), dstate_out=st[1:].clone())
    torch.cuda.synchronize()
    assert torch.equal(y[-n:], y1) and torch.equal(out[1:], out1) and torch.equal(dx[-n:], g1[0])
    assert torch.equal(y[4096 * 3:4096 * 4], y[4096 * 500:4096 * 501]) and torch.equal(dx[4096 * 3:4096 * 4 - 3], dx[4096 * 500:4096 * 501 - 3])


def test_scan_past_32_bits():
    """More than 2^31 elements: the last sequence as it is by itself (a head a group: its
    sums are divided alike)."""
    H, N, P, n, dt = 8, 64, 128, 300, torch.bfloat16
    T = (1 << 21) + 5 * 4096 + n
    s = dict(x=tiled(T, H, P, dtype=dt, seed=1), B=tiled(T, H, N, dtype=dt, seed=2), C=tiled(T, H, N, dtype=dt, seed=3),
             dy=tiled(T, H, P, dtype=dt, seed=4), dt=tiled(T, H, dtype=torch.float32, seed=5), A=-torch.linspace(1, 16, H, device="cuda"),
             D=rand(H, seed=6), dt_bias=torch.linspace(-5, -2, H, device="cuda"), h0=rand(2, H, N, P, seed=7), dhT=rand(2, H, N, P, seed=8))
    assert s["x"].numel() > 1 << 31
    cu = [0, T - n, T]
    y, hT = forward(s, cu)
    got = dict(zip(GRADS, backward(s, cu)))
    one = {k: v[-n:].clone() if k in ("x", "B", "C", "dy", "dt") else v[1:].clone() if k in ("h0", "dhT") else v for k, v in s.items()}
    y1, hT1 = forward(one, [0, n])
    want = dict(zip(GRADS, backward(one, [0, n])))
    torch.cuda.synchronize()
    assert torch.equal(y[-n:], y1) and torch.equal(hT[1:], hT1)
    for k in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(got[k][-n:], want[k]), k
    assert torch.equal(got["dh0"][1:], want["dh0"])
    assert all(torch.isfinite(v).all() for v in (y, hT, *got.values()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_that_grow(dtype):
    """A of either sign, and steps of either sign without softplus: decays above 1, a
    state that grows by up to e^20 within a sequence."""
    import gated_delta_rule_52_amd as gdn
    cu, dt = [0, 150, 170, 171], DT[dtype]
    for softplus in (True, False):
        s = make(171, 3, 2, 1, 64, 64, dt)
        s["A"] = torch.tensor([0.4, -3.0], device="cuda")
        if not softplus:
            s["dt"], s["dt_bias"] = s["dt"] * 0.4, torch.tensor([0.01, -0.02], device="cuda")
        a = (s["x"], s["dt"], s["A"], s["B"], s["C"], ints(cu))
        kw = dict(D=s["D"], dt_bias=s["dt_bias"], softplus=softplus, h0=s["h0"])
        y, hT = gdn.gdn_ssm_forward(*a, **kw)
        got = dict(zip(GRADS, gdn.gdn_ssm_backward(*a, s["dy"], dhT=s["dhT"], **kw)), y=y, hT=hT)
        torch.cuda.synchronize()
        want = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["D"], s["dt_bias"], softplus, s["h0"], s["dy"], s["dhT"])
        errs = {k: worst(v, *want[k]) for k, v in got.items()}
        log(f"growing {dtype} softplus {softplus}: " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
        assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_tokens_as_a_packed_call(dtype):
    """Sequences of one token each: what the step calls make of them."""
    import gated_delta_rule_52_amd as gdn
    B, dt = 70, DT[dtype]
    s = make(B, B, 4, 2, 128, 64, dt)
    cu = list(range(B + 1))
    y, hT = forward(s, cu)
    st = s["h0"].clone()
    y1 = gdn.gdn_ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], st, D=s["D"], dt_bias=s["dt_bias"])
    torch.cuda.synchronize()
    want = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["D"], s["dt_bias"], True, s["h0"])
    errs = [worst(a, *want[k]) for k, a in (("y", y), ("hT", hT), ("y", y1), ("hT", st))]
    x, w, b, cs = rand(B, 136, dtype=dt), rand(136, 3, seed=1), rand(136, seed=2), rand(B, 2, 136, dtype=dt, seed=3)
    z, out = gdn.gdn_conv_forward(x, w, ints(cu), b, cs)
    z1 = gdn.gdn_conv_step(x, w, cs, b)
    torch.cuda.synchronize()
    log(f"single tokens {dtype}: " + " ".join(f"{e:.2f}" for e in errs))
    assert max(errs) <= 1 and torch.equal(z, z1) and torch.equal(out, cs)
