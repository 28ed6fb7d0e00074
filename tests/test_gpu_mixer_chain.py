"""A state-space layer's training step as it is run: the convolution, the scan on slices
of its output, and their gradients one behind the other, the scan's dx, dB and dC side
by side as the convolution's dy."""
import pytest
import torch

import mixer_reference as ref
import ssm_checks
from gpu_util import log
from mixer_reference import f64, worst
from test_gpu_attention import DT, cumulate, ints, rand
from test_gpu_ssm import GRADS

pytestmark = pytest.mark.gpu

H, G, N, P = 4, 2, 64, 64
CHAN = H * P + 2 * G * N
LEAVES = ("x", "weight", "bias", "state", "dt", "A", "D", "dt_bias", "h0")


def layer(lens, dt):
    T, B = sum(lens), len(lens)
    return dict(x=rand(T, CHAN + 64, dtype=dt)[:, :CHAN], weight=rand(CHAN, 4, std=0.5, seed=1), bias=rand(CHAN, seed=2),
                state=rand(B, 3, CHAN, dtype=dt, seed=3), dt=rand(T, H, std=0.5, seed=4), A=-torch.linspace(1, 8, H, device="cuda"),
                D=rand(H, seed=5), dt_bias=torch.linspace(-4, -2, H, device="cuda"), h0=rand(B, H, N, P, seed=6),
                dy=rand(T, H, P, dtype=dt, seed=7), dstate=rand(B, 3, CHAN, dtype=dt, seed=8), dhT=rand(B, H, N, P, std=0.3, seed=9))


def split(y):
    return (y[:, :H * P].unflatten(1, (H, P)), y[:, H * P:H * P + G * N].unflatten(1, (G, N)),
            y[:, H * P + G * N:].unflatten(1, (G, N)))


def step(s, cu):
    """(results, gradients, what went from the scan's gradients to the convolution's)"""
    import gated_delta_rule_52_amd as gdn
    c = ints(cu)
    z, st = gdn.gdn_conv_forward(s["x"], s["weight"], c, s["bias"], s["state"])
    x, Bm, Cm = split(z)
    a, kw = (x, s["dt"], s["A"], Bm, Cm, c), dict(D=s["D"], dt_bias=s["dt_bias"], h0=s["h0"])
    y, hT = gdn.gdn_ssm_forward(*a, **kw)
    g = dict(zip(GRADS, gdn.gdn_ssm_backward(*a, s["dy"], dhT=s["dhT"], **kw)))
    dz = torch.cat([g[k].flatten(1) for k in ("dx", "dB", "dC")], 1)
    dx, dw, db, ds = gdn.gdn_conv_backward(s["x"], s["weight"], c, dz, s["bias"], s["state"], dstate_out=s["dstate"])
    torch.cuda.synchronize()
    grads = dict(x=dx, weight=dw, bias=db, state=ds, dt=g["ddt"], A=g["dA"], D=g["dD"], dt_bias=g["ddt_bias"], h0=g["dh0"])
    return dict(z=z, state=st, y=y, hT=hT), grads, dict(g, dz=dz)


def plain(s, cu):
    """The layer token by token, for autograd: the loss sum(y dy) + sum(hT dhT) + sum(state dstate)."""
    T, rows, last = len(s["x"]), [], []
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        ahead = torch.cat([s["state"][b], s["x"][a:e]])
        z = s["bias"] + sum(s["weight"][:, j] * ahead[j:j + e - a] for j in range(4))
        rows.append(z * torch.sigmoid(z))
        last.append(ahead[e - a:])
    z, st = torch.cat(rows), torch.stack(last)
    x, Bm, Cm = split(z)
    y, hT = ref.ssm_serial(x, s["dt"], s["A"], Bm, Cm, cu, s["D"], s["dt_bias"], True, s["h0"])
    assert len(z) == T
    return (y * s["dy"]).sum() + (hT * s["dhT"]).sum() + (st * s["dstate"]).sum()


@pytest.mark.parametrize("lens", [[40, 2, 75], [1, 0, 200]], ids=str)
def test_gradients_of_the_whole_layer(lens):
    """float32 against autograd of the 64-bit form.  Four operators one behind the other,
    each within 2^-18 of its results' 2-norm (ssm_checks.py), and each passing on what
    it gets within the size of its own: 2^-16."""
    cu = cumulate(lens)
    s = layer(lens, torch.float32)
    _, grads, _ = step(s, cu)
    wide = {k: f64(v) for k, v in s.items()}
    for k in LEAVES:
        wide[k] = wide[k].clone().requires_grad_()
    plain(wide, cu).backward()
    errs = {k: float((f64(grads[k]) - wide[k].grad).norm() / (2.0 ** -16 * wide[k].grad.norm())) for k in LEAVES}
    log(f"layer {lens}: " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


def test_gradients_of_the_whole_layer_against_differences():
    """The kernels' own loss along each gradient, as in the scan's test: a step of 2^-6
    along a unit vector leaves third derivatives below 1 %, and rounding less."""
    lens = [40, 35]
    cu = cumulate(lens)
    s = layer(lens, torch.float32)
    _, grads, _ = step(s, cu)

    def loss(s):
        r, _, _ = step(s, cu)
        return float((r["y"].double() * s["dy"].double()).sum() + (r["hT"].double() * s["dhT"].double()).sum()
                     + (r["state"].double() * s["dstate"].double()).sum())

    for k in LEAVES:
        g = grads[k]
        u = g / g.norm()
        d = (loss(dict(s, **{k: s[k] + 2.0 ** -6 * u})) - loss(dict(s, **{k: s[k] - 2.0 ** -6 * u}))) * 32
        want = float((g.double() * u.double()).sum())
        log(f"  {k}: {d:.6f} against {want:.6f}")
        assert abs(d - want) <= 0.01 * abs(want), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[150, 0, 40, 3], [1100]], ids=str)
def test_each_operator_in_the_step(dtype, lens):
    """Every operator of the step against its plain form on the inputs that it had."""
    cu, dt = cumulate(lens), DT[dtype]
    s = layer(lens, dt)
    r, grads, scan = step(s, cu)
    x, Bm, Cm = split(r["z"])
    few = torch.tensor([0, H * P - 1, H * P + 5, CHAN - 1], device="cuda")  # channels are independent
    pick = lambda t, d=-1: t.index_select(t.dim() + d, few)  # noqa: E731
    a = (pick(s["x"]), pick(s["weight"], -2), cu)
    wz, bz, wst = ref.conv(*a, pick(s["bias"]), pick(s["state"]))
    errs = {"z": worst(pick(r["z"]), wz, bz)}
    assert torch.equal(pick(r["state"]).cpu().double(), wst)
    want = ref.conv_backward(*a, pick(scan["dz"]), pick(s["bias"]), pick(s["state"]), pick(s["dstate"]))
    for k, name, d in (("x", "dx", -1), ("weight", "dweight", -2), ("bias", "dbias", -1), ("state", "dstate", -1)):
        errs[name] = worst(pick(grads[k], d), *want[name])
    t = dict(x=x, B=Bm, C=Cm, **{k: s[k] for k in ("dt", "A", "D", "dt_bias", "h0", "dy", "dhT")})
    want, size = ssm_checks.definition(t, cu)
    errs.update({"scan " + k: v for k, v in ssm_checks.shares(dict({k: scan[k] for k in GRADS}, y=r["y"], hT=r["hT"]), want, size).items()})
    log(f"step {dtype} {lens}: " + " ".join(f"{k}={v:.3f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs
