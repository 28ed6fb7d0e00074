"""Norms before and after a block against the plain 64-bit forms.  A bound is
HALF (half a step of the stored type) times the value plus fp32 arithmetic:
2^-24 for each of the width + 16 operations a row takes (rows more for the sums
over rows), times the sizes of what is summed."""
import pytest
import torch

import block_reference as ref
from block_reference import HALF, U32, f64, worst
from gpu_util import log

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rand(*shape, dtype=torch.float32, std=1.0, mean=0.0, seed=0):
    g = torch.Generator().manual_seed(seed + 17 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()


def block_bounds(dt, x, y, a, w, dn, dh):
    h, n, r = ref.norm_block(x, w, y, a)
    W, rows = x.shape[-1], x.numel() // x.shape[-1]
    u = (W + 16) * U32
    hs = f64(x).abs() + (0 if y is None else f64(y).abs() * (1 if a is None else f64(a).abs()))  # sizes in h
    r1 = r[..., None]
    xs = hs * r1
    out = {"h": HALF[dt] * h.abs() + 4 * U32 * hs, "n": HALF[dt] * n.abs() + u * (n.abs() + xs * f64(w).abs()),
           "rstd": u * r * (1 + (hs * hs).sum(-1) / (h * h).sum(-1).clamp(min=1e-30))}
    gs = f64(dn).abs() * f64(w).abs()
    dxs = r1 * (gs + xs * (gs * xs).mean(-1, keepdim=True)) * 4 + (0 if dh is None else f64(dh).abs())
    dx, dy, dw, da = ref.norm_block_backward(dn, dh, x, w, y, a)
    out["dx"] = HALF[dt] * dx.abs() + u * dxs
    if a is not None:
        out["dy"] = HALF[dt] * dy.abs() + u * dxs * f64(a).abs()
        out["dres_scale"] = (u + rows * U32) * (dxs * f64(y).abs()).reshape(rows, W).sum(0)
    out["dweight"] = (2 * u + rows * U32) * (f64(dn).abs() * xs).reshape(rows, W).sum(0)
    return (h, n, r), (dx, dy, dw, da), out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 8), (3, 64), (2, 5, 768), (7, 1000), (130, 2048), (2, 4104), (1, 8192),
                                   (2100, 136), (5000, 768)])
@pytest.mark.parametrize("mode", ["scaled", "added", "alone"])
def test_norm_block(dtype, shape, mode):
    import gated_delta_rule_52_amd as gdn
    dt = DT[dtype]
    log(f"norm_block {dtype} {shape} {mode}")
    W = shape[-1]
    x, w = rand(*shape, dtype=dt, std=2.0), rand(W, std=0.2, mean=1.0, seed=1)
    y = None if mode == "alone" else rand(*shape, dtype=dt, seed=2)
    a = rand(W, std=0.3, mean=0.5, seed=3) if mode == "scaled" else None
    dn, dh = rand(*shape, dtype=dt, seed=4), None if mode == "added" else rand(*shape, dtype=dt, seed=5)
    (h, n, r), grads, b = block_bounds(dt, x, y, a, w, dn, dh)
    gh, gn, gr = gdn.gdn_norm_block(x, w, y, a)
    got = gdn.gdn_norm_block_backward(dn, x, w, gr, y, a, dh=dh)
    again = gdn.gdn_norm_block_backward(dn, x, w, gr, y, a, dh=dh)
    torch.cuda.synchronize()
    assert all(p is None or torch.equal(p, q) for p, q in zip(got, again))
    errs = {"n": worst(gn, n, b["n"]), "rstd": worst(gr, r, b["rstd"])}
    if mode == "alone":
        assert gh is x and got[1] is None and got[3] is None
    else:
        errs["h"] = worst(gh, h, b["h"])
    if mode == "added":
        assert got[1] is got[0] and got[3] is None
    for i, name in enumerate(("dx", "dy", "dweight", "dres_scale")):
        if got[i] is not None and name in b:
            errs[name] = worst(got[i], grads[i], b[name])
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("shape", [(3, 16384), (600, 10000)])
def test_norm_block_wide(shape):
    """The widest rows, more of them than there are workgroups."""
    import gated_delta_rule_52_amd as gdn
    W = shape[-1]
    x, y, dn, dh = (rand(*shape, dtype=torch.bfloat16, seed=i) for i in range(4))
    w, a = rand(W, std=0.2, mean=1.0, seed=5), rand(W, std=0.3, mean=0.5, seed=6)
    (h, n, r), grads, b = block_bounds(torch.bfloat16, x, y, a, w, dn, dh)
    gh, gn, gr = gdn.gdn_norm_block(x, w, y, a)
    got = gdn.gdn_norm_block_backward(dn, x, w, gr, y, a, dh=dh)
    torch.cuda.synchronize()
    errs = {"h": worst(gh, h, b["h"]), "n": worst(gn, n, b["n"]), "rstd": worst(gr, r, b["rstd"])}
    for name, t, want in zip(("dx", "dy", "dweight", "dres_scale"), got, grads):
        errs[name] = worst(t, want, b[name])
    log(f"wide {shape}: " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs
    with pytest.raises(gdn.GdnError):
        gdn.gdn_norm_block(torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda"), torch.ones(16392, device="cuda"))


def test_norm_block_edges():
    """Rows of zeros, no rows, outputs in place of the inputs, only n."""
    import gated_delta_rule_52_amd as gdn
    w = rand(64, mean=1.0)
    z = torch.zeros(3, 64, device="cuda")
    h, n, r = gdn.gdn_norm_block(z, w, z)
    assert torch.equal(n, z) and torch.equal(h, z) and torch.allclose(r, torch.full_like(r, 1e3))
    e = torch.zeros(0, 64, device="cuda", dtype=torch.bfloat16)
    h, n, r = gdn.gdn_norm_block(e, w, e)
    dx, _, dw, da = gdn.gdn_norm_block_backward(e, e, w, r, e, w)
    assert dx.shape == e.shape and torch.equal(dw, torch.zeros_like(w)) and torch.equal(da, torch.zeros_like(w))
    x, y = rand(40, 640, dtype=torch.bfloat16), rand(40, 640, dtype=torch.bfloat16, seed=1)
    w, a = rand(640), rand(640, seed=2)
    h, n, r = gdn.gdn_norm_block(x, w, y, a)
    xx, yy = x.clone(), y.clone()
    gdn.gdn_norm_block(xx, w, yy, a, out=(xx, yy, None))
    n2 = torch.empty_like(x)
    gdn.gdn_norm_block(x, w, y, a, out=(None, n2, None))
    assert torch.equal(xx, h) and torch.equal(yy, n) and torch.equal(n2, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens,heads,stride", [(1, 1, 0), (5, 3, 0), (257, 6, 2), (33, 16, 3), (9000, 1, 0)])
def test_norm_gate(dtype, D, tokens, heads, stride):
    import gated_delta_rule_52_amd as gdn
    dt = DT[dtype]
    log(f"norm_gate {dtype} D={D} tokens={tokens} heads={heads} stride={stride}")
    o, w, dy = rand(tokens, heads, D, dtype=dt, std=0.3), rand(D, mean=1.0, std=0.2), rand(tokens, heads, D, dtype=dt, seed=3)
    z = rand(tokens, max(stride, 1), heads, D, dtype=dt, std=3.0, seed=2)[:, -1]
    assert stride == 0 or tokens == 1 or not z.is_contiguous()
    y, r = ref.norm_gate(o, z, w)
    do, dz, dw = ref.norm_gate_backward(dy, o, z, w)
    gy, gr = gdn.gdn_norm_gate(o, z, w)
    got = gdn.gdn_norm_gate_backward(dy, o, z, w, gr)
    again = gdn.gdn_norm_gate_backward(dy, o, z, w, gr)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    # the exponent's error: |z| 2^-24 twice (its scaling and the hardware's argument), so the factors take |z| more steps
    u = (D + 24 + 4 * float(z.float().abs().max())) * U32
    s = 1 / (1 + torch.exp(-f64(z)))
    oh, act, d64 = f64(o) * r[..., None], f64(z) * s, f64(dy).abs()
    gs = d64 * act.abs() * f64(w).abs()
    errs = {
        "y": worst(gy, y, (HALF[dt] + u) * y.abs()),
        "rstd": worst(gr, r, u * r),
        "do": worst(got[0], do, HALF[dt] * do.abs() + u * r[..., None] * (gs + oh.abs() * (gs * oh.abs()).mean(-1, keepdim=True))),
        "dz": worst(got[1], dz, HALF[dt] * dz.abs() + u * d64 * oh.abs() * f64(w).abs() * s * (1 + f64(z).abs())),
        "dw": worst(got[2], dw, (u + tokens * heads * U32) * (d64 * act.abs() * oh.abs()).sum((0, 1))),
    }
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


def test_norm_gate_no_tokens_and_batches():
    """No tokens: the weight's gradient is zero.  [B, T, H, D] with a gate whose
    tokens have one stride is taken as it is, with two it is refused."""
    import gated_delta_rule_52_amd as gdn
    w = rand(32, mean=1.0)
    e = torch.zeros(0, 2, 32, device="cuda")
    y, r = gdn.gdn_norm_gate(e, e, w)
    do, dz, dw = gdn.gdn_norm_gate_backward(e, e, e, w, r)
    torch.cuda.synchronize()
    assert y.shape == e.shape and torch.equal(dw, torch.zeros_like(w))
    o = rand(3, 5, 2, 32)
    z = rand(3, 5, 4, 32, seed=1)[:, :, 2:]
    y, r = gdn.gdn_norm_gate(o, z, w)
    want, _ = gdn.gdn_norm_gate(o.view(15, 2, 32), z.reshape(15, 2, 32), w)
    assert torch.equal(y.view(15, 2, 32), want) and r.shape == (3, 5, 2)
    with pytest.raises(ValueError):
        gdn.gdn_norm_gate(o, rand(5, 3, 2, 32).transpose(0, 1), w)


def test_norm_gate_extreme_gates():
    """Gates far out: silu is 0 below and the gate itself above, with no NaN."""
    import gated_delta_rule_52_amd as gdn
    z = torch.tensor([-1e4, -200.0, -100.0, 0.0, 100.0, 1e4] + [1.0] * 10, device="cuda").repeat(2, 1, 1)
    o, w = torch.ones_like(z), torch.ones(16, device="cuda")
    y, r = gdn.gdn_norm_gate(o, z, w)
    do, dz, dw = gdn.gdn_norm_gate_backward(torch.ones_like(z), o, z, w, r)
    want = ref.norm_gate(o, z, w)[0]
    # below the last exponent the value is 0 where the plain form has at most 1e4 exp(-100) < 1e-39
    assert worst(y, want, 600 * U32 * want.abs() + 1e-36) <= 1
    assert torch.isfinite(do).all() and torch.isfinite(dz).all() and torch.isfinite(dw).all()


def test_other_stream_and_graph():
    """On a side stream, and captured: every replay gives the eager bits."""
    import gated_delta_rule_52_amd as gdn
    x, y, dn = (rand(700, 768, dtype=torch.bfloat16, seed=i) for i in range(3))
    w, a = rand(768, mean=1.0), rand(768, seed=9)
    ws = torch.empty(1 << 23, dtype=torch.uint8, device="cuda")
    fwd = (torch.empty_like(x), torch.empty_like(x), torch.empty(700, device="cuda"))
    bwd = (torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w))

    def step():
        gdn.gdn_norm_block(x, w, y, a, out=fwd)
        gdn.gdn_norm_block_backward(dn, x, w, fwd[2], y, a, out=bwd, ws=ws)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in fwd + bwd]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in fwd + bwd:
            t.fill_(float("nan"))
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(fwd + bwd, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for t in fwd + bwd:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(fwd + bwd, want)), i
        step()
        torch.cuda.synchronize()
