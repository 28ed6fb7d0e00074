"""The norms where their launch rules take their other branches: outputs larger
than the L2, more rows than one grid of the forward holds, and both with outputs
in place of the inputs.  Bounds as in test_gpu_norm.py."""
import pytest
import torch

import block_reference as ref
from block_reference import HALF, U32, f64, worst
from gpu_util import log
from test_gpu_norm import DT, block_bounds, rand

pytestmark = pytest.mark.gpu

# rows, width: past one grid of 4096 workgroups (70001 x 8, 4200 x 4104), past 32 MB (all but 70001 x 8)
BLOCK = [("bf16", 21931, 768), ("bf16", 1101, 16384), ("bf16", 70001, 8), ("bf16", 4200, 4104), ("bf16", 66001, 264),
         ("f32", 11003, 768), ("f32", 1101, 8192), ("f32", 4200, 2052), ("f32", 70001, 128)]


@pytest.mark.parametrize("dtype,rows,width", BLOCK)
def test_norm_block_large(dtype, rows, width):
    import gated_delta_rule_52_amd as gdn
    dt = DT[dtype]
    log(f"norm_block {dtype} {rows} x {width}")
    x, y, dn, dh = (rand(rows, width, dtype=dt, seed=i) for i in range(4))
    w, a = rand(width, std=0.2, mean=1.0, seed=5), rand(width, std=0.3, mean=0.5, seed=6)
    gh, gn, gr = gdn.gdn_norm_block(x, w, y, a)
    got = gdn.gdn_norm_block_backward(dn, x, w, gr, y, a, dh=dh)
    again = gdn.gdn_norm_block_backward(dn, x, w, gr, y, a, dh=dh)
    hx, nx = x.clone(), torch.empty_like(x)
    gdn.gdn_norm_block(hx, w, y, a, out=(hx, nx, None))  # h in place of x
    hy = y.clone()
    gdn.gdn_norm_block(x, w, hy, a, out=(hy, torch.empty_like(x), None))  # h in place of y
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    assert torch.equal(hx, gh) and torch.equal(hy, gh) and torch.equal(nx, gn)
    with ref.where("cuda"):
        (h, n, r), grads, b = block_bounds(dt, x, y, a, w, dn, dh)
        errs = {"h": worst(gh, h, b["h"]), "n": worst(gn, n, b["n"]), "rstd": worst(gr, r, b["rstd"])}
        for name, t, want in zip(("dx", "dy", "dweight", "dres_scale"), got, grads):
            errs[name] = worst(t, want, b[name])
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("dtype,tokens,heads,D", [("bf16", 21931, 6, 128), ("f32", 11003, 6, 128), ("f32", 131101, 1, 64),
                                                  ("bf16", 262150, 4, 16)])
def test_norm_gate_large(dtype, tokens, heads, D):
    import gated_delta_rule_52_amd as gdn
    dt = DT[dtype]
    log(f"norm_gate {dtype} {tokens} x {heads} x {D}")
    o, w, dy = rand(tokens, heads, D, dtype=dt, std=0.3), rand(D, mean=1.0, std=0.2), rand(tokens, heads, D, dtype=dt, seed=3)
    z = rand(tokens, 2, heads, D, dtype=dt, std=3.0, seed=2)[:, 1]
    gy, gr = gdn.gdn_norm_gate(o, z, w)
    got = gdn.gdn_norm_gate_backward(dy, o, z, w, gr)
    again = gdn.gdn_norm_gate_backward(dy, o, z, w, gr)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    with ref.where("cuda"):
        y, r = ref.norm_gate(o, z, w)
        do, dz, dw = ref.norm_gate_backward(dy, o, z, w)
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
