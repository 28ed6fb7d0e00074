"""How far the scan's results may be from the 64-bit form as a whole.

The bounds of mixer_reference.py hold for any values: they sum magnitudes, also of
terms that cancel, and grow with the tokens, so over many tokens they are wider than
the steps' gradients themselves.  These are for inputs of random signs, whose sums of
terms are about as large as the root of the sum of their squares.  A term of a float32
result takes fewer than 64 roundings (three factors of its decay, each with its
exponent's, delta, the sums over N and P and along the tokens), which as often go up
as down: so the results' 2-norm is within 64 U32 = 2^-18 of its own.  A sum over all
tokens (dA, dD, ddt_bias) is off by its terms' errors, so by 2^-18 of the sum of their
magnitudes: of delta dg, of dy x, of ddt.  A bf16 result is rounded once when stored,
its pairs' factor (E G or E Z delta) once, and the states' part once: 3 HALF.
"""
import torch

import mixer_reference as ref
from mixer_reference import HALF, f64

SUMS = ("dA", "dD", "ddt_bias")


def definition(s, cu, keep=None):
    """The 64-bit form of a call's results, with the sums of the magnitudes."""
    H = s["x"].shape[1]
    size = {k: torch.zeros(H).double() for k in SUMS}

    def note(b, h, **p):
        size["dA"][h] += (p["d"] * p["dg"]).abs().sum()
        size["dD"][h] += p["yx"].abs().sum()
        size["ddt_bias"][h] += p["dd"].abs().sum()
        if keep is not None:
            keep(b, h, **p)

    out = ref.ssm(s["x"], s["dt"], s["A"], s["B"], s["C"], cu, s["D"], s["dt_bias"], True, s["h0"], s["dy"], s["dhT"], keep=note)
    return {k: v[0] for k, v in out.items()}, size


def shares(got, want, size):
    """{name: the share that a result's error has of what it may be}"""
    out = {}
    for k, v in got.items():
        if v is None:
            continue
        err = f64(v) - want[k]
        if k in SUMS:
            out[k] = float((err.abs() / (2.0 ** -18 * size[k])).max())
        else:
            may = 3 * HALF[v.dtype] if v.dtype == torch.bfloat16 else 2.0 ** -18
            out[k] = float(err.norm() / (may * want[k].norm()))
    return out
