"""The checks of ssm_checks.py let right results pass and refuse wrong ones: results
with a part left out, each as a kernel that forgets it would give them (CPU)."""
import pytest
import torch

import ssm_checks
from mixer_reference import f64

L, BLOCK = 128, 32  # a chunk of bf16 calls and its blocks
LENS = [300, 31, 330]


def inputs(dt):
    g = torch.Generator().manual_seed(3)
    r = lambda *s, std=1.0, dtype=torch.float32: (torch.randn(s, generator=g) * std).to(dtype)  # noqa: E731
    T, B, H, G, N, P = sum(LENS), len(LENS), 2, 1, 64, 64
    return dict(x=r(T, H, P, dtype=dt), dt=r(T, H, std=0.5), A=-torch.linspace(1, 16, H), B=r(T, G, N, dtype=dt), C=r(T, G, N, dtype=dt),
                D=r(H), dt_bias=torch.linspace(-5, -2, H), h0=r(B, H, N, P), dy=r(T, H, P, dtype=dt), dhT=r(B, H, N, P, std=0.3))


@pytest.fixture(scope="module")
def case():
    s, kept = inputs(torch.bfloat16), {}
    cu = [0]
    for n in LENS:
        cu.append(cu[-1] + n)
    want, size = ssm_checks.definition(s, cu, lambda b, h, **p: kept.update({(b, h): p}))
    return s, cu, want, size, kept


def stored(want):
    """As a call of bf16 inputs returns them."""
    return {k: v.to(torch.bfloat16 if k in ("y", "dx", "dB", "dC") else torch.float32) for k, v in want.items()}


def without(case, missing):
    """The results whose dg lacks missing(pieces, n): [n] of a sequence and head."""
    s, cu, want, size, kept = case
    got = {k: f64(v).clone() for k, v in want.items()}
    for (b, h), p in kept.items():
        less = missing(p, len(p["d"]))
        ddt = p["A"] * less * p["slope"]
        got["ddt"][cu[b]:cu[b + 1], h] -= ddt
        got["dA"][h] -= (p["d"] * less).sum()
        got["ddt_bias"][h] -= ddt.sum()
    return stored(got)


def pairs_over(p, n, unit, outside):
    """For every token, the sum of the pairs from before its unit to behind it, within
    its `outside` (a multiple of the unit)."""
    out = torch.zeros(n).double()
    for a in range(0, n, unit):
        e, lo = min(a + unit, n), a // outside * outside
        out[a:e] = p["M"][e:lo + outside, lo:a].sum()
    return out


def test_right_results_pass(case):
    s, cu, want, size, kept = case
    errs = ssm_checks.shares(stored(want), want, size)
    assert max(errs.values()) < 0.5, errs
    noise = {k: f64(v) * (1 + 2.0 ** -22 * torch.randn(v.shape).double()) for k, v in want.items()}
    errs = ssm_checks.shares({k: v.float() for k, v in noise.items() if k in ("hT", "ddt", "dh0")}, want, size)
    assert max(errs.values()) < 1, errs


@pytest.mark.parametrize("name", ["dA", "dD", "ddt_bias", "ddt", "hT", "dh0", "y", "dx", "dB", "dC"])
def test_zeros_are_refused(case, name):
    s, cu, want, size, kept = case
    got = stored(want)
    got[name] = torch.zeros_like(got[name])
    assert ssm_checks.shares(got, want, size)[name] > 1


@pytest.mark.parametrize("name", ["dA", "dD", "ddt_bias"])
@pytest.mark.parametrize("seq,chunk", [(0, 0), (0, 2), (1, 0), (2, 1)])
def test_a_sum_that_lacks_a_chunk_is_refused(case, name, seq, chunk):
    s, cu, want, size, kept = case
    got = stored(want)
    for h in range(2):
        p = kept[seq, h]
        term = {"dA": p["d"] * p["dg"], "dD": p["yx"], "ddt_bias": p["dd"]}[name]
        got[name][h] -= term[chunk * L:(chunk + 1) * L].sum().float()
    assert ssm_checks.shares(got, want, size)[name] > 1


@pytest.mark.parametrize("missing", [
    lambda p, n: pairs_over(p, n, L, 1 << 20),                             # from before a chunk to behind it: <S, dS>
    lambda p, n: pairs_over(p, n, BLOCK, L),                               # over a block within its chunk
    lambda p, n: torch.full((n,), 1.0).double() * p["through"],            # from the first state to the last gradient
    lambda p, n: torch.cat([p["dg"][:L] * 0, p["dg"][L:L + 1], p["dg"][L + 1:] * 0]),  # one token's
], ids=["chunk", "block", "states", "token"])
def test_step_gradients_that_lack_a_part_are_refused(case, missing):
    s, cu, want, size, kept = case
    errs = ssm_checks.shares(without(case, missing), want, size)
    assert errs["ddt"] > 1 and max(errs["dA"], errs["ddt_bias"]) > 1, errs


def test_the_pairs_are_those_of_the_definition(case):
    """dg less the pairs within 32 tokens, by the pieces above, adds up: what the
    mutants leave out is really in it."""
    s, cu, want, size, kept = case
    for (b, h), p in kept.items():
        n = len(p["d"])
        over = torch.stack([p["M"][t:, :t].sum() for t in range(n)])
        t = n // 2
        a, e = t // L * L, min(t // L * L + L, n)
        parts = p["M"][e:, :a].sum() + p["M"][t:e, a:t].sum() + p["M"][e:, a:t].sum() + p["M"][t:e, :a].sum()
        assert abs(float(over[t] - parts)) <= 1e-9 * float(p["M"].abs().sum())
