"""Host side: outputs that are inputs which a later launch, or another workgroup, still
reads are refused before any launch (no pointer below is ever followed)."""
import ctypes

import pytest

import gated_delta_rule_52_amd as gdn
from test_block_abi import BIG
from test_mixer_abi import conv, ssm

CONV = ("x", "weight", "bias", "cu", "state", "dy", "dstate_out", "dx", "dweight", "dbias", "dstate", "ws")


def at(names):
    return {n: ctypes.c_void_p(4096 * (i + 1)) for i, n in enumerate(names)}


@pytest.mark.parametrize("out,of", [("dx", "x"), ("dx", "dy"), ("dstate", "dstate_out"), ("dweight", "weight"), ("dbias", "bias")])
def test_conv_backward_refuses_outputs_that_are_inputs(out, of):
    """dstate's rows are sums with rows of dstate_out that an earlier one would have
    replaced, and its launch reads weight and bias behind the one that writes their
    gradients."""
    p = at(CONV)
    p[out] = p[of]
    assert gdn.lib().gdn_conv_backward(conv(), *p.values(), BIG, None) == 1


SCAN = ("x", "dt", "A", "B", "C", "D", "dt_bias", "cu", "h0", "dy", "dhT", "dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0", "ws")


@pytest.mark.parametrize("out,of", [(o, i) for o in ("dx", "dB", "dC") for i in ("x", "B", "C", "dy")]
                         + [("dx", "dB"), ("dx", "dC"), ("dB", "dC"), ("dh0", "h0"), ("dh0", "dhT")])
def test_scan_backward_refuses_outputs_that_are_inputs(out, of):
    """One head a group and N = P: x and B are of one size."""
    p = at(SCAN)
    p[out] = p[of]
    assert gdn.lib().gdn_ssm_backward(ssm(H=2, G=2), *p.values(), BIG, None) == 1


@pytest.mark.parametrize("of", ["x", "B", "C"])
def test_scan_refuses_outputs_that_are_inputs(of):
    p = at(("x", "dt", "A", "B", "C", "D", "dt_bias", "cu", "h0", "y", "hT", "ws"))
    p["y"] = p[of]
    assert gdn.lib().gdn_ssm_forward(ssm(H=2, G=2), *p.values(), BIG, None) == 1
    p = at(("x", "dt", "A", "B", "C", "D", "dt_bias", "state", "y"))
    p["y"] = p[of]
    assert gdn.lib().gdn_ssm_step(ssm(T=2, H=2, G=2), *p.values(), None) == 1
