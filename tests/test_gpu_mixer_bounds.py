"""Sequence bounds that decrease, in the state-space layer's operators: a bound below
an earlier one counts as that one, whatever the size of the call, so that the given
bounds and their running maximum have the same results, bit for bit."""
from itertools import accumulate

import pytest
import torch

from gpu_util import log
from test_gpu_attention import DT, ints
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
