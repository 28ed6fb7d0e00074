"""The scan's results as a whole over many chunks and segments: within what their
roundings leave of random inputs (ssm_checks.py), the sums over all tokens among them."""
import pytest
import torch

import ssm_checks
from gpu_util import log
from test_gpu_attention import DT, cumulate
from test_gpu_ssm import GRADS, backward, forward, make

pytestmark = pytest.mark.gpu

AMONG = [1, 0, 2] * 20  # short sequences, before a long one


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,decay", [
    ([300, 31, 33], (3, 1, 64, 128), 1.0), ([127, 128, 129, 1], (2, 2, 128, 64), 1.0),  # a few chunks
    ([2500, 40, 700], (4, 1, 128, 64), 1.0), ([1700], (8, 2, 64, 64), 1.0), ([513, 1025, 129], (2, 1, 128, 128), 1.0),  # segments
    (AMONG + [8700] + [1] * 30 + [130, 0, 3], (2, 1, 64, 64), 0.1),  # one long sequence's segments
    ([(97 * b) % 500 for b in range(150)], (6, 2, 64, 64), 1.0), ([(97 * b) % 300 for b in range(110)], (4, 1, 64, 128), 1.0),  # all of a group's heads
], ids=lambda v: str(v)[:24])
def test_results_as_a_whole(dtype, lens, heads, decay):
    dt = DT[dtype]
    if dtype == "f32" and max(lens) > 5000:
        lens = AMONG + [4400] + [1] * 30 + [130, 0, 3]
    cu = cumulate(lens)
    log(f"whole {dtype} {len(lens)} sequences, {cu[-1]} tokens {heads}")
    s = make(cu[-1], len(lens), *heads, dt, decay=decay)
    got = dict(zip(GRADS, backward(s, cu)))
    got["y"], got["hT"] = forward(s, cu)
    torch.cuda.synchronize()
    want, size = ssm_checks.definition(s, cu)
    errs = ssm_checks.shares(got, want, size)
    log("  " + " ".join(f"{k}={v:.4f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs
