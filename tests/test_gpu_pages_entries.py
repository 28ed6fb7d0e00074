"""The page step on lengths and entries that no pool in order has."""
import pytest
import torch

from test_gpu_attention import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [True, False])
def test_release_takes_a_length_below_zero_as_zero(in_place):
    """As gdn_pages_take does: a sequence that goes on begins at position 0."""
    import gated_delta_rule_52_amd as gdn
    kv, table, free, count = ints([-7, 20, -1, 5]), ints([[1, -1], [2, 3], [4, -1], [0, -1]]), ints([9] * 6), ints([1])
    new = {} if in_place else dict(kv_out=torch.full_like(kv, 77), count_out=torch.full_like(count, 77))
    kv1, c1 = gdn.gdn_pages_release(ints([0, 0, 1, 1]), kv, table, free, count, 16, **new)
    torch.cuda.synchronize()
    assert kv1.tolist() == [0, 20, 0, 0] and c1.tolist() == [2] and free.tolist() == [9, 0, 9, 9, 9, 9]
