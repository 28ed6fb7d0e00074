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


def test_entries_that_are_no_pages_are_handed_on():
    """A length that claims a page which the table does not have: -1 goes on the stack as
    it stands, and a token that gets it has no slot; the others keep theirs.  Names of
    pages are not held to the stack's room."""
    import gated_delta_rule_52_amd as gdn
    kv, table, free, count = ints([40, 0]), ints([[5, -1, 300, -1], [-1, -1, -1, -1]]), ints([9] * 4), ints([1])
    gdn.gdn_pages_release(ints([1, 0]), kv, table, free, count, 16)
    assert kv.tolist() == [0, 0] and count.tolist() == [4] and free.tolist() == [9, 5, -1, 300]
    _, _, cu, pos, slots = gdn.gdn_pages_take(ints([0, 40]), kv, table, free, count, 16, 40)
    torch.cuda.synchronize()
    assert kv.tolist() == [0, 40] and count.tolist() == [1] and cu.tolist() == [0, 0, 40] and pos.tolist() == list(range(40))
    assert table.tolist()[1] == [300, -1, 5, -1]
    assert slots.tolist() == [4800 + i for i in range(16)] + [-1] * 16 + [80 + i for i in range(8)]


def test_slots_of_no_page_are_not_written():
    """What gdn_attn_append does with such a table: the tokens without a page, and those
    whose page the cache does not have, leave it as it was."""
    import gated_delta_rule_52_amd as gdn
    kc = torch.full((6, 16, 1, 64), 7.0, device="cuda")
    vc = kc.clone()
    k = torch.randn(40, 1, 64, device="cuda")
    gdn.gdn_attn_append(None, k, k, None, None, ints([0, 40]), ints([40]), ints([[300, -1, 5, -1]]), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc[5, :8], k[32:]) and (kc[5, 8:] == 7.0).all() and (kc[:5] == 7.0).all() and torch.equal(kc, vc)
