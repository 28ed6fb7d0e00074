"""The page step against the plain form in lists: whole numbers, equal."""
import random

import pytest
import torch

import mixer_reference as ref
from gpu_util import log
from test_gpu_attention import ints

pytestmark = pytest.mark.gpu


def pool(lens, ps, spare, width, seed):
    rng = random.Random(seed)
    held = [-(-n // ps) for n in lens]
    order = list(range(sum(held) + spare))
    rng.shuffle(order)
    table, at = [[-1] * width for _ in lens], 0
    for b, n in enumerate(held):
        table[b][:n] = order[at:at + n]
        at += n
    return table, order[at:] + [-1] * at, spare


def step(lens, done, want, ps, spare, width, rows, seed, in_place):
    import gated_delta_rule_52_amd as gdn
    table, free, count = pool(lens, ps, spare, width, seed)
    t, f, kv, c = ints(table), ints(free), ints(lens), ints([count])
    new = (lambda x: None) if in_place else torch.empty_like
    kv1, c1 = gdn.gdn_pages_release(ints(done), kv, t, f, c, ps, kv_out=new(kv), count_out=new(c))
    kv2, c2, cu, pos, slots = gdn.gdn_pages_take(ints(want), kv1, t, f, c1, ps, rows, kv_out=new(kv), count_out=new(c))
    torch.cuda.synchronize()
    if in_place:
        assert kv2 is kv and c2 is c
    else:
        assert kv.tolist() == lens and c.tolist() == [count]
    wkv, wc, wfree = ref.pages_release(done, lens, table, free, count, ps)
    if not in_place:
        assert kv1.tolist() == wkv and c1.tolist() == [wc]
    assert f.tolist() == wfree
    wkv, wc, wtable, wcu, wpos, wslots = ref.pages_take(want, wkv, table, wfree, wc, ps, rows)
    assert kv2.tolist() == wkv and c2.tolist() == [wc] and cu.tolist() == wcu and t.tolist() == wtable
    n = wcu[-1]
    assert pos.tolist() == wpos + [-1] * (rows - n) and slots.tolist() == wslots + [-1] * (rows - n)
    return wcu


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("B,ps,most,new,spare", [(1, 16, 40, 1, 3), (3, 16, 5, 60, 4), (64, 32, 300, 1, 10), (256, 16, 700, 1, 5),
                                                 (70, 64, 500, 300, 200), (1000, 16, 50, 3, 100), (1025, 128, 20, 2, 30),
                                                 (2500, 16, 30, 40, 3000), (5, 1024, 3000, 5000, 12), (1, 16, 0, 20000, 1300)])
def test_step(B, ps, most, new, spare, in_place):
    rng = random.Random(B + ps)
    for kind in range(4):
        lens = [rng.randint(0, most) for _ in range(B)]
        done = [int(rng.random() < 0.2) for _ in range(B)]
        want = [new if kind == 0 else rng.randint(0, new) for _ in range(B)]
        width = -(-(most + new) // ps) + (0 if kind != 2 else -1)  # too narrow for some
        width = max(width, -(-max(lens + [1]) // ps))
        rows = sum(want) if kind != 3 else max(1, sum(want) // 2)
        cu = step(lens, done, want, ps, spare, width, rows, kind, in_place)
        log(f"pages B={B} ps={ps} kind={kind}: {cu[-1]} of {sum(want)} tokens")


def test_odd_values():
    """Lengths and counts out of range, sequences that want nothing, no rows at all."""
    import gated_delta_rule_52_amd as gdn
    t, f = ints([[3, -1], [1, 2], [-1, -1]]), ints([0, 4, 5, 6])
    kv, c, cu, pos, slots = gdn.gdn_pages_take(ints([5, -3, 1]), ints([-7, 32, 16]), t, f, ints([99]), 16, 8, kv_out=ints([9] * 3),
                                               count_out=ints([9]))
    # a count past the pool is the pool; a length below 0 is 0; position 16 of the third has a new page
    assert kv.tolist() == [5, 32, 17] and c.tolist() == [2] and cu.tolist() == [0, 5, 5, 6]
    assert t.tolist() == [[6, -1], [1, 2], [-1, 5]]
    assert pos.tolist() == [0, 1, 2, 3, 4, 16, -1, -1] and slots.tolist() == [96, 97, 98, 99, 100, 80, -1, -1]
    kv, c, cu, pos, slots = gdn.gdn_pages_take(ints([1]), ints([3]), ints([[-1]]), f, ints([2]), 16, 4)
    assert pos.tolist()[0] == 3 and slots.tolist() == [-1] * 4  # the page that the length claims is not there
    kv, c, cu, pos, slots = gdn.gdn_pages_take(ints([1]), ints([0]), ints([[-1]]), f, ints([2]), 16, 0)
    assert kv.tolist() == [0] and c.tolist() == [2] and cu.tolist() == [0, 0] and pos.numel() == 0
    kv, c, cu, pos, slots = gdn.gdn_pages_take(ints([1]), ints([0]), ints([[-1]]), f, ints([2]), 16, 4, want_maps=False)
    assert kv.tolist() == [1] and pos is None and slots is None
    # more pages come back than the stack has room for: it ends full
    f = ints([9, 9, 9])
    kv, c = gdn.gdn_pages_release(ints([1, 1]), ints([30, 40]), ints([[5, 6], [7, 8]]), f, ints([1]), 16)
    assert kv.tolist() == [0, 0] and c.tolist() == [3] and f.tolist() == [9, 5, 6]
    kv, c = gdn.gdn_pages_release(ints([1]), ints([-4]), ints([[5, 6]]), f, ints([-1]), 16)
    assert kv.tolist() == [0] and c.tolist() == [0]


def test_binding_refusals():
    import gated_delta_rule_52_amd as gdn
    a = [ints([1, 1]), ints([0, 0]), ints([[-1], [-1]]), ints([0, 1]), ints([2])]
    take = lambda i, t: gdn.gdn_pages_take(*a[:i], t, *a[i + 1:], 16, 4)  # noqa: E731
    for i, t in enumerate((ints([1]), ints([0]), ints([[-1]]), ints([[0]]), ints([2, 2]))):
        with pytest.raises(ValueError):
            take(i, t)
    for i in range(5):
        with pytest.raises(TypeError):
            take(i, a[i].long())
    with pytest.raises(ValueError):
        gdn.gdn_pages_take(*a, 16, 4, slots=torch.empty(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_pages_take(*a, 24, 4)
