"""Infinities and NaN reach the results that depend on them, and no others.  What
does not depend on them has the bits that it has without them: a masked value
takes part in no sum.  (A score moves the running maximum of its own row, and with
it when the other 31 rows of a wave are rescaled: where a key is not finite, the
rows before it are compared with the 64-bit form.  So are the gradients of keys in
a masked tile with a row that is not finite: that tile is then summed last.)"""
import pytest
import torch

import block_reference as ref
from gpu_util import log
from test_gpu_attention import DT, cumulate, ints, make_cache, qkv, rand

pytestmark = pytest.mark.gpu

NAN = float("nan")
VALUES = {"nan": NAN, "inf": float("inf"), "-inf": -float("inf")}
LENS = [[1, 37], [64, 3], [131], [700, 260]]


def spots(n):
    return sorted({0, 1, n // 3, min(31, n - 1), min(32, n - 1), n - 2 if n > 1 else 0, n - 1})


def same(a, b, rows, what):
    assert torch.equal(a[rows], b[rows]), what


def seen_column(got, clean, rows, heads, col, what):
    """Rows that see the value: not finite in its column, the same in the others."""
    x = got[rows][:, heads]
    assert not torch.isfinite(x[..., col].float()).any(), what
    keep = [c for c in range(x.shape[-1]) if c != col]
    assert torch.equal(x[..., keep], clean[rows][:, heads][..., keep]), what


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,heads", [(64, (4, 2)), (128, (3, 3)), (128, (16, 4))])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompt_values_and_keys(dtype, D, heads, lens):
    import gated_delta_rule_52_amd as gdn
    dt, (Hq, Hkv) = DT[dtype], heads
    G, cu = Hq // Hkv, cumulate(lens)
    log(f"not finite, prompt {dtype} D={D} heads={heads} {lens}")
    q, k, v = (t.contiguous() for t in qkv(cu[-1], Hq, Hkv, D, dt, True))
    c = ints(cu)
    clean, lse = gdn.gdn_attn_forward(q, k, v, c)
    with ref.where("cuda"):
        want, wl, bo, bl = ref.prompt(q, k, v, cu)
    hk, col = Hkv - 1, 5
    mine = list(range(hk * G, Hq))
    others = list(range(hk * G))
    a, e = cu[-2], cu[-1]  # the last sequence
    for n, i in enumerate(spots(e - a)):
        value = list(VALUES.values())[n % 3]
        bad = v.clone()
        bad[a + i, hk, col] = value
        o, l = gdn.gdn_attn_forward(q, k, bad, c)
        assert torch.equal(l, lse)
        same(o, clean, slice(0, a + i), (i, value))
        same(o[:, others], clean[:, others], slice(None), (i, value))
        seen_column(o, clean, slice(a + i, e), mine, col, (i, value))
        bad = k.clone()
        bad[a + i, hk, col] = VALUES["nan"]
        o, l = gdn.gdn_attn_forward(q, bad, v, c)
        before = slice(0, a + i)
        with ref.where("cuda"):
            assert ref.worst(o[before], want[before], bo[before]) <= 1 and ref.worst(l[before], wl[before], bl[before]) <= 1
        same(o, clean, slice(0, a), i)
        same(o[:, others], clean[:, others], slice(None), i)
        assert torch.isnan(o[a + i:e, mine].float()).all() and torch.isnan(l[a + i:e, mine]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,heads", [(64, (4, 2)), (128, (8, 2))])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompt_gradients(dtype, D, heads, lens):
    import gated_delta_rule_52_amd as gdn
    dt, (Hq, Hkv) = DT[dtype], heads
    G, cu = Hq // Hkv, cumulate(lens)
    log(f"not finite, gradients {dtype} D={D} heads={heads} {lens}")
    q, k, v = (t.contiguous() for t in qkv(cu[-1], Hq, Hkv, D, dt, True))
    dO, c = rand(cu[-1], Hq, D, dtype=dt, seed=8), ints(cu)
    o, lse = gdn.gdn_attn_forward(q, k, v, c)
    clean = gdn.gdn_attn_backward(q, k, v, c, o, lse, dO)
    with ref.where("cuda"):
        exact = ref.prompt_backward(q, k, v, cu, dO)

    def keys_behind(got, name, row, hk, i):
        """dk or dv: keys of other heads and sequences have their bits; those of the
        last sequence behind `row` are within the bounds."""
        want = clean[1 if name == "dk" else 2]
        same(got, want, slice(0, cu[-2]), i)
        same(got[:, :hk], want[:, :hk], slice(None), i)
        x, bound = exact[name]
        with ref.where("cuda"):
            assert ref.worst(got[row + 1:], x[row + 1:], bound[row + 1:]) <= 1, (i, name)

    h, hk, col = Hq - 1, Hkv - 1, 7
    a, e = cu[-2], cu[-1]
    for n, i in enumerate(spots(e - a)):
        value = list(VALUES.values())[n % 3]
        row = a + i
        away = [x for x in range(cu[-1]) if x != row]
        # dO of one row: its own dq, and dk, dv of the keys up to it
        bad = dO.clone()
        bad[row, h, col] = value
        dq, dk, dv = gdn.gdn_attn_backward(q, k, v, c, o, lse, bad)
        same(dq, clean[0], away, i)
        for got, name in ((dk, "dk"), (dv, "dv")):
            keys_behind(got, name, row, hk, i)
        x, bound = exact["dv"]
        assert not torch.isfinite(dv[a:row + 1, hk, col].float()).any(), i
        keep = [d for d in range(D) if d != col]
        with ref.where("cuda"):
            assert ref.worst(dv[a:row + 1, hk][:, keep], x[a:row + 1, hk][:, keep], bound[a:row + 1, hk][:, keep]) <= 1, i
        # q of one row
        bad = q.clone()
        bad[row, h, col] = VALUES["nan"]
        bo, bl = o.clone(), lse.clone()
        bo[row, h], bl[row, h] = NAN, NAN
        dq, dk, dv = gdn.gdn_attn_backward(bad, k, v, c, bo, bl, dO)
        same(dq, clean[0], away, i)
        for got, name in ((dk, "dk"), (dv, "dv")):
            keys_behind(got, name, row, hk, i)
            assert torch.isnan(got[a:row + 1, hk].float()).all()
        # k and v of one row: dq of the rows before it; v leaves dv alone
        for which in (0, 1):
            kk, vv = k.clone(), v.clone()
            (kk, vv)[which][row, hk, col] = value
            bo, bl = o.clone(), lse.clone()
            bo[row:e, hk * G:] = gdn.gdn_attn_forward(q, kk, vv, c)[0][row:e, hk * G:]
            if which == 0:
                bl[row:e, hk * G:] = NAN
            dq, dk, dv = gdn.gdn_attn_backward(q, kk, vv, c, bo, bl, dO)
            same(dq, clean[0], slice(0, row), i)
            same(dk, clean[1], slice(0, a), i)
            same(dv, clean[2], slice(0, a), i)
            if which == 1:
                x, bound = exact["dv"]
                with ref.where("cuda"):
                    assert ref.worst(dv, x, bound) <= 1, i
            assert not torch.isfinite(dq[row:e, hk * G:].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,heads", [(64, (4, 2)), (128, (8, 2))])
@pytest.mark.parametrize("new,whole", [([5, 1], [70, 300]), ([200], [333]), ([40, 9], [40, 2000])], ids=str)
def test_paged_values(dtype, D, heads, new, whole):
    """A value behind a new token's position, and values that pages hold behind a
    missing page or behind the end."""
    import gated_delta_rule_52_amd as gdn
    dt, (Hq, Hkv) = DT[dtype], heads
    G, cu, page = Hq // Hkv, cumulate(new), 16
    log(f"not finite, paged {dtype} D={D} {new} {whole}")
    kc, vc, table = make_cache(whole, page, Hkv, D, dt)
    q = rand(cu[-1], Hq, D, dtype=dt)
    args = table, ints(cu), ints(whole)
    clean = gdn.gdn_attn_paged(q, kc, vc, *args)
    assert torch.isfinite(clean.float()).all()
    hk, col = Hkv - 1, 5
    mine = list(range(hk * G, Hq))
    for n, i in enumerate(spots(new[0])):  # at the i-th new token of the first sequence
        value = list(VALUES.values())[n % 3]
        p = whole[0] - new[0] + i
        at = int(table[0, p // page]), p % page
        bad = vc.clone()
        bad[at][hk, col] = value
        o = gdn.gdn_attn_paged(q, kc, bad, *args)
        same(o, clean, slice(0, i), i)
        same(o, clean, slice(cu[1], None), i)
        seen_column(o, clean, slice(i, cu[1]), mine, col, i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 150])
def test_paged_beside_a_missing_page(dtype, new):
    """Values of cached tokens in tiles that a missing page makes masked ones: seen
    by every new token, in their column alone; in a missing page itself: by none."""
    import gated_delta_rule_52_amd as gdn
    dt, D, page, whole = DT[dtype], 64, 16, [400, 700]
    log(f"not finite beside a missing page {dtype} new={new}")
    kc, vc, table = make_cache(whole, page, 2, D, dt)
    gone = vc.clone()
    gone[int(table[0, 2]), 3, 1, 9] = NAN  # in page 2 of sequence 0, which is taken out
    table[0, 2] = table[1, 7] = -1
    q, cu = rand(2 * new, 4, D, dtype=dt), ints([0, new, 2 * new])
    clean = gdn.gdn_attn_paged(q, kc, vc, table, cu, ints(whole))
    assert torch.isfinite(clean.float()).all()
    assert torch.equal(gdn.gdn_attn_paged(q, kc, gone, table, cu, ints(whole)), clean)
    for n, (b, pos) in enumerate([(0, 50), (0, 63), (1, 96), (1, 111)]):  # pages 3 and 6, beside the missing ones
        value = list(VALUES.values())[n % 3]
        bad = vc.clone()
        bad[int(table[b, pos // page]), pos % page, 1, 5] = value
        o = gdn.gdn_attn_paged(q, kc, bad, table, cu, ints(whole))
        rows, others = slice(b * new, (b + 1) * new), slice((1 - b) * new, (2 - b) * new)
        same(o, clean, others, (b, pos))
        assert torch.equal(o[rows, :2], clean[rows, :2])
        seen_column(o, clean, rows, [2, 3], 5, (b, pos))
