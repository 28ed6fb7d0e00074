"""Attention at the sizes from which its launch rules take their other branches:
pieces of the key axis longer than the window of page numbers that a wave holds,
with pages missing behind its refill; pieces of sequences past the first waves of
64; fp32 prompts in 128-row blocks, their keys whole and cut up; products of rows
and keys that 24 bits do not hold; appends that write more than the L2 holds.
Against the plain 64-bit forms, within the bounds that block_reference.py derives."""
import pytest
import torch

import block_reference as ref
from block_reference import worst
from gpu_util import log
from test_gpu_attention import DT, cumulate, ints, make_cache, qkv, rand

pytestmark = pytest.mark.gpu


def check_paged(dt, D, heads, page, new, whole, drop):
    """`drop`: (sequence, position) whose pages are taken out of the table."""
    import gated_delta_rule_52_amd as gdn
    Hq, Hkv = heads
    cu = cumulate(new)
    kc, vc, table = make_cache(whole, page, Hkv, D, dt)
    for b, pos in drop:
        table[b, pos // page] = -1
    q = rand(cu[-1], Hq, D, dtype=dt)
    o = gdn.gdn_attn_paged(q, kc, vc, table, ints(cu), ints(whole))
    again = gdn.gdn_attn_paged(q, kc, vc, table, ints(cu), ints(whole))
    torch.cuda.synchronize()
    assert torch.equal(o, again)
    with ref.where("cuda"):
        want, bound = ref.paged(q, kc, vc, table, cu, whole)
        e = worst(o, want, bound)
    log(f"  o={e:.2f}")
    assert e <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,heads", [(64, (8, 4)), (128, (4, 4))])
def test_single_tokens_past_a_page_window(dtype, D, heads):
    """129 sequences over 4 key heads: the key axis is not cut up, and a wave of the
    32-row blocks refills its window of 32 tiles' pages (2048 keys for two waves,
    4096 for four) up to four times."""
    log(f"page window, single tokens {dtype} D={D}")
    whole = [1 + (13 * b) % 40 for b in range(129)]
    whole[5], whole[70], whole[128] = 9001, 4613, 8193
    drop = [(5, 0), (5, 4096), (5, 4300), (5, 7001), (5, 9000), (70, 2100), (128, 8192), (128, 6000)]
    check_paged(DT[dtype], D, heads, 16, [1] * 129, whole, drop)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_chunk_past_a_page_window(dtype, D):
    """2000 new tokens at the end of 9001, 16 heads over 8: 128-row blocks whose
    pieces (2600 keys and more) refill the window of 16 tiles' pages."""
    log(f"page window, chunk {dtype} D={D}")
    check_paged(DT[dtype], D, (16, 8), 16, [2000, 3], [9001, 500], [(0, 1100), (0, 2047), (0, 5000), (0, 8992), (1, 499)])


def test_rows_and_keys_past_24_bits():
    """Blocks times keys of more than 2^24, of which fp32 holds a rounded value: the
    attention and the join of its pieces find the same pieces from it."""
    log("rows and keys past 24 bits")
    check_paged(torch.bfloat16, 64, (16, 1), 64, [4001, 1, 1], [70003, 69999, 5], [(0, 65536), (1, 0)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cut_sequences_past_64(dtype):
    """Sequences that are cut into several pieces in every run of 64 that a wave
    looks at, the last of them among them."""
    log(f"cut sequences past 64 {dtype}")
    new = [1 + b % 2 for b in range(150)]
    whole = [n + (37 * b) % 90 for b, n in enumerate(new)]
    for b in (3, 63, 64, 75, 130, 149):
        whole[b] += 3000 + 11 * b
    check_paged(DT[dtype], 64, (2, 1), 16, new, whole, [(64, 3000), (149, 0)])


@pytest.mark.parametrize("D,heads,lens", [(64, (8, 4), [2100, 2533]), (128, (8, 4), [2100, 2533]), (64, (8, 2), [4101, 1, 4200])])
def test_prompt_fp32_in_large_blocks(D, heads, lens):
    """fp32 prompts with enough rows for 128-row blocks (T Hq >= 32768), and with
    enough that no query block's keys are cut up in the backward (T Hq > 65536)."""
    import gated_delta_rule_52_amd as gdn
    Hq, Hkv = heads
    cu = cumulate(lens)
    log(f"fp32 prompt D={D} heads={heads} {lens}")
    q, k, v = qkv(cu[-1], Hq, Hkv, D, torch.float32, True)
    dO = rand(cu[-1], Hq, D, seed=8)
    o, lse = gdn.gdn_attn_forward(q, k, v, ints(cu))
    got = gdn.gdn_attn_backward(q, k, v, ints(cu), o, lse, dO)
    torch.cuda.synchronize()
    with ref.where("cuda"):
        wo, wl, bo, bl = ref.prompt(q, k, v, cu)
        errs = {"o": worst(o, wo, bo), "lse": worst(lse, wl, bl)}
        for (name, (want, bound)), x in zip(ref.prompt_backward(q, k, v, cu, dO).items(), got):
            errs[name] = worst(x, want, bound)
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


def plain32(q, k, v, dO, cu):
    """o, lse, dq, dk, dv in elementary fp32 operations, a head at a time."""
    T, Hq, D = q.shape
    G, scale = Hq // k.shape[1], D ** -0.5
    o, lse = torch.empty_like(q), torch.empty(T, Hq, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, e in zip(cu[:-1], cu[1:]):
        hide = torch.ones(e - a, e - a, dtype=torch.bool, device=q.device).triu(1)
        for h in range(Hq):
            qq, kk, vv, do = q[a:e, h], k[a:e, h // G], v[a:e, h // G], dO[a:e, h]
            s = (qq @ kk.T.contiguous() * scale).masked_fill(hide, -float("inf"))
            m = s.amax(1, keepdim=True)
            x = torch.exp(s - m)
            z = x.sum(1, keepdim=True)
            p = x / z
            o[a:e, h], lse[a:e, h] = p @ vv, (m + torch.log(z))[:, 0]
            ds = p * (do @ vv.T.contiguous() - (do * o[a:e, h]).sum(1, keepdim=True)) * scale
            dq[a:e, h] = ds @ kk
            dk[a:e, h // G] += ds.T.contiguous() @ qq
            dv[a:e, h // G] += p.T.contiguous() @ do
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


@pytest.mark.parametrize("D,heads,lens", [(64, (4, 2), [300, 77]), (128, (4, 2), [515]), (64, (8, 4), [2100, 2533])])
def test_fp32_error_in_the_norm(D, heads, lens):
    """The whole error of a tensor, in the Euclidean norm, where roundings average
    out and a lost digit does not hide under a bound for the worst element: at most
    four times what elementary fp32 operations leave.  Both take the same number of
    roundings a value; the base-2 exponent adds one to a score and one to a
    log-sum, a sum in another order changes a partial sum's size by a factor of two
    at most here, and two such norms of independent roundings differ by less than
    the factor of two that remains."""
    import gated_delta_rule_52_amd as gdn
    Hq, Hkv = heads
    cu = cumulate(lens)
    q, k, v = (t.contiguous() for t in qkv(cu[-1], Hq, Hkv, D, torch.float32, True))
    dO = rand(cu[-1], Hq, D, seed=8)
    o, lse = gdn.gdn_attn_forward(q, k, v, ints(cu))
    dq, dk, dv = gdn.gdn_attn_backward(q, k, v, ints(cu), o, lse, dO)
    plain = plain32(q, k, v, dO, cu)
    with ref.where("cuda"):
        wo, wl, _, _ = ref.prompt(q, k, v, cu)
        want = {"o": wo, "lse": wl, **{n: x for n, (x, _) in ref.prompt_backward(q, k, v, cu, dO).items()}}
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        size = want[name].norm()
        here, there = float((got.double() - want[name]).norm() / size), float((plain[name].double() - want[name]).norm() / size)
        log(f"  D={D} {lens} {name}: {here:.1e} against {there:.1e}")
        assert here <= 4 * there, name


@pytest.mark.parametrize("dtype,tokens", [("bf16", 7001), ("f32", 3501)])
def test_append_past_the_l2(dtype, tokens):
    """More than 32 MB written: 24 heads of 128 a token."""
    import gated_delta_rule_52_amd as gdn
    dt, new = DT[dtype], [tokens, 1, 500]
    log(f"append past the L2 {dtype} {new}")
    cu, whole = cumulate(new), [tokens, 65, 700]
    q, k, v = qkv(cu[-1], 16, 4, 128, dt, True)
    kc, vc, table = make_cache(whole, 64, 4, 128, dt, poison=3.0)
    table[2, 9] = -1
    ang = torch.rand(max(whole), 64, generator=torch.Generator().manual_seed(1)).double() * 1e4
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    qo = torch.full_like(q, 5.0, memory_format=torch.contiguous_format)
    assert (qo.numel() + 2 * k.numel()) * qo.element_size() > 32 << 20
    wk, wv, wq = ref.append(q, k, v, cos, sin, cu, whole, table, kc, vc, qo)
    gdn.gdn_attn_append(q, k, v, cos, sin, ints(cu), ints(whole), table, kc, vc, q_out=qo)
    torch.cuda.synchronize()
    # a rotated value: two products and a sum in fp32, then half a step
    size = 2 * max(float(q.float().abs().max()), float(k.float().abs().max()))
    lim = lambda w: ref.HALF[dt] * w.abs() + 3 * ref.U32 * size
    e = worst(qo, wq, lim(wq)), worst(kc, wk, lim(wk))
    log(f"  q={e[0]:.2f} k={e[1]:.2f}")
    assert max(e) <= 1, e
    assert torch.equal(ref.f64(vc), wv)
