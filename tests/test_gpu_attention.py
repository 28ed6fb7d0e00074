"""Packed and paged softmax attention and the cache's append against the plain
64-bit forms, within the bounds that block_reference.py derives."""
import pytest
import torch

import block_reference as ref
from block_reference import worst
from gpu_util import log

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAN = float("nan")


def rand(*shape, dtype=torch.float32, std=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * len(shape) + sum(shape))
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def cumulate(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def qkv(T, Hq, Hkv, D, dt, fused, std=1.0):
    if fused:  # slices of one projection's output
        x = rand(T, Hq + 2 * Hkv, D, dtype=dt, std=std)
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    return tuple(rand(T, h, D, dtype=dt, std=std, seed=i) for i, h in enumerate((Hq, Hkv, Hkv)))


LENS = [[1], [2, 1, 3], [31, 32, 33], [64, 65, 0, 127, 1, 128, 129], [0, 0, 5], [300], [513, 40]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (4, 2), (6, 2), (8, 1)])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_prompt(dtype, D, heads, lens):
    import gated_delta_rule_52_amd as gdn
    dt, (Hq, Hkv) = DT[dtype], heads
    tail = 3  # rows of no sequence
    cu = cumulate(lens)
    n, T = cu[-1], cu[-1] + tail
    log(f"prompt {dtype} D={D} heads={heads} {lens}")
    q, k, v = qkv(T, Hq, Hkv, D, dt, fused=Hq != 4, std=1.5)
    for t in (q, k, v):
        t[n:] = NAN
    o = torch.full((T, Hq, D), 7.0, dtype=dt, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    gdn.gdn_attn_forward(q, k, v, ints(cu), o=o, lse=lse)
    dO = rand(T, Hq, D, dtype=dt, seed=8)
    out = tuple(torch.full((T, h, D), 7.0, dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv))
    gdn.gdn_attn_backward(q, k, v, ints(cu), o, lse, dO, out=out)
    first = [t.clone() for t in out]
    gdn.gdn_attn_backward(q, k, v, ints(cu), o, lse, dO, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    for t in (o, lse) + out:
        assert (t[n:] == 7.0).all(), "a row of no sequence was written"
    q, k, v, o, lse, dO = (t[:n] for t in (q, k, v, o, lse, dO))
    wo, wl, bo, bl = ref.prompt(q, k, v, cu)
    errs = {"o": worst(o, wo, bo), "lse": worst(lse, wl, bl)}
    back = ref.prompt_backward(q, k, v, cu, dO)
    for name, got in zip(("dq", "dk", "dv"), out):
        want, bound = back[name]
        errs[name] = worst(got[:n], want, bound)
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("dtype,D,heads,lens", [
    ("bf16", 128, (16, 4), [2100, 700, 1500]), ("bf16", 64, (24, 3), [1111, 2500]), ("f32", 128, (8, 8), [1300, 900])])
def test_prompt_long(dtype, D, heads, lens):
    """Enough blocks that the keys of a query block are not cut up (and those of a
    key block less), and rows of more than 512 keys."""
    import gated_delta_rule_52_amd as gdn
    dt, (Hq, Hkv) = DT[dtype], heads
    cu = cumulate(lens)
    log(f"long prompts {dtype} D={D} heads={heads} {lens}")
    q, k, v = qkv(cu[-1], Hq, Hkv, D, dt, True)
    o, lse = gdn.gdn_attn_forward(q, k, v, ints(cu))
    dO = rand(cu[-1], Hq, D, dtype=dt, seed=8)
    got = gdn.gdn_attn_backward(q, k, v, ints(cu), o, lse, dO)
    torch.cuda.synchronize()
    with ref.where("cuda"):
        wo, wl, bo, bl = ref.prompt(q, k, v, cu)
        errs = {"o": worst(o, wo, bo), "lse": worst(lse, wl, bl)}
        for (name, (want, bound)), x in zip(ref.prompt_backward(q, k, v, cu, dO).items(), got):
            errs[name] = worst(x, want, bound)
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("scale", [0.01, 3.0])
def test_prompt_scale_and_large_scores(scale):
    """Scores of a hundred and more: the running maximum moves, and nearly all
    weight falls on single keys."""
    import gated_delta_rule_52_amd as gdn
    q, k, v = qkv(200, 2, 1, 64, torch.float32, False, std=2.0)
    k = k * torch.linspace(0.1, 2, 200, device="cuda")[:, None, None]  # later keys score higher
    o, lse = gdn.gdn_attn_forward(q, k, v, ints([0, 200]), scale=scale)
    wo, wl, bo, bl = ref.prompt(q, k, v, [0, 200], scale)
    e = worst(o, wo, bo), worst(lse, wl, bl)
    log(f"scale {scale}: o={e[0]:.2f} lse={e[1]:.2f}")
    assert max(e) <= 1


def test_prompt_gradient_against_differences():
    """The kernels' own loss along a direction: central differences of fp32
    outputs, summed in 64 bits.  The step h = 2^-5 leaves h^2 / 6 of third
    derivatives (of the order of the loss's size here) and 2^-24 / h of the
    outputs' rounding a summed output, together below 1 % of a directional
    derivative of this size."""
    import gated_delta_rule_52_amd as gdn
    cu = ints([0, 40, 75])
    q, k, v = (t * 0.5 for t in qkv(75, 4, 2, 64, torch.float32, False))
    dO = rand(75, 4, 64, seed=9)
    o, lse = gdn.gdn_attn_forward(q, k, v, cu)
    grads = gdn.gdn_attn_backward(q, k, v, cu, o, lse, dO)
    loss = lambda *a: float((gdn.gdn_attn_forward(*a, cu)[0].double() * dO.double()).sum())
    h = 2.0 ** -5
    for i, g in enumerate(grads):
        u = g / g.norm()  # along the gradient itself
        up, down = [q, k, v], [q, k, v]
        up[i], down[i] = up[i] + h * u, down[i] - h * u
        d, want = (loss(*up) - loss(*down)) / (2 * h), float((g.double() * u.double()).sum())
        log(f"  {'qkv'[i]}: {d:.6f} against {want:.6f}")
        assert abs(d - want) <= 0.01 * abs(want)


def test_prompt_bounds_of_cu_are_clamped():
    """Sequence bounds outside the rows reach nothing outside the buffers."""
    import gated_delta_rule_52_amd as gdn
    q, k, v = qkv(50, 2, 2, 64, torch.bfloat16, False)
    o, _ = gdn.gdn_attn_forward(q, k, v, ints([-5, 20, 9999]))
    want, _ = gdn.gdn_attn_forward(q, k, v, ints([0, 20, 50]))
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def make_cache(lens, page, Hkv, D, dt, extra=2, poison=NAN):
    """A pool whose pages are handed out in a mixed order; what no sequence owns
    holds `poison`."""
    pages = [-(-n // page) for n in lens]
    num = sum(pages) + 3
    g = torch.Generator().manual_seed(sum(lens) + page)
    order = torch.randperm(num, generator=g).tolist()
    table = torch.full((len(lens), max(pages + [1]) + extra), -1, dtype=torch.int32)
    kc = torch.full((num, page, Hkv, D), poison, dtype=dt, device="cuda")
    vc = kc.clone()
    at = 0
    for b, n in enumerate(lens):
        for i in range(pages[b]):
            table[b, i] = order[at]
            m = min(page, n - i * page)
            kc[order[at], :m] = rand(m, Hkv, D, dtype=dt, std=1.2, seed=at)
            vc[order[at], :m] = rand(m, Hkv, D, dtype=dt, seed=at + 1000)
            at += 1
    return kc, vc, table.cuda()


PAGED = [  # new tokens and whole lengths
    ([1], [1]), ([1, 1, 1], [1, 17, 300]), ([1, 0, 2], [64, 40, 65]), ([5, 3], [5, 90]), ([130, 1], [130, 700]),
    ([200], [264]), ([33, 64, 7], [1000, 64, 129]), ([1, 1], [0, 20]), ([10, 4], [6, 4]), ([1], [5000]), ([300], [4000]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,heads,page", [(128, (8, 2), 16), (64, (6, 2), 32), (128, (4, 4), 64), (64, (16, 1), 256)])
@pytest.mark.parametrize("new,whole", PAGED, ids=lambda x: str(x))
def test_paged(dtype, D, heads, page, new, whole):
    import gated_delta_rule_52_amd as gdn
    dt, (Hq, Hkv) = DT[dtype], heads
    cu = cumulate(new)
    n, T = cu[-1], cu[-1] + 2
    log(f"paged {dtype} D={D} heads={heads} page={page} new={new} whole={whole}")
    kc, vc, table = make_cache(whole, page, Hkv, D, dt)
    q = rand(T, Hq, D, dtype=dt)
    o = torch.full((T, Hq, D), 7.0, dtype=dt, device="cuda")
    gdn.gdn_attn_paged(q, kc, vc, table, ints(cu), ints(whole), o=o)
    o2 = torch.full_like(o, 7.0)
    gdn.gdn_attn_paged(q, kc, vc, table, ints(cu), ints(whole), o=o2)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and (o[n:] == 7.0).all()
    want, bound = ref.paged(q[:n], kc, vc, table, cu, whole)
    e = worst(o[:n], want, bound)
    log(f"  o={e:.2f}")
    assert e <= 1


@pytest.mark.parametrize("B", [64, 65, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype, B):
    """More sequences than a wave has lanes (and just as many): prompt, append and
    paged, the key axis in one piece and in several."""
    import gated_delta_rule_52_amd as gdn
    dt = DT[dtype]
    log(f"many sequences {dtype} B={B}")
    lens = [(7 * b) % 40 for b in range(B)]
    cu = cumulate(lens)
    q, k, v = qkv(cu[-1], 4, 2, 64, dt, True)
    o, lse = gdn.gdn_attn_forward(q, k, v, ints(cu))
    dO = rand(cu[-1], 4, 64, dtype=dt, seed=4)
    got = gdn.gdn_attn_backward(q, k, v, ints(cu), o, lse, dO)
    torch.cuda.synchronize()
    wo, wl, bo, bl = ref.prompt(q, k, v, cu)
    errs = {"o": worst(o, wo, bo), "lse": worst(lse, wl, bl)}
    for (name, (want, bound)), x in zip(ref.prompt_backward(q, k, v, cu, dO).items(), got):
        errs[name] = worst(x, want, bound)
    new = [b % 3 for b in range(B)]
    whole = [n + (37 * b) % 90 for b, n in enumerate(new)]
    whole[B // 2] += 3000  # one that is cut into pieces
    cu = cumulate(new)
    q, k, v = qkv(cu[-1], 2, 1, 64, dt, True)
    kc, vc, table = make_cache(whole, 16, 1, 64, dt, poison=0.0)
    wk, wv, wq = ref.append(q, k, v, None, None, cu, whole, table, kc, vc, torch.zeros_like(q))
    qo = gdn.gdn_attn_append(q, k, v, None, None, ints(cu), ints(whole), table, kc, vc)
    x = gdn.gdn_attn_paged(qo, kc, vc, table, ints(cu), ints(whole))
    torch.cuda.synchronize()
    assert torch.equal(ref.f64(kc), wk) and torch.equal(ref.f64(vc), wv) and torch.equal(ref.f64(qo), wq)
    want, bound = ref.paged(qo, kc, vc, table, cu, whole)
    errs["paged"] = worst(x, want, bound)
    log("  " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


def test_cache_past_32_bits():
    """Pages whose first byte lies past 2^32 and whose first element past 2^31."""
    import gated_delta_rule_52_amd as gdn
    dt, Hkv, D, page, num = torch.bfloat16, 8, 128, 16, 140000
    kc = torch.empty(num, page, Hkv, D, dtype=dt, device="cuda")
    vc = torch.empty_like(kc)
    assert kc[num - 4:].storage_offset() * 2 > 2 ** 32 and kc.numel() > 2 ** 31
    whole, new = [70, 33], [2, 1]
    at = [num - 1, 5, num - 3, num - 2, 132000, num - 7, 131500, 7]
    for i in at:
        kc[i] = rand(page, Hkv, D, dtype=dt, seed=i)
        vc[i] = rand(page, Hkv, D, dtype=dt, seed=i + 1)
    table = ints([at[:5], at[5:] + [-1, -1]])
    q, k, v = qkv(3, 16, Hkv, D, dt, True)
    gdn.gdn_attn_append(None, k, v, None, None, ints([0, 2, 3]), ints(whole), table, kc, vc)
    torch.cuda.synchronize()
    for t, (b, p) in enumerate(((0, 68), (0, 69), (1, 32))):
        pg = int(table[b, p // page])
        assert torch.equal(kc[pg, p % page], k[t]) and torch.equal(vc[pg, p % page], v[t])
    o = gdn.gdn_attn_paged(q, kc, vc, table, ints([0, 2, 3]), ints(whole))
    small = ints([[0, 1, 2, 3, 4], [5, 6, 7, -1, -1]])
    want, bound = ref.paged(q, kc[at], vc[at], small, [0, 2, 3], whole)
    e = worst(o, want, bound)
    log(f"past 32 bits: {e:.2f}")
    assert e <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 100])
def test_paged_missing_pages(dtype, new):
    """Pages that do not exist (-1, and past the pool) are absent keys; a table
    shorter than the length ends it; shared pages are read by both."""
    import gated_delta_rule_52_amd as gdn
    dt = DT[dtype]
    whole = [200, 333, 160]  # the third ends with a page: nothing unset is in reach of its length below
    kc, vc, table = make_cache(whole, 16, 2, 64, dt, extra=0)
    table[0, 3] = -1
    table[0, 12] = kc.shape[0]
    table[1, :5] = -7
    table[2, :4] = table[1, 8:12]
    kv = [200, 333, 4000]  # the third is longer than its table
    cu = cumulate([new] * 3)
    q = rand(cu[-1], 4, 64, dtype=dt)
    o = gdn.gdn_attn_paged(q, kc, vc, table, ints(cu), ints(kv))
    torch.cuda.synchronize()
    want, bound = ref.paged(q, kc, vc, table, cu, kv)
    e = worst(o, want, bound)
    log(f"missing pages {dtype} new={new}: {e:.2f}")
    assert e <= 1
    table.fill_(-1)  # nothing is there
    o = gdn.gdn_attn_paged(q, kc, vc, table, ints(cu), ints(kv))
    torch.cuda.synchronize()
    assert torch.equal(o, torch.zeros_like(o))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,rot,heads", [(128, 128, (8, 2)), (64, 32, (3, 3)), (128, 0, (2, 1)), (64, 64, (5, 1))])
@pytest.mark.parametrize("new,whole", [([1], [1]), ([1, 1, 1], [5, 64, 65]), ([40, 0, 17], [40, 9, 200]), ([700], [900]),
                                       ([2200, 3], [2200, 50])], ids=lambda x: str(x))
def test_append(dtype, D, rot, heads, new, whole):
    import gated_delta_rule_52_amd as gdn
    dt, (Hq, Hkv) = DT[dtype], heads
    cu = cumulate(new)
    T = cu[-1] + 2
    log(f"append {dtype} D={D} rot={rot} heads={heads} {new} {whole}")
    q, k, v = qkv(T, Hq, Hkv, D, dt, fused=True)
    kc, vc, table = make_cache(whole, 16, Hkv, D, dt, poison=3.0)
    ang = torch.rand(max(whole), rot // 2, generator=torch.Generator().manual_seed(1)).double() * 1e4
    cos, sin = (ang.cos().float().cuda(), ang.sin().float().cuda()) if rot else (None, None)
    qo = torch.full((T, Hq, D), 5.0, dtype=dt, device="cuda")
    wk, wv, wq = ref.append(q, k, v, cos, sin, cu, whole, table, kc, vc, qo)
    gdn.gdn_attn_append(q, k, v, cos, sin, ints(cu), ints(whole), table, kc, vc, q_out=qo)
    torch.cuda.synchronize()
    # a rotated value: two products and a sum in fp32, then half a step
    size = 2 * max(float(q.float().abs().max()), float(k.float().abs().max()))
    lim = lambda w: ref.HALF[dt] * w.abs() + 3 * ref.U32 * size
    e = worst(qo, wq, lim(wq)), worst(kc, wk, lim(wk))
    assert max(e) <= 1, e
    assert torch.equal(ref.f64(vc), wv)
    if not rot:
        assert torch.equal(ref.f64(kc), wk) and torch.equal(ref.f64(qo), wq)


def test_append_leaves_out():
    """Tokens without a position, a page or an angle write nothing; q may be absent."""
    import gated_delta_rule_52_amd as gdn
    new, kv = [6, 3, 4, 2], [4, 40, 70, 33]
    cu = cumulate(new)
    q, k, v = qkv(cu[-1], 2, 2, 64, torch.bfloat16, True)
    kc, vc, table = make_cache([20, 48, 80, 48], 16, 2, 64, torch.bfloat16, extra=0, poison=3.0)
    table[1, 2] = -1
    table[2, 4] = 10000
    ang = torch.rand(34, 32)  # no angle for positions from 34 on
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    qo = torch.full((cu[-1], 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    wk, wv, wq = ref.append(q, k, v, cos, sin, cu, kv, table, kc, vc, qo)
    k0, v0 = kc.clone(), vc.clone()
    gdn.gdn_attn_append(q, k, v, cos, sin, ints(cu), ints(kv), table, kc, vc, q_out=qo)
    torch.cuda.synchronize()
    assert (qo[:2] == 5.0).all() and (qo[6:13] == 5.0).all() and not (qo[13:] == 5.0).all()
    for got, want in ((qo, wq), (kc, wk)):
        assert worst(got, want, ref.HALF[torch.bfloat16] * want.abs() + 30 * ref.U32) <= 1
    assert torch.equal(ref.f64(vc), wv)
    assert gdn.gdn_attn_append(None, k, v, cos, sin, ints(cu), ints(kv), table, k0, v0) is None
    torch.cuda.synchronize()
    assert torch.equal(k0, kc) and torch.equal(v0, vc)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(dtype):
    """As a server runs them: a prompt enters the cache in two pieces, then
    single tokens follow; every output equals one packed prompt's over the same
    rotated tokens, within both sides' bounds.  The cached keys are the packed
    side's input, so both see the same bits."""
    import gated_delta_rule_52_amd as gdn
    dt = DT[dtype]
    lens, pieces = [70, 41], [[32, 40], [30, 0], [1, 1], [7, 0]]
    Hq, Hkv, D, page = 4, 2, 64, 16
    cu = cumulate(lens)
    q, k, v = qkv(cu[-1], Hq, Hkv, D, dt, True)
    ang = torch.rand(128, 32, generator=torch.Generator().manual_seed(2)).double() * 100
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    kc, vc, table = make_cache(lens, page, Hkv, D, dt)
    kc.fill_(NAN), vc.fill_(NAN)
    done, got, qr = [0, 0], torch.zeros(cu[-1], Hq, D, dtype=dt, device="cuda"), torch.zeros_like(q)
    for new in pieces:
        rows = torch.tensor([cu[b] + done[b] + i for b in range(2) for i in range(new[b])], device="cuda")
        done = [d + n for d, n in zip(done, new)]
        c, w = ints(cumulate(new)), ints(done)
        x = gdn.gdn_attn_append(q[rows], k[rows], v[rows], cos, sin, c, w, table, kc, vc)
        got[rows] = gdn.gdn_attn_paged(x, kc, vc, table, c, w)
        qr[rows] = x
    assert done == lens
    flat = [s for b in range(2) for s in ref.slots(table.cpu(), b, lens[b], page, kc.shape[0])]
    kr, vr = kc.view(-1, Hkv, D)[flat], vc.view(-1, Hkv, D)[flat]
    assert torch.equal(vr, v)
    o, lse = gdn.gdn_attn_forward(qr, kr, vr, ints(cu))
    torch.cuda.synchronize()
    wo, _, bo, _ = ref.prompt(qr, kr, vr, cu)
    e = worst(got, wo, bo), worst(o, wo, bo)
    log(f"in pieces {dtype}: paged={e[0]:.2f} packed={e[1]:.2f}")
    assert max(e) <= 1


def test_block_of_a_hybrid_stack():
    """The operators together, around both kinds of mixer, forward and backward:
    norm, delta rule, gated norm, residual norm, attention, with gradients that
    reach the input; two passes give the same bits."""
    import gated_delta_rule_52_amd as gdn
    B, T, H, D = 2, 96, 2, 64
    W = H * D
    x = rand(B * T, W, dtype=torch.bfloat16)
    w1, w2, wg, a = (rand(n, seed=i, std=0.1) + 1 for i, n in enumerate((W, W, D, W)))
    gate = rand(B * T, 2 * H, D, dtype=torch.bfloat16, seed=5)[:, H:]
    g = -torch.rand(B, T, H, generator=torch.Generator().manual_seed(6)).cuda()
    beta = torch.rand(B, T, H, generator=torch.Generator().manual_seed(7)).cuda()
    cu = ints([0, T, 2 * T])
    dO = rand(B * T, H, D, dtype=torch.bfloat16, seed=8)

    def step():
        _, n1, r1 = gdn.gdn_norm_block(x, w1)
        u = n1.view(B, T, H, D)
        m, _, ws = gdn.gdn_forward_train(u, u, u, g, beta, use_qk_l2norm=True)
        m = m.view(B * T, H, D)
        y, rg = gdn.gdn_norm_gate(m, gate, wg)
        h, n2, r2 = gdn.gdn_norm_block(x, w2, y.view(B * T, W), a)
        s = n2.view(B * T, H, D)
        o, lse = gdn.gdn_attn_forward(s, s, s, cu)
        ds = sum(t.float() for t in gdn.gdn_attn_backward(s, s, s, cu, o, lse, dO)).bfloat16().view(B * T, W)
        dx, dy, dw2, da = gdn.gdn_norm_block_backward(ds, x, w2, r2, y.view(B * T, W), a)
        dm, dgate, dwg = gdn.gdn_norm_gate_backward(dy.view(B * T, H, D), m, gate, wg, rg)
        dq, dk, dv, dg, dbeta, _ = gdn.gdn_backward_train(u, u, u, g, beta, dm.view(B, T, H, D), ws, use_qk_l2norm=True)
        du = (dq.float() + dk.float() + dv.float()).bfloat16().view(B * T, W)
        dxx, _, dw1, _ = gdn.gdn_norm_block_backward(du, x, w1, r1, dh=dx)
        return o, lse, dxx, dw1, dw2, da, dgate, dwg, dg, dbeta

    first, second = step(), step()
    torch.cuda.synchronize()
    for p, q in zip(first, second):
        assert torch.isfinite(p.float()).all() and p.float().abs().max() > 0
        assert torch.equal(p, q)


def test_graphs_streams():
    """A decode step and a training step captured: replays give the eager bits
    while lengths move on between them (the lengths are device data), and
    so does a side stream."""
    import gated_delta_rule_52_amd as gdn
    dt = torch.bfloat16
    kc, vc, table = make_cache([300, 1000], 16, 2, 128, dt, poison=0.0)
    q, k, v = qkv(2, 8, 2, 128, dt, True)
    ang = torch.rand(1024, 64)
    cos, sin = ang.cos().cuda(), ang.sin().cuda()
    cu, kv = ints([0, 1, 2]), ints([200, 900])
    qo, o = torch.empty(2, 8, 128, dtype=dt, device="cuda"), torch.empty(2, 8, 128, dtype=dt, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def decode():
        gdn.gdn_attn_append(q, k, v, cos, sin, cu, kv, table, kc, vc, q_out=qo)
        gdn.gdn_attn_paged(qo, kc, vc, table, cu, kv, o=o, ws=ws)

    Q, K, V = qkv(150, 4, 2, 128, dt, True)
    dO = rand(150, 4, 128, dtype=dt)
    c2 = ints([0, 100, 150])
    to, tl = torch.empty(150, 4, 128, dtype=dt, device="cuda"), torch.empty(150, 4, device="cuda")
    tg = tuple(torch.empty(150, h, 128, dtype=dt, device="cuda") for h in (4, 2, 2))

    def train():
        gdn.gdn_attn_forward(Q, K, V, c2, o=to, lse=tl)
        gdn.gdn_attn_backward(Q, K, V, c2, to, tl, dO, out=tg, ws=ws)

    decode(), train()
    torch.cuda.synchronize()
    gd, gt = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gd):
        decode()
    with torch.cuda.graph(gt):
        train()
    for i in range(3):
        decode()
        want = [t.clone() for t in (qo, o)]
        train()
        want += [t.clone() for t in (to, tl) + tg]
        for t in (qo, o, to, tl) + tg:
            t.fill_(NAN)
        gd.replay(), gt.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(want, (qo, o, to, tl) + tg)), i
        kv += 7
    side = torch.cuda.Stream()
    decode()
    want = o.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        o.fill_(NAN)
        decode()
    side.synchronize()
    assert torch.equal(o, want)


def test_two_streams_at_once():
    """Two calls under way together, each with its own outputs and workspace, give
    what each gives alone."""
    import gated_delta_rule_52_amd as gdn
    dt, jobs = torch.bfloat16, []
    for i, lens in enumerate(([900, 300], [50, 700, 450])):
        cu = cumulate(lens)
        q, k, v = qkv(cu[-1], 8, 2, 128, dt, True)
        jobs.append((q, k, v, ints(cu), rand(cu[-1], 8, 128, dtype=dt, seed=i)))
    kc, vc, table = make_cache([3000, 500], 32, 2, 128, dt)
    qd, cd, kv = rand(2, 8, 128, dtype=dt), ints([0, 1, 2]), ints([3000, 500])

    def work(job):
        q, k, v, cu, dO = job
        o, lse = gdn.gdn_attn_forward(q, k, v, cu)
        return (o, lse) + gdn.gdn_attn_backward(q, k, v, cu, o, lse, dO) + (
            gdn.gdn_attn_paged(qd, kc, vc, table, cd, kv),)

    want = [work(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(3):
        for j, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(work(j))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2])), i


def test_refusals():
    import gated_delta_rule_52_amd as gdn
    dt = torch.bfloat16
    q, k, v = qkv(6, 4, 2, 64, dt, False)
    cu = ints([0, 6])
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q, k[:, :, :32], v, cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q, k, v[:5], cu)
    with pytest.raises(TypeError):
        gdn.gdn_attn_forward(q, k.float(), v, cu)
    with pytest.raises(TypeError):
        gdn.gdn_attn_forward(q, k, v, cu.long())
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q.transpose(1, 2), k, v, cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q, k, v, cu, o=torch.empty(6, 4, 128, dtype=dt, device="cuda"))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_attn_forward(q[:, :3], k, v, cu)  # 3 query heads over 2
    with pytest.raises(gdn.GdnError):
        gdn.gdn_attn_forward(*qkv(6, 4, 2, 80, dt, False), cu)
    with pytest.raises(ValueError):
        gdn.gdn_attn_forward(q[:1].expand(6, 4, 64), k, v, cu)  # one token seen six times
    with pytest.raises(ValueError):
        gdn.gdn_norm_gate(q, q[:1].expand(6, 4, 64), torch.ones(64, device="cuda"))
    kc = torch.zeros(4, 16, 2, 64, dtype=dt, device="cuda")
    table, kv = ints([[0, 1]]), ints([6])
    with pytest.raises(ValueError):
        gdn.gdn_attn_paged(q, kc, kc[:3], table, cu, kv)
    with pytest.raises(ValueError):
        gdn.gdn_attn_paged(q, kc, kc, table[0], cu, kv)
    with pytest.raises(ValueError):
        gdn.gdn_attn_paged(q, kc, kc, table, cu, ints([6, 6]))
    with pytest.raises(gdn.GdnError):
        gdn.gdn_attn_paged(q, kc.view(8, 8, 2, 64), kc.view(8, 8, 2, 64), table, cu, kv)
    with pytest.raises(gdn.GdnError):
        gdn.gdn_attn_paged(q, kc, kc, ints([[0] * 4096]), cu, kv, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    cos = torch.ones(16, 32, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_attn_append(q, k, v, cos, None, cu, kv, table, kc, kc.clone())
    with pytest.raises(ValueError):
        gdn.gdn_attn_append(q, k, v, cos, cos[:8], cu, kv, table, kc, kc.clone())
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_norm_block(x[:, ::2], torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_norm_block(x, torch.ones(32, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_norm_block(x, torch.ones(64, device="cuda"), None, torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_norm_gate(x.view(4, 1, 64), x[:3].view(3, 1, 64), torch.ones(64, device="cuda"))
