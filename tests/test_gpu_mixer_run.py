"""The state-space layer's operators and the page step as they are used: together in
a serving loop, captured into graphs, on other streams, two at once, and in batches
large enough for the other divisions of their work."""
import pytest
import torch

import block_reference
import mixer_reference as ref
from gpu_util import log
from mixer_reference import worst
from test_gpu_attention import DT, NAN, cumulate, ints, rand
from test_gpu_ssm import GRADS, backward, blank, forward, make

pytestmark = pytest.mark.gpu

H, G, N, P = 2, 1, 64, 64
CHAN = H * P + 2 * G * N


def split(y):
    """A convolution's output as the scan takes it."""
    return (y[:, :H * P].unflatten(1, (H, P)), y[:, H * P:H * P + G * N].unflatten(1, (G, N)),
            y[:, H * P + G * N:].unflatten(1, (G, N)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hybrid_serving(dtype):
    """Prompts in pieces, then single tokens, through one pool of pages: pages, then a
    convolution and the scan, then attention over the cache; one sequence ends and
    another takes its place and its pages.  Every operator's results over all of a
    sequence are held to its plain form over the whole, on the inputs that it had."""
    import gated_delta_rule_52_amd as gdn
    dt, B, ps, width, pool = DT[dtype], 3, 16, 12, 22
    weight, bias = rand(CHAN, 4, std=0.5, seed=1), rand(CHAN, seed=2)
    A, D, dt_bias = -torch.linspace(1, 4, H, device="cuda"), rand(H, seed=3), torch.linspace(-4, -2, H, device="cuda")
    kc = torch.full((pool, ps, 1, 64), NAN, dtype=dt, device="cuda")
    vc = torch.full_like(kc, NAN)
    table, kv = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), ints([0] * B)
    free, count = torch.arange(pool, dtype=torch.int32, device="cuda"), ints([pool])
    cs, ss = torch.zeros(B, 3, CHAN, dtype=dt, device="cuda"), torch.zeros(B, H, N, P, device="cuda")
    # sequence: its rows of the projections, made once, and what came out
    total = [150, 40, 180, 70]
    rows = [dict(x=rand(n, CHAN, dtype=dt, seed=10 * i), dt=rand(n, H, std=0.5, seed=10 * i + 1),
                 qkv=rand(n, 4, 64, dtype=dt, seed=10 * i + 2)) for i, n in enumerate(total)]
    seen = [dict(y=[], s=[], o=[]) for _ in total]
    who, length, hold = [0, 1, 2], [0, 0, 0], 64
    ends = {}

    def step(want):
        gdn.gdn_pages_take(ints(want), kv, table, free, count, ps, hold, cu_seqlens=(cu := torch.empty(B + 1, dtype=torch.int32, device="cuda")),
                           positions=(pos := torch.full((hold,), -1, dtype=torch.int32, device="cuda")),
                           slots=(slots := torch.full((hold,), -1, dtype=torch.int64, device="cuda")))
        at = cu.tolist()
        assert at == cumulate(want) and kv.tolist() == [length[b] + want[b] for b in range(B)]
        n = at[-1]
        part = {k: torch.cat([rows[who[b]][k][length[b]:length[b] + want[b]] for b in range(B)]) for k in ("x", "dt", "qkv")}
        assert pos[:n].tolist() == [length[b] + i for b in range(B) for i in range(want[b])]
        q, k, v = part["qkv"][:, :2], part["qkv"][:, 2:3], part["qkv"][:, 3:]
        if want == [1] * B:
            y = gdn.gdn_conv_step(part["x"], weight, cs, bias)
            x, Bm, Cm = split(y)
            s = gdn.gdn_ssm_step(x, part["dt"], A, Bm, Cm, ss, D=D, dt_bias=dt_bias)
        else:
            y, _ = gdn.gdn_conv_forward(part["x"], weight, cu, bias, cs, state_out=cs)
            x, Bm, Cm = split(y)
            s, _ = gdn.gdn_ssm_forward(x, part["dt"], A, Bm, Cm, cu, D=D, dt_bias=dt_bias, h0=ss, hT=ss)
        gdn.gdn_attn_append(q, k, v, None, None, cu, kv, table, kc, vc, q_out=(qo := torch.empty(n, 2, 64, dtype=dt, device="cuda")))
        o = gdn.gdn_attn_paged(qo, kc, vc, table, cu, kv)
        torch.cuda.synchronize()
        assert torch.equal(kc.flatten(0, 1)[slots[:n]], k) and torch.equal(vc.flatten(0, 1)[slots[:n]], v)
        for b in range(B):
            for name, t in (("y", y), ("s", s), ("o", o)):
                seen[who[b]][name].append(t[at[b]:at[b + 1]])
            length[b] += want[b]

    for want in ([30, 1, 20], [34, 0, 30], [40, 20, 4], [1, 1, 1], [1, 1, 1], [20, 5, 39], [1, 1, 1]):
        step(want)
    ends[1] = ss[1].clone()
    before = count.item()
    gdn.gdn_pages_release(ints([0, 1, 0]), kv, table, free, count, ps)
    assert kv.tolist() == [length[0], 0, length[2]] and count.item() == before + -(-length[1] // ps)
    who[1], length[1] = 3, 0
    cs[1], ss[1] = 0, 0
    for want in ([0, 60, 0], [1, 1, 1], [1, 1, 1], [10, 3, 20], [1, 1, 1]):
        step(want)
    for b in range(B):
        ends[who[b]] = ss[b].clone()
    errs = {}
    for i, r in enumerate(rows):
        y, s, o = (torch.cat(seen[i][k]) for k in ("y", "s", "o"))
        n = len(y)
        wy, by, _ = ref.conv(r["x"][:n], weight, [0, n], bias)
        x, Bm, Cm = split(y)
        want = ref.ssm(x, r["dt"][:n], A, Bm, Cm, [0, n], D, dt_bias, True)
        wo, _, bo, _ = block_reference.prompt(r["qkv"][:n, :2], r["qkv"][:n, 2:3], r["qkv"][:n, 3:], [0, n])
        for name, e in (("conv", worst(y, wy, by)), ("scan", worst(s, *want["y"])), ("state", worst(ends[i][None], *want["hT"])),
                        ("attention", worst(o, wo, bo))):
            errs[name] = max(errs.get(name, 0.0), e)
    log(f"serving {dtype} " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


def test_decode_step_in_a_graph():
    """One decode step captured: replays move lengths, pages and states on as eager
    steps of the same inputs do, bit for bit, with eager steps between them."""
    import gated_delta_rule_52_amd as gdn
    dt, B, ps, pool = torch.bfloat16, 5, 16, 200
    weight, bias = rand(CHAN, 4, std=0.5, seed=1), rand(CHAN, seed=2)
    A, D, dt_bias = -torch.linspace(1, 4, H, device="cuda"), rand(H, seed=3), torch.linspace(-4, -2, H, device="cuda")
    x, delta = rand(B, CHAN, dtype=dt), rand(B, H, std=0.5)
    done, want = ints([0, 0, 1, 0, 0]), ints([1] * B)

    def fresh():
        return dict(kv=ints([15, 30, 100, 16, 0]), table=torch.arange(B * 20, dtype=torch.int32, device="cuda").view(B, 20),
                    free=torch.arange(100, 100 + pool, dtype=torch.int32, device="cuda"), count=ints([50]),
                    cs=rand(B, 3, CHAN, dtype=dt, seed=5), ss=rand(B, H, N, P, seed=6), y=torch.empty(B, CHAN, dtype=dt, device="cuda"),
                    s=torch.empty(B, H, P, dtype=dt, device="cuda"), cu=ints([0] * (B + 1)), pos=ints([0] * B),
                    slots=torch.zeros(B, dtype=torch.int64, device="cuda"))

    def step(v):
        gdn.gdn_pages_release(done, v["kv"], v["table"], v["free"], v["count"], ps)
        gdn.gdn_pages_take(want, v["kv"], v["table"], v["free"], v["count"], ps, B, cu_seqlens=v["cu"], positions=v["pos"], slots=v["slots"])
        gdn.gdn_conv_step(x, weight, v["cs"], bias, y=v["y"])
        xs, Bm, Cm = split(v["y"])
        gdn.gdn_ssm_step(xs, delta, A, Bm, Cm, v["ss"], D=D, dt_bias=dt_bias, y=v["s"])

    a, b = fresh(), fresh()
    step(fresh())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for i in range(6):
        x.add_(0.125)
        step(a)
        graph.replay()
        torch.cuda.synchronize()
        for k in a:
            assert torch.equal(a[k], b[k]), (i, k)
        if i % 2:
            step(a), step(b)  # an eager step of both
            torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,lens", [("bf16", [900, 40]), ("f32", [150, 40, 0, 3]), ("bf16", [2600])])
def test_training_step_in_a_graph_and_on_a_stream(dtype, lens):
    """Forward and backward captured: replays give the eager bits, and so does a side
    stream.  (2600 tokens of two heads: several segments.)"""
    import gated_delta_rule_52_amd as gdn
    dt, cu = DT[dtype], cumulate(lens)
    T, B = cu[-1], len(lens)
    cui = ints(cu)
    weight, bias, state = rand(CHAN, 4, std=0.5, seed=1), rand(CHAN, seed=2), rand(B, 3, CHAN, dtype=dt, seed=3)
    x, dy = rand(T, CHAN, dtype=dt), rand(T, CHAN, dtype=dt, seed=4)
    s = make(T, B, H, G, N, P, dt)
    y, st = torch.empty_like(x), torch.empty_like(state)
    cg = (torch.empty_like(x), torch.empty_like(weight), torch.empty_like(bias), torch.empty_like(state))
    sy, hT, sg = torch.empty(T, H, P, dtype=dt, device="cuda"), torch.empty_like(s["h0"]), blank(s, dt)
    ws, ws2 = (torch.empty(1 << 27, dtype=torch.uint8, device="cuda") for _ in range(2))
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"], cui)
    kw = dict(D=s["D"], dt_bias=s["dt_bias"], h0=s["h0"])

    def train():
        gdn.gdn_conv_forward(x, weight, cui, bias, state, y=y, state_out=st)
        gdn.gdn_ssm_forward(*args, y=sy, hT=hT, ws=ws, **kw)
        gdn.gdn_ssm_backward(*args, s["dy"], dhT=s["dhT"], out=sg, ws=ws, **kw)
        gdn.gdn_conv_backward(x, weight, cui, dy, bias, state, dstate_out=st, out=cg, ws=ws2)

    outs = (y, st, sy, hT) + sg + cg
    train()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train()
    for i in range(4):
        for t in outs:
            t.fill_(NAN)
        ws.fill_(255), ws2.fill_(255)  # nothing is expected of a workspace
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (i, k)
        train()
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for t in outs:
        t.fill_(NAN)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    """Calls under way together, each with its own outputs and workspace."""
    import gated_delta_rule_52_amd as gdn
    jobs = []
    for lens, heads, dt in (([700, 130], (4, 2, 64, 64), torch.bfloat16), ([3000], (2, 1, 128, 64), torch.bfloat16)):
        cu = cumulate(lens)
        jobs.append((make(cu[-1], len(lens), *heads, dt), cu, rand(cu[-1], 512, dtype=dt), rand(512, 4, std=0.5)))

    def work(job):
        s, cu, x, w = job
        y, hT = forward(s, cu)
        cy, _ = gdn.gdn_conv_forward(x, w, ints(cu), want_state=False)
        return (y, hT, cy) + backward(s, cu) + gdn.gdn_conv_backward(x, w, ints(cu), cy)[:2]

    want = [work(j) for j in jobs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], []
    for _ in range(3):
        for j, st in zip(jobs, streams):
            with torch.cuda.stream(st):
                got.append(work(j))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for k, (a, b) in enumerate(zip(g, want[i % 2])):
            assert torch.equal(a, b), (i, k)


@pytest.mark.parametrize("dtype,B,heads", [("bf16", 300, (1, 1, 64, 64)), ("bf16", 280, (6, 2, 64, 64)), ("f32", 150, (4, 1, 64, 64)),
                                           ("bf16", 260, (4, 2, 128, 64)), ("bf16", 140, (4, 1, 64, 128))])
def test_many_chunks(dtype, B, heads):
    """Batches in which a workgroup has several slices or all of a group's heads; some
    of the sequences against the plain form.  (Groups of 1 and 3 slices: odd.)"""
    dt = DT[dtype]
    lens = [(97 * b) % 500 for b in range(B)]
    cu = cumulate(lens)
    s = make(cu[-1], B, *heads, dt)
    y, hT = forward(s, cu)
    got = dict(zip(GRADS, backward(s, cu)), y=y, hT=hT)
    torch.cuda.synchronize()
    errs = {}
    for b in (0, 1, 2, B // 2, B - 1):
        at = slice(cu[b], cu[b + 1])
        p = {k: v[at] if k in ("x", "dt", "B", "C", "dy") else v[b:b + 1] if k in ("h0", "dhT") else v for k, v in s.items()}
        want = ref.ssm(p["x"], p["dt"], p["A"], p["B"], p["C"], [0, lens[b]], p["D"], p["dt_bias"], True, p["h0"], p["dy"], p["dhT"])
        for k in ("y", "dx", "ddt", "dB", "dC"):
            errs[k] = max(errs.get(k, 0.0), worst(got[k][at], *want[k]))
        for k in ("hT", "dh0"):
            errs[k] = max(errs.get(k, 0.0), worst(got[k][b:b + 1], *want[k]))
    log(f"many chunks {dtype} B={B} {heads}: " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1, errs


@pytest.mark.parametrize("C,T", [(8, 3000), (24, 700), (520, 90), (8 * 63, 40), (8 * 65, 40), (8 * 130, 2000)])
def test_conv_widths(C, T):
    """Widths about those at which a workgroup's division changes, rows of many strips."""
    import gated_delta_rule_52_amd as gdn
    dt = torch.bfloat16
    cu = [0, T // 3, T // 3 + 1, T // 3 + 1, T - 1]
    x, dy, w, b = rand(T, C, dtype=dt), rand(T, C, dtype=dt, seed=1), rand(C, 4, std=0.5, seed=2), rand(C, seed=3)
    st = rand(4, 3, C, dtype=dt, seed=4)
    y, out = gdn.gdn_conv_forward(x, w, ints(cu), b, st)
    got = gdn.gdn_conv_backward(x, w, ints(cu), dy, b, st, dstate_out=st)
    torch.cuda.synchronize()
    n = cu[-1]
    wy, by, wst = ref.conv(x, w, cu, b, st)
    errs = {"y": worst(y[:n], wy[:n], by[:n])}
    for (k, (want, bound)), g in zip(ref.conv_backward(x, w, cu, dy, b, st, st).items(), got):
        errs[k] = worst(g[:n], want[:n], bound[:n]) if k == "dx" else worst(g, want, bound)
    log(f"conv C={C} T={T} " + " ".join(f"{k}={v:.2f}" for k, v in errs.items()))
    assert max(errs.values()) <= 1 and torch.equal(out.cpu().double(), wst), errs
