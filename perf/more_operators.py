"""What a state-space layer adds to a hybrid stack, and the page step that feeds all its layers, as cases to time.

  conv   the short causal convolution along the tokens (depthwise, with silu) that stands before a recurrent layer,
         over packed sequences, with its gradients, and one token a sequence with the state updated
  ssm    the selective state space scan, S <- exp(delta A) S + delta B x^T, y = S^T C + D x, heads in groups that
         share B and C: over packed sequences, with its gradients, and one token a sequence
  pages  one step of continuous batching: pages of finished sequences go back to the pool, new tokens get pages,
         and the call's sequence bounds, positions and slots are built from the lengths

Sizes: 6 heads of 128, 8 x 4096 tokens and 256 sequences with 16 heads are this
repository's benchmark sizes; the rest are generic.  A convolution's channels are
x, B and C side by side (heads x dim + 2 groups x state), and the scan takes them
as slices of that, so their token stride is wider than they are.

`run` is the operators in elementary torch operations where `own` is false, and
the library's calls where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 128  # of the plain scan


def listed():
    return [
        # a decode step of 256 sequences before the scan's 16 heads
        {"name": "conv, decode step", "op": "conv_step", "seqs": 256, "chan": 1280, "taps": 4, "dtype": "bf16"},
        # the training benchmark's tokens before 6 heads of 128, forward and backward
        {"name": "conv, training", "op": "conv", "seqs": 8, "new": 4096, "chan": 1024, "taps": 4, "state": False, "train": True, "even": True, "dtype": "bf16"},
        # pieces of prompts of odd lengths that go on from a state
        {"name": "conv, prompt pieces", "op": "conv", "seqs": 13, "new": 700, "chan": 1792, "taps": 4, "state": True, "train": False, "even": False, "dtype": "f32"},
        # the decode benchmark's batch
        {"name": "scan, decode step", "op": "ssm_step", "seqs": 256, "heads": 16, "groups": 1, "state_dim": 128, "dim": 64, "dtype": "bf16"},
        # one sequence, all latency
        {"name": "scan, decode one", "op": "ssm_step", "seqs": 1, "heads": 6, "groups": 1, "state_dim": 128, "dim": 128, "dtype": "f32"},
        # prompts of different lengths, some of them pieces that go on from a state
        {"name": "scan, prompts", "op": "ssm", "seqs": 8, "new": 4096, "heads": 16, "groups": 1, "state_dim": 128, "dim": 64, "state": True, "train": False, "even": False, "dtype": "bf16"},
        # one long prompt
        {"name": "scan, long prompt", "op": "ssm", "seqs": 1, "new": 32768, "heads": 8, "groups": 2, "state_dim": 128, "dim": 64, "state": False, "train": False, "even": True, "dtype": "bf16"},
        # the training benchmark's batch, 6 heads of 128, forward and backward
        {"name": "scan, training", "op": "ssm", "seqs": 8, "new": 4096, "heads": 6, "groups": 1, "state_dim": 128, "dim": 128, "state": False, "train": True, "even": True, "dtype": "bf16"},
        # more and smaller heads, sequences of odd lengths, gradients of the states too
        {"name": "scan, training packed", "op": "ssm", "seqs": 5, "new": 2777, "heads": 24, "groups": 2, "state_dim": 64, "dim": 64, "state": True, "train": True, "even": False, "dtype": "bf16"},
        # a short odd batch in fp32, forward and backward
        {"name": "scan, short fp32", "op": "ssm", "seqs": 3, "new": 333, "heads": 6, "groups": 1, "state_dim": 64, "dim": 64, "state": True, "train": True, "even": False, "dtype": "f32"},
        # every sequence of a full batch one token further
        {"name": "pages, decode step", "op": "pages", "seqs": 256, "new": 1, "context": 4096, "page": 16, "done": 4, "spare": 64},
        # prompts come in for finished sequences, more of them than the pool holds
        {"name": "pages, prompts", "op": "pages", "seqs": 512, "new": 2048, "context": 2048, "page": 16, "done": 100, "spare": 20000},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0), w["bytes"] * 300 + w["flops"])
    while True:
        op = rng.choice(("conv", "conv_step", "ssm", "ssm", "ssm_step", "pages"))
        c = {"op": op}
        if op == "pages":
            c.update(seqs=log(1, 512), new=log(1, 2048), context=log(16, 4096), page=rng.choice((16, 32, 64, 128)))
            c.update(done=rng.randint(0, c["seqs"] // 2), spare=log(8, 20000))
        else:
            c.update(dtype=rng.choice(("bf16", "bf16", "f32")))
            if op.startswith("conv"):
                c.update(seqs=log(1, 256), chan=8 * log(4, 256), taps=rng.choice((2, 3, 4, 4)))
            else:
                groups = rng.choice((1, 1, 2, 4))
                c.update(seqs=log(1, 256 if op == "ssm_step" else 16), heads=groups * rng.randint(1, 8), groups=groups,
                         state_dim=rng.choice((64, 128)), dim=rng.choice((64, 128)))
            if not op.endswith("step"):
                c.update(new=log(1, 4096), state=rng.random() < 0.5, train=rng.random() < 0.6, even=rng.random() < 0.3)
        w = work(c)
        if w["bytes"] * 300 + w["flops"] <= most[op] and w["bytes"] < 2e9:
            return c


# ---------------------------------------------------------------------------
# lengths of a case's sequences: the longest first, the others spread below it
# ---------------------------------------------------------------------------
def spread(n, lo, hi, turn):
    out = [hi]
    for i in range(1, n):
        x = i * 0.6180339887498949 + turn
        out.append(lo + int((hi - lo) * (x - math.floor(x))))
    return out


def lengths(case):
    if case.get("even"):
        return [case["new"]] * case["seqs"]
    return spread(case["seqs"], max(1, case["new"] // 4), case["new"], 0.37)


def work(case):
    op = case["op"]
    if op == "pages":
        new, old = lengths(case), page_context(case)
        t = sum(new)
        back = sum(-(-x // case["page"]) for x in old[: case["done"]])
        return {"bytes": case["seqs"] * 20 + back * 8 + t // case["page"] * 8 + t * 12, "flops": t}
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("conv"):
        c, w = case["chan"], case["taps"]
        t = case["seqs"] if op == "conv_step" else sum(lengths(case))
        st = case["seqs"] * (w - 1) * c * e
        by, fl = 2 * t * c * e + c * (w + 1) * 4, (2 * w + 5) * t * c
        by += 2 * st if op == "conv_step" else st * (2 if case["state"] else 1)
        if case.get("train"):  # x, dy -> dx, and the weights' gradients
            by += 3 * t * c * e + c * (w + 1) * 8 + (2 * st if case["state"] else 0)
            fl += (6 * w + 12) * t * c
        return {"bytes": by, "flops": fl}
    h, g, n, p = case["heads"], case["groups"], case["state_dim"], case["dim"]
    if op == "ssm_step":
        b = case["seqs"]
        return {"bytes": 2 * b * h * n * p * 4 + b * (2 * h * p + 2 * g * n) * e + b * h * 4, "flops": 6 * b * h * n * p}
    t, st = sum(lengths(case)), case["seqs"] * h * n * p * 4
    by = t * (2 * h * p + 2 * g * n) * e + t * h * 4 + st * (2 if case["state"] else 1)
    fl = t * h * 4 * n * p  # the state's two products; those inside a chunk depend on its length
    if case["train"]:  # x, B, C, dy, dt -> dx, dB, dC, ddt
        by += t * (3 * h * p + 4 * g * n) * e + 2 * t * h * 4 + (3 * st if case["state"] else 0)
        fl += t * h * 10 * n * p
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
def page_context(case):
    return spread(case["seqs"], case["context"] // 4, case["context"], 0.11)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s, op = dict(case=case), case["op"]
    if op == "pages":
        old, ps, b = page_context(case), case["page"], case["seqs"]
        held = [-(-x // ps) for x in old]
        pool = sum(held) + case["spare"]
        order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)  # pages as a pool hands them out
        shift = torch.randint(0, 3, (b,), generator=g, device=DEV, dtype=torch.int32)  # requests of another seed are others
        table = torch.full((b, max(-(-(x + n + 2) // ps) for x, n in zip(old, lengths(case)))), -1, dtype=torch.int32, device=DEV)
        at = torch.repeat_interleave(torch.arange(b, device=DEV), torch.tensor(held, device=DEV))
        first = torch.tensor([sum(held[:i]) for i in range(b)], device=DEV)
        table[at, torch.arange(sum(held), device=DEV) - first[at]] = order[: sum(held)]
        free = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
        free[: case["spare"]] = order[sum(held):]
        done = ints([1] * case["done"] + [0] * (b - case["done"]))
        want = ints(lengths(case))
        rows = sum(lengths(case)) + 2 * b if case["new"] > 1 else b
        s.update(ps=ps, done=done, want=want + shift if case["new"] > 1 else want - (shift == 2).int(), rows=rows, kv_len=ints(old), table=table, free=free, count=ints([case["spare"]]),
                 kv_mid=torch.empty(b, dtype=torch.int32, device=DEV), count_mid=torch.empty(1, dtype=torch.int32, device=DEV),
                 kv_out=torch.empty(b, dtype=torch.int32, device=DEV), count_out=torch.empty(1, dtype=torch.int32, device=DEV),
                 cu=torch.empty(b + 1, dtype=torch.int32, device=DEV), positions=torch.full((rows,), -1, dtype=torch.int32, device=DEV),
                 slots=torch.full((rows,), -1, dtype=torch.int64, device=DEV))
        return s
    dt = TYPES[case["dtype"]]

    def rand(*shape, mean=0.0, std=1.0, dtype=None):
        x = torch.empty(shape, dtype=torch.float32, device=DEV)
        return x.normal_(mean, std, generator=g).to(dtype or dt)

    def even(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=g, device=DEV) * (hi - lo) + lo

    b = case["seqs"]
    if not op.endswith("step"):
        cu = [0]
        for n in lengths(case):
            cu.append(cu[-1] + n)
        s["cu"], t = ints(cu), cu[-1]
    else:
        t = b
    if op.startswith("conv"):
        c, w = case["chan"], case["taps"]
        s.update(weight=even(c, w, lo=-w ** -0.5, hi=w ** -0.5), bias=even(c, lo=-0.2, hi=0.2), x=rand(t, c + 64)[:, :c])  # beside other outputs of the projection
        s["y"] = torch.empty(t, c, dtype=dt, device=DEV)
        s["state"] = rand(b, w - 1, c) if op == "conv_step" or case["state"] else None
        if op == "conv":
            s["state_out"] = torch.empty(b, w - 1, c, dtype=dt, device=DEV)
            if case["train"]:
                s.update(dy=rand(t, c), dx=torch.empty(t, c, dtype=dt, device=DEV), dweight=torch.empty(c, w, device=DEV), dbias=torch.empty(c, device=DEV))
                if case["state"]:
                    s.update(dstate_out=rand(b, w - 1, c), dstate=torch.empty(b, w - 1, c, dtype=dt, device=DEV))
        return s
    h, gr, n, p = case["heads"], case["groups"], case["state_dim"], case["dim"]
    xbc = rand(t, h * p + 2 * gr * n)
    s.update(x=xbc[:, : h * p].view(t, h, p), B=xbc[:, h * p: h * p + gr * n].view(t, gr, n), C=xbc[:, h * p + gr * n:].view(t, gr, n))
    step = torch.exp(even(h, lo=math.log(0.001), hi=math.log(0.1)))  # softplus(dt_bias), as such layers are initialised
    s.update(dt=rand(t, h, std=0.5, dtype=torch.float32), dt_bias=torch.log(torch.expm1(step)), A=-even(h, lo=1.0, hi=16.0), D=rand(h, mean=1.0, std=0.2, dtype=torch.float32))
    s["y"] = torch.empty(t, h, p, dtype=dt, device=DEV)
    if op == "ssm_step":
        s["state"] = rand(b, h, n, p, std=0.3, dtype=torch.float32)
        return s
    s["hT"] = torch.empty(b, h, n, p, device=DEV)
    s["h0"] = rand(b, h, n, p, std=0.3, dtype=torch.float32) if case["state"] else None
    if case["train"]:
        s.update(dy=rand(t, h, p), dhT=rand(b, h, n, p, std=0.1, dtype=torch.float32) if case["state"] else None)
        s["out"] = (torch.empty(t, h, p, dtype=dt, device=DEV), torch.empty(t, h, device=DEV), torch.empty(h, device=DEV),
                    torch.empty(t, gr, n, dtype=dt, device=DEV), torch.empty(t, gr, n, dtype=dt, device=DEV), torch.empty(h, device=DEV),
                    torch.empty(h, device=DEV), torch.empty(b, h, n, p, device=DEV) if case["state"] else None)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"conv": own_conv, "conv_step": own_conv_step, "ssm": own_ssm, "ssm_step": own_ssm_step, "pages": own_pages}[op](s)
    return {"conv": plain_conv, "conv_step": plain_conv_step, "ssm": plain_ssm, "ssm_step": plain_ssm_step, "pages": plain_pages}[op](s)


def own_conv(s):
    import gated_delta_rule_52_amd as gdn
    y, st = gdn.gdn_conv_forward(s["x"], s["weight"], s["cu"], s["bias"], s["state"], silu=True, y=s["y"], state_out=s["state_out"])
    out = {"y": y, "state": st}
    if s["case"]["train"]:
        dx, dw, db, ds = gdn.gdn_conv_backward(s["x"], s["weight"], s["cu"], s["dy"], s["bias"], s["state"], silu=True, dstate_out=s.get("dstate_out"),
                                               out=(s["dx"], s["dweight"], s["dbias"], s.get("dstate")))
        out.update(dx=dx, dweight=dw, dbias=db, dstate=ds)
    return out


def own_conv_step(s):
    import gated_delta_rule_52_amd as gdn
    return {"y": gdn.gdn_conv_step(s["x"], s["weight"], s["state"], s["bias"], silu=True, y=s["y"]), "state": s["state"]}


def own_ssm(s):
    import gated_delta_rule_52_amd as gdn
    a = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"])
    y, hT = gdn.gdn_ssm_forward(*a, D=s["D"], dt_bias=s["dt_bias"], softplus=True, h0=s["h0"], y=s["y"], hT=s["hT"])
    out = {"y": y, "hT": hT}
    if s["case"]["train"]:
        names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")
        out.update(zip(names, gdn.gdn_ssm_backward(*a, s["dy"], D=s["D"], dt_bias=s["dt_bias"], softplus=True, h0=s["h0"], dhT=s["dhT"], out=s["out"])))
    return out


def own_ssm_step(s):
    import gated_delta_rule_52_amd as gdn
    y = gdn.gdn_ssm_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], dt_bias=s["dt_bias"], softplus=True, y=s["y"])
    return {"y": y, "state": s["state"]}


def own_pages(s):
    import gated_delta_rule_52_amd as gdn
    gdn.gdn_pages_release(s["done"], s["kv_len"], s["table"], s["free"], s["count"], s["ps"], kv_out=s["kv_mid"], count_out=s["count_mid"])
    gdn.gdn_pages_take(s["want"], s["kv_mid"], s["table"], s["free"], s["count_mid"], s["ps"], s["rows"], kv_out=s["kv_out"], count_out=s["count_out"],
                       cu_seqlens=s["cu"], positions=s["positions"], slots=s["slots"])
    return page_outputs(s)


def page_outputs(s):
    return {"kv_len": s["kv_out"], "count": s["count_out"], "table": s["table"], "free": s["free"], "cu": s["cu"], "positions": s["positions"], "slots": s["slots"]}


def of_tokens(cu, t):
    """Sequence of every token, and its place there."""
    tok = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    return b, tok - cu[b]


def plain_conv(s):
    cu, w, x = s["cu"], s["weight"], s["x"]
    b, t, (c, taps) = len(cu) - 1, len(x), w.shape
    k, dt = taps - 1, x.dtype
    sb, _ = of_tokens(cu, t)
    at = torch.arange(t, device=DEV) + sb * k  # window of every token in the sequences with their states before them
    ahead = (cu[:-1] + torch.arange(b, device=DEV) * k)[:, None] + torch.arange(k, device=DEV)
    last = (cu[1:] + torch.arange(b, device=DEV) * k)[:, None] + torch.arange(k, device=DEV)
    e = torch.zeros(t + b * k, c, dtype=torch.float32, device=DEV)
    e[at + k] = x.float()
    if s["state"] is not None:
        e[ahead] = s["state"].float()
    z = s["bias"] + sum(w[:, j] * e[at + j] for j in range(taps))
    sig = 1.0 / (1.0 + torch.exp(-z))
    out = {"y": (z * sig).to(dt), "state": e[last].to(dt)}
    if s["case"]["train"]:
        dz = s["dy"].float() * sig * (1.0 + z * (1.0 - sig))
        de = torch.zeros_like(e)
        for j in range(taps):
            de[at + j] += w[:, j] * dz
        if s["state"] is not None:
            de[last] += s["dstate_out"].float()
        dw = torch.stack([(dz * e[at + j]).sum(0, dtype=torch.float64) for j in range(taps)], 1)
        out.update(dx=de[at + k].to(dt), dweight=dw.float(), dbias=dz.sum(0, dtype=torch.float64).float(), dstate=None if s["state"] is None else de[ahead].to(dt))
    return out


def plain_conv_step(s):
    dt = s["x"].dtype
    e = torch.cat([s["state"], s["x"][:, None]], 1)
    z = s["bias"] + (e.float() * s["weight"].T).sum(1)
    s["state"].copy_(e[:, 1:])
    return {"y": (z / (1.0 + torch.exp(-z))).to(dt), "state": s["state"]}


def softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(v.clamp(max=20.0))))


def chunks(x, at, live):
    """[T, H, ...] as [B, H, n, CHUNK, ...] in fp32, zeros behind a sequence's end."""
    x = x[at].float() * live.reshape(live.shape + (1,) * (x.dim() - 1))  # [B, n CHUNK, H, ...]
    return x.unflatten(1, (-1, CHUNK)).movedim(3, 1).contiguous()


def plain_ssm(s):
    cu, t, case = s["cu"], len(s["x"]), s["case"]
    h, gr, b, dt = case["heads"], case["groups"], case["seqs"], s["x"].dtype
    most = -(-case["new"] // CHUNK) * CHUNK
    place = torch.arange(most, device=DEV)
    live = place < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + place).clamp(max=t - 1)
    sb, i = of_tokens(cu, t)
    v = s["dt"] + s["dt_bias"]
    x, B, C = chunks(s["x"], at, live), chunks(s["B"], at, live), chunks(s["C"], at, live)
    B, C = B.repeat_interleave(h // gr, 1), C.repeat_interleave(h // gr, 1)
    d = chunks(softplus(v), at, live)  # [B, H, n, L], 0 behind the end: nothing changes there
    cum = (d.double() * s["A"].double()[:, None, None]).cumsum(-1)  # 64 bits: differences of large sums
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()

    def decay(c, see):  # exp(c_t - c_s) where see, 0 elsewhere
        return torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~see, -math.inf).float())

    E = decay(cum, lower)
    W = E * torch.matmul(C, B.transpose(-1, -2))
    u = x * d[..., None]
    end, start = torch.exp((cum[..., -1:] - cum).float())[..., None], torch.exp(cum.float())[..., None]
    # states at the chunks' starts and at the end: of chunk n, what h0 and the chunks before it have left
    nc = d.shape[2]
    local = torch.matmul((B * end).transpose(-1, -2), u)  # [B, H, n, N, P]
    ends = torch.nn.functional.pad(cum[..., -1].cumsum(-1), (1, 0))  # [B, H, n + 1]
    h0 = torch.zeros(b, h, 1, *local.shape[3:], device=DEV) if s["h0"] is None else s["h0"][:, :, None]
    carry = decay(ends, torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=DEV).tril())
    S = torch.matmul(carry, torch.cat([h0, local], 2).flatten(3)).unflatten(3, local.shape[3:])
    y = torch.matmul(W, u) + start * torch.matmul(C, S[:, :, :-1])
    y = y + s["D"][:, None, None, None] * x

    def packed(a):  # [B, H, n, L, ...] -> [T, H, ...]
        return a.movedim(1, 3).flatten(1, 2)[sb, i]

    out = {"y": packed(y).to(dt), "hT": S[:, :, -1].contiguous()}
    if not case["train"]:
        return out
    dy = chunks(s["dy"], at, live)
    dhT = torch.zeros(b, h, 1, *local.shape[3:], device=DEV) if s["dhT"] is None else s["dhT"][:, :, None]
    back = torch.matmul((C * start).transpose(-1, -2), dy)  # what a chunk adds to its start's gradient
    dS = torch.matmul(carry.transpose(-1, -2), torch.cat([back, dhT], 2).flatten(3)).unflatten(3, local.shape[3:])
    S_in, dS_out = S[:, :, :-1], dS[:, :, 1:]
    Z = torch.matmul(dy, x.transpose(-1, -2))
    du_far = end * torch.matmul(B, dS_out)
    du = torch.matmul(W.transpose(-1, -2), dy) + du_far
    Zd = E * Z
    dC_far = start * torch.matmul(dy, S_in.transpose(-1, -2))
    dC = torch.matmul(Zd * d[..., None, :], B) + dC_far
    dB = d[..., None] * (torch.matmul(Zd.transpose(-1, -2), C) + end * torch.matmul(x, dS_out.transpose(-1, -2)))
    # gradient of the log-decays: every pair whose span holds the token
    M = (W * Z * d[..., None, :]).double()
    r, q = (C * dC_far).sum(-1).double(), (u * du_far).sum(-1).double()
    through = torch.exp(cum[..., -1].float()) * (S_in * dS_out).sum((-1, -2))
    over = (M.sum(-1) - M.sum(-2) + r).flip(-1).cumsum(-1).flip(-1)
    dg = over + q.cumsum(-1) - q + through.double()[..., None]
    ddelta = dg * s["A"].double()[:, None, None] + (x * du).sum(-1).double()
    dv = packed(ddelta) / (1.0 + torch.exp(-v.double()))
    out.update(dx=packed(d[..., None] * du + s["D"][:, None, None, None] * dy).to(dt), ddt=dv.float(), dA=(d.double() * dg).sum((0, 2, 3)).float(),
               dB=packed(dB.unflatten(1, (gr, -1)).sum(2)).to(dt), dC=packed(dC.unflatten(1, (gr, -1)).sum(2)).to(dt),
               dD=(x * dy).sum((0, 2, 3, 4), dtype=torch.float64).float(), ddt_bias=dv.sum(0).float(), dh0=None if s["h0"] is None else dS[:, :, 0].contiguous())
    return out


def plain_ssm_step(s):
    h, gr = s["case"]["heads"], s["case"]["groups"]
    x, d = s["x"].float(), softplus(s["dt"] + s["dt_bias"])
    B, C = (a.float().repeat_interleave(h // gr, 1) for a in (s["B"], s["C"]))
    st = s["state"]
    st.copy_(st * torch.exp(d * s["A"])[..., None, None] + (d[..., None] * B)[..., None] * x[:, :, None])
    y = (st * C[..., None]).sum(2) + s["D"][:, None] * x
    return {"y": y.to(s["x"].dtype), "state": st}


def plain_pages(s):
    ps, table, free, b, width = s["ps"], s["table"], s["free"], len(s["want"]), s["table"].shape[1]
    # pages of finished sequences go back, in the order of the sequences
    back = torch.where(s["done"] != 0, (s["kv_len"] + ps - 1) // ps, 0)
    rows = s["count"] + back.cumsum(0) - back
    col = torch.arange(width, device=DEV)
    sq, k = torch.nonzero(col < back[:, None], as_tuple=True)
    free[rows[sq] + k] = table[sq, k]
    kv, count = torch.where(s["done"] != 0, 0, s["kv_len"]), s["count"] + back.sum()
    # a sequence gets all its tokens or none: its table has room, the pool has pages for it and all before it, the rows hold it
    have, need = (kv + ps - 1) // ps, (kv + s["want"] + ps - 1) // ps
    fits = need <= width
    fresh = torch.where(fits, need - have, 0)
    ok = fits & ((fresh == 0) | (fresh.cumsum(0) <= count))
    n = torch.where(ok, s["want"], 0)
    ok &= n.cumsum(0) <= s["rows"]
    n, fresh = torch.where(ok, s["want"], 0), torch.where(ok, fresh, 0)
    first = count - (fresh.cumsum(0) - fresh)
    sq, k = torch.nonzero(col < fresh[:, None], as_tuple=True)
    table[sq, have[sq] + k] = free[first[sq] - 1 - k]
    s["kv_out"].copy_(kv + n)
    s["count_out"].copy_(count - fresh.sum())
    s["cu"].copy_(torch.nn.functional.pad(n.cumsum(0), (1, 0)))
    sq = torch.repeat_interleave(torch.arange(b, device=DEV), n)
    tok = torch.arange(len(sq), device=DEV)
    pos = kv[sq] + tok - s["cu"][sq]
    s["positions"][tok] = pos.to(torch.int32)
    s["slots"][tok] = table[sq, pos // ps].long() * ps + pos % ps
    return page_outputs(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a sequence and a head at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    lens = [1] * case["seqs"] if op.endswith("step") else lengths(case)
    if op.startswith("conv"):
        return exact_conv(case, s, lens)
    h, per = case["heads"], case["heads"] // case["groups"]
    d = torch.nn.functional.softplus(s["dt"] + s["dt_bias"], threshold=700.0)
    if op == "ssm_step":
        y, st = torch.empty_like(s["x"]), torch.empty_like(s["state"])
        for k in range(h):
            at = torch.exp(d[:, k] * s["A"][k])
            st[:, k] = at[:, None, None] * s["state"][:, k] + torch.einsum("b,bn,bp->bnp", d[:, k], s["B"][:, k // per], s["x"][:, k])
            y[:, k] = torch.einsum("bn,bnp->bp", s["C"][:, k // per], st[:, k]) + s["D"][k] * s["x"][:, k]
        return {"y": y, "state": st}
    train, zero = case["train"], torch.zeros(case["state_dim"], case["dim"], dtype=torch.float64, device=DEV)
    out = {"y": torch.empty_like(s["x"]), "hT": torch.empty_like(s["hT"])}
    if train:
        out.update(dx=torch.empty_like(s["x"]), ddt=torch.empty_like(s["dt"]), dA=torch.zeros_like(s["A"]), dB=torch.zeros_like(s["B"].contiguous()),
                   dC=torch.zeros_like(s["C"].contiguous()), dD=torch.zeros_like(s["A"]), ddt_bias=None, dh0=torch.empty_like(s["hT"]) if case["state"] else None)
    lo = 0
    for b, n in enumerate(lens):
        hi = lo + n
        for k in range(h):
            g, A = k // per, s["A"][k]
            x, B, C, dl = s["x"][lo:hi, k], s["B"][lo:hi, g], s["C"][lo:hi, g], d[lo:hi, k]
            c = torch.cumsum(dl * A, 0)
            S0 = s["h0"][b, k] if case["state"] else zero
            u = dl[:, None] * x
            tail = torch.exp(c[-1] - c)
            out["hT"][b, k] = torch.exp(c[-1]) * S0 + (tail[:, None] * B).T @ u
            y = torch.exp(c)[:, None] * (C @ S0) + s["D"][k] * x
            if train:
                dy = s["dy"][lo:hi, k]
                dS = s["dhT"][b, k] if case["state"] else zero
                dC = torch.exp(c)[:, None] * (dy @ S0.T)
                du = tail[:, None] * (B @ dS)
                dBk = tail[:, None] * (u @ dS.T)
                # the gradient of c_t: what decays from t on, less what t itself has put in; the end's whole state at the last one
                dc = (C * dC).sum(1) - (u * du).sum(1)
                dc[-1] += torch.sum(out["hT"][b, k] * dS)
            for r0 in range(0, n, 2048):  # blocks of rows of the whole triangle
                r1 = min(n, r0 + 2048)
                gap = c[r0:r1, None] - c[:r1]
                E = torch.exp(gap.masked_fill(torch.arange(r1, device=DEV) > torch.arange(r0, r1, device=DEV)[:, None], -math.inf))
                W = (C[r0:r1] @ B[:r1].T) * E
                y[r0:r1] += W @ u[:r1]
                if train:
                    dyr = dy[r0:r1]
                    du[:r1] += W.T @ dyr
                    EZ = (dyr @ u[:r1].T) * E
                    dC[r0:r1] += EZ @ B[:r1]
                    dBk[:r1] += EZ.T @ C[r0:r1]
                    M = W * (dyr @ u[:r1].T)
                    dc[r0:r1] += M.sum(1)
                    dc[:r1] -= M.sum(0)
            out["y"][lo:hi, k] = y
            if train:
                dg = dc.flip(0).cumsum(0).flip(0)
                out["dx"][lo:hi, k] = dl[:, None] * du + s["D"][k] * dy
                out["dB"][lo:hi, g] += dBk
                out["dC"][lo:hi, g] += dC
                out["ddt"][lo:hi, k] = (A * dg + (x * du).sum(1)) * torch.sigmoid(s["dt"][lo:hi, k] + s["dt_bias"][k])
                out["dA"][k] += torch.sum(dl * dg)
                out["dD"][k] += torch.sum(dy * x)
                if case["state"]:
                    out["dh0"][b, k] = torch.exp(c[-1]) * dS + (torch.exp(c)[:, None] * C).T @ dy
        lo = hi
    if train:
        out["ddt_bias"] = out["ddt"].sum(0)
    return out


def exact_conv(case, s, lens):
    w, k = s["weight"], case["taps"] - 1
    out = {"y": torch.empty_like(s["y"]), "state": torch.empty(case["seqs"], k, case["chan"], dtype=torch.float64, device=DEV)}
    train = case.get("train")
    if train:
        out.update(dx=torch.empty_like(s["y"]), dweight=torch.zeros_like(w), dbias=torch.zeros_like(s["bias"]), dstate=torch.empty_like(out["state"]) if case["state"] else None)
    lo = 0
    for b, n in enumerate(lens):
        before = torch.zeros(k, case["chan"], dtype=torch.float64, device=DEV) if s["state"] is None else s["state"][b]
        e = torch.cat([before, s["x"][lo:lo + n]])
        windows = e.unfold(0, k + 1, 1)  # [n, C, taps]
        z = (windows * w).sum(2) + s["bias"]
        out["y"][lo:lo + n] = z * torch.sigmoid(z)
        out["state"][b] = e[n:]
        if train:
            sg = torch.sigmoid(z)
            dz = s["dy"][lo:lo + n] * (sg + z * sg * (1 - sg))
            out["dweight"] += (windows * dz[..., None]).sum(0)
            out["dbias"] += dz.sum(0)
            wide = torch.nn.functional.pad(dz, (0, 0, k, k)).unfold(0, k + 1, 1)  # dz_{i - k} .. dz_i for every row i of e
            de = (wide * w.flip(1)).sum(2)
            if case["state"]:
                de[n:] += s["dstate_out"][b]
                out["dstate"][b] = de[:k]
            out["dx"][lo:lo + n] = de[k:]
        lo += n
    return out
