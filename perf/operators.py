"""The operators around the gated delta-rule layer in a hybrid stack, as cases to time.

A stack that mixes gated delta-rule layers with softmax-attention layers needs,
next to the delta rule itself, four things:

  norm_block  residual add with a residual scale per channel, then RMS norm: what stands before a block
  norm_gate   RMS norm of every head's output, times a weight, times silu of the gate: what stands after it
  append      new keys and values into a paged cache, keys (and the queries handed on) rotated by position
  paged       causal attention of each sequence's new tokens over its pages (one token: decoding)
  prompt      causal attention over packed prompts, with its gradients

Sizes: width 768 = 6 heads of 128, 8 x 4096 tokens and 256 sequences with 16 heads
are this repository's benchmark sizes, 131072 tokens its longest context; the
rest are generic.  q, k and v are slices of one projection's output, so their
token stride is wider than their heads.

`run` is the operators in elementary torch operations where `own` is false, and
the library's calls where it is true.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode step of 32 sequences: all latency
        {"name": "block norm, decode step", "op": "norm_block", "rows": 32, "width": 2048, "dtype": "bf16", "train": False},
        # the training benchmark's tokens and width, forward and backward
        {"name": "block norm, training", "op": "norm_block", "rows": 32768, "width": 768, "dtype": "bf16", "train": True},
        # the decode benchmark's heads, fp32
        {"name": "gated norm, decode step", "op": "norm_gate", "rows": 256, "heads": 16, "dim": 128, "dtype": "f32", "train": False},
        # the training benchmark's layer output, forward and backward
        {"name": "gated norm, training", "op": "norm_gate", "rows": 32768, "heads": 6, "dim": 128, "dtype": "bf16", "train": True},
        # one token for each of 256 sequences in the middle of their contexts
        {"name": "append, decode step", "op": "append", "seqs": 256, "new": 1, "context": 2048, "hq": 16, "hkv": 4, "dim": 128, "page": 16, "dtype": "bf16"},
        # eight prompts of different lengths enter the cache
        {"name": "append, prompts", "op": "append", "seqs": 8, "new": 4096, "context": 0, "hq": 16, "hkv": 4, "dim": 128, "page": 64, "dtype": "bf16"},
        # decoding, a full batch of ordinary contexts
        {"name": "paged, decode batch", "op": "paged", "seqs": 256, "new": 1, "context": 4096, "hq": 16, "hkv": 4, "dim": 128, "page": 16, "dtype": "bf16"},
        # decoding, two very long contexts and few heads
        {"name": "paged, decode long", "op": "paged", "seqs": 2, "new": 1, "context": 131072, "hq": 16, "hkv": 2, "dim": 128, "page": 64, "dtype": "bf16"},
        # prompts that arrive in pieces: 512 more tokens on contexts up to 16384
        {"name": "paged, chunks", "op": "paged", "seqs": 4, "new": 512, "context": 16384, "hq": 16, "hkv": 4, "dim": 128, "page": 32, "dtype": "bf16"},
        # a short odd batch in fp32, forward and backward
        {"name": "prompt, short fp32", "op": "prompt", "seqs": 3, "new": 333, "hq": 6, "hkv": 2, "dim": 64, "dtype": "f32", "train": True},
        # the training benchmark's batch, packed: eight sequences up to 4096, six heads
        {"name": "prompt, training packed", "op": "prompt", "seqs": 8, "new": 4096, "hq": 6, "hkv": 2, "dim": 128, "dtype": "bf16", "train": True},
        # one long sequence, forward and backward
        {"name": "prompt, training long", "op": "prompt", "seqs": 1, "new": 8192, "hq": 16, "hkv": 4, "dim": 128, "dtype": "bf16", "train": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = max(most.get(c["op"], 0), w["bytes"] * 300 + w["flops"])
    while True:
        op = rng.choice(("norm_block", "norm_gate", "append", "paged", "prompt"))
        c = {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32"))}
        if op == "norm_block":
            c.update(rows=log(1, 32768), width=8 * log(8, 1024), train=rng.random() < 0.6)
        elif op == "norm_gate":
            c.update(rows=log(1, 32768), heads=rng.randint(1, 16), dim=rng.choice((16, 32, 64, 128)), train=rng.random() < 0.6)
        else:
            hkv = rng.choice((1, 2, 3, 4, 8))
            c.update(hq=hkv * rng.choice((1, 2, 3, 4, 6, 8)), hkv=hkv, dim=rng.choice((64, 128)))
            if op == "prompt":
                c.update(seqs=log(1, 16), new=log(1, 8192), train=rng.random() < 0.7)
            else:
                new = 1 if rng.random() < 0.4 else log(2, 2048)
                c.update(seqs=log(1, 256), new=new, context=log(16, 65536), page=rng.choice((16, 32, 64, 128)))
        w = work(c)
        if w["bytes"] * 300 + w["flops"] <= most[op] and w["bytes"] < 3e9 and w["flops"] < 3e12:
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
    """New tokens and whole context (the new ones among them) of every sequence."""
    new = spread(case["seqs"], max(1, case["new"] // 4), case["new"], 0.37)
    ctx = case.get("context", 0)
    old = spread(case["seqs"], ctx // 4, ctx, 0.11)
    return new, [a + b for a, b in zip(new, old)]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "norm_block":
        n, d = case["rows"] * case["width"], case["width"]
        by = n * 4 * e + 2 * d * 4  # x, y -> h, n
        fl = 7 * n
        if case["train"]:  # x, y, dn, dh -> dx, dy, and the two weights' gradients
            by += n * 6 * e + 4 * d * 4
            fl += 15 * n
        return {"bytes": by, "flops": fl}
    if op == "norm_gate":
        n, d = case["rows"] * case["heads"] * case["dim"], case["dim"]
        by, fl = n * 3 * e + d * 4, 10 * n
        if case["train"]:  # dy, o, gate -> do, dgate
            by += n * 5 * e + 2 * d * 4
            fl += 25 * n
        return {"bytes": by, "flops": fl}
    new, whole = lengths(case)
    t, hq, hkv, d = sum(new), case["hq"], case["hkv"], case["dim"]
    if op == "append":
        return {"bytes": 2 * t * (hq + 2 * hkv) * d * e + t * d * 4 + t * 8, "flops": 3 * t * (hq + hkv) * d}
    pairs = sum(n * (w - n) + n * (n + 1) // 2 for n, w in zip(new, whole))
    if op == "paged":
        return {"bytes": 2 * t * hq * d * e + 2 * sum(whole) * hkv * d * e, "flops": 4 * pairs * hq * d}
    by, fl = (2 * hq + 2 * hkv) * t * d * e + t * hq * 4, 4 * pairs * hq * d
    if case["train"]:  # q, k, v, o, do, lse -> dq, dk, dv: five products for two
        by += (4 * hq + 4 * hkv) * t * d * e - hq * t * d * e + t * hq * 4
        fl += 10 * pairs * hq * d
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------------------
# what a program has in hand before the call
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def rand(*shape, mean=0.0, std=1.0, dtype=None):
        x = torch.empty(shape, dtype=torch.float32, device=DEV)
        return x.normal_(mean, std, generator=g).to(dtype or dt)

    s = dict(case=case)
    op = case["op"]
    if op == "norm_block":
        r, d = case["rows"], case["width"]
        s.update(x=rand(r, d, std=2.0), y=rand(r, d), weight=rand(d, mean=1.0, std=0.1, dtype=torch.float32),
                 res_scale=rand(d, mean=0.5, std=0.1, dtype=torch.float32))
        s.update(h=torch.empty_like(s["x"]), n=torch.empty_like(s["x"]), rstd=torch.empty(r, dtype=torch.float32, device=DEV))
        if case["train"]:
            s.update(dn=rand(r, d), dh=rand(r, d), dx=torch.empty_like(s["x"]), dy=torch.empty_like(s["x"]),
                     dweight=torch.empty_like(s["weight"]), dres_scale=torch.empty_like(s["weight"]))
        return s
    if op == "norm_gate":
        r, h, d = case["rows"], case["heads"], case["dim"]
        s.update(o=rand(r, h, d, std=0.3), weight=rand(d, mean=1.0, std=0.1, dtype=torch.float32))
        s["gate"] = rand(r, 2, h, d)[:, 1]  # a projection's output holds the gate beside something else
        s.update(y=torch.empty_like(s["o"]), rstd=torch.empty(r, h, dtype=torch.float32, device=DEV))
        if case["train"]:
            s.update(dy=rand(r, h, d), do=torch.empty_like(s["o"]), dgate=torch.empty_like(s["o"]), dweight=torch.empty_like(s["weight"]))
        return s
    new, whole = lengths(case)
    t, b, hq, hkv, d = sum(new), case["seqs"], case["hq"], case["hkv"], case["dim"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if op == "prompt":
        qkv = rand(t, hq + 2 * hkv, d)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        s.update(o=torch.empty(t, hq, d, dtype=dt, device=DEV), lse=torch.empty(t, hq, dtype=torch.float32, device=DEV))
        if case["train"]:
            s.update(do=rand(t, hq, d), dq=torch.empty(t, hq, d, dtype=dt, device=DEV),
                     dk=torch.empty(t, hkv, d, dtype=dt, device=DEV), dv=torch.empty(t, hkv, d, dtype=dt, device=DEV))
        return s
    ps = case["page"]
    pages = [-(-w // ps) for w in whole]
    order = torch.randperm(sum(pages), generator=g, device=DEV).to(torch.int32)  # pages as a pool hands them out
    table = torch.full((b, max(pages)), -1, dtype=torch.int32, device=DEV)
    at = torch.repeat_interleave(torch.arange(b, device=DEV), torch.tensor(pages, device=DEV))
    first = torch.tensor([sum(pages[:i]) for i in range(b)], device=DEV)
    table[at, torch.arange(len(order), device=DEV) - first[at]] = order
    s.update(table=table, kv_len=torch.tensor(whole, dtype=torch.int32, device=DEV))
    s.update(k_cache=rand(len(order), ps, hkv, d), v_cache=rand(len(order), ps, hkv, d))
    if op == "append":
        qkv = rand(t, hq + 2 * hkv, d)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], q_out=torch.empty(t, hq, d, dtype=dt, device=DEV))
        freq = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
        ang = torch.arange(max(whole), dtype=torch.float64, device=DEV)[:, None] * freq
        s.update(cos=ang.cos().float(), sin=ang.sin().float())
    else:
        s.update(q=rand(t, hq, d), o=torch.empty(t, hq, d, dtype=dt, device=DEV))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm_block": own_norm_block, "norm_gate": own_norm_gate, "append": own_append, "paged": own_paged, "prompt": own_prompt}[op](s)
    return {"norm_block": plain_norm_block, "norm_gate": plain_norm_gate, "append": plain_append, "paged": plain_paged, "prompt": plain_prompt}[op](s)


def own_norm_block(s):
    import gated_delta_rule_52_amd as gdn
    h, n, rstd = gdn.gdn_norm_block(s["x"], s["weight"], s["y"], s["res_scale"], eps=EPS, out=(s["h"], s["n"], s["rstd"]))
    if not s["case"]["train"]:
        return {"h": h, "n": n}
    dx, dy, dw, drs = gdn.gdn_norm_block_backward(s["dn"], s["x"], s["weight"], rstd, s["y"], s["res_scale"], dh=s["dh"],
                                                  out=(s["dx"], s["dy"], s["dweight"], s["dres_scale"]))
    return {"h": h, "n": n, "dx": dx, "dy": dy, "dweight": dw, "dres_scale": drs}


def own_norm_gate(s):
    import gated_delta_rule_52_amd as gdn
    y, rstd = gdn.gdn_norm_gate(s["o"], s["gate"], s["weight"], eps=EPS, out=(s["y"], s["rstd"]))
    if not s["case"]["train"]:
        return {"y": y}
    do, dgate, dw = gdn.gdn_norm_gate_backward(s["dy"], s["o"], s["gate"], s["weight"], rstd, out=(s["do"], s["dgate"], s["dweight"]))
    return {"y": y, "do": do, "dgate": dgate, "dweight": dw}


def own_append(s):
    import gated_delta_rule_52_amd as gdn
    q = gdn.gdn_attn_append(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["cu"], s["kv_len"], s["table"], s["k_cache"], s["v_cache"], q_out=s["q_out"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def own_paged(s):
    import gated_delta_rule_52_amd as gdn
    return {"o": gdn.gdn_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], o=s["o"])}


def own_prompt(s):
    import gated_delta_rule_52_amd as gdn
    o, lse = gdn.gdn_attn_forward(s["q"], s["k"], s["v"], s["cu"], o=s["o"], lse=s["lse"])
    if not s["case"]["train"]:
        return {"o": o, "lse": lse}
    dq, dk, dv = gdn.gdn_attn_backward(s["q"], s["k"], s["v"], s["cu"], o, lse, s["do"], out=(s["dq"], s["dk"], s["dv"]))
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def plain_norm_block(s):
    dt, w, rs = s["x"].dtype, s["weight"], s["res_scale"]
    y = s["y"].float()
    h = s["x"].float() + rs * y
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    xh = h * r
    out = {"h": h.to(dt), "n": (xh * w).to(dt)}
    if s["case"]["train"]:
        dn = s["dn"].float()
        g = dn * w
        dx = s["dh"].float() + r * (g - xh * (g * xh).mean(-1, keepdim=True))
        out.update(dx=dx.to(dt), dy=(dx * rs).to(dt), dweight=(dn * xh).sum(0), dres_scale=(dx * y).sum(0))
    return out


def plain_norm_gate(s):
    dt, w = s["o"].dtype, s["weight"]
    o, z = s["o"].float(), s["gate"].float()
    r = torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS)
    oh, sig = o * r, 1.0 / (1.0 + torch.exp(-z))
    silu = z * sig
    out = {"y": (oh * w * silu).to(dt)}
    if s["case"]["train"]:
        dy = s["dy"].float()
        g = dy * silu * w
        do = r * (g - oh * (g * oh).mean(-1, keepdim=True))
        dz = dy * oh * w * (sig + silu * (1.0 - sig))
        out.update(do=do.to(dt), dgate=dz.to(dt), dweight=(dy * silu * oh).sum((0, 1)))
    return out


def of_tokens(cu, t):
    """Sequence of every token, and its place there."""
    tok = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    return tok, b, tok - cu[b]


def plain_append(s):
    q, k, v = s["q"], s["k"], s["v"]
    tok, b, i = of_tokens(s["cu"], len(q))
    n = s["cu"][1:] - s["cu"][:-1]
    pos = (s["kv_len"] - n)[b] + i
    ps = s["k_cache"].shape[1]
    page, slot = s["table"][b, pos // ps].long(), pos % ps
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]

    def rotate(x):
        x1, x2 = x.float().chunk(2, -1)
        return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).to(x.dtype)

    s["k_cache"][page, slot] = rotate(k)
    s["v_cache"][page, slot] = v
    return {"q": rotate(q), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def padded(x, cu, n):
    """[T, H, D] as [B, H, n, D] in fp32; places behind a sequence's end repeat some token."""
    at = (cu[:-1, None] + torch.arange(n, device=cu.device)).clamp(max=len(x) - 1)
    return x[at].float().transpose(1, 2)


def softmax(sc, see):
    sc = sc.masked_fill(~see, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    z = p.sum(-1, keepdim=True)
    return p / z, (m + torch.log(z)).squeeze(-1)


def plain_paged(s):
    c, cu = s["case"], s["cu"]
    hkv, d, ps = c["hkv"], c["dim"], c["page"]
    g, n, b = c["hq"] // hkv, c["new"], c["seqs"]
    width = s["table"].shape[1] * ps
    at = torch.arange(width, device=DEV)
    rows = s["table"][:, at // ps].clamp(min=0).long() * ps + at % ps
    k = s["k_cache"].view(-1, hkv, d)[rows].float().permute(0, 2, 3, 1)  # [B, Hkv, D, L]
    v = s["v_cache"].view(-1, hkv, d)[rows].float().transpose(1, 2)
    q = padded(s["q"], cu, n).reshape(b, hkv, g * n, d)
    pos = (s["kv_len"] - (cu[1:] - cu[:-1]))[:, None] + torch.arange(n, device=DEV)  # [B, n]
    see = (at <= pos[:, :, None])[:, None].repeat(1, 1, g, 1)
    p, _ = softmax(torch.matmul(q, k) * d ** -0.5, see)
    o = torch.matmul(p, v).reshape(b, c["hq"], n, d)
    _, sb, i = of_tokens(cu, len(s["q"]))
    return {"o": o[sb, :, i].to(s["q"].dtype)}


def plain_prompt(s):
    c, cu, dt = s["case"], s["cu"], s["q"].dtype
    hq, hkv, d, n, b = c["hq"], c["hkv"], c["dim"], c["new"], c["seqs"]
    g, scale = hq // hkv, d ** -0.5
    q = padded(s["q"], cu, n).reshape(b, hkv, g * n, d)
    k, v = padded(s["k"], cu, n).contiguous(), padded(s["v"], cu, n).contiguous()
    at = torch.arange(n, device=DEV)
    see = (at <= at[:, None]).repeat(g, 1)
    p, lse = softmax(torch.matmul(q, k.transpose(-1, -2)) * scale, see)
    o = torch.matmul(p, v)
    _, sb, i = of_tokens(cu, len(s["q"]))

    def packed(x, h):
        return x.reshape(b, h, n, -1)[sb, :, i]

    out = {"o": packed(o, hq).to(dt), "lse": packed(lse, hq).squeeze(-1)}
    if c["train"]:
        do = padded(s["do"], cu, n) * (at < (cu[1:] - cu[:-1])[:, None])[:, None, :, None]
        do = do.reshape(b, hkv, g * n, d)
        dv = torch.matmul(p.transpose(-1, -2), do)
        ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * scale
        out.update(dq=packed(torch.matmul(ds, k), hq).to(dt), dk=packed(torch.matmul(ds.transpose(-1, -2), q), hkv).to(dt),
                   dv=packed(dv, hkv).to(dt))
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits, a sequence and a head at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op == "norm_block":
        h = torch.addcmul(s["x"], s["y"], s["res_scale"].expand_as(s["y"]))
        norm = ((h * h).sum(1) / case["width"] + EPS).sqrt()
        u = h / norm[:, None]
        out = {"h": h, "n": u * s["weight"]}
        if case["train"]:
            a = s["dn"] * s["weight"]
            dot = (a * u).sum(1) / case["width"]
            dx = s["dh"] + (a - dot[:, None] * u) / norm[:, None]
            out.update(dx=dx, dy=dx * s["res_scale"], dweight=(s["dn"] * u).sum(0), dres_scale=(dx * s["y"]).sum(0))
        return out
    if op == "norm_gate":
        norm = ((s["o"] ** 2).sum(2) / case["dim"] + EPS).sqrt()
        u = s["o"] / norm[..., None]
        sig = torch.sigmoid(s["gate"])
        act = s["gate"] * sig
        out = {"y": u * s["weight"] * act}
        if case["train"]:
            a = s["dy"] * act * s["weight"]
            do = (a - u * ((a * u).sum(2) / case["dim"])[..., None]) / norm[..., None]
            dgate = s["dy"] * u * s["weight"] * sig * (1 + s["gate"] * (1 - sig))
            out.update(do=do, dgate=dgate, dweight=(s["dy"] * act * u).flatten(0, 1).sum(0))
        return out
    new, whole = lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["dim"]
    ends = torch.tensor(new).cumsum(0).tolist()
    if op == "append":
        ps, half = case["page"], d // 2
        out = {"q": s["q"].clone(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        for b, (n, w, e) in enumerate(zip(new, whole, ends)):
            turn = torch.complex(s["cos"][w - n:w], s["sin"][w - n:w])[:, None]
            for x in (s["q"], s["k"]):
                part = x[e - n:e]
                z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
                z = torch.cat([z.real, z.imag], -1)
                if x is s["q"]:
                    out["q"][e - n:e] = z
                else:
                    key = z
            pos = torch.arange(w - n, w, device=DEV)
            flat = s["table"][b].long()[pos // ps] * ps + pos % ps
            out["k_cache"].view(-1, hkv, d)[flat] = key
            out["v_cache"].view(-1, hkv, d)[flat] = s["v"][e - n:e]
        return out
    train = case.get("train", False)
    t = sum(new)
    out = {"o": torch.empty(t, hq, d, dtype=torch.float64, device=DEV)}
    if op == "prompt":
        out["lse"] = torch.empty(t, hq, dtype=torch.float64, device=DEV)
        if train:
            for name, h in (("dq", hq), ("dk", hkv), ("dv", hkv)):
                out[name] = torch.zeros(t, h, d, dtype=torch.float64, device=DEV)
    for b, (n, w, e) in enumerate(zip(new, whole, ends)):
        a = e - n
        if op == "paged":
            used = s["table"][b, : -(-w // case["page"])].long()
            keys, values = (s[x][used].reshape(-1, hkv, d)[:w] for x in ("k_cache", "v_cache"))
        else:
            keys, values = s["k"][a:e], s["v"][a:e]
        hide = torch.ones(n, w, dtype=torch.bool, device=DEV).triu(w - n + 1)
        for h in range(hq):
            m = h * hkv // hq
            kk, vv, qq = keys[:, m], values[:, m], s["q"][a:e, h]
            sc = (qq @ kk.T / math.sqrt(d)).masked_fill(hide, -math.inf)
            lse = torch.logsumexp(sc, 1)
            p = torch.exp(sc - lse[:, None])
            o = p @ vv
            out["o"][a:e, h] = o
            if op == "prompt":
                out["lse"][a:e, h] = lse
            if train:
                do = s["do"][a:e, h]
                out["dv"][a:e, m] += p.T @ do
                ds = p * (do @ vv.T - (do * o).sum(1)[:, None]) / math.sqrt(d)
                out["dq"][a:e, h] = ds @ kk
                out["dk"][a:e, m] += ds.T @ qq
    return out
