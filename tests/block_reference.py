"""Plain 64-bit forms of the operators around the layer, on the CPU (or, for the
long cases, wherever `where` says), a sequence and a head at a time, and how far a result may be from them.

Bounds count roundings.  Storing a value in type t moves it by at most half a
step, HALF[t] = eps(t) / 2 relative; an operand of a matrix product that is
rounded to t first moves every product by the same, so the sum by HALF[t] times
the sum of the products' sizes.  fp32 arithmetic adds 2^-24 for every operation
on the way; `steps32` counts them for a score of d products, its exponential
(whose argument's absolute error is the score's) and a sum of n terms.
"""
import contextlib

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U32 = 2.0 ** -24


_where = "cpu"


@contextlib.contextmanager
def where(device):
    """Compute the plain forms on `device` inside."""
    global _where
    _where = device
    try:
        with torch.device(device):
            yield
    finally:
        _where = "cpu"


def f64(t):
    return t.detach().to(_where).double()


def norm_block(x, weight, y=None, a=None, eps=1e-6):
    h = f64(x)
    if y is not None:
        h = h + (f64(a) * f64(y) if a is not None else f64(y))
    r = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h, h * r[..., None] * f64(weight), r


def norm_block_backward(dn, dh, x, weight, y=None, a=None, eps=1e-6):
    h, _, r = norm_block(x, weight, y, a, eps)
    xh = h * r[..., None]
    g = f64(dn) * f64(weight)
    dx = r[..., None] * (g - xh * (g * xh).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + f64(dh)
    rows = tuple(range(x.dim() - 1))
    dw = (f64(dn) * xh).sum(rows)
    if a is None:
        return dx, dx if y is not None else None, dw, None
    return dx, dx * f64(a), dw, (dx * f64(y)).sum(rows)


def norm_gate(o, z, weight, eps=1e-6):
    o, z = f64(o), f64(z)
    r = 1 / torch.sqrt((o * o).mean(-1) + eps)
    return o * r[..., None] * f64(weight) * z / (1 + torch.exp(-z)), r


def norm_gate_backward(dy, o, z, weight, eps=1e-6):
    _, r = norm_gate(o, z, weight, eps)
    oh, z, dy, w = f64(o) * r[..., None], f64(z), f64(dy), f64(weight)
    s = 1 / (1 + torch.exp(-z))
    g = dy * z * s * w
    do = r[..., None] * (g - oh * (g * oh).mean(-1, keepdim=True))
    dz = dy * oh * w * s * (1 + z * (1 - s))
    return do, dz, (dy * z * s * oh).sum(tuple(range(o.dim() - 1)))


def steps32(d, n, smax):
    """fp32 roundings that a probability-weighted sum can take: d products a score
    (twice: the product and the sum), each worth the score's size in the
    exponent, n terms summed, and a handful for exp2, scale and division."""
    return U32 * ((2 * d + 8) * (1 + smax) + n + 16)


def attention_head(q, k, v, see, scale):
    """One head: q [n, D], k, v [w, D], see [n, w].  Returns o, lse, p and the
    elementwise sizes behind the bounds (P |v|, largest |score| sum)."""
    s = q @ k.T * scale
    s = torch.where(see, s, torch.full_like(s, -np.inf))
    any_ = see.any(1)
    m = torch.where(any_, s.max(1).values if s.shape[1] else torch.zeros(len(q)).double(), torch.zeros(len(q)).double())
    e = torch.where(see, torch.exp(s - m[:, None]), torch.zeros_like(s))
    z = e.sum(1)
    p = torch.where(any_[:, None], e / torch.where(any_, z, torch.ones_like(z))[:, None], torch.zeros_like(e))
    lse = torch.where(any_, m + torch.log(torch.where(any_, z, torch.ones_like(z))), torch.full_like(m, -np.inf))
    v0 = torch.where(see.any(0)[:, None], v, torch.zeros_like(v))  # what nobody sees is not used
    size = float((q.abs() @ torch.where(see.any(0)[:, None], k, torch.zeros_like(k)).abs().T * scale).max()) if see.any() else 0.0
    return p @ v0, lse, p, p @ v0.abs(), size


def attention_head_backward(q, k, v, see, scale, o, lse, do):
    """Gradients from the given o and lse, and the sizes behind their bounds:
    (dq, dk, dv), (|ds| |k| scale, ...), (A |k| scale, ...), P^T |do|."""
    s = q @ k.T * scale
    p = torch.where(see, torch.exp(s - lse[:, None]), torch.zeros_like(s))
    delta = (do * o).sum(1)
    ds = p * (do @ v.T - delta[:, None])
    big = p * (do.abs() @ v.abs().T + (do.abs() * o.abs()).sum(1)[:, None])
    return {
        "dq": (ds @ k * scale, ds.abs() @ k.abs() * scale, big @ k.abs() * scale),
        "dk": (ds.T @ q * scale, ds.abs().T @ q.abs() * scale, big.T @ q.abs() * scale),
        "dv": (p.T @ do, p.T @ do.abs(), p.T @ do.abs()),
    }


def prompt(q, k, v, cu, scale=None):
    """o, lse and the bound of o's error, all [T, ...] (rows of no sequence: NaN)."""
    dt = q.dtype
    q, k, v = f64(q), f64(k), f64(v)
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    o = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    lse, bo, bl = o[..., 0].clone(), o.clone(), o[..., 0].clone()
    for a, e in zip(cu[:-1], cu[1:]):
        see = torch.ones(e - a, e - a, dtype=torch.bool).tril()
        for h in range(Hq):
            x, l, _, pv, size = attention_head(q[a:e, h], k[a:e, h // G], v[a:e, h // G], see, scale)
            u = steps32(D, e - a, size)
            o[a:e, h], lse[a:e, h] = x, l
            bo[a:e, h] = HALF[dt] * x.abs() + (HALF[dt] + u) * pv * (1 + HALF[dt])
            bl[a:e, h] = u * (1 + l.abs())
    return o, lse, bo, bl


def prompt_backward(q, k, v, cu, do, scale=None):
    """{name: (gradient, bound)}: the gradients of the 64-bit forward.

    do . o is taken from the stored o, whose error is at most bo, so it is off by
    at most e_i = |do_i| . bo_i and ds_ij by p_ij e_i; in bf16 that holds for rows
    of more than 512 keys only (the others take it from the row sums of p (do . v),
    in fp32)."""
    dt = q.dtype
    o, lse, bo, _ = prompt(q, k, v, cu, scale)
    q, k, v, do = (f64(t) for t in (q, k, v, do))
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    g = {n: [torch.zeros(T, H, D, dtype=torch.float64) for _ in range(2)] for n, H in (("dq", Hq), ("dk", Hkv), ("dv", Hkv))}
    for a, e in zip(cu[:-1], cu[1:]):
        see = torch.ones(e - a, e - a, dtype=torch.bool).tril()
        for h in range(Hq):
            qq, kk = q[a:e, h], k[a:e, h // G]
            r = attention_head_backward(qq, kk, v[a:e, h // G], see, scale, o[a:e, h], lse[a:e, h], do[a:e, h])
            size = float((qq.abs() @ kk.abs().T * scale).max()) if e > a else 0.0
            u = 2 * steps32(D, (e - a) * G, size)
            off = (do[a:e, h].abs() * bo[a:e, h]).sum(1)
            if dt == torch.bfloat16:
                off = torch.where(torch.arange(e - a) < 512, torch.zeros_like(off), off)
            s = torch.where(see, qq @ kk.T * scale, torch.full(see.shape, -np.inf, dtype=torch.float64))
            pe = torch.exp(s - lse[a:e, h][:, None]) * off[:, None] * scale
            more = {"dq": pe @ kk.abs(), "dk": pe.T @ qq.abs(), "dv": 0.0}
            for n, (x, rounded, big) in r.items():
                hh = h if n == "dq" else h // G
                g[n][0][a:e, hh] += x
                g[n][1][a:e, hh] += HALF[dt] * rounded + u * (1 + HALF[dt]) * big + more[n]
    return {n: (x, b + HALF[dt] * x.abs()) for n, (x, b) in g.items()}


def slots(table, b, n, page, num_pages):
    """Flat slots of positions 0 .. n - 1, -1 where there is no page."""
    out = []
    for p in range(n):
        pg = int(table[b, p // page]) if p // page < table.shape[1] else -1
        out.append(pg * page + p % page if 0 <= pg < num_pages else -1)
    return out


def paged(q, k_cache, v_cache, table, cu, kv_len, scale=None):
    dt = q.dtype
    q, kc, vc, table = f64(q), f64(k_cache), f64(v_cache), table.cpu()
    num, page, Hkv, D = kc.shape
    T, Hq, _ = q.shape
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    kc, vc = kc.view(-1, Hkv, D), vc.view(-1, Hkv, D)
    o = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    bo = o.clone()
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        w = max(0, int(kv_len[b]))
        at = torch.tensor(slots(table, b, w, page, num), dtype=torch.long)
        have = at >= 0
        n = e - a
        pos = int(kv_len[b]) - n + torch.arange(n)
        see = (torch.arange(w)[None, :] <= pos[:, None]) & have[None, :]
        keys = torch.where(have[:, None, None], kc[at.clamp(min=0)], torch.zeros(1, 1, 1).double())
        vals = torch.where(have[:, None, None], vc[at.clamp(min=0)], torch.zeros(1, 1, 1).double())
        for h in range(Hq):
            x, _, _, pv, size = attention_head(q[a:e, h], keys[:, h // G], vals[:, h // G], see, scale)
            u = steps32(D, w + 64, size)
            o[a:e, h] = x
            bo[a:e, h] = HALF[dt] * x.abs() + (HALF[dt] + u) * pv * (1 + HALF[dt])
    return o, bo


def rotate(x, c, s, rot):
    h = rot // 2
    a, b = x[..., :h], x[..., h:rot]
    return torch.cat([a * c - b * s, b * c + a * s, x[..., rot:]], -1)


def append(q, k, v, cos, sin, cu, kv_len, table, k_cache, v_cache, q_out):
    """(k_cache, v_cache, q_out) after the call, from their values before it; rows
    that the call leaves out keep them."""
    kc, vc, qo, table = f64(k_cache).clone(), f64(v_cache).clone(), f64(q_out).clone(), table.cpu()
    num, page, Hkv, D = kc.shape
    rot = 0 if cos is None else 2 * cos.shape[1]
    flat_k, flat_v = kc.view(-1, Hkv, D), vc.view(-1, Hkv, D)
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        for t in range(a, e):
            p = int(kv_len[b]) - (e - a) + t - a
            if p < 0 or p >= table.shape[1] * page or (rot and p >= cos.shape[0]):
                continue
            c, s = (f64(cos[p]), f64(sin[p])) if rot else (torch.zeros(0), torch.zeros(0))
            qo[t] = rotate(f64(q[t]), c, s, rot)
            pg = int(table[b, p // page])
            if 0 <= pg < num:
                flat_k[pg * page + p % page] = rotate(f64(k[t]), c, s, rot)
                flat_v[pg * page + p % page] = f64(v[t])
    return kc, vc, qo


def worst(got, want, bound):
    """Largest error in units of the bound (0 where both agree)."""
    d = (f64(got) - want).abs()
    assert torch.isfinite(f64(got)).all(), "not finite"
    if d.numel() == 0:
        return 0.0
    return float(torch.where(d == 0, torch.zeros_like(d), d / bound.clamp(min=1e-300)).max())
