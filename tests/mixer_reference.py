"""Plain 64-bit forms of the state-space layer's operators and of the page step, on
the CPU, and how far a result may be from them.

Bounds count roundings, as in block_reference.py: HALF[t] relative for a value
stored in type t, and for a product's operand that is rounded to it; U32 for every
fp32 operation on the way, the more of them the longer the sums.  A decay
exp(c_t - c_s) is off by (1 + |c_t - c_s|) roundings of fp32: those of its exponent
and of the exponential; one below 2^-126, the smallest normal number, may be 0, which
is off by less than U32 times FLOOR = 2^-102.  The sizes that these factors multiply are sums of
magnitudes, term by term those of the result.
"""
import torch

from block_reference import HALF, U32, f64, worst  # noqa: F401

FLOOR = 2.0 ** -102


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------
def conv(x, w, cu, bias=None, state=None, silu=True):
    """(y, its bound, the new states); rows of no sequence are NaN."""
    dt = x.dtype
    x, w = f64(x), f64(w)
    T, C = x.shape
    K = w.shape[1] - 1
    B = len(cu) - 1
    y = torch.full((T, C), float("nan"), dtype=torch.float64)
    by, out = y.clone(), torch.zeros(B, K, C, dtype=torch.float64)
    for b in range(B):
        a, e = cu[b], cu[b + 1]
        rows = torch.cat([torch.zeros(K, C).double() if state is None else f64(state[b]), x[a:e]])
        out[b] = rows[e - a:]
        for t in range(e - a):
            z = sum(w[:, j] * rows[t + j] for j in range(K + 1))
            size = sum(w[:, j].abs() * rows[t + j].abs() for j in range(K + 1))
            if bias is not None:
                z, size = z + f64(bias), size + f64(bias).abs()
            off = U32 * (K + 3) * size
            y[a + t] = z * torch.sigmoid(z) if silu else z
            # the slope of z s(z) is below 1.1; s has an exponential of z, a reciprocal and a product
            by[a + t] = HALF[dt] * y[a + t].abs() + 1.1 * off + U32 * (8 + z.abs()) * y[a + t].abs()
    return y, by, out


def conv_backward(x, w, cu, dy, bias=None, state=None, dstate_out=None, silu=True):
    """{name: (gradient, bound)}"""
    dt = x.dtype
    x, w, dy = f64(x), f64(w), f64(dy)
    T, C = x.shape
    K = w.shape[1] - 1
    B = len(cu) - 1
    nan = torch.full((T, C), float("nan"), dtype=torch.float64)
    dx, bx, dw, bw = nan, nan.clone(), torch.zeros_like(w), torch.zeros_like(w)
    db, bb = torch.zeros(C).double(), torch.zeros(C).double()
    ds, bs = torch.zeros(B, K, C).double(), torch.zeros(B, K, C).double()
    for b in range(B):
        a, e = cu[b], cu[b + 1]
        n = e - a
        rows = torch.cat([torch.zeros(K, C).double() if state is None else f64(state[b]), x[a:e]])
        de, be = torch.zeros(n + K, C).double(), torch.zeros(n + K, C).double()
        if dstate_out is not None:
            de[n:] += f64(dstate_out[b])
            be[n:] += U32 * f64(dstate_out[b]).abs()
        for t in range(n):
            z = sum(w[:, j] * rows[t + j] for j in range(K + 1))
            size = sum(w[:, j].abs() * rows[t + j].abs() for j in range(K + 1))
            if bias is not None:
                z, size = z + f64(bias), size + f64(bias).abs()
            dz, off = dy[a + t], torch.zeros(C).double()
            if silu:
                s = torch.sigmoid(z)
                slope = s * (1 + z * (1 - s))
                # its own slope is below 1/2; s (1 + |z| (1 - s)) bounds its terms
                off = dy[a + t].abs() * (0.5 * U32 * (K + 3) * size + U32 * (10 + 2 * z.abs()) * s * (1 + z.abs() * (1 - s)))
                dz = dz * slope
            db += dz
            bb += off + U32 * dz.abs() * (n + 40)
            for j in range(K + 1):
                de[t + j] += w[:, j] * dz
                be[t + j] += w[:, j].abs() * (off + U32 * (K + 4) * dz.abs())
                dw[:, j] += dz * rows[t + j]
                bw[:, j] += rows[t + j].abs() * (off + U32 * (n + 40) * dz.abs())
        be += HALF[dt] * de.abs()
        ds[b], bs[b] = de[:K], be[:K]
        dx[a:e], bx[a:e] = de[K:], be[K:]
    return {"dx": (dx, bx), "dweight": (dw, bw + U32 * dw.abs()), "dbias": (db, bb + U32 * db.abs()), "dstate": (ds, bs)}


# ---------------------------------------------------------------------------
# scan
# ---------------------------------------------------------------------------
def delta(dt, bias, softplus):
    v = f64(dt) if bias is None else f64(dt) + f64(bias)
    return torch.where(v > 30, v, torch.log1p(torch.exp(v.clamp(max=30)))) if softplus else v


def ssm_serial(x, dt, A, Bm, Cm, cu, D=None, bias=None, softplus=True, h0=None):
    """Token by token: (y, hT), for any values that autograd may follow."""
    T, H, P = x.shape
    G, N = Bm.shape[1:]
    v = dt if bias is None else dt + bias
    d = torch.nn.functional.softplus(v, threshold=700.0) if softplus else v
    ys, hs = [torch.zeros(cu[0], H, P, dtype=x.dtype)], []
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        S = torch.zeros(H, N, P, dtype=x.dtype) if h0 is None else h0[b]
        for t in range(a, e):
            BB, CC = (m[t].repeat_interleave(H // G, 0) for m in (Bm, Cm))
            S = torch.exp(d[t] * A)[:, None, None] * S + d[t][:, None, None] * BB[:, :, None] * x[t][:, None, :]
            y = (S * CC[:, :, None]).sum(1)
            ys.append((y if D is None else y + D[:, None] * x[t])[None])
        hs.append(S)
    ys.append(torch.zeros(T - cu[-1], H, P, dtype=x.dtype))
    return torch.cat(ys), torch.stack(hs)


def ssm(x, dt, A, Bm, Cm, cu, D=None, bias=None, softplus=True, h0=None, dy=None, dhT=None, keep=None):
    """{name: (value, bound)}: y and hT, and the gradients where dy is given; a sequence
    and a head at a time, every pair of tokens by itself.  Rows of no sequence: 0.
    keep(b, h, ...) is called with what the steps' gradients are made of."""
    dtype = x.dtype
    half = HALF[dtype] if dtype == torch.bfloat16 else 0.0  # a rounded operand; fp32 has none
    T, H, P = x.shape
    G, N = Bm.shape[1:]
    B = len(cu) - 1
    d_all, raw = delta(dt, bias, softplus), f64(dt) if bias is None else f64(dt) + f64(bias)
    x, A, Bm, Cm = f64(x), f64(A), f64(Bm), f64(Cm)
    z = lambda *s: (torch.zeros(s).double(), torch.zeros(s).double())  # noqa: E731
    out = {"y": z(T, H, P), "hT": z(B, H, N, P)}
    if dy is not None:
        dy = f64(dy)
        out.update(dx=z(T, H, P), ddt=z(T, H), dA=z(H), dB=z(T, G, N), dC=z(T, G, N), dD=z(H), ddt_bias=z(H), dh0=z(B, H, N, P))
    for b in range(B):
        a, e = cu[b], cu[b + 1]
        n = e - a
        # sums of N products (twice), P of them, n tokens; softplus, decay and scale on the way
        u = U32 * (2 * N + P + 2 * n + 80)
        see = torch.ones(n, n, dtype=torch.bool).tril()
        for h in range(H):
            g = h // (H // G)
            S0 = torch.zeros(N, P).double() if h0 is None else f64(h0[b, h])
            if n == 0:
                out["hT"][0][b, h] = S0
                if dy is not None:
                    out["dh0"][0][b, h] = 0 if dhT is None else f64(dhT[b, h])
                continue
            X, Bk, Ck, d = x[a:e, h], Bm[a:e, g], Cm[a:e, g], d_all[a:e, h]
            c = torch.cumsum(d * A[h], 0)
            gap = torch.where(see, c[:, None] - c[None, :], torch.zeros(n, n).double())
            E = torch.where(see, torch.exp(gap), torch.zeros(n, n).double())
            Ea = torch.where(see, E * (1 + gap.abs()) + FLOOR, E)  # with the roundings of the exponent
            ec, et = torch.exp(c), torch.exp(c[-1] - c)
            eca, eta = ec * (1 + c.abs()) + FLOOR, et * (1 + (c[-1] - c).abs()) + FLOOR
            eL, eLa = ec[-1], eca[-1]
            U = d[:, None] * X
            W, Wa = E * (Ck @ Bk.T), Ea * (Ck.abs() @ Bk.abs().T)
            y = W @ U + ec[:, None] * (Ck @ S0)
            ya = Wa @ U.abs() + eca[:, None] * (Ck.abs() @ S0.abs())
            if D is not None:
                y, ya = y + f64(D)[h] * X, ya + (f64(D)[h] * X).abs()
            out["y"][0][a:e, h] = y
            out["y"][1][a:e, h] = HALF[dtype] * y.abs() + (half + u) * (1 + half) * ya
            S = eL * S0 + (et[:, None] * Bk).T @ U
            Sa = eLa * S0.abs() + (eta[:, None] * Bk.abs()).T @ U.abs()
            out["hT"][0][b, h], out["hT"][1][b, h] = S, u * Sa
            if dy is None:
                continue
            Y = dy[a:e, h]
            dS = torch.zeros(N, P).double() if dhT is None else f64(dhT[b, h])
            Z, Za = Y @ X.T, Y.abs() @ X.abs().T
            far, fara = et[:, None] * (Bk @ dS), eta[:, None] * (Bk.abs() @ dS.abs())
            du, dua = W.T @ Y + far, Wa.T @ Y.abs() + fara
            dx, dxa = d[:, None] * du, d[:, None].abs() * dua
            if D is not None:
                dx, dxa = dx + f64(D)[h] * Y, dxa + (f64(D)[h] * Y).abs()
            out["dx"][0][a:e, h] = dx
            out["dx"][1][a:e, h] = HALF[dtype] * dx.abs() + (half + u) * (1 + half) * dxa
            r0, r0a = ec[:, None] * (Y @ S0.T), eca[:, None] * (Y.abs() @ S0.abs().T)
            out["dC"][0][a:e, g] += (E * Z * d) @ Bk + r0
            out["dC"][1][a:e, g] += (half + u) * (1 + half) * ((Ea * Za * d.abs()) @ Bk.abs() + r0a)
            out["dB"][0][a:e, g] += d[:, None] * ((E * Z).T @ Ck + et[:, None] * (X @ dS.T))
            out["dB"][1][a:e, g] += (half + u) * (1 + half) * d[:, None].abs() * (
                (Ea * Za).T @ Ck.abs() + eta[:, None] * (X.abs() @ dS.abs().T))
            M, Ma = W * Z * d, Wa * Za * d.abs()
            r, ra = (Ck * r0).sum(1), (Ck.abs() * r0a).sum(1)
            q, qa = d * (X * far).sum(1), d.abs() * (X.abs() * fara).sum(1)
            thr, thra = eL * (S0 * dS).sum(), eLa * (S0.abs() * dS.abs()).sum()
            back = lambda v: v.flip(0).cumsum(0).flip(0)  # noqa: E731
            dg = back(M.sum(1) - M.sum(0) + r) + torch.cumsum(q, 0) - q + thr
            dga = back(Ma.sum(1) + Ma.sum(0) + ra) + torch.cumsum(qa, 0) + thra
            s = torch.sigmoid(raw[a:e, h]) if softplus else torch.ones(n).double()
            dd = (A[h] * dg + (X * du).sum(1)) * s
            bd = (u * (A[h].abs() * dga + (X.abs() * dua).sum(1)) + U32 * 8 * dd.abs()) * s + U32 * 4 * dd.abs()
            out["ddt"][0][a:e, h], out["ddt"][1][a:e, h] = dd, bd
            if keep is not None:
                keep(b, h, d=d, A=A[h], slope=s, dg=dg, dd=dd, M=M, yx=Z.diagonal(), through=thr)
            out["dA"][0][h] += (d * dg).sum()
            out["dA"][1][h] += u * (d.abs() * dga).sum() * 2
            out["dD"][0][h] += Z.diagonal().sum()
            out["dD"][1][h] += u * Za.diagonal().sum()
            out["ddt_bias"][0][h] += dd.sum()
            out["ddt_bias"][1][h] += bd.sum() + u * dd.abs().sum()
            out["dh0"][0][b, h] = eL * dS + (ec[:, None] * Ck).T @ Y
            out["dh0"][1][b, h] = u * (eLa * dS.abs() + (eca[:, None] * Ck.abs()).T @ Y.abs())
    if dy is not None:
        for k in ("dB", "dC"):  # stored once, behind the sum over the heads
            out[k][1].add_(HALF[dtype] * out[k][0].abs())
    return out


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def pages_release(done, kv_len, table, free, count, ps):
    """Lists in, lists out: (kv_out, count_out, free), one page at a time."""
    free, kv, width, pool = list(free), list(kv_len), len(table[0]), len(free)
    count = min(max(count, 0), pool)
    for b in range(len(kv)):
        if done[b]:
            for k in range(min(-(-max(kv[b], 0) // ps), width)):
                if count < pool:
                    free[count] = table[b][k]
                    count += 1
            kv[b] = 0
    return kv, count, free


def pages_take(want, kv_len, table, free, count, ps, rows):
    """(kv_out, count_out, table, cu, positions, slots)"""
    table, pool = [list(r) for r in table], len(free)
    count = min(max(count, 0), pool)
    kv, cu, positions, slots = [], [0], [], []
    asked = wanted = used = 0
    for b in range(len(kv_len)):
        n, w = max(kv_len[b], 0), max(want[b], 0)
        have, need = -(-n // ps), -(-(n + w) // ps)
        ok = need <= len(table[b])
        if ok:
            asked += need - have
            ok = need == have or asked <= count
        if ok:
            wanted += w
            ok = wanted <= rows
        if ok:
            for k in range(have, need):
                table[b][k] = free[count - 1 - used]
                used += 1
            for p in range(n, n + w):
                page = table[b][p // ps]
                positions.append(p)
                slots.append(-1 if page < 0 else page * ps + p % ps)
        kv.append(n + (w if ok else 0))
        cu.append(cu[-1] + (w if ok else 0))
    return kv, count - used, table, cu, positions, slots
