"""The operators of a state-space layer and the page step (include/gdn.h).

    gdn_conv_forward(x, weight, cu_seqlens, bias=None, state=None)  -> (y, state_out)
    gdn_conv_backward(x, weight, cu_seqlens, dy, bias, state)       -> (dx, dweight, dbias, dstate)
    gdn_conv_step(x, weight, state, bias=None)                      -> y   (state updated in place)
    gdn_ssm_forward(x, dt, A, B, C, cu_seqlens, ...)                -> (y, hT)
    gdn_ssm_backward(x, dt, A, B, C, cu_seqlens, dy, ...)
                                     -> (dx, ddt, dA, dB, dC, dD, ddt_bias, dh0)
    gdn_ssm_step(x, dt, A, B, C, state, ...)                        -> y   (state updated in place)
    gdn_pages_release(done, kv_len, page_table, free_pages, free_count, page_size)
                                                                    -> (kv_len, free_count)
    gdn_pages_take(want, kv_len, page_table, free_pages, free_count, page_size, rows)
                                     -> (kv_len, free_count, cu_seqlens, positions, slots)

Argument marshalling only, as in block.py: every computation runs in the library's
HIP kernels, on the current stream of the tensors' device.  x, y, B, C and the
convolution's states share one dtype, float32 or bfloat16; weights, dt, A, D and the
scan's states are float32, lengths and tables int32.  x, B and C may be slices of a
wider tensor: dense within a token, any token stride.

Outputs are allocated unless passed.  Rows that belong to no sequence (behind
cu_seqlens[-1]) are left as they were in outputs that are passed, and are zeros in
outputs that are allocated here.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import GdnError, lib
from .block import _alike, _dtype, _gpu, _p, _run, _sequences, _take, _too_large

GDN_SSM_FORWARD, GDN_SSM_BACKWARD = 0, 1
_F32, _I32 = torch.float32, torch.int32


class GdnConvShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int), ("W", ctypes.c_int),
                ("dtype", ctypes.c_int), ("silu", ctypes.c_int), ("x_stride", ctypes.c_longlong)]


class GdnSsmShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("G", ctypes.c_int),
                ("N", ctypes.c_int), ("P", ctypes.c_int), ("dtype", ctypes.c_int), ("softplus", ctypes.c_int),
                ("x_stride", ctypes.c_longlong), ("b_stride", ctypes.c_longlong), ("c_stride", ctypes.c_longlong)]


class GdnPagesShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("rows", ctypes.c_int)]


# The shapes of sizes, to be read only: a decoding step's calls are short enough for
# the host to count, and a structure's fields take it longer than to find it.
_conv_sizes = lru_cache(maxsize=256)(GdnConvShape)
_ssm_sizes = lru_cache(maxsize=256)(GdnSsmShape)
_pages_sizes = lru_cache(maxsize=256)(GdnPagesShape)


def declare(L):
    """Argument types of the entry points, for the library handle."""
    vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    cs, ss, ps = (ctypes.POINTER(t) for t in (GdnConvShape, GdnSsmShape, GdnPagesShape))
    for name, args, res in (
            ("gdn_conv_workspace_bytes", [cs], sz), ("gdn_conv_forward", [cs] + [vp] * 8, i),
            ("gdn_conv_backward", [cs] + [vp] * 12 + [sz, vp], i), ("gdn_conv_step", [cs] + [vp] * 6, i),
            ("gdn_ssm_workspace_bytes", [ss, i], sz), ("gdn_ssm_forward", [ss] + [vp] * 12 + [sz, vp], i),
            ("gdn_ssm_backward", [ss] + [vp] * 20 + [sz, vp], i), ("gdn_ssm_step", [ss] + [vp] * 10, i),
            ("gdn_pages_release", [ps] + [vp] * 8, i), ("gdn_pages_take", [ps] + [vp] * 11, i)):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res


def _room(n, ws, device, name):
    """The workspace, allocated unless passed, and its size."""
    if n == 0:
        raise GdnError(2, name)
    if ws is None:
        return torch.empty(n, dtype=torch.uint8, device=device), n
    if ws.get_device() != device.index or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous and on {device}")
    return ws, ws.numel() * ws.element_size()


# ---------------------------------------------------------------------------
# short causal convolution
# ---------------------------------------------------------------------------
def _conv_shape(x, weight, bias, state, B, silu, dev):
    shape, taps, dtype = x.shape, weight.shape, x.dtype
    if len(shape) != 2:
        raise ValueError(f"x must be [T, C], got {tuple(shape)}")
    T, C = shape
    if len(taps) != 2 or taps[0] != C:
        raise ValueError(f"weight must be [{C}, W], got {tuple(taps)}")
    W = taps[1]
    if (B | T | C | W) >> 31:
        raise _too_large(B, T, C, W)
    stride = 0
    if not x.is_contiguous() or x.get_device() != dev.index:
        stride = _take(x.unsqueeze(1), "x", (T, 1, C), dtype, dev, stride=True)
    _alike(dev, taps, _F32, ("weight",), weight)
    if bias is not None:
        _alike(dev, (C,), _F32, ("bias",), bias)
    if state is not None:
        _alike(dev, (B, W - 1, C), dtype, ("state",), state)
    return _conv_sizes(B, T, C, W, _dtype(x, "x"), int(bool(silu)), stride)


def gdn_conv_forward(x, weight, cu_seqlens, bias=None, state=None, *, silu=True, y=None, state_out=None,
                     want_state=True):
    """Causal convolution of packed rows x [T, C] with weight [C, W] (W = 2..4), then
    silu; state [B, W - 1, C] holds each sequence's last rows before these.  Returns
    (y, state_out), state_out None when want_state is False; it may be state."""
    dev = _gpu(x, "x")
    B = _sequences(cu_seqlens, dev)
    sh = _conv_shape(x, weight, bias, state, B, silu, dev)
    if y is None:
        y = torch.zeros(x.shape, dtype=x.dtype, device=dev)
    if state_out is None and want_state:
        state_out = torch.empty((B, sh.W - 1, sh.C), dtype=x.dtype, device=dev)
    _alike(dev, x.shape, x.dtype, ("y",), y)
    _alike(dev, (B, sh.W - 1, sh.C), x.dtype, ("state_out",), state_out)
    _run(lib().gdn_conv_forward, "gdn_conv_forward", dev, ctypes.byref(sh), _p(x), _p(weight), _p(bias), _p(cu_seqlens),
         _p(state), _p(y), _p(state_out))
    return y, state_out


def gdn_conv_backward(x, weight, cu_seqlens, dy, bias=None, state=None, *, silu=True, dstate_out=None, out=None, ws=None):
    """Gradients (dx, dweight, dbias, dstate) of gdn_conv_forward from dy and
    dstate_out (None = zero).  dbias and dstate are None without bias and state; out
    takes them."""
    dev = _gpu(x, "x")
    B = _sequences(cu_seqlens, dev)
    sh = _conv_shape(x, weight, bias, state, B, silu, dev)
    if out is None:
        out = (torch.zeros(x.shape, dtype=x.dtype, device=dev), torch.empty_like(weight),
               None if bias is None else torch.empty_like(bias), None if state is None else torch.empty_like(state))
    dx, dw, db, ds = out
    if dx is None or dw is None:
        raise ValueError("out: dx and dweight are required")
    _alike(dev, x.shape, x.dtype, ("dy", "dx"), dy, dx)
    _alike(dev, weight.shape, _F32, ("dweight",), dw)
    _alike(dev, weight.shape[:1], _F32, ("dbias",), db)
    _alike(dev, (B, sh.W - 1, sh.C), x.dtype, ("dstate_out", "dstate"), dstate_out, ds)
    L = lib()
    ws, n = _room(int(L.gdn_conv_workspace_bytes(ctypes.byref(sh))), ws, dev, "gdn_conv_workspace_bytes")
    _run(L.gdn_conv_backward, "gdn_conv_backward", dev, ctypes.byref(sh), _p(x), _p(weight), _p(bias), _p(cu_seqlens),
         _p(state), _p(dy), _p(dstate_out), _p(dx), _p(dw), _p(db), _p(ds), _p(ws), n)
    return dx, dw, db, ds


def gdn_conv_step(x, weight, state, bias=None, *, silu=True, y=None):
    """One row a sequence, x [B, C]; state [B, W - 1, C] is updated in place.  Returns y."""
    dev = _gpu(x, "x")
    if state is None:
        raise ValueError("state is required")
    sh = _conv_shape(x, weight, bias, state, x.shape[0], silu, dev)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _alike(dev, x.shape, x.dtype, ("y",), y)
    if sh.T == 0:
        return y
    _run(lib().gdn_conv_step, "gdn_conv_step", dev, ctypes.byref(sh), _p(x), _p(weight), _p(bias), _p(state), _p(y))
    return y


# ---------------------------------------------------------------------------
# selective state space scan
# ---------------------------------------------------------------------------
def _ssm_shape(x, dt, A, Bm, Cm, D, dt_bias, B, softplus, dev):
    shape, pairs, dtype = x.shape, Bm.shape, x.dtype
    if len(shape) != 3 or len(pairs) != 3:
        raise ValueError(f"x must be [T, H, P] and B [T, G, N], got {tuple(shape)} and {tuple(pairs)}")
    T, H, P = shape
    _, G, N = pairs
    if (B | T | H | P | G | N) >> 31:
        raise _too_large(B, T, H, P, G, N)
    xs = _take(x, "x", shape, dtype, dev, stride=True)
    bs = _take(Bm, "B", (T, G, N), dtype, dev, stride=True)
    cs = _take(Cm, "C", (T, G, N), dtype, dev, stride=True)
    _alike(dev, (T, H), _F32, ("dt",), dt)
    _alike(dev, (H,), _F32, ("A", "D", "dt_bias"), A, D, dt_bias)
    return _ssm_sizes(B, T, H, G, N, P, _dtype(x, "x"), int(bool(softplus)), xs, bs, cs)


def gdn_ssm_forward(x, dt, A, B, C, cu_seqlens, *, D=None, dt_bias=None, softplus=True, h0=None, y=None, hT=None,
                    want_state=True, ws=None):
    """Scan of packed sequences: x [T, H, P], dt [T, H], A [H], B, C [T, G, N].
    Returns (y, hT), hT [B, H, N, P] None when want_state is False; it may be h0."""
    dev = _gpu(x, "x")
    nb = _sequences(cu_seqlens, dev)
    sh = _ssm_shape(x, dt, A, B, C, D, dt_bias, nb, softplus, dev)
    states = (nb, sh.H, sh.N, sh.P)
    if y is None:
        y = torch.zeros(x.shape, dtype=x.dtype, device=dev)
    if hT is None and want_state:
        hT = torch.empty(states, dtype=_F32, device=dev)
    _alike(dev, x.shape, x.dtype, ("y",), y)
    _alike(dev, states, _F32, ("h0", "hT"), h0, hT)
    L = lib()
    ws, n = _room(int(L.gdn_ssm_workspace_bytes(ctypes.byref(sh), GDN_SSM_FORWARD)), ws, dev, "gdn_ssm_workspace_bytes")
    _run(L.gdn_ssm_forward, "gdn_ssm_forward", dev, ctypes.byref(sh), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias),
         _p(cu_seqlens), _p(h0), _p(y), _p(hT), _p(ws), n)
    return y, hT


def gdn_ssm_backward(x, dt, A, B, C, cu_seqlens, dy, *, D=None, dt_bias=None, softplus=True, h0=None, dhT=None, out=None,
                     ws=None):
    """Gradients (dx, ddt, dA, dB, dC, dD, ddt_bias, dh0) of sum(y dy) + sum(hT dhT).
    dD, ddt_bias and dh0 are None without D, dt_bias and h0 (or where out has None)."""
    dev = _gpu(x, "x")
    nb = _sequences(cu_seqlens, dev)
    sh = _ssm_shape(x, dt, A, B, C, D, dt_bias, nb, softplus, dev)
    states, dtype = (nb, sh.H, sh.N, sh.P), x.dtype
    if out is None:
        new = lambda t: None if t is None else torch.zeros(t.shape, dtype=t.dtype, device=dev)  # noqa: E731
        out = tuple(new(t) for t in (x, dt, A, B, C, D, dt_bias, h0))
    dx, ddt, dA, dB, dC, dD, db, dh0 = out
    for t, name in ((dx, "dx"), (ddt, "ddt"), (dA, "dA"), (dB, "dB"), (dC, "dC")):
        if t is None:
            raise ValueError(f"out: {name} is required")
    _alike(dev, x.shape, dtype, ("dy", "dx"), dy, dx)
    _alike(dev, dt.shape, _F32, ("ddt",), ddt)
    _alike(dev, A.shape, _F32, ("dA", "dD", "ddt_bias"), dA, dD, db)
    _alike(dev, B.shape, dtype, ("dB", "dC"), dB, dC)
    _alike(dev, states, _F32, ("h0", "dhT", "dh0"), h0, dhT, dh0)
    L = lib()
    ws, n = _room(int(L.gdn_ssm_workspace_bytes(ctypes.byref(sh), GDN_SSM_BACKWARD)), ws, dev, "gdn_ssm_workspace_bytes")
    _run(L.gdn_ssm_backward, "gdn_ssm_backward", dev, ctypes.byref(sh), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias),
         _p(cu_seqlens), _p(h0), _p(dy), _p(dhT), _p(dx), _p(ddt), _p(dA), _p(dB), _p(dC), _p(dD), _p(db), _p(dh0), _p(ws), n)
    return dx, ddt, dA, dB, dC, dD, db, dh0


def gdn_ssm_step(x, dt, A, B, C, state, *, D=None, dt_bias=None, softplus=True, y=None):
    """One token a sequence: x [B, H, P], dt [B, H], B, C [B, G, N]; state [B, H, N, P]
    is updated in place.  Returns y."""
    dev = _gpu(x, "x")
    sh = _ssm_shape(x, dt, A, B, C, D, dt_bias, x.shape[0], softplus, dev)
    if state is None:
        raise ValueError("state is required")
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _alike(dev, x.shape, x.dtype, ("y",), y)
    _alike(dev, (sh.B, sh.H, sh.N, sh.P), _F32, ("state",), state)
    if sh.T == 0:
        return y
    _run(lib().gdn_ssm_step, "gdn_ssm_step", dev, ctypes.byref(sh), _p(x), _p(dt), _p(A), _p(B), _p(C), _p(D), _p(dt_bias),
         _p(state), _p(y))
    return y


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def _pages_shape(flags, kv_len, page_table, free_pages, free_count, page_size, rows, kv_out, count_out, names):
    dev = _gpu(kv_len, "kv_len")
    lens, table, stack = kv_len.shape, page_table.shape, free_pages.shape
    if len(lens) != 1 or len(table) != 2 or table[0] != lens[0]:
        raise ValueError(f"kv_len must be [B] and page_table [B, max_pages], got {tuple(lens)} and {tuple(table)}")
    if len(stack) != 1:
        raise ValueError(f"free_pages must be [num_pages], got {tuple(stack)}")
    (B, width), pool = table, stack[0]
    if (B | width | pool | page_size | rows) >> 31:
        raise _too_large(B, width, pool, page_size, rows)
    # kv_out and count_out are kv_len and free_count where they are updated in place
    _alike(dev, lens, _I32, names, flags, kv_len, None if kv_out is kv_len else kv_out)
    _alike(dev, table, _I32, ("page_table",), page_table)
    _alike(dev, stack, _I32, ("free_pages",), free_pages)
    _alike(dev, (1,), _I32, ("free_count", "count_out"), free_count, None if count_out is free_count else count_out)
    return _pages_sizes(B, pool, page_size, width, rows), dev


def gdn_pages_release(done, kv_len, page_table, free_pages, free_count, page_size, *, kv_out=None, count_out=None):
    """Pages of the sequences with done[b] != 0 back on the stack of free ones.
    Returns (kv_out, count_out): kv_len and free_count, updated in place, unless passed."""
    kv_out = kv_len if kv_out is None else kv_out
    count_out = free_count if count_out is None else count_out
    sh, dev = _pages_shape(done, kv_len, page_table, free_pages, free_count, page_size, 0, kv_out, count_out,
                           ("done", "kv_len", "kv_out"))
    _run(lib().gdn_pages_release, "gdn_pages_release", dev, ctypes.byref(sh), _p(done), _p(kv_len), _p(page_table),
         _p(free_pages), _p(free_count), _p(kv_out), _p(count_out))
    return kv_out, count_out


def gdn_pages_take(want, kv_len, page_table, free_pages, free_count, page_size, rows, *, kv_out=None, count_out=None,
                   cu_seqlens=None, positions=None, slots=None, want_maps=True):
    """Pages for want[b] new tokens of every sequence, in place in page_table, and the
    step's bounds: (kv_out, count_out, cu_seqlens, positions, slots) for at most `rows`
    tokens.  kv_out and count_out are kv_len and free_count, updated in place, unless
    passed; positions and slots are -1 behind the last token where they are allocated
    here, and None when want_maps is False and they are not passed."""
    kv_out = kv_len if kv_out is None else kv_out
    count_out = free_count if count_out is None else count_out
    sh, dev = _pages_shape(want, kv_len, page_table, free_pages, free_count, page_size, rows, kv_out, count_out,
                           ("want", "kv_len", "kv_out"))
    if cu_seqlens is None:
        cu_seqlens = torch.empty(sh.B + 1, dtype=_I32, device=dev)
    if want_maps and positions is None:
        positions = torch.full((rows,), -1, dtype=_I32, device=dev)
    if want_maps and slots is None:
        slots = torch.full((rows,), -1, dtype=torch.int64, device=dev)
    _alike(dev, (sh.B + 1,), _I32, ("cu_seqlens",), cu_seqlens)
    _alike(dev, (rows,), _I32, ("positions",), positions)
    _alike(dev, (rows,), torch.int64, ("slots",), slots)
    _run(lib().gdn_pages_take, "gdn_pages_take", dev, ctypes.byref(sh), _p(want), _p(kv_len), _p(page_table), _p(free_pages),
         _p(free_count), _p(kv_out), _p(count_out), _p(cu_seqlens), _p(positions), _p(slots))
    return kv_out, count_out, cu_seqlens, positions, slots
