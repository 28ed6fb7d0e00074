"""The operators around the layer (include/gdn.h): norms before and after a
block, causal softmax attention over packed sequences, and a paged cache.

    gdn_norm_block(x, weight, y=None, res_scale=None)          -> (h, n, rstd)
    gdn_norm_block_backward(dn, x, weight, rstd, y, res_scale) -> (dx, dy, dweight, dres_scale)
    gdn_norm_gate(o, gate, weight)                             -> (y, rstd)
    gdn_norm_gate_backward(dy, o, gate, weight, rstd)          -> (do, dgate, dweight)
    gdn_attn_forward(q, k, v, cu_seqlens)                      -> (o, lse)
    gdn_attn_backward(q, k, v, cu_seqlens, o, lse, dO)         -> (dq, dk, dv)
    gdn_attn_append(q, k, v, cos, sin, cu_seqlens, kv_len, page_table, k_cache, v_cache) -> q_out
    gdn_attn_paged(q, k_cache, v_cache, page_table, cu_seqlens, kv_len) -> o

Argument marshalling only, as in the package's other calls: every computation
runs in the library's HIP kernels, on the current stream of the tensors' device
(which need not be the current device).  x, y, q, k, v and the caches share one
dtype, float32 or bfloat16; weights, cos, sin, rstd and lse are float32,
cu_seqlens, kv_len and page_table int32.  q, k, v and gate may be slices of a
wider projection's output: dense within a token, any token stride.

Outputs are allocated unless passed.  Rows of q, k, v that belong to no sequence
(behind cu_seqlens[-1]) are left as they were in outputs that are passed, and
are zeros in outputs that are allocated here.
"""
from __future__ import annotations

import ctypes

import torch

from . import GDN_BF16, GDN_F32, GdnError, lib

GDN_ATTN_PAGED, GDN_ATTN_BACKWARD = 0, 1


class GdnNormShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int), ("heads", ctypes.c_int), ("width", ctypes.c_int),
                ("dtype", ctypes.c_int), ("eps", ctypes.c_float), ("gate_stride", ctypes.c_longlong)]


class GdnAttnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong),
                ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("max_pos", ctypes.c_int)]


def declare(L):
    """Argument types of the entry points, for the library handle."""
    vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    ns, at = ctypes.POINTER(GdnNormShape), ctypes.POINTER(GdnAttnShape)
    for name, args, res in (
            ("gdn_norm_workspace_bytes", [ns, i], sz), ("gdn_norm_block", [ns] + [vp] * 8, i),
            ("gdn_norm_block_backward", [ns] + [vp] * 12 + [sz, vp], i), ("gdn_norm_gate", [ns] + [vp] * 6, i),
            ("gdn_norm_gate_backward", [ns] + [vp] * 9 + [sz, vp], i), ("gdn_attn_workspace_bytes", [at, i], sz),
            ("gdn_attn_forward", [at] + [vp] * 7, i), ("gdn_attn_backward", [at] + [vp] * 11 + [sz, vp], i),
            ("gdn_attn_append", [at] + [vp] * 12, i), ("gdn_attn_paged", [at] + [vp] * 8 + [sz, vp], i)):
        fn = getattr(L, name)
        fn.argtypes, fn.restype = args, res


def _too_large(*counts):
    """The C shapes hold 32-bit counts, and ctypes drops higher bits silently: every
    call refuses a size with any of them first, (a | b | ...) >> 31."""
    return ValueError(f"sizes must be at most 2147483647, got {counts}")


_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _p(t):
    return None if t is None else t.data_ptr()


# the current stream's handle by device index; the public call makes a Stream object for it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _take(t, name, shape, dtype, device, *, stride=False):
    """Check a tensor: its shape, type and device, dense (or, with stride, a
    [T, H, D] that is dense within its tokens).  Returns the elements between
    tokens, 0 for dense."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device.index:
        raise ValueError(f"{name} must be on {device}, a GPU, and is on {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    if not stride:
        raise ValueError(f"{name} must be contiguous")
    step, row, one = t.stride()  # [T, H, D]
    if (one != 1 and shape[2] > 1) or (row != shape[2] and shape[1] > 1):
        raise ValueError(f"{name} must be contiguous within a token")
    if shape[0] < 2:
        return 0  # one token has no stride of its own
    if step < shape[1] * shape[2]:  # an expanded tensor: its tokens are one, and 0 would say dense
        raise ValueError(f"{name}: its tokens overlap (stride {step})")
    return step


def _alike(device, shape, dtype, names, *tensors):
    """_take for dense tensors of one shape and type (None ones are left out), in
    one call: a decoding step's calls are short enough for the host to count."""
    index = device.index
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != index or t.shape != shape
                              or not t.is_contiguous()):
            for t, name in zip(tensors, names):
                if t is not None:
                    _take(t, name, shape, dtype, device)


def _run(fn, name, device, *args):
    """Call on the device's current stream, with that device current."""
    index = device.index
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        raise GdnError(rc, name)


def _gpu(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.device


def _workspace(query, shape, arg, ws, device, name):
    n = int(query(ctypes.byref(shape), arg))
    if n == 0:
        raise GdnError(2, name)
    if ws is None:
        return torch.empty(n, dtype=torch.uint8, device=device), n
    if ws.get_device() != device.index or not ws.is_contiguous():
        raise ValueError(f"ws must be contiguous and on {device}")
    return ws, ws.numel() * ws.element_size()


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
def gdn_norm_block(x, weight, y=None, res_scale=None, *, eps=1e-6, out=None):
    """h = x + res_scale * y; n = rmsnorm(h) * weight over the last dimension.
    Returns (h, n, rstd); out = (h, n, rstd) takes them (h, rstd may be None: not
    wanted).  Without y, h is x."""
    dt, dev = _dtype(x, "x"), _gpu(x, "x")
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    lead, channels = shape[:-1], shape[-1:]
    tokens, width = lead.numel(), shape[-1]
    if (tokens | width) >> 31:
        raise _too_large(tokens, width)
    if res_scale is not None and y is None:
        raise ValueError("res_scale scales y: pass y too")
    if out is None:
        h = torch.empty_like(x) if y is not None else None
        n, rstd = torch.empty_like(x), torch.empty(lead, dtype=f32, device=dev)
    else:
        h, n, rstd = out
        if n is None:
            raise ValueError("out: n is required")
    _alike(dev, shape, dtype, ("x", "y", "h", "n"), x, y, h, n)
    _alike(dev, channels, f32, ("weight", "res_scale"), weight, res_scale)
    _alike(dev, lead, f32, ("rstd",), rstd)
    sh = GdnNormShape(tokens, 1, width, dt, eps, 0)
    _run(lib().gdn_norm_block, "gdn_norm_block", dev, ctypes.byref(sh), _p(x), _p(y), _p(res_scale), _p(weight), _p(h),
         _p(n), _p(rstd))
    return (x if h is None and y is None else h), n, rstd


def gdn_norm_block_backward(dn, x, weight, rstd, y=None, res_scale=None, *, dh=None, out=None, ws=None):
    """Gradients of gdn_norm_block: (dx, dy, dweight, dres_scale) from dn and dh
    (None = zero).  dy and dres_scale are None without y and res_scale; with y
    but no res_scale dy is dx.  out = (dx, dy, dweight, dres_scale)."""
    dt, dev = _dtype(x, "x"), _gpu(x, "x")
    shape, dtype, f32 = x.shape, x.dtype, torch.float32
    lead, channels, scaled = shape[:-1], shape[-1:], res_scale is not None
    tokens, width = lead.numel(), shape[-1]
    if (tokens | width) >> 31:
        raise _too_large(tokens, width)
    if scaled and y is None:
        raise ValueError("res_scale scales y: pass y too")
    if out is None:
        out = (torch.empty_like(x), torch.empty_like(x) if scaled else None, torch.empty_like(weight),
               torch.empty_like(weight) if scaled else None)
    dx, dy, dw, da = out
    if not scaled:
        dy = da = None
    if dx is None or dw is None or (scaled and (dy is None or da is None)):
        raise ValueError("out: dx and dweight are required, dy and dres_scale with res_scale")
    _alike(dev, shape, dtype, ("x", "dn", "y", "dh", "dx", "dy"), x, dn, y, dh, dx, dy)
    _alike(dev, channels, f32, ("weight", "res_scale", "dweight", "dres_scale"), weight, res_scale, dw, da)
    _alike(dev, lead, f32, ("rstd",), rstd)
    sh = GdnNormShape(tokens, 1, width, dt, 1e-6, 0)  # the saved rstd holds the forward's eps
    L = lib()
    ws, n = _workspace(L.gdn_norm_workspace_bytes, sh, 0, ws, dev, "gdn_norm_workspace_bytes")
    _run(L.gdn_norm_block_backward, "gdn_norm_block_backward", dev, ctypes.byref(sh), _p(dn), _p(dh), _p(x), _p(y),
         _p(res_scale), _p(weight), _p(rstd), _p(dx), _p(dy), _p(dw), _p(da), _p(ws), n)
    return dx, (dx if dy is None and y is not None else dy), dw, da


def _gate_shape(o, gate, weight, dev, eps):
    shape, dtype = o.shape, o.dtype
    if len(shape) < 3:
        raise ValueError(f"o must be [..., H, D], got {tuple(shape)}")
    tokens, (H, D) = shape[:-2].numel(), shape[-2:]
    if (tokens | H | D) >> 31:
        raise _too_large(tokens, H, D)
    if gate.shape != shape:
        raise ValueError(f"gate must have shape {tuple(shape)}, got {tuple(gate.shape)}")
    if not gate.is_contiguous() and len(shape) > 3:
        try:
            gate = gate.view(tokens, H, D)
        except RuntimeError:
            raise ValueError("gate must have one token stride") from None
    stride = _take(gate, "gate", gate.shape, dtype, dev, stride=True)
    _alike(dev, shape[-1:], torch.float32, ("weight",), weight)
    return GdnNormShape(tokens, H, D, _dtype(o, "o"), eps, stride)


def gdn_norm_gate(o, gate, weight, *, eps=1e-6, out=None):
    """y = rmsnorm(o) * weight * silu(gate) for o, gate [..., H, D], the norm over
    D.  Returns (y, rstd); out = (y, rstd), rstd None: not wanted."""
    dev, shape = _gpu(o, "o"), o.shape
    sh = _gate_shape(o, gate, weight, dev, eps)
    if out is None:
        out = torch.empty_like(o), torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    y, rstd = out
    if y is None:
        raise ValueError("out: y is required")
    _alike(dev, shape, o.dtype, ("o", "y"), o, y)
    _alike(dev, shape[:-1], torch.float32, ("rstd",), rstd)
    _run(lib().gdn_norm_gate, "gdn_norm_gate", dev, ctypes.byref(sh), _p(o), _p(gate), _p(weight), _p(y), _p(rstd))
    return y, rstd


def gdn_norm_gate_backward(dy, o, gate, weight, rstd, *, out=None, ws=None):
    """Gradients of gdn_norm_gate: (do, dgate, dweight); out takes them."""
    dev, shape = _gpu(o, "o"), o.shape
    sh = _gate_shape(o, gate, weight, dev, 1e-6)  # the saved rstd holds the forward's eps
    do, dgate, dw = out if out is not None else (torch.empty_like(o), torch.empty_like(o), torch.empty_like(weight))
    if rstd is None or do is None or dgate is None or dw is None:
        raise ValueError("rstd, and do, dgate and dweight of out, are required")
    _alike(dev, shape, o.dtype, ("dy", "o", "do", "dgate"), dy, o, do, dgate)
    _alike(dev, shape[:-1], torch.float32, ("rstd",), rstd)
    _alike(dev, shape[-1:], torch.float32, ("dweight",), dw)
    L = lib()
    ws, n = _workspace(L.gdn_norm_workspace_bytes, sh, 1, ws, dev, "gdn_norm_workspace_bytes")
    _run(L.gdn_norm_gate_backward, "gdn_norm_gate_backward", dev, ctypes.byref(sh), _p(dy), _p(o), _p(gate), _p(weight),
         _p(rstd), _p(do), _p(dgate), _p(dw), _p(ws), n)
    return do, dgate, dw


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _heads(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, D], got {tuple(t.shape)}")
    return t.shape


def _sequences(cu, dev):
    if cu.dim() != 1 or cu.shape[0] < 2:
        raise ValueError(f"cu_seqlens must be [B + 1] with B >= 1, got {tuple(cu.shape)}")
    _take(cu, "cu_seqlens", cu.shape, torch.int32, dev)
    return cu.shape[0] - 1


def _prompt_shape(q, k, v, cu, scale):
    dt, dev = _dtype(q, "q"), _gpu(q, "q")
    T, Hq, D = _heads(q, "q")
    Hkv = _heads(k, "k")[1]
    qs = _take(q, "q", q.shape, q.dtype, dev, stride=True)
    ks = _take(k, "k", (T, Hkv, D), q.dtype, dev, stride=True)
    vs = _take(v, "v", (T, Hkv, D), q.dtype, dev, stride=True)
    B = _sequences(cu, dev)
    if (B | T | Hq | Hkv | D) >> 31:
        raise _too_large(B, T, Hq, Hkv, D)
    return GdnAttnShape(B, T, Hq, Hkv, D, dt, 0.0 if scale is None else scale, qs, ks, vs), dev


def gdn_attn_forward(q, k, v, cu_seqlens, *, scale=None, o=None, lse=None):
    """Causal attention of packed sequences: q [T, Hq, D], k, v [T, Hkv, D],
    cu_seqlens [B + 1].  Returns (o, lse)."""
    sh, dev = _prompt_shape(q, k, v, cu_seqlens, scale)
    if o is None:
        o = torch.zeros(q.shape, dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.zeros(q.shape[:2], dtype=torch.float32, device=dev)
    _alike(dev, q.shape, q.dtype, ("o",), o)
    _alike(dev, q.shape[:2], torch.float32, ("lse",), lse)
    _run(lib().gdn_attn_forward, "gdn_attn_forward", dev, ctypes.byref(sh), _p(q), _p(k), _p(v), _p(cu_seqlens), _p(o),
         _p(lse))
    return o, lse


def gdn_attn_backward(q, k, v, cu_seqlens, o, lse, dO, *, scale=None, out=None, ws=None):
    """Gradients (dq, dk, dv) of sum(o * dO); o, lse from gdn_attn_forward."""
    sh, dev = _prompt_shape(q, k, v, cu_seqlens, scale)
    _take(o, "o", q.shape, q.dtype, dev)
    _take(dO, "dO", q.shape, q.dtype, dev)
    _take(lse, "lse", q.shape[:2], torch.float32, dev)
    if out is None:
        out = tuple(torch.zeros(t.shape, dtype=q.dtype, device=dev) for t in (q, k, v))
    dq, dk, dv = out
    _take(dq, "dq", q.shape, q.dtype, dev)
    _take(dk, "dk", k.shape, q.dtype, dev)
    _take(dv, "dv", k.shape, q.dtype, dev)
    if sh.T == 0:
        return dq, dk, dv
    L = lib()
    ws, n = _workspace(L.gdn_attn_workspace_bytes, sh, GDN_ATTN_BACKWARD, ws, dev, "gdn_attn_workspace_bytes")
    _run(L.gdn_attn_backward, "gdn_attn_backward", dev, ctypes.byref(sh), _p(q), _p(k), _p(v), _p(cu_seqlens), _p(o),
         _p(lse), _p(dO), _p(dq), _p(dk), _p(dv), _p(ws), n)
    return dq, dk, dv


def _cache(sh, k_cache, v_cache, page_table, kv_len, dtype, dev):
    shape, table = k_cache.shape, page_table.shape
    if len(shape) != 4 or shape[2:] != (sh.Hkv, sh.D):
        raise ValueError(f"k_cache must be [num_pages, page_size, {sh.Hkv}, {sh.D}], got {tuple(shape)}")
    if len(table) != 2 or table[0] != sh.B:
        raise ValueError(f"page_table must be [{sh.B}, max_pages], got {tuple(table)}")
    _alike(dev, shape, dtype, ("k_cache", "v_cache"), k_cache, v_cache)
    _take(page_table, "page_table", table, torch.int32, dev)
    _take(kv_len, "kv_len", (sh.B,), torch.int32, dev)
    if (shape[0] | shape[1] | table[1]) >> 31:
        raise _too_large(shape[0], shape[1], table[1])
    sh.num_pages, sh.page_size, sh.max_pages = shape[0], shape[1], table[1]


def gdn_attn_append(q, k, v, cos, sin, cu_seqlens, kv_len, page_table, k_cache, v_cache, *, q_out=None):
    """New tokens' k (rotated) and v into the cache, in place; returns q rotated
    (q None: only the cache, returns None).  cos, sin [max_pos, rot_dim / 2], or
    both None: no rotation."""
    T, Hkv, D = _heads(k, "k")
    dt, dev = _dtype(k, "k"), _gpu(k, "k")
    ks = _take(k, "k", k.shape, k.dtype, dev, stride=True)
    vs = _take(v, "v", k.shape, k.dtype, dev, stride=True)
    Hq, qs = Hkv, 0
    if q is not None:
        Hq = _heads(q, "q")[1]
        qs = _take(q, "q", (T, Hq, D), k.dtype, dev, stride=True)
        if q_out is None:
            q_out = torch.zeros(q.shape, dtype=q.dtype, device=dev)
        _take(q_out, "q_out", q.shape, k.dtype, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    B = _sequences(cu_seqlens, dev)
    if (B | T | Hq | Hkv | D) >> 31:
        raise _too_large(B, T, Hq, Hkv, D)
    sh = GdnAttnShape(B, T, Hq, Hkv, D, dt, 0.0, qs, ks, vs)
    _cache(sh, k_cache, v_cache, page_table, kv_len, k.dtype, dev)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        angles = cos.shape
        if len(angles) != 2:
            raise ValueError(f"cos must be [max_pos, rot_dim / 2], got {tuple(angles)}")
        _alike(dev, angles, torch.float32, ("cos", "sin"), cos, sin)
        if (angles[0] | 2 * angles[1]) >> 31:
            raise _too_large(*angles)
        sh.max_pos, sh.rot_dim = angles[0], 2 * angles[1]
    _run(lib().gdn_attn_append, "gdn_attn_append", dev, ctypes.byref(sh), _p(q), _p(k), _p(v), _p(cos), _p(sin),
         _p(cu_seqlens), _p(kv_len), _p(page_table), _p(k_cache), _p(v_cache), _p(q_out))
    return q_out


def gdn_attn_paged(q, k_cache, v_cache, page_table, cu_seqlens, kv_len, *, scale=None, o=None, ws=None):
    """Causal attention of every sequence's new tokens (the rows of q [T, Hq, D])
    over its cached positions, the new ones among them.  Returns o."""
    dt, dev = _dtype(q, "q"), _gpu(q, "q")
    T, Hq, D = _heads(q, "q")
    qs = _take(q, "q", q.shape, q.dtype, dev, stride=True)
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache must be [num_pages, page_size, Hkv, D], got {tuple(k_cache.shape)}")
    B, Hkv = _sequences(cu_seqlens, dev), k_cache.shape[2]
    if (B | T | Hq | Hkv | D) >> 31:
        raise _too_large(B, T, Hq, Hkv, D)
    sh = GdnAttnShape(B, T, Hq, Hkv, D, dt, 0.0 if scale is None else scale, qs)
    _cache(sh, k_cache, v_cache, page_table, kv_len, q.dtype, dev)
    if o is None:
        o = torch.zeros(q.shape, dtype=q.dtype, device=dev)
    _take(o, "o", q.shape, q.dtype, dev)
    if T == 0:
        return o
    L = lib()
    ws, n = _workspace(L.gdn_attn_workspace_bytes, sh, GDN_ATTN_PAGED, ws, dev, "gdn_attn_workspace_bytes")
    _run(L.gdn_attn_paged, "gdn_attn_paged", dev, ctypes.byref(sh), _p(q), _p(k_cache), _p(v_cache), _p(page_table),
         _p(cu_seqlens), _p(kv_len), _p(o), _p(ws), n)
    return o
