"""The paged-cache calls on torch tensors: argument checks and marshalling only, as
in ``binding``.

A decoding step makes these calls once per layer and its kernels run for a few
microseconds, so the checks are written as one condition per call; what it was
that failed is worked out only when it does.
"""
from __future__ import annotations

import ctypes

from . import binding as B_

try:
    import torch
except ImportError:  # the library can be built without it
    torch = None

class RopeSpec:
    """How a rotary embedding turns (medusa_rope_plan): built once, passed to
    medusa_rope and medusa_paged_append.  scaling is "none", "linear", "bands" or
    "ramp"; see include/medusa.h for the formulas."""

    SCALINGS = ("none", "linear", "bands", "ramp")

    def __init__(self, rotary_dim: int, interleaved: bool = False, base: float = 10000.0, scaling: str = "none",
                 factor: float = 1.0, low: float = 1.0, high: float = 4.0, original_len: int = 4096,
                 magnitude: float = 1.0):
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling must be one of {self.SCALINGS}")
        self.st = B_.medusa_rope_plan()
        self.ref = ctypes.byref(self.st)
        B_._check("medusa_rope_plan_init", B_.lib().medusa_rope_plan_init(
            rotary_dim, int(interleaved), float(base), self.SCALINGS.index(scaling), float(factor), float(low),
            float(high), original_len, float(magnitude), self.ref))

    rotary_dim = property(lambda self: self.st.rotary_dim)
    interleaved = property(lambda self: bool(self.st.interleaved))


def _refuse(what: str, dev, shapes, dense, strided=()):
    """Raises for the first of `dense` (name, tensor, dtype) or `strided` (name,
    tensor, dtype) that does not fit, else for `shapes`, the call's own rule."""
    for name, t, dt in (*dense, *strided):
        if t is None:
            continue
        if not t.is_cuda or t.device != dev:
            raise ValueError(f"{what}: {name} must be on the GPU of the other tensors ({dev}), not on {t.device}")
        if t.dtype != dt:
            raise ValueError(f"{what}: {name} must be {dt}, not {t.dtype}")
    for name, t, _ in dense:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be dense")
    raise ValueError(f"{what}: {shapes}")


def _token_stride(what: str, name: str, t, nl: int, T: int, H: int, d: int) -> int:
    """Elements from one token to the next of t [nl, T, H, d], whose heads are dense
    and whose layers are T tokens apart."""
    s0, s1, s2, s3 = t.stride()
    ld = s1 if T > 1 else (s0 if nl > 1 else H * d)
    if t.shape != (nl, T, H, d):
        raise ValueError(f"{what}: {name} must be [{nl}, {T}, {H}, {d}], not {list(t.shape)}")
    if s3 != 1 or (H > 1 and s2 != d) or (nl > 1 and s0 != T * ld):
        raise ValueError(f"{what}: {name} must have dense heads and evenly spaced tokens (strides {t.stride()})")
    return ld


def _code(what: str, t) -> int:
    if t.dtype is torch.bfloat16:
        return B_.MEDUSA_BF16
    if t.dtype is torch.float32:
        return B_.MEDUSA_F32
    raise TypeError(f"{what}: tensors must be bfloat16 or float32, not {t.dtype}")


def _call(what: str, fn, dev, stream, args):
    """fn(*args, stream) with the tensors' device current."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
    else:
        raw = stream.cuda_stream
    if dev.index == torch.cuda.current_device():
        code = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, raw)
    if code:
        raise B_.MedusaError(what, code)


def _fresh(stream, shape, dtype, dev):
    """A new tensor out of the memory of the stream that the call runs on: what that
    memory held before is done with there, and a workspace dropped on return goes
    to nothing but later work of the same stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _given(what: str, name: str, t, shape, dtype, dev):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be dense {dtype} {list(shape)} on {dev}")
    return t


def _workspace(what: str, nbytes: int, dev, ws, stream):
    if ws is None:
        return _fresh(stream, nbytes, torch.uint8, dev), nbytes
    have = ws.numel() * ws.element_size()
    if ws.device != dev or not ws.is_contiguous() or have < nbytes:
        raise ValueError(f"{what}: the workspace must be {nbytes} dense bytes on {dev}")
    return ws, have


def medusa_rope(q, k, pos, rope: RopeSpec, q_out=None, k_out=None, inverse: bool = False, stream=None):
    """Rotary embedding of q [nl, T, Hq, d] and k [nl, T, Hkv, d] (or None) at pos
    [T] int32; returns (q_out, k_out), new tensors unless given (q_out may be q,
    k_out may be k).  inverse=True maps gradients of the outputs to those of the
    inputs."""
    what = "medusa_rope"
    nl, T, Hq, d = q.shape
    dt, dev = _code(what, q), q.device
    ldq = _token_stride(what, "q", q, nl, T, Hq, d)
    Hkv = ldk = 0
    if k is not None:
        Hkv = k.shape[2]
        ldk = _token_stride(what, "k", k, nl, T, Hkv, d)
    if not (q.is_cuda and pos.dtype is torch.int32 and pos.device == dev and pos.is_contiguous() and pos.numel() == T
            and (k is None or (k.dtype is q.dtype and k.device == dev)) and (k is not None or k_out is None)):
        _refuse(what, dev, "pos must hold one position per token, and k_out needs k", [("pos", pos, torch.int32)],
                [("q", q, q.dtype), ("k", k, q.dtype)])
    q_out = _fresh(stream, (nl, T, Hq, d), q.dtype, dev) if q_out is None else _given(what, "q_out", q_out, q.shape, q.dtype, dev)
    if k is not None:
        k_out = _fresh(stream, (nl, T, Hkv, d), q.dtype, dev) if k_out is None else _given(what, "k_out", k_out, k.shape, q.dtype, dev)
    _call(what, B_.lib().medusa_rope, dev, stream, (
        q.data_ptr(), ldq, None if k is None else k.data_ptr(), ldk, pos.data_ptr(), rope.ref, 1 if inverse else 0, nl, T,
        Hq, Hkv, d, dt, q_out.data_ptr(), None if k is None else k_out.data_ptr()))
    return q_out, k_out


def medusa_paged_append(k, v, k_pages, v_pages, page_table, q_start, prefix_len, q=None, pos=None,
                        rope: RopeSpec | None = None, q_out=None, d_status=None, stream=None):
    """Enters the chunk's k, v [nl, T, Hkv, d] (k rotated by `rope`, at pos [T] or at
    the row numbers) into the pages behind prefix_len [B] rows; returns q
    [nl, T, Hq, d] rotated into q_out (new unless given), or None without q.
    q, k and v may be slices of one projection's output."""
    what = "medusa_paged_append"
    nl, n_pages, ps, Hkv, d = k_pages.shape
    B, max_pages = page_table.shape
    dt, dev, ty, i32 = _code(what, k), k_pages.device, k.dtype, torch.int32
    T = k.shape[1]
    ldk, ldv = _token_stride(what, "k", k, nl, T, Hkv, d), _token_stride(what, "v", v, nl, T, Hkv, d)
    if not (k_pages.is_cuda and k_pages.dtype is ty and v_pages.dtype is ty and v_pages.device == dev and k.device == dev
            and v.device == dev and v.dtype is ty and v_pages.shape == k_pages.shape and k_pages.is_contiguous()
            and v_pages.is_contiguous() and page_table.dtype is i32 and page_table.device == dev
            and page_table.is_contiguous() and q_start.dtype is i32 and q_start.device == dev and q_start.is_contiguous()
            and q_start.numel() == B + 1 and prefix_len.dtype is i32 and prefix_len.device == dev
            and prefix_len.is_contiguous() and prefix_len.numel() == B
            and (pos is None or (pos.dtype is i32 and pos.device == dev and pos.is_contiguous() and pos.numel() == T))
            and (d_status is None or (d_status.dtype is i32 and d_status.device == dev))
            and (q is not None or q_out is None)):
        _refuse(what, dev, "v_pages must be like k_pages, q_start [B + 1], prefix_len [B] and pos [T], and q_out needs q",
                [("k_pages", k_pages, ty), ("v_pages", v_pages, ty), ("page_table", page_table, i32), ("q_start", q_start, i32),
                 ("prefix_len", prefix_len, i32), ("pos", pos, i32), ("d_status", d_status, i32)], [("k", k, ty), ("v", v, ty)])
    Hq = ldq = 0
    if q is not None:
        Hq = q.shape[2]
        ldq = _token_stride(what, "q", q, nl, T, Hq, d)
        if q.dtype is not ty or q.device != dev:
            raise ValueError(f"{what}: q must have the cache's dtype and device")
        q_out = _fresh(stream, (nl, T, Hq, d), ty, dev) if q_out is None else _given(what, "q_out", q_out, q.shape, ty, dev)
    _call(what, B_.lib().medusa_paged_append, dev, stream, (
        None if q is None else q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
        None if pos is None else pos.data_ptr(), None if rope is None else rope.ref, page_table.data_ptr(),
        q_start.data_ptr(), prefix_len.data_ptr(), nl, T, B, Hq, Hkv, d, n_pages, ps, max_pages, dt,
        None if q is None else q_out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        None if d_status is None else d_status.data_ptr()))
    return q_out


def medusa_paged_attention(q, k_pages, v_pages, page_table, q_start, prefix_len, scale: float | None = None, out=None,
                           lse=None, want_lse: bool = False, ws=None, d_status=None, stream=None):
    """Causal attention of the chunk q [nl, T, Hq, d] over the paged cache, which
    already holds the chunk's rows; returns (out like q, lse fp32 [nl, T, Hq] or
    None).  q may be a slice of a projection's output."""
    what = "medusa_paged_attention"
    nl, n_pages, ps, Hkv, d = k_pages.shape
    B, max_pages = page_table.shape
    _, T, Hq, _ = q.shape
    dt, dev, ty, i32 = _code(what, q), k_pages.device, q.dtype, torch.int32
    ldq = _token_stride(what, "q", q, nl, T, Hq, d)
    if not (k_pages.is_cuda and k_pages.dtype is ty and v_pages.dtype is ty and v_pages.device == dev and q.device == dev
            and v_pages.shape == k_pages.shape and k_pages.is_contiguous() and v_pages.is_contiguous()
            and page_table.dtype is i32 and page_table.device == dev and page_table.is_contiguous()
            and q_start.dtype is i32 and q_start.device == dev and q_start.is_contiguous() and q_start.numel() == B + 1
            and prefix_len.dtype is i32 and prefix_len.device == dev and prefix_len.is_contiguous()
            and prefix_len.numel() == B and (d_status is None or (d_status.dtype is i32 and d_status.device == dev))):
        _refuse(what, dev, "v_pages must be like k_pages, q_start [B + 1] and prefix_len [B]",
                [("k_pages", k_pages, ty), ("v_pages", v_pages, ty), ("page_table", page_table, i32), ("q_start", q_start, i32),
                 ("prefix_len", prefix_len, i32), ("d_status", d_status, i32)], [("q", q, ty)])
    shape = (nl, T, Hq, d)
    out = _fresh(stream, shape, ty, dev) if out is None else _given(what, "out", out, shape, ty, dev)
    if lse is not None:
        _given(what, "lse", lse, shape[:3], torch.float32, dev)
    elif want_lse:
        lse = _fresh(stream, shape[:3], torch.float32, dev)
    L = B_.lib()
    ws, nbytes = _workspace(what, L.medusa_paged_attention_workspace_size(nl, T, B, Hq, Hkv, d, ps, dt), dev, ws, stream)
    _call(what, L.medusa_paged_attention, dev, stream, (
        q.data_ptr(), ldq, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), q_start.data_ptr(),
        prefix_len.data_ptr(), nl, T, B, Hq, Hkv, d, n_pages, ps, max_pages, d ** -0.5 if scale is None else scale, dt,
        out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(), nbytes,
        None if d_status is None else d_status.data_ptr()))
    return out, lse


def medusa_paged_tree_attention(q, k_pages, v_pages, page_table, kt, vt, mask, prefix_len, scale: float | None = None,
                                out=None, lse=None, want_lse: bool = False, ws=None, d_status=None, stream=None):
    """Tree attention of q [nl, B, N, Hq, d] over a paged prefix and the tree rows
    kt, vt [nl, B, N, Hkv, d]; returns (out like q, lse fp32 [nl, B, N, Hq] or None)."""
    what = "medusa_paged_tree_attention"
    nl, n_pages, ps, Hkv, d = k_pages.shape
    B, max_pages = page_table.shape
    N, Hq = q.shape[2], q.shape[3]
    dt, dev, ty, i32 = _code(what, q), k_pages.device, q.dtype, torch.int32
    shape, rows = (nl, B, N, Hq, d), (nl, B, N, Hkv, d)
    if not (k_pages.is_cuda and k_pages.dtype is ty and v_pages.dtype is ty and v_pages.device == dev and q.device == dev
            and kt.dtype is ty and kt.device == dev and vt.dtype is ty and vt.device == dev
            and v_pages.shape == k_pages.shape and q.shape == shape and kt.shape == rows and vt.shape == rows
            and k_pages.is_contiguous() and v_pages.is_contiguous() and q.is_contiguous() and kt.is_contiguous()
            and vt.is_contiguous() and page_table.dtype is i32 and page_table.device == dev and page_table.is_contiguous()
            and mask.dtype is i32 and mask.device == dev and mask.is_contiguous() and mask.shape == (N, (N + 31) // 32)
            and prefix_len.dtype is i32 and prefix_len.device == dev and prefix_len.is_contiguous()
            and prefix_len.numel() == B and (d_status is None or (d_status.dtype is i32 and d_status.device == dev))):
        _refuse(what, dev, "q must be [nl, B, N, Hq, d], kt and vt [nl, B, N, Hkv, d], mask [N, ceil(N / 32)], prefix_len [B]",
                [("q", q, ty), ("k_pages", k_pages, ty), ("v_pages", v_pages, ty), ("kt", kt, ty), ("vt", vt, ty),
                 ("page_table", page_table, i32), ("mask", mask, i32), ("prefix_len", prefix_len, i32), ("d_status", d_status, i32)])
    out = _fresh(stream, shape, ty, dev) if out is None else _given(what, "out", out, shape, ty, dev)
    if lse is not None:
        _given(what, "lse", lse, shape[:4], torch.float32, dev)
    elif want_lse:
        lse = _fresh(stream, shape[:4], torch.float32, dev)
    L = B_.lib()
    ws, nbytes = _workspace(what, L.medusa_paged_attention_workspace_size(nl, B * N, B, Hq, Hkv, d, ps, dt), dev, ws, stream)
    _call(what, L.medusa_paged_tree_attention, dev, stream, (
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kt.data_ptr(), vt.data_ptr(),
        mask.data_ptr(), prefix_len.data_ptr(), nl, B, N, Hq, Hkv, d, n_pages, ps, max_pages,
        d ** -0.5 if scale is None else scale, dt, out.data_ptr(), None if lse is None else lse.data_ptr(),
        ws.data_ptr(), nbytes, None if d_status is None else d_status.data_ptr()))
    return out, lse


def medusa_paged_compact(k_pages, v_pages, page_table, kt, vt, path_nodes, accept_len, prefix_len, new_len=None,
                         d_status=None, stream=None):
    """Appends the accepted paths path_nodes [B, Dmax + 1], accept_len [B] of the tree
    rows kt, vt [nl, B, N, Hkv, d] to the pages; returns new_len [B] (new unless
    given; may be prefix_len)."""
    what = "medusa_paged_compact"
    nl, n_pages, ps, Hkv, d = k_pages.shape
    B, max_pages = page_table.shape
    N = kt.shape[2]
    dt, dev, ty, i32 = _code(what, kt), k_pages.device, kt.dtype, torch.int32
    rows = (nl, B, N, Hkv, d)
    if not (k_pages.is_cuda and k_pages.dtype is ty and v_pages.dtype is ty and v_pages.device == dev and kt.device == dev
            and vt.dtype is ty and vt.device == dev and v_pages.shape == k_pages.shape and kt.shape == rows
            and vt.shape == rows and k_pages.is_contiguous() and v_pages.is_contiguous() and kt.is_contiguous()
            and vt.is_contiguous() and page_table.dtype is i32 and page_table.device == dev and page_table.is_contiguous()
            and path_nodes.dtype is i32 and path_nodes.device == dev and path_nodes.is_contiguous() and path_nodes.dim() == 2
            and path_nodes.shape[0] == B and accept_len.dtype is i32 and accept_len.device == dev
            and accept_len.is_contiguous() and accept_len.numel() == B and prefix_len.dtype is i32
            and prefix_len.device == dev and prefix_len.is_contiguous() and prefix_len.numel() == B
            and (d_status is None or (d_status.dtype is i32 and d_status.device == dev))):
        _refuse(what, dev, "kt and vt must be [nl, B, N, Hkv, d], path_nodes [B, Dmax + 1], accept_len and prefix_len [B]",
                [("k_pages", k_pages, ty), ("v_pages", v_pages, ty), ("kt", kt, ty), ("vt", vt, ty),
                 ("page_table", page_table, i32), ("path_nodes", path_nodes, i32), ("accept_len", accept_len, i32),
                 ("prefix_len", prefix_len, i32), ("d_status", d_status, i32)])
    new_len = _fresh(stream, (B,), i32, dev) if new_len is None else _given(what, "new_len", new_len, (B,), i32, dev)
    _call(what, B_.lib().medusa_paged_compact, dev, stream, (
        k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kt.data_ptr(), vt.data_ptr(), path_nodes.data_ptr(),
        accept_len.data_ptr(), prefix_len.data_ptr(), new_len.data_ptr(), nl, B, N, Hkv, d, n_pages, ps, max_pages,
        path_nodes.shape[1] - 1, dt, None if d_status is None else d_status.data_ptr()))
    return new_len
