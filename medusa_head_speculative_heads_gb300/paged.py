"""The paged-cache calls on torch tensors.  csrc/python/paged_binding.cpp checks and
marshals their arguments: a decoding step makes these calls once per layer and
their kernels run for a few microseconds.

Everywhere: what is not given (outputs, workspace) is allocated, on the stream that
the call runs on: the current one of the tensors' device, or `stream`.  Gradients are
recorded by medusa_rope where it makes its outputs, and by no other call.
"""
from __future__ import annotations

import ctypes

from . import binding as B_
from .build import load_binding

try:
    import torch
except ImportError:  # the library can be built without it
    torch = None

_native = None


def _load():
    """The compiled binding (raises if it has not been built)."""
    global _native
    _native = load_binding("paged_binding")
    return _native


def _on(stream, t, call, *args):
    """call(*args) with `stream` current, which must be of t's device."""
    if stream.device != t.device:
        raise ValueError(f"{call.__name__}: the stream is of {stream.device}, the tensors are on {t.device}")
    with torch.cuda.stream(stream):
        return call(*args)


def _token_stride(what: str, name: str, t, nl: int, T: int, H: int, d: int) -> int:
    """Elements from one token to the next of t [nl, T, H, d], as the calls see it."""
    return (_native or _load()).token_stride(what, name, t, nl, T, H, d)


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
        self.ref, self.addr = ctypes.byref(self.st), ctypes.addressof(self.st)
        B_._check("medusa_rope_plan_init", B_.lib().medusa_rope_plan_init(
            rotary_dim, int(interleaved), float(base), self.SCALINGS.index(scaling), float(factor), float(low),
            float(high), original_len, float(magnitude), self.ref))

    rotary_dim = property(lambda self: self.st.rotary_dim)
    interleaved = property(lambda self: bool(self.st.interleaved))


class _Rope(torch.autograd.Function if torch is not None else object):
    """medusa_rope of tensors that require grad: its gradient is the turn by the opposite angle."""

    @staticmethod
    def forward(ctx, q, k, pos, rope, inverse):
        outs = medusa_rope(q, k, pos, rope, inverse=inverse)
        ctx.save_for_backward(pos)
        ctx.rope, ctx.inverse = rope, inverse
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(*(o for o, need in zip(outs, ctx.needs_input_grad) if o is not None and not need))
        return outs

    @staticmethod
    def backward(ctx, *grads):
        pos, = ctx.saved_tensors
        back = [g.contiguous() for g, need in zip(grads, ctx.needs_input_grad) if g is not None and need]
        back = iter(medusa_rope(back[0], back[1] if len(back) > 1 else None, pos, ctx.rope, inverse=not ctx.inverse) if back else ())
        return *(next(back) if g is not None and need else None for g, need in zip(grads, ctx.needs_input_grad)), None, None, None


def medusa_rope(q, k, pos, rope: RopeSpec, q_out=None, k_out=None, inverse: bool = False, stream=None):
    """Rotary embedding of q [nl, T, Hq, d] and k [nl, T, Hkv, d] (or None) at pos
    [T] int32; returns (q_out, k_out), new tensors unless given (q_out may be q,
    k_out may be k).  inverse=True maps gradients of the outputs to those of the
    inputs; outputs of inputs that require grad do so by themselves, unless q_out or
    k_out is given (nothing is recorded then)."""
    if stream is not None:
        return _on(stream, q, medusa_rope, q, k, pos, rope, q_out, k_out, inverse)
    if q_out is None and k_out is None and torch.is_grad_enabled() and (
            getattr(q, "requires_grad", False) or getattr(k, "requires_grad", False)):
        return _Rope.apply(q, k, pos, rope, inverse)
    r = (_native or _load()).rope(q, k, pos, rope.addr, q_out, k_out, inverse)
    if type(r) is int:
        raise B_.MedusaError("medusa_rope", r)
    return r


def medusa_paged_append(k, v, k_pages, v_pages, page_table, q_start, prefix_len, q=None, pos=None,
                        rope: RopeSpec | None = None, q_out=None, d_status=None, stream=None):
    """Enters the chunk's k, v [nl, T, Hkv, d] (k rotated by `rope`, at pos [T] or at
    the row numbers) into the pages behind prefix_len [B] rows; returns q
    [nl, T, Hq, d] rotated into q_out (new unless given), or None without q.
    q, k and v may be slices of one projection's output."""
    if stream is not None:
        return _on(stream, k, medusa_paged_append, k, v, k_pages, v_pages, page_table, q_start, prefix_len, q, pos, rope,
                   q_out, d_status)
    r = (_native or _load()).append(k, v, k_pages, v_pages, page_table, q_start, prefix_len, q, pos,
                                    None if rope is None else rope.addr, q_out, d_status)
    if type(r) is int:
        raise B_.MedusaError("medusa_paged_append", r)
    return r[0]


def medusa_paged_attention(q, k_pages, v_pages, page_table, q_start, prefix_len, scale: float | None = None, out=None,
                           lse=None, want_lse: bool = False, ws=None, d_status=None, stream=None):
    """Causal attention of the chunk q [nl, T, Hq, d] over the paged cache, which
    already holds the chunk's rows; returns (out like q, lse fp32 [nl, T, Hq] or
    None).  q may be a slice of a projection's output.  ws:
    medusa_paged_attention_workspace_size() bytes."""
    if stream is not None:
        return _on(stream, q, medusa_paged_attention, q, k_pages, v_pages, page_table, q_start, prefix_len, scale, out, lse,
                   want_lse, ws, d_status)
    r = (_native or _load()).attention(q, k_pages, v_pages, page_table, q_start, prefix_len, scale, out, lse, want_lse, ws,
                                       d_status)
    if type(r) is int:
        raise B_.MedusaError("medusa_paged_attention", r)
    return r


def medusa_paged_tree_attention(q, k_pages, v_pages, page_table, kt, vt, mask, prefix_len, scale: float | None = None,
                                out=None, lse=None, want_lse: bool = False, ws=None, d_status=None, stream=None):
    """Tree attention of q [nl, B, N, Hq, d] over a paged prefix and the tree rows
    kt, vt [nl, B, N, Hkv, d]; returns (out like q, lse fp32 [nl, B, N, Hq] or None)."""
    if stream is not None:
        return _on(stream, q, medusa_paged_tree_attention, q, k_pages, v_pages, page_table, kt, vt, mask, prefix_len, scale,
                   out, lse, want_lse, ws, d_status)
    r = (_native or _load()).tree_attention(q, k_pages, v_pages, page_table, kt, vt, mask, prefix_len, scale, out, lse,
                                            want_lse, ws, d_status)
    if type(r) is int:
        raise B_.MedusaError("medusa_paged_tree_attention", r)
    return r


def medusa_paged_compact(k_pages, v_pages, page_table, kt, vt, path_nodes, accept_len, prefix_len, new_len=None,
                         d_status=None, stream=None):
    """Appends the accepted paths path_nodes [B, Dmax + 1], accept_len [B] of the tree
    rows kt, vt [nl, B, N, Hkv, d] to the pages; returns new_len [B] (new unless
    given; may be prefix_len)."""
    if stream is not None:
        return _on(stream, kt, medusa_paged_compact, k_pages, v_pages, page_table, kt, vt, path_nodes, accept_len, prefix_len,
                   new_len, d_status)
    r = (_native or _load()).compact(k_pages, v_pages, page_table, kt, vt, path_nodes, accept_len, prefix_len, new_len,
                                     d_status)
    if type(r) is int:
        raise B_.MedusaError("medusa_paged_compact", r)
    return r[0]
