"""The calls around a verify pass's output on torch tensors: linear layers with 4-bit
weights, the logits as requests want them, and the counts that go with them.
csrc/python/verify_binding.cpp checks and marshals their arguments.

Everywhere: outputs that are not given are allocated, on the stream that
the call runs on: the current one of the tensors' device, or `stream`.  No gradients
are recorded.
"""
from __future__ import annotations

import ctypes

from . import binding as B_
from .build import load_binding
from .paged import _on

try:
    import torch
except ImportError:  # the library can be built without it
    torch = None

_native = None


def _load():
    """The compiled binding (raises if it has not been built)."""
    global _native
    _native = load_binding("verify_binding")
    return _native


def _topology(topo, like):
    """The address of a device topology's description, which must be on `like`'s device, or None."""
    if topo is None:
        return None
    held = topo.buf if isinstance(topo.buf, torch.Tensor) else topo.buf[0]
    if held.device != like.device:
        raise ValueError(f"medusa_logits_process: topo is on {held.device}, logits are on {like.device}")
    return ctypes.addressof(topo.st)


def medusa_w4_quantize(w, group: int = 128, symmetric: bool = False, stream=None):
    """w [Nout, K] bf16 or fp32 in 4 bits: (qweight int32 [Nout, K / 8], scales bf16
    [K / group, Nout], zeros uint8 like scales, or None when symmetric).  group is 32, 64 or
    128; see include/medusa.h for the formulas."""
    if stream is not None:
        return _on(stream, w, medusa_w4_quantize, w, group, symmetric)
    r = (_native or _load()).quantize(w, group, symmetric)
    if type(r) is int:
        raise B_.MedusaError("medusa_w4_quantize", r)
    return r


def medusa_linear_w4(x, qweight, scales, zeros=None, y=None, out_dtype=None, d_status=None, stream=None):
    """y [T, Nout] = x [T, K] @ W^T with W in 4 bits (qweight, scales, zeros as
    medusa_w4_quantize makes them; zeros None: 8).  x is bf16, its rows may be spaced; y is
    bf16, or fp32 with out_dtype=torch.float32 or a y of that type."""
    if stream is not None:
        return _on(stream, x, medusa_linear_w4, x, qweight, scales, zeros, y, out_dtype, d_status)
    r = (_native or _load()).linear_w4(x, qweight, scales, zeros, y, out_dtype is torch.float32 if out_dtype in _OUT else out_dtype, d_status)
    if type(r) is int:
        raise B_.MedusaError("medusa_linear_w4", r)
    return r


_OUT = () if torch is None else (None, torch.bfloat16, torch.float32)


def medusa_logits_process(logits, counts=None, prompt_bits=None, repetition=None, frequency=None, presence=None, bias=None,
                          mask=None, mask_row=None, tokens=None, topo=None, out=None, d_status=None, stream=None):
    """logits [B, N, V] (fp32 or bf16, rows may be spaced) as the requests want them: fp32
    [B, N, V], new unless given (out may be logits).  counts int32 [B, V] and prompt_bits
    int32 [B, ceil(V / 32)] are what medusa_count_tokens and medusa_count_accepted keep;
    repetition, frequency and presence fp32 [B]; bias fp32 [V] or [B, V]; mask int32
    [M, ceil(V / 32)], bits of the tokens that may follow, with mask_row int32 [B, N] (-1: no
    mask), or [B * N, ceil(V / 32)] without.  With topo (DevTopology) and tokens [B, N] the tokens
    on a node's path count as said.  See include/medusa.h for the formulas."""
    if stream is not None:
        return _on(stream, logits, medusa_logits_process, logits, counts, prompt_bits, repetition, frequency, presence, bias, mask,
                   mask_row, tokens, topo, out, d_status)
    r = (_native or _load()).logits(logits, counts, prompt_bits, repetition, frequency, presence, bias, mask, mask_row, tokens,
                                    _topology(topo, logits), out, d_status)
    if type(r) is int:
        raise B_.MedusaError("medusa_logits_process", r)
    return r


def medusa_count_tokens(tokens, V: int, counts=None, prompt_bits=None, d_status=None, stream=None):
    """Enters tokens int32 [B, S] (negative: padding) into counts int32 [B, V] and / or
    prompt_bits int32 [B, ceil(V / 32)], in place; returns (counts, prompt_bits)."""
    if stream is not None:
        return _on(stream, tokens, medusa_count_tokens, tokens, V, counts, prompt_bits, d_status)
    r = (_native or _load()).count_tokens(tokens, V, counts, prompt_bits, d_status)
    if r:
        raise B_.MedusaError("medusa_count_tokens", r)
    return counts, prompt_bits


def medusa_count_accepted(counts, tokens, path_nodes, accept_len, d_status=None, stream=None):
    """Counts the accepted paths' tokens, in place: counts int32 [B, V], tokens [B, N],
    path_nodes [B, Dmax + 1] and accept_len [B] as medusa_typical_accept leaves them; returns counts."""
    if stream is not None:
        return _on(stream, counts, medusa_count_accepted, counts, tokens, path_nodes, accept_len, d_status)
    r = (_native or _load()).count_accepted(counts, tokens, path_nodes, accept_len, d_status)
    if r:
        raise B_.MedusaError("medusa_count_accepted", r)
    return counts
