"""Inputs and error bounds of the tests of the calls around a verify pass's output.

Bounds, from the arithmetic (u = 2^-24, half a step of fp32):
 - 4-bit linear layer: the weights are exact bf16 values and so are the products in fp32.  A
   product instruction adds 16 columns to a sum: the 16 terms are brought to the largest one's
   exponent and cut off there (2 u of it each at most), the sum is cut off (2 u).  K / 16
   instructions one after the other, their results added over at most 64 parts more, each rounded: every
   intermediate is at most S = sum |x w|, so |error| <= (K / 16 * (2 u + 2 u) + 64 u) S, terms cut
   off within an instruction counted once, as their sum is at most S over all instructions: + 2 u S.
   Then y rounds: u |y| or 2^-8 |y|.
 - logits: five operations, each off by u of its result at most, none larger than the sum `size` of the
   sizes of what is added up: |error| <= 6 u size.
"""
import numpy as np

import workloads as wl
from oracle import verify as ov
from tests.helpers import to_dev, to_host

U = 2.0 ** -24


def matrix(rng, N, K, G, zeros=True, spread=2.6):
    """(words, scale bits, zeros or None) as quantizing normal weights leaves them."""
    q = np.clip(np.rint(rng.standard_normal((N, K)) * spread + 7.5), 0, 15).astype(int)
    s = wl.to_bf16_bits((0.008 + 0.004 * rng.random((K // G, N))).astype(np.float32))
    return ov.pack(q), s, rng.integers(0, 16, (K // G, N)).astype(np.uint8) if zeros else None


def dev_words(w):
    return to_dev(np.ascontiguousarray(w).view(np.int32))


def dev_matrix(m):
    return dev_words(m[0]), to_dev(m[1]), None if m[2] is None else to_dev(m[2])


def bf16(rng, *shape):
    return wl.to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def linear_bound(y, size, K, out):
    return (K / 16 * 4 + 66) * U * size + (U if out == "f32" else 2.0 ** -8) * np.abs(y) + 1e-37


def value(t):
    """A tensor as float64."""
    return t.double().cpu().numpy()


def check_linear(got, x, m, out):
    y, size = ov.linear_w4(x, *m)
    g = value(got)
    assert g.shape == y.shape
    off = np.abs(g - y)
    assert np.all(off <= linear_bound(y, size, x.shape[1], out)), (float(np.max(off / linear_bound(y, size, x.shape[1], out))), np.argwhere(off > linear_bound(y, size, x.shape[1], out))[:4])


def host_words(t):
    return to_host(t).view(np.uint32)
