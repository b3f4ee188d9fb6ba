"""Inputs and error bounds of the paged-cache tests.

Bounds, from the arithmetic of the calls (u = 2^-24, a rounding to fp32; e =
half a step of the output type, eps / 2: 2^-24 for fp32 and 2^-8 for bf16):
 - rotation: the angle is rounded once to fp32 within an eighth of a turn
   (u pi / 4 < u), sincospif is within 2 ulp (2^-23 of a value at most 1), the
   magnitude's product rounds once, the two products and their sum once each:
   |error| <= 8 u m (|x0| + |x1|) + e |y|.
 - attention: a score is a sum of d products in fp32, off by at most
   ds = (d + 4) u scale sum |q k| (scale and log2 e rounded in), the
   probabilities by a factor e^ds each, so a quotient of sums by e^(2 ds);
   2^x is within 2 ulp, the sums of n terms within n u, rescaling by running
   maxima within n / 16 u more: at most r = 2 ds + (1.1 n + 32) u of
   sum p |v|.  The tensor-core kernel rounds p to bf16: 2^-8 of sum p |v| more.
   Then the output rounds: e |out|.
 - lse: ds + (1.1 n + 32) u + u |lse| * 4 (the log2 domain's factors).
"""
from __future__ import annotations

import numpy as np

import workloads as wl
from oracle.paged import f64
from tests.helpers import to_dev

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def values(rng, shape, dtype):
    x = rng.standard_normal(shape).astype(np.float32)
    return wl.to_bf16_bits(x) if dtype == "bf16" else x


def pool(rng, lens, *, nl, page, hkv, d, dtype, spare=2):
    """(k_pages, v_pages, page_table) with room for lens[b] rows each: pages in
    random order, NaN wherever no row lies, -1 behind each sequence's last page."""
    need = [-(-n // page) for n in lens]
    n_pages, wide = max(1, sum(need)) + spare, max(1, *need)
    order = rng.permutation(n_pages)
    table = np.full((len(lens), wide), -1, np.int32)
    nan = np.uint16(0x7FC0) if dtype == "bf16" else np.float32(np.nan)
    kp = np.full((nl, n_pages, page, hkv, d), nan)
    vp = kp.copy()
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for r in range(n):
            pg = table[b, r // page]
            kp[:, pg, r % page], vp[:, pg, r % page] = values(rng, (nl, hkv, d), dtype), values(rng, (nl, hkv, d), dtype)
    return kp, vp, table


def starts(chunk):
    return np.concatenate(([0], np.cumsum(chunk))).astype(np.int32)


def score_error(q, k_rows_max, d, scale):
    """ds of the module's text for every q row: q [..., d], the largest |k| row norm."""
    return (d + 4) * U * scale * np.linalg.norm(f64(q), axis=-1) * k_rows_max


def attention_bound(q, k_norm, d, scale, n, mag, out, dtype, rounded_p):
    ds = score_error(q, k_norm, d, scale)[..., None]
    r = 2 * ds + (1.1 * n + 32) * U + (2.0 ** -8 if rounded_p else 0.0)
    return r * mag + HALF[dtype] * np.abs(out) + 1e-30


def lse_bound(q, k_norm, d, scale, n, lse):
    return score_error(q, k_norm, d, scale) + (1.1 * n + 32) * U + 4 * U * np.abs(lse)


def dev_ints(a):
    return to_dev(np.ascontiguousarray(a, np.int32))
