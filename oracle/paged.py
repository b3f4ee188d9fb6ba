"""The paged-cache calls in float64 numpy, one sequence and one head at a time,
from their definitions: row r of sequence b is row r % page_size of page
page_table[b][r // page_size].  Arrays are float32, or uint16 holding bf16 bits;
inputs are never modified."""
from __future__ import annotations

import numpy as np


def f64(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return a.astype(np.float64)


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original_len=4096):
    """Radians a position of the rotary_dim / 2 pairs."""
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    f = np.float64(base) ** (-2.0 * i / rotary_dim)
    if scaling == "none":
        return f
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        wave = 2.0 * np.pi / f
        t = (original_len / wave - low) / (high - low)
        return np.where(wave > original_len / low, f / factor,
                        np.where(wave < original_len / high, f, (1.0 - t) * f / factor + t * f))
    if scaling == "ramp":
        def pair(turns):
            return rotary_dim * np.log(original_len / (2.0 * np.pi * turns)) / (2.0 * np.log(base))
        a, b = max(np.floor(pair(high)), 0.0), min(np.ceil(pair(low)), rotary_dim - 1.0)
        t = np.clip((i - a) / max(b - a, 0.001), 0.0, 1.0)
        return t * f / factor + (1.0 - t) * f
    raise ValueError(scaling)


def rope(x, pos, freq, interleaved=False, magnitude=1.0, inverse=False):
    """x [nl, T, H, d] at positions pos [T]: the leading 2 len(freq) elements turn."""
    y = f64(x).copy()
    angle = np.asarray(pos, np.float64)[:, None] * freq * (-1.0 if inverse else 1.0)
    c, s = magnitude * np.cos(angle)[:, None], magnitude * np.sin(angle)[:, None]
    h = len(freq)
    i0, i1 = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    x0, x1 = y[..., i0].copy(), y[..., i1].copy()
    y[..., i0], y[..., i1] = x0 * c - x1 * s, x1 * c + x0 * s
    return y


def rows_of(page_table, b, first, n, page_size):
    """Pool rows of rows first .. first + n - 1 of sequence b."""
    r = np.arange(first, first + n)
    return np.asarray(page_table)[b, r // page_size].astype(np.int64) * page_size + r % page_size


def paged_append(k, v, k_pages, v_pages, page_table, q_start, prefix_len, turn=lambda x, pos: f64(x)):
    """float64 pools with the chunk's rows entered; `turn(x, pos)` rotates [nl, n, H, d]."""
    k2, v2 = f64(k_pages), f64(v_pages)
    ps = k2.shape[2]
    kf, vf = k2.reshape(k2.shape[0], -1, *k2.shape[3:]), v2.reshape(v2.shape[0], -1, *v2.shape[3:])
    for b, L in enumerate(prefix_len):
        a, e = int(q_start[b]), int(q_start[b + 1])
        at = rows_of(page_table, b, int(L), e - a, ps)
        kf[:, at] = turn(k[:, a:e], np.arange(L, L + e - a))
        vf[:, at] = f64(v[:, a:e])
    return k2, v2


def _softmax_rows(q, k, v, see, scale):
    """q [n, d], k, v [m, d], see [n, m] -> (out, lse, sum of p |v|); nothing seen: zeros and -inf;
    a score seen that is NaN or +inf, or none that is more than -inf: NaN."""
    with np.errstate(divide="ignore", invalid="ignore"):
        s = np.where(see, scale * (q @ k.T), -np.inf)
        m = s.max(-1, initial=-np.inf, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        l = p.sum(-1, keepdims=True)
        w = np.where(see.any(-1, keepdims=True), p / l, 0.0)
        return w @ v, (np.log(l) + m)[:, 0], w @ np.abs(v)


def paged_attention(q, k_pages, v_pages, page_table, q_start, prefix_len, scale=None):
    """(out, lse, bound) for q [nl, T, Hq, d]: bound is the sum of p |v| an error
    estimate needs.  Tokens of no sequence keep NaN."""
    nl, T, Hq, d = q.shape
    ps, Hkv = k_pages.shape[2], k_pages.shape[3]
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out, lse, mag = np.full(q.shape, np.nan), np.full(q.shape[:-1], np.nan), np.full(q.shape, np.nan)
    for b, L in enumerate(prefix_len):
        a, e, L = int(q_start[b]), int(q_start[b + 1]), int(L)
        n = e - a
        at = rows_of(page_table, b, 0, L + n, ps)
        see = np.arange(L + n) < L + 1 + np.arange(n)[:, None]
        for l in range(nl):
            kl, vl = (f64(x[l].reshape(-1, Hkv, d)[at]) for x in (k_pages, v_pages))
            for h in range(Hq):
                out[l, a:e, h], lse[l, a:e, h], mag[l, a:e, h] = _softmax_rows(
                    f64(q[l, a:e, h]), kl[:, h // G], vl[:, h // G], see, scale)
    return out, lse, mag


def paged_tree_attention(q, k_pages, v_pages, page_table, kt, vt, mask, prefix_len, scale=None):
    """(out, lse, bound) for q [nl, B, N, Hq, d], tree rows kt, vt, mask words [N, W]."""
    nl, B, N, Hq, d = q.shape
    ps, Hkv = k_pages.shape[2], k_pages.shape[3]
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    words = np.ascontiguousarray(mask).view(np.uint32)
    n = np.arange(N)
    bits = (words[:, n // 32] >> (n % 32).astype(np.uint32)) & 1 == 1
    out, lse, mag = np.empty(q.shape), np.empty(q.shape[:-1]), np.empty(q.shape)
    for b, L in enumerate(prefix_len):
        L = int(L)
        at = rows_of(page_table, b, 0, L, ps)
        see = np.concatenate((np.ones((N, L), bool), bits), 1)
        for l in range(nl):
            kl, vl = (np.concatenate((f64(x[l].reshape(-1, Hkv, d)[at]), f64(t[l, b]))) for x, t in ((k_pages, kt), (v_pages, vt)))
            for h in range(Hq):
                out[l, b, :, h], lse[l, b, :, h], mag[l, b, :, h] = _softmax_rows(
                    f64(q[l, b, :, h]), kl[:, h // G], vl[:, h // G], see, scale)
    return out, lse, mag


def paged_compact(k_pages, v_pages, page_table, kt, vt, path_nodes, accept_len, prefix_len):
    """(k_pages', v_pages', new_len), bit for bit."""
    k2, v2 = np.array(k_pages, copy=True), np.array(v_pages, copy=True)
    ps = k2.shape[2]
    for b, L in enumerate(prefix_len):
        A = int(accept_len[b])
        at = rows_of(page_table, b, int(L), A, ps)
        for pool, tree in ((k2, kt), (v2, vt)):
            pool.reshape(pool.shape[0], -1, *pool.shape[3:])[:, at] = tree[:, b, path_nodes[b][:A]]
    return k2, v2, np.asarray(prefix_len, np.int32) + np.asarray(accept_len, np.int32)
