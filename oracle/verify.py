"""float64 oracle of the calls around a verify pass's output: weights in 4 bits and the linear
layers with them, the logits as requests want them, and counts of tokens.  numpy alone, element by
element from the definitions."""
from __future__ import annotations

import numpy as np


def bf16_value(bits):
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def round_bf16(x):
    """float64 to the nearest bf16's value, halves to even (subnormals and overflow as bf16 has them)."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
        step = np.exp2(np.maximum(e - 8, -133).astype(np.float64))
        r = np.where(np.isfinite(x), np.rint(x / step) * step, x)
        return np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, x), r)


def bf16_bits(x):
    """Values that bf16 has, as its bits."""
    return (np.asarray(x, np.float64).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def pack(q):
    """Elements 0 .. 15 [N, K] -> words [N, K / 8]: element 2i of eight in bits 4i, element 2i + 1 in bits 16 + 4i."""
    q = np.asarray(q, np.uint32).reshape(q.shape[0], -1, 8)
    words = np.zeros(q.shape[:2], np.uint32)
    for e in range(8):
        words |= q[:, :, e] << np.uint32(4 * (e // 2) + 16 * (e % 2))
    return words


def unpack(words):
    words = np.ascontiguousarray(words).view(np.uint32)
    q = np.zeros(words.shape + (8,), np.int64)
    for e in range(8):
        q[..., e] = (words >> np.uint32(4 * (e // 2) + 16 * (e % 2))) & np.uint32(15)
    return q.reshape(words.shape[0], -1)


def weights(words, scales, zeros=None):
    """The bf16 matrix [N, K] that words, scales (bf16 bits [K / G, N]) and zeros [K / G, N] stand for."""
    q = unpack(words)
    G = q.shape[1] // scales.shape[0]
    s = np.repeat(bf16_value(scales).T, G, 1)
    z = 8 if zeros is None else np.repeat(np.asarray(zeros, np.int64).T & 127, G, 1)
    with np.errstate(invalid="ignore"):
        return round_bf16(s * (q - z))


def linear_w4(x, words, scales, zeros=None):
    """(y, sum of |x w|), x bf16 bits [T, K]."""
    w, x = weights(words, scales, zeros), bf16_value(x)
    with np.errstate(invalid="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T


def quantize(w, G, symmetric):
    """fp32 values [N, K] -> (elements [N, K], scale values [K / G, N], zeros [K / G, N]), in fp32 steps as defined."""
    f = np.float32
    N, K = w.shape
    v = np.asarray(w, f).reshape(N, K // G, G)
    with np.errstate(all="ignore"):
        lo, hi = np.minimum(np.fmin.reduce(v, -1), f(0)), np.maximum(np.fmax.reduce(v, -1), f(0))
        lo, hi = np.where(np.isnan(lo), f(0), lo), np.where(np.isnan(hi), f(0), hi)
        step = np.maximum(hi, -lo) / f(7) if symmetric else (hi - lo) / f(15)
        s = round_bf16(step).astype(f)
        none = s == 0
        bad = ~np.isfinite(v).all(-1) | ~np.isfinite(s)
        s = np.where(none, f(1), s)
        z = np.full(s.shape, 8, f) if symmetric else np.clip(np.rint(-lo / s), 0, 15).astype(f)
        q = np.clip(np.rint(v / s[..., None]) + z[..., None], 0, 15)
        q = np.where(none[..., None], z[..., None], q)
    s = np.where(bad, f(np.nan), s)
    return np.where(bad[..., None], 0, q).astype(np.int64).reshape(N, K), s.T, z.T, bad.T


def bit(words, V):
    """Words [..., W] -> truth values [..., V]."""
    words = np.ascontiguousarray(words).view(np.uint32)
    v = np.arange(V)
    return (words[..., v // 32] >> (v % 32).astype(np.uint32)) & 1 == 1


def words_of(bits):
    bits = np.asarray(bits, bool)
    V = bits.shape[-1]
    out = np.zeros(bits.shape[:-1] + ((V + 31) // 32,), np.uint32)
    for v in range(V):
        out[..., v // 32] |= bits[..., v].astype(np.uint32) << np.uint32(v % 32)
    return out


def path(parent, n):
    p = []
    while n >= 0:
        p.append(n)
        n = int(parent[n])
    return p[::-1]


def process(logits, counts=None, prompt=None, repetition=None, frequency=None, presence=None, bias=None, mask=None, mask_row=None,
            tokens=None, parent=None):
    """logits [B, N, V] values; prompt and mask words.  Returns (processed float64, a bound of the sizes of what was added up)."""
    z = np.array(logits, np.float64)
    B, N, V = z.shape
    size = np.zeros_like(z)
    with np.errstate(invalid="ignore"):
        for b in range(B):
            for n in range(N):
                c = np.zeros(V) if counts is None else counts[b].astype(np.float64)
                if parent is not None:
                    for j in path(parent, n):
                        t = int(tokens[b, j])
                        if 0 <= t < V:
                            c[t] += 1
                said = c > 0
                if prompt is not None:
                    said = said | bit(prompt[b], V)
                x = z[b, n]
                if repetition is not None:
                    r = float(repetition[b])
                    x = np.where(said, np.where(x > 0, x / r, x * r), x)
                s = np.abs(x)
                for w, times in ((frequency, c), (presence, (c > 0).astype(np.float64))):
                    if w is not None:
                        x = x - float(w[b]) * times
                        s = s + np.abs(float(w[b]) * times)
                if bias is not None:
                    e = np.asarray(bias if np.ndim(bias) == 1 else bias[b], np.float64)
                    x, s = x + e, s + np.abs(e)
                if mask is not None:
                    m = b * N + n if mask_row is None else int(mask_row[b, n])
                    if m >= 0:
                        x = np.where(bit(mask[m], V), x, -np.inf)
                z[b, n], size[b, n] = x, s
    return z, size


def count_tokens(tokens, V, counts=None, prompt=None):
    counts = None if counts is None else np.array(counts)
    prompt = None if prompt is None else np.array(prompt).view(np.uint32)
    for b, row in enumerate(np.asarray(tokens)):
        for t in row:
            if 0 <= t < V:
                if counts is not None:
                    counts[b, t] += 1
                if prompt is not None:
                    prompt[b, t // 32] |= np.uint32(1 << (t % 32))
    return counts, prompt


def count_accepted(counts, tokens, path_nodes, accept_len):
    counts = np.array(counts)
    B, V = counts.shape
    N, D1 = tokens.shape[1], path_nodes.shape[1]
    for b in range(B):
        n = int(accept_len[b])
        if not 1 <= n <= D1:
            continue
        nodes = [int(x) for x in path_nodes[b, :n]]
        if any(not 0 <= x < N or not 0 <= tokens[b, x] < V for x in nodes):
            continue
        for x in nodes:
            counts[b, tokens[b, x]] += 1
    return counts
