"""Pins of the float64 paged-cache functions that the GPU tests compare with:
against torch's attention, the contiguous oracle and closed forms (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import paged
from oracle import topology as otopo
from tests.paged import pool, starts, values

torch = pytest.importorskip("torch")


def test_chunk_attention_is_causal_attention_of_the_gathered_rows():
    rng = np.random.default_rng(1)
    prefix, chunk = [5, 0, 17], [4, 9, 1]
    kp, vp, table = pool(rng, [p + c for p, c in zip(prefix, chunk)], nl=2, page=4, hkv=2, d=8, dtype="f32")
    q0 = starts(chunk)
    q = values(rng, (2, int(q0[-1]), 4, 8), "f32")
    out, lse, mag = paged.paged_attention(q, kp, vp, table, q0, prefix)
    for b in range(3):
        n, m = chunk[b], prefix[b] + chunk[b]
        at = [table[b, r // 4] * 4 + r % 4 for r in range(m)]
        for l in range(2):
            k, v = (torch.tensor(x[l].reshape(-1, 2, 8)[at], dtype=torch.float64).repeat_interleave(2, 1).transpose(0, 1)
                    for x in (kp, vp))
            qq = torch.tensor(q[l, q0[b]:q0[b + 1]], dtype=torch.float64).transpose(0, 1)
            see = torch.ones(n, m, dtype=torch.bool).tril(prefix[b])
            ref = torch.nn.functional.scaled_dot_product_attention(qq, k, v, attn_mask=see).transpose(0, 1)
            np.testing.assert_allclose(out[l, q0[b]:q0[b + 1]], ref.numpy(), rtol=1e-12, atol=1e-13)
            s = (qq @ k.transpose(1, 2) / np.sqrt(8)).masked_fill(~see, -np.inf)
            np.testing.assert_allclose(lse[l, q0[b]:q0[b + 1]], torch.logsumexp(s, -1).T.numpy(), rtol=1e-12)


def test_tree_attention_over_pages_equals_the_contiguous_oracle():
    rng = np.random.default_rng(2)
    t = otopo.dense([3, 2], 10)
    prefix = np.array([7, 0], np.int32)
    kp, vp, table = pool(rng, [7, 0], nl=1, page=3, hkv=2, d=32, dtype="bf16")
    kt, vt, q = (values(rng, (1, 2, 10, h, 32), "bf16") for h in (2, 2, 4))
    _, _, mask = otopo.tree_build(t, np.zeros(2, np.int32), np.zeros((2, 2, 10), np.int32), prefix)
    kc, vc = np.zeros((1, 2, 8, 2, 32), np.uint16), np.zeros((1, 2, 8, 2, 32), np.uint16)
    at = paged.rows_of(table, 0, 0, 7, 3)
    kc[0, 0, :7], vc[0, 0, :7] = kp[0].reshape(-1, 2, 32)[at], vp[0].reshape(-1, 2, 32)[at]
    out, _, _ = paged.paged_tree_attention(q, kp, vp, table, kt, vt, mask, prefix)
    np.testing.assert_allclose(out, oracle.tree_attention(q, kc, vc, kt, vt, mask, prefix), rtol=1e-12, atol=1e-13)


def test_a_node_that_sees_nothing_is_zero():
    rng = np.random.default_rng(3)
    kp, vp, table = pool(rng, [0], nl=1, page=4, hkv=1, d=4, dtype="f32")
    kt, vt, q = (values(rng, (1, 1, 2, 1, 4), "f32") for _ in range(3))
    out, lse, _ = paged.paged_tree_attention(q, kp, vp, table, kt, vt, np.array([[1], [0]], np.int32), [0])
    np.testing.assert_allclose(out[0, 0, 0, 0], vt[0, 0, 0, 0])
    assert np.all(out[0, 0, 1] == 0) and np.isneginf(lse[0, 0, 1, 0])


def test_rotation_matches_the_tree_rope_oracle_and_its_layouts_agree():
    rng = np.random.default_rng(4)
    x = values(rng, (2, 6, 3, 16), "f32")
    pos = np.array([0, 1, 7, 100, 4095, 131071], np.int32)
    f = paged.rope_frequencies(16)
    half = paged.rope(x, pos, f)
    np.testing.assert_allclose(half, oracle.tree_rope(x.reshape(2, 1, 6, 3, 16), pos.reshape(1, 6)).reshape(x.shape),
                               rtol=1e-9, atol=1e-9)
    order = np.concatenate((np.arange(0, 16, 2), np.arange(1, 16, 2)))  # (2i, 2i + 1) -> (i, i + 8)
    inter = paged.rope(x, pos, f, interleaved=True)
    np.testing.assert_allclose(inter[..., order], paged.rope(np.ascontiguousarray(x[..., order]), pos, f), rtol=1e-12, atol=1e-12)
    part = paged.rope(x, pos, paged.rope_frequencies(8))
    assert np.array_equal(part[..., 8:], x[..., 8:].astype(np.float64))
    np.testing.assert_allclose(paged.rope(half.astype(np.float64).astype(np.float32), pos, f, inverse=True), x, atol=1e-6)


@pytest.mark.parametrize("scaling", ["linear", "bands", "ramp"])
def test_scaled_frequencies_lie_between_the_plain_and_the_slowed_ones(scaling):
    f = paged.rope_frequencies(128, 10000.0)
    g = paged.rope_frequencies(128, 10000.0, scaling, factor=8.0, low=1.0, high=32.0, original_len=4096)
    assert np.all(g <= f * (1 + 1e-12)) and np.all(g >= f / 8 * (1 - 1e-12)) and np.all(np.diff(g) < 0)
    if scaling == "linear":
        np.testing.assert_allclose(g, f / 8)
    else:
        turns = 4096 * f / (2 * np.pi)
        np.testing.assert_allclose(g[turns > 40], f[turns > 40])
        np.testing.assert_allclose(g[turns < 0.7], f[turns < 0.7] / 8)


def test_append_and_compaction_touch_their_rows_only():
    rng = np.random.default_rng(5)
    prefix, chunk = [3, 6], [2, 3]
    kp, vp, table = pool(rng, [5, 9], nl=2, page=4, hkv=2, d=4, dtype="f32")
    kp[:], vp[:] = 1.0, 2.0
    k, v = values(rng, (2, 5, 2, 4), "f32"), values(rng, (2, 5, 2, 4), "f32")
    k2, v2 = paged.paged_append(k, v, kp, vp, table, starts(chunk), prefix)
    kc, vc, n = paged.paged_compact(kp, vp, table, k.reshape(2, 1, 5, 2, 4)[:, [0, 0]], v.reshape(2, 1, 5, 2, 4)[:, [0, 0]],
                                    np.array([[0, 4, -1], [1, 2, 3]]), [2, 3], prefix)
    assert n.tolist() == [5, 9]
    flat = k2.reshape(2, -1, 2, 4)
    assert np.array_equal(flat[:, table[1, 1] * 4 + 2], k[:, 2]) and np.array_equal(flat[:, table[1, 2] * 4], k[:, 4])
    assert np.array_equal(kc.reshape(2, -1, 2, 4)[:, table[0, 1] * 4], k[:, 4])
    for new, old, rows in ((k2, kp, 5), (v2, vp, 5), (kc, kp, 5), (vc, vp, 5)):
        assert int(np.any(new != old, axis=(0, 3, 4)).sum()) == rows
