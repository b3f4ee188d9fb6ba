"""The oracle of the calls around a verify pass's output, pinned by worked values, torch's bf16 and brute force."""
import numpy as np
import pytest

import workloads as wl
from oracle import verify as ov

torch = pytest.importorskip("torch")


def test_round_bf16_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(2000) * 10.0 ** rng.integers(-42, 38, 2000), [0.0, -0.0, np.inf, -np.inf, 3.4e38, 1e-45, 2.0 ** -133, 2.0 ** -134]]).astype(np.float32)
    want = torch.from_numpy(x).bfloat16().double().numpy()
    np.testing.assert_array_equal(ov.round_bf16(x), want)
    assert np.isnan(ov.round_bf16(np.nan))
    np.testing.assert_array_equal(ov.bf16_value(ov.bf16_bits(want)), want)


def test_words_have_neighbours_sixteen_bits_apart():
    q = np.arange(16).reshape(1, 16) % 16
    assert [hex(w) for w in ov.pack(q)[0]] == ["0x75316420", "0xfdb9eca8"]
    r = np.random.default_rng(1).integers(0, 16, (5, 96))
    np.testing.assert_array_equal(ov.unpack(ov.pack(r)), r)


def test_weights_by_hand():
    q = np.zeros((1, 32), int)
    q[0, :4] = [0, 15, 9, 8]
    s = wl.to_bf16_bits(np.array([[0.3]], np.float32))
    v = float(ov.bf16_value(s)[0, 0])
    assert v == 0.30078125
    assert ov.weights(ov.pack(q), s)[0, :4].tolist() == [-8 * v, 2.109375, v, 0.0]  # 7 * 0.30078125 = 2.10546875, up to even
    assert ov.weights(ov.pack(q), s, np.array([[128 + 9]]))[0, 2] == 0.0  # a zero's top bit is ignored
    y, size = ov.linear_w4(wl.to_bf16_bits(np.ones((1, 32), np.float32)), ov.pack(q), s)
    assert y[0, 0] == ov.weights(ov.pack(q), s).sum() and size[0, 0] == np.abs(ov.weights(ov.pack(q), s)).sum()


@pytest.mark.parametrize("symmetric", [False, True])
def test_quantizing_is_off_by_half_a_step_at_most(symmetric):
    rng = np.random.default_rng(2)
    w = rng.standard_normal((6, 128)).astype(np.float32)
    w[2, 32:64] = 0.0
    w[3, 64:96] = np.abs(w[3, 64:96])
    w[4, :32] = np.nan
    q, s, z, bad = ov.quantize(w, 32, symmetric)
    assert bad.T.tolist() == [[False] * 4] * 4 + [[True] + [False] * 3] + [[False] * 4]
    back = ov.weights(ov.pack(q), ov.bf16_bits(s), z.astype(np.uint8))
    assert np.isnan(back[4, :32]).all() and (back[2, 32:64] == 0).all()
    step = np.repeat(s.T.astype(np.float64), 32, 1)
    ok = np.isfinite(w)
    # half a step, the zero's own half step where there is one, the ends cut off by the scale's rounding (15 steps of 2^-9) and the product's rounding
    assert np.all(np.abs(back - w)[ok] <= (step * (0.5 + (0.0 if symmetric else 0.5) + 15 * 2.0 ** -8) + 2.0 ** -8 * np.abs(back))[ok])


def test_processing_by_hand():
    V, parent = 40, [-1, 0, 0, 1]
    z = np.zeros((1, 4, V))
    z[:] = np.arange(V) - 20.0
    counts = np.zeros((1, V), np.int32)
    counts[0, 30] = 2
    prompt = ov.words_of(np.arange(V)[None] == 35)
    tokens = np.array([[7, 30, 8, 7]])
    mask = ov.words_of(np.arange(V)[None] != 39)
    out, _ = ov.process(z, counts, prompt, [2.0], [0.5], [0.25], np.full(V, 1.0), mask, np.array([[-1, 0, -1, 0]]), tokens, parent)
    assert out[0, 0, 30] == 10 / 2 - 1.0 - 0.25 + 1.0 and out[0, 0, 35] == 15 / 2 + 1.0 and out[0, 0, 7] == -13 * 2 - 0.5 - 0.25 + 1.0
    assert out[0, 1, 30] == 10 / 2 - 1.5 - 0.25 + 1.0 and out[0, 2, 30] == out[0, 0, 30] and out[0, 3, 7] == -26 - 1.0 - 0.25 + 1.0
    assert out[0, 2, 8] == -24 - 0.5 - 0.25 + 1.0 and out[0, 1, 8] == -12 + 1.0
    assert out[0, 1, 39] == -np.inf == out[0, 3, 39] and out[0, 0, 39] == 20.0
    plain, _ = ov.process(z)
    np.testing.assert_array_equal(plain, z)


def test_counting_by_hand():
    c, p = ov.count_tokens([[3, 3, -1, 40], [0, 39, 50, 2]], 41, np.zeros((2, 41), np.int32), np.zeros((2, 2), np.uint32))
    assert c.sum() == 6 and c[0, 3] == 2 and c[0, 40] == 1 and p.tolist() == [[8, 256], [5, 128]]
    a = ov.count_accepted(c, np.array([[3, 4, 5], [3, 41, 5]]), np.array([[0, 2, -1], [0, 1, -1]]), [2, 2])
    assert a[0, 3] == 3 and a[0, 5] == 1 and (a[1] == c[1]).all()
