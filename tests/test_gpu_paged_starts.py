"""Starts that decrease or leave [0, T]: a sequence is entered and attended to by its own
starts, one that begins before the end of an earlier one is refused, so that a token is one
sequence's, and nothing of a refused sequence is read or written."""
import numpy as np
import pytest

from oracle import paged as ref
from tests.helpers import bf16_to_f64, to_dev, to_host
from tests.paged import HALF, U, attention_bound, dev_ints, pool, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

OVERFLOW, BAD_LENGTH = 2, 5


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


def host64(t):
    a = to_host(t)
    return bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def holders(q0, T):
    """The sequences whose starts are in order and not before the end of an earlier such sequence."""
    fine = [b for b in range(len(q0) - 1) if 0 <= q0[b] <= q0[b + 1] <= T]
    return [b for b in fine if all(j >= b or q0[j + 1] <= q0[b] for j in fine)]


def many():
    q0 = list(range(901))
    q0[5] = 700  # sequence 4 holds 4 .. 699, 5 decreases, 6 .. 699 come too late
    return q0


CASES = {
    "neighbour": (8, [0, 5, 2, 8], [3, 0, 1]),
    "late": (9, [0, 2, 1, 6, 9], [10, 20, 7, 2]),
    "back to the start": (64, [0, 50, 0, 5], [0, 1, 10]),
    "outside, then back": (12, [0, 20, 4, 12], [1, 2, 3]),
    "negative": (10, [0, -4, 3, 10], [1, 0, 2]),
    "inside another": (30, [0, 20, 6, 9, 9, 30], [0, 2, 4, 0, 5]),
    "many sequences": (900, many(), [1] * 900),
    "back in a later round": (900, [*range(500), 450, *range(501, 901)], [1] * 900),
    "before all others": (20, [0, 0, 9, 12, 3, 6, 12, 20], [2, 0, 1, 4, 0, 3, 5]),
}


def inputs(name, dtype, page=16, hq=2, hkv=1, d=64):
    T, q0, prefix = CASES[name]
    rng = np.random.default_rng(len(q0) + T)
    good = holders(q0, T)
    lens = [prefix[b] + (q0[b + 1] - q0[b] if b in good else 0) for b in range(len(prefix))]
    kp, vp, table = pool(rng, lens, nl=2, page=page, hkv=hkv, d=d, dtype=dtype)
    return T, q0, prefix, good, kp, vp, table, values(rng, (2, T, hq, d), dtype), values(rng, (2, T, hkv, d), dtype), values(rng, (2, T, hkv, d), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", CASES)
def test_append(mg, name, dtype):
    T, q0, prefix, good, kp, vp, table, q, k, v = inputs(name, dtype)
    dk, dv, st = to_dev(kp), to_dev(vp), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=dk.dtype, device="cuda")
    mg.medusa_paged_append(to_dev(k), to_dev(v), dk, dv, dev_ints(table), dev_ints(q0), dev_ints(prefix), q=to_dev(q), rope=mg.RopeSpec(64), q_out=out, d_status=st)
    assert mg.medusa_status_check(st) == BAD_LENGTH
    k2, v2, f = ref.f64(kp), ref.f64(vp), ref.rope_frequencies(64)
    want, held = np.full(q.shape, 7.0), np.zeros(T, bool)
    for b in good:
        a, e, L = q0[b], q0[b + 1], prefix[b]
        at, pos = ref.rows_of(table, b, L, e - a, 16), np.arange(L, L + e - a)
        k2.reshape(2, -1, 1, 64)[:, at], v2.reshape(2, -1, 1, 64)[:, at] = ref.rope(k[:, a:e], pos, f), ref.f64(v[:, a:e])
        want[:, a:e] = ref.rope(q[:, a:e], pos, f)
        held[a:e] = True
    assert np.array_equal(host64(dv), v2, equal_nan=True)
    g = host64(dk)
    assert np.array_equal(np.isnan(g), np.isnan(k2)) and np.nanmax(np.abs(g - k2)) <= 8 * U * 2 * 5.5 + HALF[dtype] * 5.5 * 1.5
    g = host64(out)
    assert np.all(g[:, ~held] == 7.0) and np.max(np.abs(g - want)) <= 8 * U * 2 * 5.5 + HALF[dtype] * 5.5 * 1.5


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", CASES)
def test_attention(mg, name, dtype, d):
    T, q0, prefix, good, kp, vp, table, q, _, _ = inputs(name, dtype, d=d)
    want, mag, held = np.zeros(q.shape), np.zeros(q.shape), np.zeros(T, bool)
    for b in good:
        a, e = q0[b], q0[b + 1]
        if e > a:
            want[:, a:e], _, mag[:, a:e] = ref.paged_attention(q[:, a:e], kp, vp, table[b:b + 1], [0, e - a], [prefix[b]])
            held[a:e] = True
    k64 = ref.f64(kp)
    limit = attention_bound(q, np.sqrt(np.nanmax(np.nansum(k64 * k64, -1))), d, d ** -0.5, table.shape[1] * 16, mag, want, dtype, dtype == "bf16")
    first = None
    for _ in range(2):
        st, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full(q.shape, 7.0, dtype=to_dev(q[:1, :1]).dtype, device="cuda")
        mg.medusa_paged_attention(to_dev(q), to_dev(kp), to_dev(vp), dev_ints(table), dev_ints(q0), dev_ints(prefix), out=out, d_status=st)
        assert mg.medusa_status_check(st) == BAD_LENGTH
        g = host64(out)
        assert np.all(g[:, ~held] == 7.0)
        assert np.all(np.abs(g - want)[:, held] <= limit[:, held])
        assert first is None or np.array_equal(g, first)
        first = g


def test_a_token_behind_its_sequence_reaches_no_page(mg):
    """Starts [0, 50, 0, 5] and a page each: token 40 is none of sequence 2's five, whose table has one
    page; its 50 tokens are sequence 0's, which has no room for them."""
    rng = np.random.default_rng(7)
    kp, vp, table = pool(rng, [16, 1, 15], nl=1, page=16, hkv=1, d=16, dtype="bf16")
    assert table.shape[1] == 1
    k = values(rng, (1, 64, 1, 16), "bf16")
    dk, dv, st = to_dev(kp), to_dev(vp), torch.zeros(1, dtype=torch.int32, device="cuda")
    q, out = values(rng, (1, 64, 1, 16), "bf16"), torch.full((1, 64, 1, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    mg.medusa_paged_append(to_dev(k), to_dev(k), dk, dv, dev_ints(table), dev_ints([0, 50, 0, 5]), dev_ints([0, 1, 10]), q=to_dev(q), q_out=out, d_status=st)
    assert mg.medusa_status_check(st) in (OVERFLOW, BAD_LENGTH)  # the first to be seen
    assert np.array_equal(to_host(dk), kp) and np.array_equal(to_host(dv), vp)
    assert np.array_equal(to_host(out)[:, :50], q[:, :50]) and torch.all(out[:, 50:] == 7.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_hundred_thousand_sequences_one_of_them_bad(mg, dtype):
    """One token each, which sees its own row alone; sequence 7's starts decrease and 8 begins before 6's end."""
    B, dt = 100000, torch.bfloat16 if dtype == "bf16" else torch.float32
    q0 = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    q0[8] = 6
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v, q = (torch.randn((1, B, 1, 64), generator=g, device="cuda").to(dt) for _ in range(3))
    kp, vp = (torch.full((1, B, 8, 1, 64), 3.0, dtype=dt, device="cuda") for _ in range(2))
    table, prefix = torch.arange(B, dtype=torch.int32, device="cuda").flip(0).view(B, 1).contiguous(), torch.zeros(B, dtype=torch.int32, device="cuda")
    st, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full_like(q, 7.0)
    mg.medusa_paged_append(k, v, kp, vp, table, q0, prefix, d_status=st)
    assert mg.medusa_status_check(st) == BAD_LENGTH
    mg.medusa_paged_attention(q, kp, vp, table, q0, prefix, out=out, d_status=st)
    assert mg.medusa_status_check(st) == BAD_LENGTH
    live = torch.ones(B, dtype=torch.bool, device="cuda")
    live[7:9] = False
    assert torch.equal(out[:, live], v[:, live]) and torch.all(out[:, ~live] == 7.0)
    rows = kp.flip(1)[0, :, 0], vp.flip(1)[0, :, 0]
    assert torch.equal(rows[0][live], k[0][live]) and torch.equal(rows[1][live], v[0][live])
    assert torch.all(rows[0][~live] == 3.0) and torch.all(kp[:, :, 1:] == 3.0)
