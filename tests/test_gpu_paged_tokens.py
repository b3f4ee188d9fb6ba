"""Rotation and append where a CTA takes several tokens (few vectors a token, more than
four tokens an SM): against the float64 definitions, bounds of tests/paged.py."""
import numpy as np
import pytest

from oracle import paged as ref
from tests.helpers import bf16_to_f64, to_dev, to_host
from tests.paged import HALF, U, dev_ints, pool, starts, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


def host64(t):
    a = to_host(t)
    return bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def bound(x, want, r, inter, m, dtype):
    """8 u m (|x0| + |x1|) + half a step of the result; elements behind the turned part are copies."""
    y = np.abs(ref.f64(x))
    h = r // 2
    i0, i1 = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, h), slice(h, r))
    b = np.zeros_like(y)
    b[..., i0] = b[..., i1] = 8 * U * m * (y[..., i0] + y[..., i1])
    b[..., :r] += HALF[dtype] * np.abs(want[..., :r]) + 1e-38
    return b


CASES = [
    # one task a token: a single head of two vectors of 16, 8, 4 and 2 bytes; CTAs across the layers' boundary
    dict(dtype="bf16", nl=1, T=1301, hq=1, hkv=0, d=16, r=16),
    dict(dtype="bf16", nl=1, T=2603, hq=1, hkv=0, d=8, r=8),
    dict(dtype="bf16", nl=3, T=871, hq=1, hkv=0, d=4, r=4),
    dict(dtype="bf16", nl=2, T=1301, hq=1, hkv=0, d=2, r=2),
    dict(dtype="f32", nl=2, T=651, hq=1, hkv=0, d=8, r=8),
    dict(dtype="f32", nl=1, T=2603, hq=1, hkv=0, d=4, r=4),
    dict(dtype="f32", nl=1, T=1301, hq=1, hkv=0, d=2, r=2),
    # 2, 3, 5, 16, 20, 63 and 64 tasks a token
    dict(dtype="bf16", nl=2, T=1301, hq=1, hkv=1, d=16, r=16),
    dict(dtype="f32", nl=1, T=2603, hq=2, hkv=1, d=8, r=8),
    dict(dtype="bf16", nl=3, T=401, hq=1, hkv=0, d=80, r=48),
    dict(dtype="bf16", nl=1, T=2603, hq=1, hkv=1, d=128, r=128),
    dict(dtype="f32", nl=2, T=701, hq=1, hkv=1, d=80, r=40),
    dict(dtype="bf16", nl=1, T=1301, hq=6, hkv=1, d=144, r=80),
    dict(dtype="bf16", nl=2, T=651, hq=6, hkv=2, d=128, r=64),
]
IDS = lambda c: f"{c['dtype']}-nl{c['nl']}-T{c['T']}-{c['hq']}+{c['hkv']}-d{c['d']}"  # noqa: E731


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_rotation_of_several_tokens_a_cta(mg, c, inter):
    rng = np.random.default_rng(c["d"] + c["T"] + inter)
    q = values(rng, (c["nl"], c["T"], c["hq"], c["d"]), c["dtype"])
    k = values(rng, (c["nl"], c["T"], c["hkv"], c["d"]), c["dtype"]) if c["hkv"] else None
    pos = rng.integers(-5, 1 << 16, c["T"]).astype(np.int32)
    spec = mg.RopeSpec(c["r"], interleaved=inter, magnitude=1.25)
    freq = ref.rope_frequencies(c["r"])
    for inverse in (False, True):
        got = mg.medusa_rope(to_dev(q), None if k is None else to_dev(k), dev_ints(pos), spec, inverse=inverse)
        assert (got[1] is None) == (k is None)
        for g, x in zip(got, (q, k)):
            if x is None:
                continue
            want = ref.rope(x, pos, freq, inter, 1.25, inverse)
            # a frequency's own rounding (2^-53 relative) at these positions
            slack = 2.0 ** -53 * 4 * 2.0 ** 16 * 1.25 * np.abs(ref.f64(x)).max()
            assert np.all(np.abs(host64(g) - want) <= bound(x, want, c["r"], inter, 1.25, c["dtype"]) + slack * (np.arange(c["d"]) < c["r"]))


APPENDS = [
    dict(dtype="bf16", nl=1, hq=0, hkv=1, d=16, page=16, prefix=[3, 0, 40], chunk=[700, 1, 603]),
    dict(dtype="f32", nl=2, hq=1, hkv=1, d=8, page=7, prefix=[0, 11], chunk=[330, 325]),
    dict(dtype="bf16", nl=2, hq=2, hkv=1, d=64, page=24, prefix=[5] * 40, chunk=[17, 0, 31, 18] * 10),
    dict(dtype="f32", nl=3, hq=0, hkv=3, d=16, page=32, prefix=[1, 2], chunk=[300, 151]),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("c", APPENDS, ids=lambda c: f"{c['dtype']}-nl{c['nl']}-{c['hq']}+{c['hkv']}-d{c['d']}-B{len(c['chunk'])}")
def test_append_of_several_tokens_a_cta(mg, c, inter):
    rng = np.random.default_rng(c["d"] + inter)
    kp, vp, table = pool(rng, [p + n for p, n in zip(c["prefix"], c["chunk"])], nl=c["nl"], page=c["page"], hkv=c["hkv"], d=c["d"], dtype=c["dtype"])
    q0 = starts(c["chunk"])
    T = int(q0[-1]) + 5  # five tokens behind the last sequence
    k, v = (values(rng, (c["nl"], T, c["hkv"], c["d"]), c["dtype"]) for _ in range(2))
    q = values(rng, (c["nl"], T, c["hq"], c["d"]), c["dtype"]) if c["hq"] else None
    dk, dv = to_dev(kp), to_dev(vp)
    spec = mg.RopeSpec(c["d"], interleaved=inter, base=1000.0)
    f = ref.rope_frequencies(c["d"], 1000.0)
    out = None if q is None else torch.full(q.shape, 7.0, dtype=dk.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mg.medusa_paged_append(to_dev(k), to_dev(v), dk, dv, dev_ints(table), dev_ints(q0), dev_ints(c["prefix"]), q=None if q is None else to_dev(q),
                           rope=spec, q_out=out, d_status=st)
    assert mg.medusa_status_check(st) == 0
    k2, v2 = ref.paged_append(k, v, kp, vp, table, q0, c["prefix"], lambda x, pos: ref.rope(x, pos, f, inter))
    assert np.array_equal(host64(dv), v2, equal_nan=True)
    kept = ref.f64(kp).reshape(c["nl"], -1, c["hkv"], c["d"])
    got, want = (x.reshape(kept.shape) for x in (host64(dk), k2))
    entered = np.zeros(kept.shape[1], bool)
    for b, L in enumerate(c["prefix"]):
        a, e = q0[b], q0[b + 1]
        at = ref.rows_of(table, b, L, e - a, c["page"])
        entered[at] = True
        assert np.all(np.abs(got[:, at] - want[:, at]) <= bound(k[:, a:e], want[:, at], c["d"], inter, 1.0, c["dtype"]))
        if q is not None:
            w = ref.rope(q[:, a:e], np.arange(L, L + e - a), f, inter)
            assert np.all(np.abs(host64(out)[:, a:e] - w) <= bound(q[:, a:e], w, c["d"], inter, 1.0, c["dtype"]))
    assert np.array_equal(got[:, ~entered], kept[:, ~entered], equal_nan=True)
    if q is not None:
        assert torch.all(out[:, T - 5:] == 7.0)
