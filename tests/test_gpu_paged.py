"""The paged-cache calls against their float64 definitions (oracle/paged.py);
the error bounds are derived in tests/paged.py."""
import numpy as np
import pytest

import oracle
from oracle import paged as ref
from oracle import topology as otopo
from tests.helpers import bf16_to_f64, to_dev, to_host
from tests.paged import HALF, U, attention_bound, dev_ints, lse_bound, pool, starts, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BAD_INDEX, OVERFLOW, BAD_LENGTH = 1, 2, 5


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


def host64(t):
    a = to_host(t)
    return bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotation

ROPES = [
    # 16-byte vectors; 8 (d 80, half of it turned), 4 and 2 bytes; fp32 16 and 8 bytes
    dict(dtype="bf16", nl=2, T=37, hq=8, hkv=2, d=128, r=128),
    dict(dtype="bf16", nl=1, T=1, hq=3, hkv=1, d=80, r=40),
    dict(dtype="bf16", nl=1, T=5, hq=2, hkv=2, d=36, r=36),
    dict(dtype="bf16", nl=3, T=2, hq=1, hkv=1, d=6, r=2),
    dict(dtype="f32", nl=1, T=300, hq=4, hkv=4, d=64, r=32),
    dict(dtype="f32", nl=2, T=9, hq=7, hkv=1, d=256, r=256),
    dict(dtype="f32", nl=1, T=3, hq=1, hkv=1, d=10, r=10),
]
SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(base=500000.0, scaling="bands", factor=8.0, original_len=8192),
            dict(scaling="ramp", factor=16.0, high=32.0, original_len=4096)]


def turned_bound(x, want, r, inter, m, dtype):
    y = np.abs(ref.f64(x))
    h = r // 2
    i0, i1 = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, h), slice(h, r))
    b = np.zeros_like(y)
    b[..., i0] = b[..., i1] = 8 * U * abs(m) * (y[..., i0] + y[..., i1])
    b[..., :r] += HALF[dtype] * np.abs(want[..., :r]) + 1e-38
    return b


@pytest.mark.parametrize("scale", SCALINGS, ids=lambda s: s.get("scaling", "none"))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("c", ROPES, ids=lambda c: f"{c['dtype']}-d{c['d']}-r{c['r']}")
def test_rotation(mg, c, inter, scale):
    rng = np.random.default_rng(c["d"] + inter)
    q, k = (values(rng, (c["nl"], c["T"], h, c["d"]), c["dtype"]) for h in (c["hq"], c["hkv"]))
    pos = rng.integers(-5, 1 << 20, c["T"]).astype(np.int32)
    pos[0] = 2 ** 31 - 1 if c["T"] > 8 else 0
    m = 1.25
    spec = mg.RopeSpec(c["r"], interleaved=inter, magnitude=m, **scale)
    freq = ref.rope_frequencies(c["r"], **scale)
    for inverse in (False, True):
        got = mg.medusa_rope(to_dev(q), to_dev(k), dev_ints(pos), spec, inverse=inverse)
        for g, x in zip(got, (q, k)):
            # at 2^31 a frequency's own rounding (2^-53 relative) is 2.4e-7 of a radian or less
            want = ref.rope(x, pos, freq, inter, m, inverse)
            slack = 2.0 ** -53 * 4 * np.abs(pos.astype(np.float64))[:, None, None] * m * np.abs(ref.f64(x)).max()
            assert np.all(np.abs(host64(g) - want) <= turned_bound(x, want, c["r"], inter, m, c["dtype"]) + slack * (np.arange(c["d"]) < c["r"]))


def test_rotation_of_slices_in_place_and_without_k(mg):
    rng = np.random.default_rng(3)
    qkv = values(rng, (2, 11, 6, 64), "bf16")
    pos = dev_ints(np.arange(100, 111))
    spec = mg.RopeSpec(64)
    d = to_dev(qkv)
    q, k = d[:, :, :4], d[:, :, 4:5]
    qo, ko = mg.medusa_rope(q, k, pos, spec)
    dense = q.contiguous()
    assert torch.equal(mg.medusa_rope(dense, None, pos, spec, q_out=dense)[0], qo) and dense.data_ptr() != qo.data_ptr()
    assert np.array_equal(to_host(d), qkv)
    back = mg.medusa_rope(qo, ko, pos, spec, inverse=True)
    assert np.max(np.abs(host64(back[1]) - bf16_to_f64(np.ascontiguousarray(qkv[:, :, 4:5])))) < 2 ** -8 * 2 * 4.5
    # the same rotation as the tree's own call
    a, b = to_dev(np.ascontiguousarray(qkv[:, :, :4]).reshape(2, 1, 11, 4, 64)), to_dev(np.ascontiguousarray(qkv[:, :, 4:5]).reshape(2, 1, 11, 1, 64))
    mg.medusa_tree_rope(a, b, pos.view(1, 11))
    assert np.max(np.abs(host64(a.view(2, 11, 4, 64)) - host64(qo))) <= 2 ** -7 * 4.5


def test_the_inverse_is_the_gradient(mg):
    """Of f(x) = sum w rope(x): against differences (f is linear: a difference quotient
    is exact but for rounding) and the transposed product."""
    rng = np.random.default_rng(4)
    for inter in (False, True):
        spec = mg.RopeSpec(8, interleaved=inter, magnitude=1.5)
        pos = dev_ints([3, 70000])
        x, w = values(rng, (1, 2, 1, 12), "f32"), values(rng, (1, 2, 1, 12), "f32")
        grad = host64(mg.medusa_rope(to_dev(w), None, pos, spec, inverse=True)[0])
        base = host64(mg.medusa_rope(to_dev(x), None, pos, spec)[0])
        assert abs((base * w).sum() - (grad * x).sum()) < 64 * U * 1.5 * np.abs(w).sum() * np.abs(x).max()
        for t, e in ((0, 0), (0, 5), (1, 3), (1, 11)):
            y = x.copy()
            y[0, t, 0, e] += 2.0
            diff = ((host64(mg.medusa_rope(to_dev(y), None, pos, spec)[0]) - base) * w).sum() / 2.0
            assert abs(diff - grad[0, t, 0, e]) < 64 * U * 1.5 * np.abs(w).sum() * np.abs(y).max()


# ------------------------------------------------------------------ append

APPENDS = [
    dict(dtype="bf16", nl=2, hq=8, hkv=2, d=128, page=16, prefix=[0, 31, 5, 16], chunk=[1, 2, 0, 40]),
    dict(dtype="bf16", nl=1, hq=4, hkv=4, d=64, page=24, prefix=[23], chunk=[1]),
    dict(dtype="f32", nl=2, hq=3, hkv=1, d=80, page=1, prefix=[2, 0], chunk=[7, 3]),
    dict(dtype="f32", nl=1, hq=2, hkv=2, d=6, page=5, prefix=[4] * 70, chunk=[1, 0, 3, 2, 0] * 14),
]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("c", APPENDS, ids=lambda c: f"{c['dtype']}-d{c['d']}-p{c['page']}-B{len(c['chunk'])}")
def test_append(mg, c, fused):
    rng = np.random.default_rng(c["d"])
    kp, vp, table = pool(rng, [p + n for p, n in zip(c["prefix"], c["chunk"])], nl=c["nl"], page=c["page"], hkv=c["hkv"], d=c["d"], dtype=c["dtype"])
    q0 = starts(c["chunk"])
    T, behind = int(q0[-1]), 3  # three tokens behind the last sequence
    qkv = values(rng, (c["nl"], T + behind, c["hq"] + 2 * c["hkv"], c["d"]), c["dtype"])
    q, k, v = (np.ascontiguousarray(x) for x in np.split(qkv, [c["hq"], c["hq"] + c["hkv"]], 2))
    dk, dv = to_dev(kp), to_dev(vp)
    spec = mg.RopeSpec(c["d"] // 2 // 2 * 2, interleaved=fused, base=1000.0)
    f = ref.rope_frequencies(spec.rotary_dim, 1000.0)
    out = torch.full(q.shape, 7.0, dtype=dk.dtype, device="cuda")
    if fused:
        d = to_dev(qkv)
        args = dict(k=d[:, :, c["hq"]:c["hq"] + c["hkv"]], v=d[:, :, c["hq"] + c["hkv"]:], q=d[:, :, :c["hq"]])
    else:
        args = dict(k=to_dev(k), v=to_dev(v), q=to_dev(q))
    st = status()
    got = mg.medusa_paged_append(k_pages=dk, v_pages=dv, page_table=dev_ints(table), q_start=dev_ints(q0), prefix_len=dev_ints(c["prefix"]),
                                 rope=spec, q_out=out, d_status=st, **args)
    assert got is out and mg.medusa_status_check(st) == 0
    turn = lambda x, pos: ref.rope(x, pos, f, fused)  # noqa: E731
    k2, v2 = ref.paged_append(k, v, kp, vp, table, q0, c["prefix"], turn)
    assert np.array_equal(host64(dv), v2, equal_nan=True)
    g = host64(dk)
    assert np.array_equal(np.isnan(g), np.isnan(k2))
    assert np.nanmax(np.abs(g - k2)) <= 8 * U * 2 * 5.5 + HALF[c["dtype"]] * 5.5 * 1.5
    old = ~np.any(np.where(np.isnan(ref.f64(vp)) & np.isnan(v2), False, ref.f64(vp) != v2), (0, 3, 4))
    assert np.array_equal(g[:, old], ref.f64(kp)[:, old], equal_nan=True)  # rows of no token
    go = host64(out)
    assert np.all(go[:, T:] == 7.0)
    for b, L in enumerate(c["prefix"]):
        a, e = q0[b], q0[b + 1]
        want = ref.rope(q[:, a:e], np.arange(L, L + e - a), f, fused)
        assert np.all(np.abs(go[:, a:e] - want) <= turned_bound(q[:, a:e], want, spec.rotary_dim, fused, 1.0, c["dtype"]))


def test_append_at_given_positions_without_rotation_and_without_q(mg):
    rng = np.random.default_rng(8)
    kp, vp, table = pool(rng, [10], nl=1, page=8, hkv=2, d=32, dtype="f32")
    k, v = values(rng, (1, 4, 2, 32), "f32"), values(rng, (1, 4, 2, 32), "f32")
    for pos, spec in ((None, None), ([9, 9, 2, 70], mg.RopeSpec(32))):
        dk, dv = to_dev(kp), to_dev(vp)
        assert mg.medusa_paged_append(to_dev(k), to_dev(v), dk, dv, dev_ints(table), dev_ints([0, 4]), dev_ints([6]),
                                      pos=None if pos is None else dev_ints(pos), rope=spec) is None
        turn = (lambda x, _: ref.f64(x)) if spec is None else (lambda x, _: ref.rope(x, pos, ref.rope_frequencies(32)))
        k2, v2 = ref.paged_append(k, v, kp, vp, table, [0, 4], [6], turn)
        assert np.array_equal(host64(dv), v2, equal_nan=True)
        np.testing.assert_allclose(host64(dk), k2, rtol=0, atol=8 * U * 2 * 5.5)


def test_append_reports_what_it_cannot_enter(mg):
    """Sequences that would overflow, lie on a page that does not exist or have a bad
    length write nothing to the cache; their neighbours do."""
    rng = np.random.default_rng(9)
    kp, vp, table = pool(rng, [16, 8, 8], nl=1, page=8, hkv=1, d=16, dtype="bf16")
    n_pages = kp.shape[1]
    k = values(rng, (1, 6, 1, 16), "bf16")
    # (page table of sequence 1, prefix lengths, starts) -> code, sequences entered
    cases = [([table[1, 0], -1], [0, 4, 0], [0, 2, 4, 6], 0, (0, 1, 2)),
             ([n_pages, -1], [0, 4, 0], [0, 2, 4, 6], BAD_INDEX, (0, 2)),
             ([-7, -1], [0, 4, 0], [0, 2, 4, 6], BAD_INDEX, (0, 2)),
             ([table[1, 0], -1], [0, 15, 0], [0, 2, 4, 6], OVERFLOW, (0, 2)),
             ([table[1, 0], -1], [0, -1, 0], [0, 2, 4, 6], BAD_LENGTH, (0, 2)),
             ([table[1, 0], -1], [0, 1000, 0], [0, 2, 4, 6], BAD_LENGTH, (0, 2)),
             ([table[1, 0], -1], [0, 4, 0], [0, 2, 4, 9], BAD_LENGTH, (0, 1))]
    for row, prefix, q0, code, entered in cases:
        t = table.copy()
        t[1] = row
        dk, dv, st = to_dev(kp), to_dev(vp), status()
        mg.medusa_paged_append(to_dev(k), to_dev(k), dk, dv, dev_ints(t), dev_ints(q0), dev_ints(prefix), d_status=st)
        assert mg.medusa_status_check(st) == code, (row, prefix, q0)
        want = kp.copy()
        for b in entered:
            at = ref.rows_of(t, b, prefix[b], 2, 8)
            want.reshape(1, -1, 1, 16)[:, at] = k[:, q0[b]:q0[b] + 2]
        assert np.array_equal(to_host(dk), want)


# ------------------------------------------------------------------ chunk attention

def attend(mg, q, kp, vp, table, q0, prefix, **kw):
    out, lse = mg.medusa_paged_attention(to_dev(q), to_dev(kp), to_dev(vp), dev_ints(table), dev_ints(q0), dev_ints(prefix), want_lse=True, **kw)
    return out, lse


def check_attention(out, lse, want, q, kp, dtype, scale, n, tensor_cores):
    o, z, mag = want
    k64 = ref.f64(kp)
    k_norm = np.sqrt(np.nanmax(np.nansum(k64 * k64, -1)))
    g, gl = host64(out), host64(lse)
    live = ~np.isnan(z)
    d = q.shape[-1]
    bound = attention_bound(q, k_norm, d, scale, n, mag, o, dtype, tensor_cores)
    err = np.abs(g - o)[live]
    assert np.all(err <= bound[live]), float(np.max(err / bound[live]))
    zero = live & np.isneginf(z)
    assert np.array_equal(gl[zero], z[zero]) and np.all(g[zero] == 0)
    some = live & ~zero
    assert np.all(np.abs(gl[some] - z[some]) <= lse_bound(q, k_norm, d, scale, n, np.where(some, z, 0))[some])
    if some.any():  # roundings do not add up in one direction: the 2-norm is far inside the bound
        rel = np.linalg.norm((g - o)[some]) / np.linalg.norm(o[some])
        assert rel <= (2.0 ** -8 if dtype == "bf16" else 2e-6), rel


ATTN = [
    # single tokens; prefix 0 and 1; pages that end inside a tile
    dict(dtype="bf16", nl=1, hq=4, hkv=4, d=128, page=16, prefix=[0, 1, 130, 127, 128], chunk=[1, 1, 1, 1, 1]),
    dict(dtype="bf16", nl=2, hq=8, hkv=1, d=64, page=24, prefix=[0, 300], chunk=[1, 1]),
    # chunks: one row, an exact tile, odd lengths, an empty sequence between, groups of 1, 3, 7
    dict(dtype="bf16", nl=1, hq=2, hkv=2, d=128, page=32, prefix=[0, 7, 64], chunk=[128, 257, 0]),
    dict(dtype="bf16", nl=1, hq=6, hkv=2, d=128, page=64, prefix=[100, 0, 3], chunk=[65, 0, 41]),
    dict(dtype="bf16", nl=2, hq=7, hkv=1, d=64, page=8, prefix=[0, 19], chunk=[70, 33]),
    dict(dtype="bf16", nl=1, hq=16, hkv=1, d=96, page=128, prefix=[300, 0], chunk=[9, 20]),
    dict(dtype="bf16", nl=1, hq=130, hkv=1, d=32, page=16, prefix=[3], chunk=[2]),
    dict(dtype="bf16", nl=1, hq=64, hkv=1, d=40, page=256, prefix=[513], chunk=[5]),
    # long: every item shared by several CTAs
    dict(dtype="bf16", nl=1, hq=4, hkv=1, d=128, page=64, prefix=[6000], chunk=[1]),
    dict(dtype="bf16", nl=1, hq=2, hkv=1, d=128, page=16, prefix=[2111], chunk=[300]),
    # shapes of the CUDA-core kernel: wide heads, a page of no multiple of 8, fp32
    dict(dtype="bf16", nl=1, hq=4, hkv=2, d=256, page=16, prefix=[70, 0], chunk=[3, 20]),
    dict(dtype="bf16", nl=1, hq=4, hkv=2, d=64, page=5, prefix=[33, 0], chunk=[1, 9]),
    dict(dtype="f32", nl=1, hq=4, hkv=2, d=64, page=16, prefix=[0, 129, 5], chunk=[1, 1, 1]),
    dict(dtype="f32", nl=2, hq=6, hkv=2, d=128, page=24, prefix=[0, 65], chunk=[67, 130]),
    dict(dtype="f32", nl=1, hq=2, hkv=1, d=36, page=1, prefix=[10], chunk=[17]),
    dict(dtype="f32", nl=1, hq=8, hkv=1, d=256, page=32, prefix=[1500], chunk=[2]),
    dict(dtype="f32", nl=1, hq=80, hkv=1, d=64, page=16, prefix=[200], chunk=[3]),
]


def _tc(c):
    return c["dtype"] == "bf16" and c["d"] <= 128 and c["d"] % 8 == 0 and c["page"] % 8 == 0 and c["hq"] // c["hkv"] <= 128


@pytest.mark.parametrize("c", ATTN, ids=lambda c: f"{c['dtype']}-{c['hq']}-{c['hkv']}-d{c['d']}-p{c['page']}-{max(c['prefix'])}-{max(c['chunk'])}")
def test_chunk_attention(mg, c):
    rng = np.random.default_rng(c["d"] + c["hq"] + max(c["prefix"]))
    kp, vp, table = pool(rng, [p + n for p, n in zip(c["prefix"], c["chunk"])], nl=c["nl"], page=c["page"], hkv=c["hkv"], d=c["d"], dtype=c["dtype"])
    q0 = starts(c["chunk"])
    q = values(rng, (c["nl"], int(q0[-1]) + 2, c["hq"], c["d"]), c["dtype"])  # two tokens behind the last sequence
    want = ref.paged_attention(q, kp, vp, table, q0, c["prefix"])
    out = torch.full(q.shape, 7.0, dtype=to_dev(q[:1, :1]).dtype, device="cuda")
    lse = torch.full(q.shape[:-1], 7.0, dtype=torch.float32, device="cuda")
    st = status()
    n = mg.lib().medusa_paged_attention_workspace_size(c["nl"], q.shape[1], len(c["chunk"]), c["hq"], c["hkv"], c["d"], c["page"], int(c["dtype"] == "bf16"))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    attend(mg, q, kp, vp, table, q0, c["prefix"], out=out, lse=lse, ws=ws, d_status=st)
    assert mg.medusa_status_check(st) == 0
    check_attention(out, lse, want, q, kp, c["dtype"], c["d"] ** -0.5, max(p + m for p, m in zip(c["prefix"], c["chunk"])), _tc(c))
    assert torch.all(out[:, int(q0[-1]):] == 7.0) and torch.all(lse[:, int(q0[-1]):] == 7.0)
    again, _ = attend(mg, q, kp, vp, table, q0, c["prefix"])
    assert torch.equal(again[:, :int(q0[-1])], out[:, :int(q0[-1])])  # the same bits on every call


def test_scores_of_every_size_find_the_right_keys(mg):
    """Keys planted so that row i attends to exactly one row (scores 60 above the rest):
    a wrong page, row, head or tile cannot pass."""
    rng = np.random.default_rng(12)
    for dtype, page in (("bf16", 16), ("f32", 16)):
        d, hkv, G, prefix, chunk = 64, 2, 2, [150, 0], [70, 131]
        kp, vp, table = pool(rng, [220, 131], nl=1, page=page, hkv=hkv, d=d, dtype=dtype)
        q0 = starts(chunk)
        q = np.zeros((1, int(q0[-1]), hkv * G, d), np.float32)
        want = np.zeros(q.shape)
        kf = ref.f64(kp).reshape(-1, hkv, d)
        for b in range(2):
            for i in range(chunk[b]):
                for h in range(hkv * G):
                    j = int(rng.integers(0, prefix[b] + i + 1))
                    at = ref.rows_of(table, b, j, 1, page)[0]
                    q[0, q0[b] + i, h] = 60.0 * kf[at, h // G] / np.linalg.norm(kf[at, h // G]) * np.sqrt(d) / 3
                    want[0, q0[b] + i, h] = ref.f64(vp).reshape(-1, hkv, d)[at, h // G]
        qv = q if dtype == "f32" else __import__("workloads").to_bf16_bits(q)
        out, _ = attend(mg, qv, kp, vp, table, q0, prefix)
        o, _, _ = ref.paged_attention(qv, kp, vp, table, q0, prefix)
        assert np.max(np.abs(host64(out) - o)) <= 2.0 ** -6
        assert np.median(np.max(np.abs(host64(out) - want), -1)) <= 0.1


def test_attention_of_a_slice_equals_that_of_its_copy(mg):
    rng = np.random.default_rng(13)
    kp, vp, table = pool(rng, [40, 9], nl=2, page=8, hkv=2, d=64, dtype="bf16")
    d = to_dev(values(rng, (2, 19, 8, 64), "bf16"))
    args = (to_dev(kp), to_dev(vp), dev_ints(table), dev_ints([0, 10, 19]), dev_ints([30, 0]))
    a, la = mg.medusa_paged_attention(d[:, :, :4], *args, want_lse=True)
    b, lb = mg.medusa_paged_attention(d[:, :, :4].contiguous(), *args, want_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_reports_bad_lengths_and_pages(mg, dtype):
    rng = np.random.default_rng(14)
    kp, vp, table = pool(rng, [20, 24, 9], nl=1, page=8, hkv=1, d=64, dtype=dtype)
    q = values(rng, (1, 6, 2, 64), dtype)
    good = ref.paged_attention(q, kp, vp, table, [0, 2, 4, 6], [10, 20, 7])[0]
    cap = table.shape[1] * 8
    for prefix, q0 in (([10, -1, 7], [0, 2, 4, 6]), ([10, cap - 1, 7], [0, 2, 4, 6]), ([10, 20, 7], [0, 2, 1, 6]), ([10, 2 ** 31 - 1, 7], [0, 2, 4, 6])):
        st, out = status(), torch.full(q.shape, 7.0, dtype=to_dev(q).dtype, device="cuda")
        attend(mg, q, kp, vp, table, q0, prefix, out=out, d_status=st)
        assert mg.medusa_status_check(st) == BAD_LENGTH
        g = host64(out)
        assert np.max(np.abs(g[:, :1] - good[:, :1])) < 0.02
        if q0[2] == 4:
            assert np.all(g[:, 2:4] == 7.0) and np.max(np.abs(g[:, 4:] - good[:, 4:])) < 0.02
    # a page that does not exist counts as zero rows
    for bad in (-1, kp.shape[1], 2 ** 31 - 1, -2 ** 31):
        t = table.copy()
        t[1, 1] = bad
        k2, v2 = (np.concatenate((x, np.zeros_like(x[:, :1])), 1) for x in (kp, vp))
        t2 = t.copy()
        t2[1, 1] = kp.shape[1]
        want = ref.paged_attention(q, k2, v2, t2, [0, 2, 4, 6], [10, 20, 7])[0]
        st = status()
        out, _ = attend(mg, q, kp, vp, t, [0, 2, 4, 6], [10, 20, 7], d_status=st)
        assert mg.medusa_status_check(st) == BAD_INDEX
        assert np.max(np.abs(host64(out) - want)) < 0.02


def test_offsets_past_32_bits(mg):
    """A pool of more than 2^32 bytes and 2^31 elements: the sequence lies at its end."""
    page, hkv, d, nl = 64, 8, 128, 2
    n_pages = (2 ** 31 // (page * hkv * d) + 40) // 2 + 1
    kp = torch.zeros((nl, n_pages, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    g = torch.Generator(device="cuda").manual_seed(5)
    tail = torch.randn((2, nl, 4, page, hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    table = dev_ints([[n_pages - 1, n_pages - 3, n_pages - 2]])
    assert kp.numel() > 2 ** 31
    q = torch.randn((nl, 5, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    kp[:, n_pages - 4:], vp[:, n_pages - 4:] = tail[0], tail[1]
    new = torch.randn((2, nl, 5, hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    mg.medusa_paged_append(new[0], new[1], kp, vp, table, dev_ints([0, 5]), dev_ints([150]))
    small = [to_host(x[:, n_pages - 4:]).copy() for x in (kp, vp)]
    t2 = np.array([[3, 1, 2]], np.int32)
    at = ref.rows_of(t2, 0, 150, 5, page)
    for x, n in zip(small, new):
        assert np.array_equal(x.reshape(nl, -1, hkv, d)[:, at], to_host(n))
    out, lse = mg.medusa_paged_attention(q, kp, vp, table, dev_ints([0, 5]), dev_ints([150]), want_lse=True)
    want = ref.paged_attention(to_host(q), *small, t2, [0, 5], [150])
    check_attention(out, lse, want, to_host(q), small[0], "bf16", d ** -0.5, 155, True)
    kt = torch.randn((2, nl, 1, 3, hkv, d), generator=g, device="cuda").to(torch.bfloat16)
    n = mg.medusa_paged_compact(kp, vp, table, kt[0], kt[1], dev_ints([[0, 2]]), dev_ints([2]), dev_ints([155]))
    at = ref.rows_of(t2, 0, 155, 2, page)
    assert n.tolist() == [157]
    for x, t in zip((kp, vp), kt):
        assert np.array_equal(to_host(x[:, n_pages - 4:]).reshape(nl, -1, hkv, d)[:, at], to_host(t[:, 0, [0, 2]]))


# ------------------------------------------------------------------ tree attention

def tree_mask(n, seed):
    rng = np.random.default_rng(seed)
    seen = np.zeros((n, n), bool)
    for i in range(n):
        if i:
            seen[i] = seen[rng.integers(max(0, i - 9), i)]
        seen[i, i] = True
    return seen


def words(seen):
    n = len(seen)
    w = np.zeros((n, (n + 31) // 32), np.uint32)
    for i, j in zip(*np.nonzero(seen)):
        w[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    return w.view(np.int32)


TREES = [
    dict(dtype="bf16", nl=2, hq=4, hkv=4, d=128, page=16, prefix=[0, 200, 128], N=64),
    dict(dtype="bf16", nl=1, hq=8, hkv=2, d=128, page=64, prefix=[1000], N=57),
    dict(dtype="bf16", nl=1, hq=3, hkv=1, d=64, page=8, prefix=[0, 77], N=256),
    dict(dtype="bf16", nl=1, hq=2, hkv=2, d=96, page=24, prefix=[5], N=1),
    dict(dtype="bf16", nl=3, hq=14, hkv=2, d=128, page=32, prefix=[33, 0], N=129),
    dict(dtype="f32", nl=1, hq=4, hkv=2, d=64, page=16, prefix=[128, 3], N=7),
    dict(dtype="f32", nl=2, hq=2, hkv=2, d=128, page=5, prefix=[0, 90], N=100),
]


@pytest.mark.parametrize("c", TREES, ids=lambda c: f"{c['dtype']}-{c['hq']}-{c['hkv']}-d{c['d']}-N{c['N']}")
def test_tree_attention_over_pages(mg, c):
    rng = np.random.default_rng(c["N"])
    B, N = len(c["prefix"]), c["N"]
    kp, vp, table = pool(rng, c["prefix"], nl=c["nl"], page=c["page"], hkv=c["hkv"], d=c["d"], dtype=c["dtype"])
    q, kt, vt = (values(rng, (c["nl"], B, N, h, c["d"]), c["dtype"]) for h in (c["hq"], c["hkv"], c["hkv"]))
    seen = tree_mask(N, 3)
    if N > 6:
        seen[5] = False  # a row that sees no tree node: nothing at all where the prefix is empty
    mask = words(seen)
    want = ref.paged_tree_attention(q, kp, vp, table, kt, vt, mask, c["prefix"])
    st = status()
    out, lse = mg.medusa_paged_tree_attention(to_dev(q), to_dev(kp), to_dev(vp), dev_ints(table), to_dev(kt), to_dev(vt), dev_ints(mask),
                                              dev_ints(c["prefix"]), want_lse=True, d_status=st)
    assert mg.medusa_status_check(st) == 0
    both = np.concatenate((np.nan_to_num(ref.f64(kp)).ravel(), ref.f64(kt).ravel())).reshape(-1, c["d"])
    check_attention(out, lse, want, q, both, c["dtype"], c["d"] ** -0.5, max(c["prefix"]) + N, _tc(c))


def test_tree_attention_agrees_with_the_contiguous_call(mg):
    rng = np.random.default_rng(21)
    t = otopo.greedy(otopo.synthetic_accuracy(4, 10), 64)
    prefix = np.array([130, 64], np.int32)
    kp, vp, table = pool(rng, prefix.tolist(), nl=2, page=16, hkv=2, d=128, dtype="bf16")
    q, kt, vt = (values(rng, (2, 2, 64, h, 128), "bf16") for h in (4, 2, 2))
    _, _, mask = otopo.tree_build(t, np.zeros(2, np.int32), np.zeros((2, t.max_depth, 10), np.int32), prefix)
    kc, vc = np.zeros((2, 2, 130, 2, 128), np.uint16), np.zeros((2, 2, 130, 2, 128), np.uint16)
    for b, L in enumerate(prefix):
        at = ref.rows_of(table, b, 0, int(L), 16)
        kc[:, b, :L], vc[:, b, :L] = kp.reshape(2, -1, 2, 128)[:, at], vp.reshape(2, -1, 2, 128)[:, at]
    a = mg.medusa_tree_attention(to_dev(q), to_dev(kc), to_dev(vc), to_dev(kt), to_dev(vt), to_dev(mask.view(np.int32)), dev_ints(prefix))
    b, _ = mg.medusa_paged_tree_attention(to_dev(q), to_dev(kp), to_dev(vp), dev_ints(table), to_dev(kt), to_dev(vt), to_dev(mask.view(np.int32)), dev_ints(prefix))
    assert np.linalg.norm(host64(a) - host64(b)) <= 2.0 ** -7 * np.linalg.norm(host64(a))


# ------------------------------------------------------------------ compaction

COMPACTS = [
    dict(dtype="bf16", nl=3, hkv=4, d=128, page=16, N=64, prefix=[0, 15, 30], acc=[1, 5, 3], Dmax=4),
    dict(dtype="f32", nl=1, hkv=1, d=6, page=3, N=20, prefix=[2, 7], acc=[17, 2], Dmax=16),
    dict(dtype="bf16", nl=1, hkv=3, d=5, page=1, N=2, prefix=[4], acc=[2], Dmax=1),
    dict(dtype="bf16", nl=1, hkv=1, d=2, page=7, N=9, prefix=list(range(40)), acc=[1, 2, 3, 4] * 10, Dmax=3),
]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("c", COMPACTS, ids=lambda c: f"{c['dtype']}-d{c['d']}-p{c['page']}-B{len(c['acc'])}")
def test_compaction(mg, c, alias):
    rng = np.random.default_rng(c["N"])
    B = len(c["acc"])
    kp, vp, table = pool(rng, [p + a for p, a in zip(c["prefix"], c["acc"])], nl=c["nl"], page=c["page"], hkv=c["hkv"], d=c["d"], dtype=c["dtype"])
    kt, vt = (values(rng, (c["nl"], B, c["N"], c["hkv"], c["d"]), c["dtype"]) for _ in range(2))
    path = np.full((B, c["Dmax"] + 1), -1, np.int32)
    for b, a in enumerate(c["acc"]):
        path[b, :a] = np.sort(rng.choice(c["N"], a, replace=False))
    k2, v2, n = ref.paged_compact(kp, vp, table, kt, vt, path, c["acc"], c["prefix"])
    dk, dv, st, pl = to_dev(kp), to_dev(vp), status(), dev_ints(c["prefix"])
    got = mg.medusa_paged_compact(dk, dv, dev_ints(table), to_dev(kt), to_dev(vt), dev_ints(path), dev_ints(c["acc"]), pl, new_len=pl if alias else None, d_status=st)
    assert mg.medusa_status_check(st) == 0 and got.tolist() == n.tolist()
    for g, w in ((dk, k2), (dv, v2)):
        assert np.array_equal(to_host(g).view(np.uint8), w.view(np.uint8))


def test_compaction_reports_what_it_cannot_enter(mg):
    rng = np.random.default_rng(31)
    kp, vp, table = pool(rng, [8, 8, 8], nl=2, page=4, hkv=1, d=8, dtype="f32")
    kt = values(rng, (2, 3, 5, 1, 8), "f32")
    n_pages = kp.shape[1]
    base = dict(path=[0, 2, 4], acc=3, prefix=4, row=table[1].tolist())
    for change, code in ((dict(acc=0), BAD_INDEX), (dict(acc=4), BAD_INDEX), (dict(path=[0, 5, 4]), BAD_INDEX), (dict(path=[0, 2, -1]), BAD_INDEX),
                         (dict(prefix=6), OVERFLOW), (dict(prefix=-1), BAD_LENGTH), (dict(prefix=2 ** 31 - 1), OVERFLOW),
                         (dict(row=[table[1, 0], n_pages]), BAD_INDEX), (dict(row=[table[1, 0], -1]), BAD_INDEX)):
        c = {**base, **change}
        t = table.copy()
        t[1] = c["row"]
        path = np.array([[0, 1, 2], c["path"], [4, -1, -1]], np.int32)
        acc, prefix = [3, c["acc"], 1], [1, c["prefix"], 0]
        k2, _, _ = ref.paged_compact(kp, kp, t[[0, 2]], kt[:, [0, 2]], kt[:, [0, 2]], path[[0, 2]], [3, 1], [1, 0])
        for alias in (False, True):
            dk, dv, st, pl = to_dev(kp), to_dev(kp), status(), dev_ints(prefix)
            n = mg.medusa_paged_compact(dk, dv, dev_ints(t), to_dev(kt), to_dev(kt), dev_ints(path), dev_ints(acc), pl, new_len=pl if alias else None, d_status=st)
            assert mg.medusa_status_check(st) == code, change
            assert n.tolist() == [4, c["prefix"], 1]
            assert np.array_equal(to_host(dk), k2, equal_nan=True) and np.array_equal(to_host(dv), k2, equal_nan=True)


# ------------------------------------------------------------------ streams and graphs

def test_another_stream_and_two_captured_graphs(mg):
    """append, attention and compaction on a side stream; two graphs with workspaces of
    their own replayed side by side, lengths changed between replays."""
    rng = np.random.default_rng(41)
    kp, vp, table = pool(rng, [300, 260], nl=1, page=16, hkv=2, d=64, dtype="bf16")
    kp, vp = np.nan_to_num(ref.f64(kp)).astype(np.float32), np.nan_to_num(ref.f64(vp)).astype(np.float32)
    kp, vp = (__import__("workloads").to_bf16_bits(x) for x in (kp, vp))
    q = [to_dev(values(rng, (1, 6, 8, 64), "bf16")) for _ in range(2)]
    new = to_dev(values(rng, (1, 6, 2, 64), "bf16"))
    pools = [(to_dev(kp), to_dev(vp)) for _ in range(2)]
    tab, q0 = dev_ints(table), dev_ints([0, 1, 6])
    lens = [dev_ints([280, 250]), dev_ints([3, 0])]
    spec = mg.RopeSpec(64)

    def both(i, ws=None, out=None, stream=None):
        qo = mg.medusa_paged_append(new, new, *pools[i], tab, q0, lens[i], q=q[i], rope=spec, stream=stream)
        return mg.medusa_paged_attention(qo, *pools[i], tab, q0, lens[i], ws=ws, out=out, stream=stream)[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = both(0, stream=s)
    s.synchronize()
    with torch.cuda.stream(s):
        assert torch.equal(both(0), side)
    s.synchronize()
    n = mg.lib().medusa_paged_attention_workspace_size(1, 6, 2, 8, 2, 64, 16, 1)
    graphs, outs = [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    keep = []
    for i in range(2):
        ws, out = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q[i])
        keep.append(ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            both(i, ws, out)
        graphs.append(g)
        outs.append(out)
    for step in range(3):
        torch.cuda.synchronize()
        for i in range(2):
            lens[i].copy_(dev_ints([[280, 250], [3, 0]][i]) + step)
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], both(i)), (step, i)
