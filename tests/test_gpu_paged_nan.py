"""Queries that are not finite: their rows are NaN however the work was divided, the other rows
keep their bits, and a row that sees no key is zeros whatever its query holds."""
import numpy as np
import pytest

from oracle import paged as ref
from tests.helpers import bf16_to_f64, to_dev, to_host
from tests.paged import dev_ints, pool, starts, values

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


# one tile and no merge; items that many CTAs share, in slots of 16, 64 and 256 rows; several layers
CASES = [
    dict(dtype="bf16", nl=1, hq=4, hkv=2, d=64, page=16, prefix=[0, 3, 40], chunk=[1, 1, 1]),
    dict(dtype="bf16", nl=1, hq=4, hkv=2, d=128, page=16, prefix=[5000, 3000], chunk=[1, 2]),
    dict(dtype="bf16", nl=2, hq=4, hkv=1, d=128, page=32, prefix=[3, 700], chunk=[150, 41]),
    dict(dtype="bf16", nl=1, hq=2, hkv=1, d=64, page=16, prefix=[0], chunk=[600]),
    dict(dtype="bf16", nl=1, hq=2, hkv=1, d=192, page=16, prefix=[0, 900], chunk=[9, 1]),
    dict(dtype="f32", nl=1, hq=4, hkv=2, d=64, page=16, prefix=[0, 1], chunk=[1, 1]),
    dict(dtype="f32", nl=1, hq=4, hkv=2, d=64, page=16, prefix=[2500], chunk=[2]),
    dict(dtype="f32", nl=1, hq=4, hkv=1, d=128, page=24, prefix=[300, 0], chunk=[90, 20]),
]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf], ids=str)
@pytest.mark.parametrize("c", CASES, ids=lambda c: f"{c['dtype']}-d{c['d']}-{max(c['prefix'])}-{max(c['chunk'])}")
def test_chunk(mg, c, bad):
    rng = np.random.default_rng(c["d"] + max(c["chunk"]))
    kp, vp, table = pool(rng, [p + n for p, n in zip(c["prefix"], c["chunk"])], nl=c["nl"], page=c["page"], hkv=c["hkv"], d=c["d"], dtype=c["dtype"])
    q0 = starts(c["chunk"])
    T = int(q0[-1])
    q = to_dev(values(rng, (c["nl"], T, c["hq"], c["d"]), c["dtype"]))
    hit = rng.random((c["nl"], T, c["hq"])) < 0.3
    hit.flat[0] = True
    hit.flat[1] = False
    broken = q.clone()
    broken[torch.from_numpy(hit).cuda().nonzero(as_tuple=True) + (torch.from_numpy(rng.integers(0, c["d"], hit.sum())).cuda(),)] = float(bad)
    args = (to_dev(kp), to_dev(vp), dev_ints(table), dev_ints(q0), dev_ints(c["prefix"]))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    clean, lse = mg.medusa_paged_attention(q, *args, want_lse=True, d_status=st)
    got, lse2 = mg.medusa_paged_attention(broken, *args, want_lse=True, d_status=st)
    assert mg.medusa_status_check(st) == 0
    at = torch.from_numpy(hit).cuda()
    assert torch.all(torch.isnan(got[at])) and not torch.any(torch.isfinite(lse2[at]))
    assert torch.equal(got[~at], clean[~at]) and torch.equal(lse2[~at], lse[~at])
    want, _, _ = ref.paged_attention(to_host(broken), kp, vp, table, q0, c["prefix"])
    assert np.array_equal(np.isnan(want), np.isnan(host64(got)))


@pytest.mark.parametrize("c", [dict(dtype="bf16", N=64, d=128, prefix=[0, 200]), dict(dtype="bf16", N=200, d=64, prefix=[0, 700]),
                               dict(dtype="f32", N=40, d=64, prefix=[0, 300])], ids=lambda c: f"{c['dtype']}-N{c['N']}")
def test_tree(mg, c):
    rng = np.random.default_rng(c["N"])
    N, d = c["N"], c["d"]
    kp, vp, table = pool(rng, c["prefix"], nl=1, page=16, hkv=2, d=d, dtype=c["dtype"])
    q, kt, vt = (to_dev(values(rng, (1, 2, N, h, d), c["dtype"])) for h in (4, 2, 2))
    seen = np.tril(rng.random((N, N)) < 0.2)
    seen[np.arange(N), np.arange(N)] = True
    seen[5] = seen[33] = False
    w = np.zeros((N, (N + 31) // 32), np.uint32)
    for i, j in zip(*np.nonzero(seen)):
        w[i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    if N % 32:
        w[5, -1] |= np.uint32(1) << np.uint32(N % 32)  # a bit of no node
    broken = q.clone()
    broken[0, :, 5, 0, 3], broken[0, :, 7, 1, 0], broken[0, :, 33, 3, 9] = float("nan"), float("nan"), float("inf")
    args = (to_dev(kp), to_dev(vp), dev_ints(table), kt, vt, dev_ints(w.view(np.int32)), dev_ints(c["prefix"]))
    clean, _ = mg.medusa_paged_tree_attention(q, *args)
    got, lse = mg.medusa_paged_tree_attention(broken, *args, want_lse=True)
    # rows 5 and 33 see no tree node: nothing at all in the first sequence, the prefix in the second
    assert torch.all(got[0, 0, [5, 33]] == 0) and torch.all(torch.isneginf(lse[0, 0, [5, 33]]))
    bad = torch.zeros(got.shape[:-1], dtype=torch.bool, device="cuda")
    bad[0, 1, 5, 0] = bad[0, :, 7, 1] = bad[0, 1, 33, 3] = True
    assert torch.all(torch.isnan(got[bad])) and not torch.any(torch.isfinite(lse[bad]))
    assert torch.equal(got[~bad], clean[~bad])
