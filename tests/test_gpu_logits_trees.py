"""medusa_logits_process where a tree's parents are bad: what a node is told of its path, against the oracle (bounds: tests/verify.py)."""
import numpy as np
import pytest

from oracle import verify as ov
from tests.helpers import to_dev
from tests.verify import U, dev_words, value

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PARENT = [-1, 0, 0, 1, 1, 2, 3, 3, 5, 6, 8]  # 8 and 10 are behind 5


def paths():
    p = [[]]
    for n in range(1, len(PARENT)):
        p.append(p[PARENT[n]] + [sum(1 for m in range(1, n) if PARENT[m] == PARENT[n])])
    return p[1:]


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("V", [64, 67, 2100])  # four logits at a time, one, several chunks
@pytest.mark.parametrize("node,parent", [(5, 5), (5, 200), (5, -1), (5, -7), (0, 0), (0, 3), (10, 11)])
def test_a_bad_parent_ends_the_path_there(mg, node, parent, V, in_place):
    rng = np.random.default_rng(V + node)
    B, N = 2, len(PARENT)
    z = (rng.standard_normal((B, N, V)) * 3).astype(np.float32)
    rules = dict(counts=rng.integers(0, 3, (B, V)).astype(np.int32), repetition=np.float32([1.5, 1.25]), frequency=np.float32([0.5, -0.75]),
                 presence=np.float32([0.25, 1.0]), bias=rng.standard_normal(V).astype(np.float32))
    mask = ov.words_of(rng.random((2, V)) < 0.7)
    rows = rng.integers(-1, 2, (B, N)).astype(np.int32)
    tokens = rng.integers(0, 9, (B, N)).astype(np.int32) * 7  # some of them again and again
    topo = mg.Topology.from_paths([list(p) for p in paths()])
    assert list(topo.parent) == PARENT
    topo = topo.upload()
    topo.buf[node] = parent
    ends = list(PARENT)
    ends[node] = -1
    want, size = ov.process(z, mask=mask, mask_row=rows, tokens=tokens, parent=ends, **rules)
    st, dz = torch.zeros(1, dtype=torch.int32, device="cuda"), to_dev(z)
    out = dz if in_place else torch.full((B, N, V), 77.0, device="cuda")
    got = value(mg.medusa_logits_process(dz, mask=dev_words(mask), mask_row=to_dev(rows), tokens=to_dev(tokens), topo=topo, out=out, d_status=st,
                                         **{k: to_dev(v) for k, v in rules.items()}))
    assert mg.medusa_status_check(st) == 4  # BAD_TOPOLOGY
    ok = np.isfinite(want)
    np.testing.assert_array_equal(got[~ok], want[~ok])
    assert np.all(np.abs(got[ok] - want[ok]) <= 6 * U * size[ok])
