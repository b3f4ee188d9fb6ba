"""Typical acceptance where all of a node's logits are -inf, as a grammar that leaves nothing makes them: nothing follows that node,
whatever the temperature, although its argmax is token 0 and a child may be just that token."""
import numpy as np
import pytest

import oracle
from oracle import topology as otopo
from tests.helpers import to_dev, to_host

torch = pytest.importorskip("torch")

DEAD = (0, 1, 2)  # of row b: the node that nothing may follow


def case(V):
    """Trees of 7 nodes, (0, (1, (3, 4)), (2, (5, 6))), all tokens 0 and every argmax token 0, so that all nodes would pass."""
    t = otopo.dense([2, 2], 7)
    logits = np.full((len(DEAD), t.n_nodes, V), -1.0, np.float32)
    logits[:, :, 0] = 30.0
    for b, n in enumerate(DEAD):
        logits[b, n] = -np.inf
    return t, logits, np.zeros((len(DEAD), t.n_nodes), np.int32)


# Nothing behind the root; behind node 1, so node 2 and its first child; behind node 2, so node 1 and its first child.
LEN, PATH = [1, 3, 3], [[0, -1, -1], [0, 2, 5], [0, 1, 3]]
TEMPERATURES = [0.0, 0.7]


@pytest.mark.parametrize("temperature", TEMPERATURES)
def test_oracle(temperature):
    t, logits, tokens = case(50)
    r = oracle.typical_accept(logits, tokens, t.parent, temperature, 0.1, 0.3, Dmax=t.max_depth)
    assert r["accept_len"].tolist() == LEN and r["path_nodes"].tolist() == PATH and r["next_tok"].tolist() == [0, 0, 0]
    dead = np.array(DEAD)[:, None] == np.asarray(t.parent)[None]
    assert (r["p_tok"][dead] == 0).all() and np.allclose(r["p_tok"][~dead], 1)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 50, 1024, 5001, 70000])  # one token, a chunk, several, single elements, two passes
@pytest.mark.parametrize("temperature", TEMPERATURES)
def test_nothing_follows(V, temperature):
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    t, logits, tokens = case(V)
    topo = mg.Topology.from_paths([list(p) for p in t.paths[1:]]).upload()
    al, pn, nt, pt, _ = (to_host(x) for x in mg.medusa_typical_accept(to_dev(logits), to_dev(tokens), topo, temperature, 0.1, 0.3, want_probs=True))
    r = oracle.typical_accept(logits, tokens, t.parent, temperature, 0.1, 0.3, Dmax=t.max_depth)
    assert al.tolist() == LEN == r["accept_len"].tolist() and pn.tolist() == PATH == r["path_nodes"].tolist() and nt.tolist() == [0, 0, 0]
    assert np.allclose(pt, r["p_tok"], rtol=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", TEMPERATURES)
def test_a_grammar_that_leaves_nothing(temperature):
    """Masked by medusa_logits_process, accepted, counted: the forbidden token is not counted."""
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    t, logits, tokens = case(40)
    logits[:] = -1.0
    logits[:, :, 0] = 30.0
    topo = mg.Topology.from_paths([list(p) for p in t.paths[1:]]).upload()
    mask = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    rows = np.full(tokens.shape, -1, np.int32)
    rows[np.arange(len(DEAD)), DEAD] = 0
    z = mg.medusa_logits_process(to_dev(logits), mask=mask, mask_row=to_dev(rows), tokens=to_dev(tokens), topo=topo)
    al, pn, *_ = mg.medusa_typical_accept(z, to_dev(tokens), topo, temperature, 0.1, 0.3)
    counts = mg.medusa_count_accepted(torch.zeros((len(DEAD), 40), dtype=torch.int32, device="cuda"), to_dev(tokens), pn, al)
    assert to_host(al).tolist() == LEN and to_host(pn).tolist() == PATH and to_host(counts)[:, 0].tolist() == LEN
