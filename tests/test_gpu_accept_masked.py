"""Typical acceptance over logits of which some are -inf, as a grammar's mask leaves them: against the oracle."""
import numpy as np
import pytest

import oracle
import workloads as wl
from oracle import topology as otopo
from tests.helpers import ACCEPT_BAND, TOL, check_accept, rel_err, to_dev, to_host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1024, 1023, 70000])  # one memory pass, single elements, two passes
@pytest.mark.parametrize("share", [0.3, 0.999])     # of a row that is -inf
def test_masked_logits_have_probability_zero(V, share):
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    t = otopo.dense([3, 2], 10)
    dt = mg.Topology.from_paths([list(p) for p in t.paths[1:]]).upload()
    c = wl.config("tiny", V=V, B=3, cfg_id=200 + V)
    tokens = wl.random_tokens(c, t.n_nodes)
    logits = wl.plant(c, wl.base_logits(c, t.n_nodes), tokens, t.parent, prob=0.7)
    rng = np.random.default_rng(V)
    top = logits.argmax(-1)
    logits[rng.random(logits.shape) < share] = -np.inf
    np.put_along_axis(logits, top[..., None], 9.0, -1)
    logits[1, :, : V // 2] = -np.inf  # whole chunks
    logits[1, :, V - 1] = 1.0
    T, eps, delta = 0.8, 0.09, 0.3
    al, pn, nt, pt, th = (to_host(x) for x in mg.medusa_typical_accept(to_dev(logits), to_dev(tokens), dt, T, eps, delta, want_probs=True))
    ref = oracle.typical_accept(logits, tokens, t.parent, T, eps, delta, Dmax=t.max_depth)
    assert np.isfinite(pt).all() and np.isfinite(th).all()
    assert rel_err(th[:, 1:], ref["thr"][:, 1:]) <= TOL["f32"] and rel_err(pt[:, 1:], ref["p_tok"][:, 1:]) <= TOL["f32"]
    assert np.max(np.abs((pt - th)[:, 1:] - (ref["p_tok"] - ref["thr"])[:, 1:])) < ACCEPT_BAND
    check_accept(al, pn, nt, logits, ref, t.parent, T, t.max_depth)


def test_a_node_that_nothing_may_follow():
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    t = otopo.dense([2], 3)
    dt = mg.Topology.from_paths([list(p) for p in t.paths[1:]]).upload()
    logits = torch.full((1, 3, 100), -np.inf, device="cuda")
    tokens = torch.tensor([[1, 2, 3]], dtype=torch.int32, device="cuda")
    for temperature in (0.7, 0.0):
        al, pn, nt, pt, _ = mg.medusa_typical_accept(logits, tokens, dt, temperature, 0.0, 0.3, want_probs=True)
        assert (al.tolist(), pn.tolist(), nt.tolist(), pt[:, 1:].tolist()) == ([1], [[0, -1]], [0], [[0.0, 0.0]])
