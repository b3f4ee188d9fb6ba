"""medusa_logits_process where counts are below zero (tokens that a caller makes more likely): the formulas hold for them too, and a
token counts as said where c > 0 alone (bounds: tests/verify.py)."""
import numpy as np
import pytest

import workloads as wl
from oracle import topology as otopo
from oracle import verify as ov
from tests.helpers import to_dev
from tests.verify import U, dev_words, value

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,tree", [(7, 132, True), (7, 131, True), (2, 1200, False), (2, 1201, False), (6, 516, False), (6, 517, False)])
def test_counts_below_zero(N, V, tree, dtype):
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    rng = np.random.default_rng(V)
    B = 3
    z = (rng.standard_normal((B, N, V)) * 3).astype(np.float32)
    bits = wl.to_bf16_bits(z) if dtype == "bf16" else z
    z = ov.bf16_value(bits) if dtype == "bf16" else z
    counts, prompt = rng.integers(-3, 4, (B, V)).astype(np.int32), ov.words_of(rng.random((B, V)) < 0.3)
    rules = dict(repetition=np.float32([1.5, 1.0, 2.0]), frequency=np.float32([0.5, -0.75, 1.0]), presence=np.float32([0.25, 1.0, -2.0]))
    t, tokens = otopo.dense([2, 2], 7), rng.integers(0, 12, (B, N)).astype(np.int32)
    counts[:, :12] = rng.integers(-3, 1, (B, 12))  # of the paths' tokens: what they add leaves some below 1
    host, dev = {}, {}
    if tree:
        host = dict(tokens=tokens, parent=t.parent)
        dev = dict(tokens=to_dev(tokens), topo=mg.Topology.from_paths([list(p) for p in t.paths[1:]]).upload())
    for left_out in ([], ["repetition"], ["frequency"], ["presence"], ["prompt"]):
        r = {k: v for k, v in rules.items() if k not in left_out}
        p = None if "prompt" in left_out else prompt
        want, size = ov.process(z, counts, p, **r, **host)
        got = mg.medusa_logits_process(to_dev(bits), to_dev(counts), None if p is None else dev_words(p), **{k: to_dev(v) for k, v in r.items()}, **dev)
        assert np.all(np.abs(value(got) - want) <= 6 * U * size), left_out
