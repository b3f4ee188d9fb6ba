"""Sizes beyond what a grid of the calls around a verify pass's output has at once, and a process whose first calls are captured."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import verify as ov
from tests.helpers import to_dev, to_host
from tests.verify import host_words

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


def test_more_sequences_than_a_grid_has_rows(mg):
    B, S, V = 150001, 3, 37
    rng = np.random.default_rng(1)
    tokens = rng.integers(-1, V, (B, S)).astype(np.int32)
    counts, bits = mg.medusa_count_tokens(to_dev(tokens), V, torch.zeros((B, V), dtype=torch.int32, device="cuda"), torch.zeros((B, 2), dtype=torch.int32, device="cuda"))
    want, said = np.zeros((B, V), np.int32), tokens >= 0
    np.add.at(want, (np.nonzero(said)[0], tokens[said]), 1)
    np.testing.assert_array_equal(to_host(counts), want)
    np.testing.assert_array_equal(host_words(bits), ov.words_of(want > 0))
    path = np.tile(np.array([[0, 2]], np.int32), (B, 1))
    length = rng.integers(1, 3, B).astype(np.int32)
    tokens = np.maximum(tokens, 0)
    mg.medusa_count_accepted(counts, to_dev(tokens), to_dev(path), to_dev(length))
    want[np.arange(B), tokens[:, 0]] += 1
    np.add.at(want, (np.nonzero(length == 2)[0], tokens[length == 2, 2]), 1)
    np.testing.assert_array_equal(to_host(counts), want)


@pytest.mark.parametrize("G,symmetric", [(32, False), (64, True), (128, False)])
def test_more_groups_than_a_grid_has_warps(mg, G, symmetric):
    rng = np.random.default_rng(G)
    N, K = 1500, 128 * 40
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    q, s, z = mg.medusa_w4_quantize(to_dev(w), G, symmetric)
    eq, es, ez, _ = ov.quantize(w, G, symmetric)
    np.testing.assert_array_equal(ov.unpack(host_words(q)), eq)
    np.testing.assert_array_equal(ov.bf16_value(to_host(s)), es)
    assert (z is None) == symmetric and (symmetric or np.array_equal(to_host(z), ez))


FIRST = """
import numpy as np, torch
import medusa_head_speculative_heads_gb300 as mg
from tests.helpers import to_dev, to_host
from tests.verify import bf16, check_linear, dev_matrix, matrix
rng = np.random.default_rng(0)
sizes = [(1, 512, 512), (40, 1024, 640), (2311, 4096, 2048)]  # each kernel of the linear layer
data = [(bf16(rng, T, K), matrix(rng, N, K, 64)) for T, K, N in sizes]
dev = [(to_dev(x), dev_matrix(m)) for x, m in data]
tokens, counts = to_dev(np.array([[3, 3, 5]], np.int32)), torch.zeros((1, 9), dtype=torch.int32, device="cuda")
z, penalty, out = torch.ones((1, 1, 9), device="cuda"), torch.ones(1, device="cuda"), torch.zeros((1, 1, 9), device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ys = [mg.medusa_linear_w4(x, *m) for x, m in dev]
    mg.medusa_count_tokens(tokens, 9, counts)
    mg.medusa_logits_process(z, counts, frequency=penalty, out=out)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
for y, (x, m) in zip(ys, data):
    check_linear(y, x, m, "bf16")
assert counts.tolist() == [[0, 0, 0, 4, 0, 2, 0, 0, 0]] and out[0, 0].tolist() == [1, 1, 1, -3, 1, -1, 1, 1, 1]
print("captured")
"""


def test_first_calls_of_a_process_captured(mg):
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "captured", r.stderr[-2000:]
