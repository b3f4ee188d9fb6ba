"""The output end of a verify pass as a server runs it: prompts counted, logits of the tree's nodes from an output head
in 4 bits, penalties, biases and grammar masks, acceptance, the accepted tokens counted; step after step, eager and captured."""
import numpy as np
import pytest

import oracle
import workloads as wl
from oracle import topology as otopo
from oracle import verify as ov
from tests.helpers import to_dev, to_host
from tests.verify import bf16, check_linear, dev_matrix, dev_words, matrix, value

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

V, K, B, D1 = 1000, 512, 3, 5
RULES = dict(repetition=[1.3, 1.0, 1.8], frequency=[0.4, 0.0, -0.3], presence=[0.2, 0.5, 0.0])


def step(mg):
    from medusa_head_speculative_heads_gb300.step import VerifyStep
    t = otopo.greedy(otopo.synthetic_accuracy(4, 10), 40)
    dt = mg.Topology.from_paths([list(p) for p in t.paths[1:]]).upload()
    c = wl.config("tiny", V=V, B=B)
    vs = VerifyStep(B=B, H=c["H"], V=V, K=4, topk=10, nl=1, Hq=2, Hkv=1, d=64, Lmax=64, dtype=torch.bfloat16, topology=dt, temperature=0.8, eps=0.2, delta=0.5)
    return vs, t


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("head_out", [torch.float32, torch.bfloat16])
def test_steps_in_a_row(captured, head_out):
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    vs, t = step(mg)
    N, rng = t.n_nodes, np.random.default_rng(4)
    m = matrix(rng, V, K, 128)
    dm = dev_matrix(m)
    prompt = rng.integers(-1, V, (B, 30)).astype(np.int32)
    mask = ov.words_of(rng.random((4, V)) < 0.7)
    bias = np.where(rng.random(V) < 0.05, rng.standard_normal(V) * 3, 0).astype(np.float32)
    dev = {k: torch.tensor(v, device="cuda") for k, v in RULES.items()}
    dev.update(bias=to_dev(bias), mask=dev_words(mask), counts=torch.zeros((B, V), dtype=torch.int32, device="cuda"),
               prompt_bits=torch.zeros((B, (V + 31) // 32), dtype=torch.int32, device="cuda"), mask_row=torch.zeros((B, N), dtype=torch.int32, device="cuda"))
    mg.medusa_count_tokens(to_dev(prompt), V, prompt_bits=dev["prompt_bits"])
    hidden = torch.empty((B * N, K), dtype=torch.bfloat16, device="cuda")
    steps = [dict(h=bf16(rng, B * N, K), tokens=rng.integers(0, 60, (B, N)).astype(np.int32), rows=rng.integers(-1, 4, (B, N)).astype(np.int32)) for _ in range(4)]

    def body():
        logits = mg.medusa_linear_w4(hidden, *dm, out_dtype=head_out, d_status=vs.status).view(B, N, V)
        raw = logits.clone()
        done = vs.constrain(logits, **dev)
        vs.accept(done)
        vs.count(dev["counts"])
        return raw, done

    graph = None
    counts, bits = np.zeros((B, V), np.int32), ov.count_tokens(prompt, V, None, np.zeros((B, (V + 31) // 32), np.uint32))[1]
    for s in steps:
        hidden.copy_(to_dev(s["h"]))
        vs.tokens.copy_(to_dev(s["tokens"]))
        dev["mask_row"].copy_(to_dev(s["rows"]))
        if not captured:
            raw, done = body()
        else:
            if graph is None:
                kept = dev["counts"].clone()
                body()  # one-time set-up
                dev["counts"].copy_(kept)
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    raw, done = body()
            graph.replay()
        torch.cuda.synchronize()
        assert vs.check() == 0
        check_linear(raw.view(B * N, V), s["h"], m, "f32" if head_out is torch.float32 else "bf16")
        want, size = ov.process(value(raw), counts, bits, **{k: np.float32(v) for k, v in RULES.items()}, bias=bias, mask=mask, mask_row=s["rows"],
                                tokens=s["tokens"], parent=t.parent)
        got = value(done)
        ok = np.isfinite(want)
        assert np.array_equal(got[~ok], want[~ok]) and np.all(np.abs(got - want)[ok] <= 6 * 2.0 ** -24 * size[ok])
        al, pn = to_host(vs.accept_len), to_host(vs.path_nodes)
        ref = oracle.typical_accept(to_host(done), s["tokens"], t.parent, 0.8, 0.2, 0.5, Dmax=t.max_depth)
        assert np.array_equal(al, ref["accept_len"]) and np.array_equal(pn, ref["path_nodes"]) and np.array_equal(to_host(vs.next_tok), ref["next_tok"])
        counts = ov.count_accepted(counts, s["tokens"], pn, al)
        np.testing.assert_array_equal(to_host(dev["counts"]), counts)
    assert counts.sum() > 4 * B  # more than the roots were accepted
