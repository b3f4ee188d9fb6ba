"""A verify step over pages whose logits are made as requests want them before acceptance, and whose accepted tokens are counted:
against the oracle's calls one after the other, eager and captured."""
import numpy as np
import pytest

import oracle
import workloads as wl
from oracle import verify as ov
from tests.helpers import to_dev, to_host
from tests.paged import dev_ints, starts
from tests.step import lib_topology, make_step_inputs
from tests.verify import U, dev_words, value

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,page,masked", [("f32", 8, True), ("bf16", 16, True), ("f32", 16, False), ("bf16", 8, False)])
def test_a_step_with_rules(dtype, page, masked, captured):
    import medusa_head_speculative_heads_gb300 as mg
    from medusa_head_speculative_heads_gb300.step import PagedVerifyStep
    mg.build()
    c = wl.config("tiny", dtype=dtype, B=3, nl=2)
    inp = make_step_inputs(c)
    t, rng = inp["topo"], np.random.default_rng(6)
    B, nl, N, V, L = len(inp["rows"]), inp["q"].shape[0], t.n_nodes, c["V"], int(inp["prefix_len"][0])
    per = -(-(L + 64) // page)
    table = rng.permutation(B * per).reshape(B, per).astype(np.int32)
    vs = PagedVerifyStep(B=B, H=c["H"], V=V, K=c["K"], topk=c["topk"], nl=nl, Hq=c["Hq"], Hkv=c["Hkv"], d=c["d"],
                         dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, topology=lib_topology(mg, c), temperature=c["T"],
                         eps=c["eps"], delta=c["delta"], page_table=dev_ints(table), page_size=page)
    d = {k: to_dev(inp[k]) for k in ("h", "w1", "w2", "root_tok", "prefix_len", "q", "kt", "vt")}
    kp, vp = (torch.zeros((nl, B * per, page, c["Hkv"], c["d"]), dtype=vs.dtype, device="cuda") for _ in range(2))
    rows = [to_dev(np.ascontiguousarray(x[:, :, :L]).reshape(nl, B * L, *x.shape[3:])) for x in (inp["kc"], inp["vc"])]
    vs.chunk(torch.zeros((nl, B * L, c["Hq"], c["d"]), dtype=vs.dtype, device="cuda"), *rows, kp, vp, dev_ints(starts([L] * B)), dev_ints([0] * B))
    # what requests ask: a row that nothing may follow, one token forbidden to row 1, penalties
    counts, bits = rng.integers(0, 3, (B, V)).astype(np.int32), ov.words_of(rng.random((B, V)) < 0.2)
    rules = dict(repetition=np.float32([1.0, 1.2, 1.5]), frequency=np.float32([0.0, 0.25, 0.5]), presence=np.float32([0.0, -0.5, 0.25]))
    mask, row = ov.words_of(rng.random((2, V)) < 0.8), rng.integers(-1, 1, (B, N)).astype(np.int32)
    mask[1], row[2, 0] = 0, 1
    if not masked:
        mask, row = None, None
    given, dc = to_dev(inp["logits"].astype(np.float32)), to_dev(counts)
    dev = dict(prompt_bits=dev_words(bits), **(dict(mask=dev_words(mask), mask_row=to_dev(row)) if masked else {}), **{k: to_dev(v) for k, v in rules.items()})
    logits = torch.empty_like(given)

    def body():
        logits.copy_(given)
        vs.heads(d["h"], d["w1"], d["w2"])
        vs.tree(d["root_tok"], d["prefix_len"])
        vs.attention(d["q"], kp, vp, d["kt"], d["vt"], d["prefix_len"])
        done = vs.constrain(logits, counts=dc, **dev)
        vs.accept(done)
        vs.compact(kp, vp, d["kt"], d["vt"], d["prefix_len"])
        assert vs.count(dc) is dc
        return done

    if captured:
        body()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            done = body()
        dc.copy_(to_dev(counts))
        for x in (vs.attn_out, vs.accept_len, vs.new_len, vs.tokens, done):
            x.zero_()
        graph.replay()
    else:
        done = body()
    assert vs.check() == 0 and done.data_ptr() == logits.data_ptr()
    tokens = to_host(vs.tokens)
    want, size = ov.process(inp["logits"], counts, bits, mask=mask, mask_row=row, tokens=tokens, parent=t.parent, **rules)
    got, ok = value(done), np.isfinite(want)
    assert np.array_equal(got[~ok], want[~ok]) and np.all(np.abs(got[ok] - want[ok]) <= 6 * U * size[ok])
    ref = oracle.typical_accept(to_host(done), tokens, t.parent, c["T"], c["eps"], c["delta"], Dmax=t.max_depth)
    al, pn = to_host(vs.accept_len), to_host(vs.path_nodes)
    assert np.array_equal(al, ref["accept_len"]) and np.array_equal(pn, ref["path_nodes"]) and (not masked or al[2] == 1)
    np.testing.assert_array_equal(to_host(dc), ov.count_accepted(counts, tokens, pn, al))
    kc, vc, new_len, _ = oracle.kv_compact(inp["kc"], inp["vc"], inp["kt"], inp["vt"], pn, al, inp["prefix_len"])
    assert np.array_equal(to_host(vs.new_len), new_len)
    for pages, flat in ((kp, kc), (vp, vc)):
        held = to_host(pages).reshape(nl, -1, c["Hkv"], c["d"])
        for b in range(B):
            n = np.arange(int(new_len[b]))
            assert np.array_equal(held[:, table[b, n // page] * page + n % page], flat[:, b, :len(n)])
