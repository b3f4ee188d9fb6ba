"""The paged calls as a server uses them: prompts entered and attended to, tokens
decoded one by one, a tree verified over the pages, its path compacted, and on;
and calls of many and of mixed sequences.  Bounds as in tests/paged.py."""
import numpy as np
import pytest

from oracle import paged as ref
from oracle import topology as otopo
import workloads as wl
from tests.helpers import TOL, bf16_to_f64, rel_err, to_dev, to_host
from tests.paged import attention_bound, dev_ints, lse_bound, pool, starts, values
from tests.step import lib_topology, make_step_inputs, run_gpu_step, run_oracle_step

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


def within(out, lse, want, q, kp, dtype, n, rounded_p, extra_keys=None):
    """out, lse against want = (out, lse, mag) of the definition on the same inputs."""
    o, z, mag = want
    d = q.shape[-1]
    k64 = ref.f64(kp)
    norms = [np.nanmax(np.nansum(k64 * k64, -1))]
    if extra_keys is not None:
        norms.append(np.max(np.sum(ref.f64(extra_keys) ** 2, -1)))
    k_norm = np.sqrt(max(norms))
    live = ~np.isnan(z)
    bound = attention_bound(q, k_norm, d, d ** -0.5, n, mag, o, dtype, rounded_p)
    assert np.all(np.abs(host64(out) - o)[live] <= bound[live])
    if lse is not None:
        assert np.all(np.abs(host64(lse) - z)[live] <= lse_bound(q, k_norm, d, d ** -0.5, n, np.where(live, z, 0))[live])


def paged_like(kc, page, max_pages, rng):
    """An empty pool for caches [nl, B, Lmax, Hkv, d], pages in random order."""
    nl, B, _, hkv, d = kc.shape
    n_pages = B * max_pages
    table = rng.permutation(n_pages).reshape(B, max_pages).astype(np.int32)
    nan = np.uint16(0x7FC0) if kc.dtype == np.uint16 else np.float32(np.nan)
    return np.full((nl, n_pages, page, hkv, d), nan), table


def gathered(pages, table, b, n):
    """Rows 0 .. n - 1 of sequence b: [nl, n, Hkv, d]."""
    p = to_host(pages)
    at = ref.rows_of(table, b, 0, n, p.shape[2])
    return p.reshape(p.shape[0], -1, *p.shape[3:])[:, at]


def paged_step(mg, c, inp, table, page, rope=None):
    from medusa_head_speculative_heads_gb300.step import PagedVerifyStep
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    return PagedVerifyStep(B=len(inp["rows"]), H=c["H"], V=c["V"], K=c["K"], topk=c["topk"], nl=inp["q"].shape[0], Hq=c["Hq"],
                           Hkv=c["Hkv"], d=c["d"], dtype=dtype, topology=lib_topology(mg, c), temperature=c["T"], eps=c["eps"],
                           delta=c["delta"], page_table=dev_ints(table), page_size=page, rope=rope)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,page", [("f32", 8), ("bf16", 16), ("bf16", 128)])
def test_the_step_over_pages_is_the_step_over_rows(mg, dtype, page, captured):
    """The whole verify step with the cache in pages against the contiguous one and the
    oracle's: the same tokens, decisions and cache rows, attention within bounds."""
    c = wl.config("tiny", dtype=dtype, B=3, nl=2)
    inp = make_step_inputs(c)
    want, flat = run_oracle_step(c, inp), run_gpu_step(mg, c, inp)
    rng = np.random.default_rng(5)
    B, nl, L = len(inp["rows"]), inp["q"].shape[0], int(inp["prefix_len"][0])
    empty, table = paged_like(inp["kc"], page, -(-(L + 64) // page), rng)
    vs = paged_step(mg, c, inp, table, page)
    kp, vp = to_dev(empty), to_dev(empty)
    # the prefix enters through the step itself
    rows = [to_dev(np.ascontiguousarray(x[:, :, :L]).reshape(nl, B * L, *x.shape[3:])) for x in (inp["kc"], inp["vc"])]
    zero = dev_ints([0] * B)
    vs.chunk(torch.zeros((nl, B * L, c["Hq"], c["d"]), dtype=kp.dtype, device="cuda"), *rows, kp, vp, dev_ints(starts([L] * B)), zero)
    d = {k: to_dev(inp[k]) for k in ("h", "w1", "w2", "root_tok", "prefix_len", "q", "kt", "vt", "logits")}
    args = (d["h"], d["w1"], d["w2"], d["root_tok"], d["prefix_len"], d["q"], kp, vp, d["kt"], d["vt"], d["logits"])
    if captured:
        g = vs.capture(*args)
        for t in (vs.attn_out, vs.accept_len, vs.new_len, vs.tokens):
            t.zero_()
        g.replay()
    else:
        vs.run(*args)
    assert vs.check() == 0
    assert np.array_equal(to_host(vs.tokens), flat["tokens"]) and np.array_equal(to_host(vs.pos), flat["pos"])
    assert np.array_equal(to_host(vs.accept_len), flat["accept_len"]) and np.array_equal(to_host(vs.new_len), flat["new_len"])
    assert rel_err(host64(vs.attn_out), want["attn_out"]) <= TOL[dtype]
    for b in range(B):
        n = int(flat["new_len"][b])
        assert np.array_equal(gathered(kp, table, b, n), flat["kc"][:, b, :n]) and np.array_equal(gathered(vp, table, b, n), flat["vc"][:, b, :n])


@pytest.mark.parametrize("dtype,hq,hkv,d", [("f32", 4, 2, 64), ("bf16", 8, 2, 128), ("bf16", 4, 4, 64)])
def test_prompt_decode_verify_compact_decode(mg, dtype, hq, hkv, d):
    """Ragged prompts in one call, two tokens decoded one by one, a tree turned, verified
    and compacted, one more token: every attention against its definition on what the
    cache then holds, the cache against rotations of what entered it, and the decoded
    tokens against the same tokens entered as one chunk."""
    from medusa_head_speculative_heads_gb300.step import PagedVerifyStep
    rng = np.random.default_rng(d + hq)
    nl, page, prompts = 2, 16, [37, 1, 130]
    B, rc = len(prompts), dtype == "bf16"
    t = otopo.dense([2, 2])
    N, W = t.n_nodes, (t.n_nodes + 31) // 32
    max_pages = 14
    table = rng.permutation(B * max_pages).reshape(B, max_pages).astype(np.int32)
    spec = mg.RopeSpec(d, base=500000.0)
    freq = ref.rope_frequencies(d, 500000.0)
    tt = torch.bfloat16 if rc else torch.float32
    vs = PagedVerifyStep(B=B, H=64, V=64, K=2, topk=2, nl=nl, Hq=hq, Hkv=hkv, d=d, dtype=tt, topology=mg.Topology.from_paths([list(p) for p in t.paths[1:]]),
                         temperature=0.7, eps=0.1, delta=0.3, page_table=dev_ints(table), page_size=page, rope=spec)
    nan = torch.full((nl, B * max_pages, page, hkv, d), float("nan"), dtype=tt, device="cuda")
    kp, vp, kp2, vp2 = nan.clone(), nan.clone(), nan.clone(), nan.clone()

    def tokens(n):
        qkv = to_dev(values(rng, (nl, n, hq + 2 * hkv, d), dtype))
        return qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]

    def chunk_checked(q, k, v, lens, prefix):
        q0 = starts(lens)
        out = vs.chunk(q, k, v, kp, vp, dev_ints(q0), dev_ints(prefix))
        pos = np.concatenate([np.arange(p, p + n) for p, n in zip(prefix, lens)])
        turned = mg.medusa_rope(q, None, dev_ints(pos), spec)[0]
        held = [to_host(kp), to_host(vp)]
        qh = to_host(turned)
        want = ref.paged_attention(qh, *held, table, q0, prefix)
        within(out, None, want, qh, held[0], dtype, 200, rc)
        for b in range(B):  # what entered: values as they were, keys turned at their rows
            rows = gathered(vp, table, b, prefix[b] + lens[b])[:, prefix[b]:]
            assert np.array_equal(rows, to_host(v[:, q0[b]:q0[b + 1]]))
            kw = ref.rope(to_host(k[:, q0[b]:q0[b + 1]]), np.arange(prefix[b], prefix[b] + lens[b]), freq)
            got = ref.f64(gathered(kp, table, b, prefix[b] + lens[b])[:, prefix[b]:])
            assert np.all(np.abs(got - kw) <= 8 * 2.0 ** -24 * 11 + (2.0 ** -8 if rc else 2.0 ** -24) * np.abs(kw) + 1e-30)
        return out

    lens = list(prompts)
    prompt = tokens(sum(prompts))
    chunk_checked(*prompt, prompts, [0] * B)
    one = [tokens(B) for _ in range(2)]
    outs = []
    for x in one:
        outs.append(chunk_checked(*x, [1] * B, lens))
        lens = [n + 1 for n in lens]
    # the same two tokens of each sequence as one chunk behind the same prompts
    vs.chunk(*prompt, kp2, vp2, dev_ints(starts(prompts)), dev_ints([0] * B))
    two = [torch.stack((a, b), 2).reshape(nl, 2 * B, a.shape[2], d) for a, b in zip(*one)]
    both = vs.chunk(*two, kp2, vp2, dev_ints(starts([2] * B)), dev_ints(prompts))
    assert torch.equal(kp.view(torch.int16 if rc else torch.int32), kp2.view(torch.int16 if rc else torch.int32))
    apart = torch.stack(outs, 2).reshape(both.shape)
    assert rel_err(host64(apart), host64(both)) <= TOL[dtype]

    q, kt, vt = (to_dev(values(rng, (nl, B, N, h, d), dtype)) for h in (hq, hkv, hkv))
    depth = np.array([len(p) for p in t.paths])
    bits = np.zeros((N, W), np.uint32)
    for i, p in enumerate(t.paths):
        for j, o in enumerate(t.paths):
            if list(o) == list(p)[:len(o)]:
                bits[i, j // 32] |= np.uint32(1 << (j % 32))
    vs.mask.copy_(to_dev(bits.view(np.int32)))
    vs.pos.copy_(dev_ints(np.array(lens)[:, None] + depth[None]))
    before = to_host(kt.view(nl, B * N, hkv, d))
    vs.rope(q, kt)
    kw = ref.rope(before, (np.array(lens)[:, None] + depth[None]).reshape(-1), freq).reshape(nl, B, N, hkv, d)
    assert np.all(np.abs(host64(kt) - kw) <= 8 * 2.0 ** -24 * 11 + (2.0 ** -8 if rc else 2.0 ** -24) * np.abs(kw) + 1e-30)
    vs.attention(q, kp, vp, kt, vt, dev_ints(lens))
    want = ref.paged_tree_attention(to_host(q), to_host(kp), to_host(vp), table, to_host(kt), to_host(vt), bits, lens)
    within(vs.attn_out, None, want, to_host(q), to_host(kp), dtype, 200, rc, to_host(kt))
    path, acc = np.zeros((B, vs.topo.max_depth + 1), np.int32), [1, 3, 2]
    deep = next(i for i, p in enumerate(t.paths) if len(p) == 2)
    chain = [next(i for i, o in enumerate(t.paths) if list(o) == list(t.paths[deep])[:n]) for n in range(3)]
    path[:] = chain
    vs.path_nodes.copy_(dev_ints(path))
    vs.accept_len.copy_(dev_ints(acc))
    k3, v3, n3 = ref.paged_compact(to_host(kp), to_host(vp), table, to_host(kt), to_host(vt), path, acc, lens)
    vs.compact(kp, vp, kt, vt, dev_ints(lens))
    assert np.array_equal(to_host(kp), k3, equal_nan=not rc) and np.array_equal(to_host(vp), v3, equal_nan=not rc)
    assert np.array_equal(to_host(vs.new_len), n3)
    chunk_checked(*tokens(B), [1] * B, n3.tolist())
    assert vs.check() == 0


MIXED = [
    # more sequences than a CTA has threads, some without a token
    dict(dtype="bf16", nl=1, hq=4, hkv=4, d=64, page=16, B=420, prefix=90, chunk=lambda r, b: int(r.integers(0, 2))),
    dict(dtype="f32", nl=1, hq=2, hkv=1, d=32, page=16, B=300, prefix=70, chunk=lambda r, b: int(r.integers(0, 2))),
    # many single tokens and one chunk (blocks of 64 rows), one long chunk and a few single tokens (of 256)
    dict(dtype="bf16", nl=1, hq=8, hkv=2, d=128, page=16, B=40, prefix=400, chunk=lambda r, b: 90 if b == 17 else 1),
    dict(dtype="bf16", nl=1, hq=8, hkv=8, d=128, page=64, B=6, prefix=260, chunk=lambda r, b: [1, 300, 0, 1, 5, 129][b]),
    # sequences that hold one tile of keys at most, and just more
    dict(dtype="bf16", nl=2, hq=8, hkv=2, d=64, page=64, B=70, prefix=60, chunk=lambda r, b: int(r.integers(1, 60)), cap=128),
    dict(dtype="f32", nl=1, hq=8, hkv=2, d=64, page=16, B=30, prefix=40, chunk=lambda r, b: int(r.integers(0, 25)), cap=64),
    dict(dtype="bf16", nl=1, hq=4, hkv=2, d=128, page=8, B=30, prefix=70, chunk=lambda r, b: int(r.integers(0, 60)), cap=136),
    # many blocks a CTA, and one sequence's rows over every CTA
    dict(dtype="bf16", nl=12, hq=16, hkv=4, d=64, page=8, B=9, prefix=130, chunk=lambda r, b: int(r.integers(1, 60))),
    dict(dtype="bf16", nl=1, hq=20, hkv=1, d=104, page=32, B=1, prefix=9000, chunk=lambda r, b: 14),
    dict(dtype="f32", nl=1, hq=3, hkv=1, d=96, page=7, B=1, prefix=5000, chunk=lambda r, b: 30),
]


@pytest.mark.parametrize("c", MIXED, ids=lambda c: f"{c['dtype']}-{c['hq']}-{c['hkv']}-d{c['d']}-B{c['B']}-{c['prefix']}")
def test_many_and_mixed_sequences(mg, c):
    rng = np.random.default_rng(c["B"] + c["d"])
    prefix = rng.integers(0, c["prefix"] + 1, c["B"]).tolist()
    if c["B"] == 1:
        prefix = [c["prefix"]]
    chunk = [c["chunk"](rng, b) for b in range(c["B"])]
    kp, vp, table = pool(rng, [p + n for p, n in zip(prefix, chunk)], nl=c["nl"], page=c["page"], hkv=c["hkv"], d=c["d"], dtype=c["dtype"])
    if "cap" in c:  # the table is as wide as `cap` rows need
        assert table.shape[1] * c["page"] <= c["cap"]
        table = np.pad(table, ((0, 0), (0, c["cap"] // c["page"] - table.shape[1])), constant_values=-1)
    q0 = starts(chunk)
    q = values(rng, (c["nl"], int(q0[-1]), c["hq"], c["d"]), c["dtype"])
    want = ref.paged_attention(q, kp, vp, table, q0, prefix)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(3):  # on memory of its own each time
        dev = [to_dev(x) for x in (q, kp, vp)] + [dev_ints(x) for x in (table, q0, prefix)]
        out, lse = mg.medusa_paged_attention(*dev, want_lse=True, d_status=st)
        assert mg.medusa_status_check(st) == 0
        if first is None:
            first = out.clone()
            rc = c["dtype"] == "bf16"
            within(out, lse, want, q, kp, c["dtype"], max(p + n for p, n in zip(prefix, chunk)), rc)
        assert torch.equal(out, first)
        del dev, out, lse
        torch.cuda.empty_cache()


@pytest.mark.parametrize("N,hq,hkv,d,B,nl", [(64, 4, 4, 128, 2, 10), (100, 6, 3, 64, 3, 5), (33, 8, 1, 96, 5, 3)])
def test_trees_of_many_layers(mg, N, hq, hkv, d, B, nl):
    rng = np.random.default_rng(N)
    prefix = rng.integers(0, 300, B).tolist()
    kp, vp, table = pool(rng, prefix, nl=nl, page=16, hkv=hkv, d=d, dtype="bf16")
    q, kt, vt = (values(rng, (nl, B, N, h, d), "bf16") for h in (hq, hkv, hkv))
    see = np.tril(rng.random((N, N)) < 0.3)
    bits = np.zeros((N, (N + 31) // 32), np.uint32)
    for i, j in zip(*np.nonzero(see)):
        bits[i, j // 32] |= np.uint32(1 << (j % 32))
    want = ref.paged_tree_attention(q, kp, vp, table, kt, vt, bits, prefix)
    first = None
    for _ in range(3):
        dev = [to_dev(x) for x in (q, kp, vp)] + [dev_ints(table), to_dev(kt), to_dev(vt), to_dev(bits.view(np.int32)), dev_ints(prefix)]
        out, lse = mg.medusa_paged_tree_attention(*dev, want_lse=True)
        if first is None:
            first = out.clone()
            sees = ~np.isneginf(want[1])
            bare = np.where(sees, want[1], np.nan)
            within(out, lse, (want[0], bare, want[2]), q, kp, "bf16", 300 + N, True, kt)
            assert np.all(host64(out)[~sees] == 0) and np.all(np.isneginf(host64(lse)[~sees]))
        assert torch.equal(out, first)
        del dev, out, lse
        torch.cuda.empty_cache()


def test_pipelined_steps_over_pages(mg):
    """The step under PipelinedSteps: inputs from pinned memory, results read back, the
    page table changed between steps (a captured step reads it on the device)."""
    from medusa_head_speculative_heads_gb300.step import PipelinedSteps
    c = wl.config("tiny", dtype="bf16", B=3, nl=2)
    inp = make_step_inputs(c)
    flat = run_gpu_step(mg, c, inp)
    rng = np.random.default_rng(6)
    page, L, B = 16, int(inp["prefix_len"][0]), 3
    empty, table = paged_like(inp["kc"], page, -(-(L + 64) // page), rng)
    vs = paged_step(mg, c, inp, table, page)

    def pools(t):
        out = []
        for x in (inp["kc"], inp["vc"]):
            p = empty.copy()
            for b in range(B):
                p.reshape(p.shape[0], -1, *p.shape[3:])[:, ref.rows_of(t, b, 0, L, page)] = x[:, b, :L]
            out.append(to_dev(p))
        return out

    kp, vp = pools(table)
    names = ("h", "root_tok", "prefix_len", "q", "kt", "vt", "logits")
    dev = {k: to_dev(inp[k]) for k in names}
    outs = [vs.accept_len, vs.next_tok, vs.new_len, vs.attn_out]
    hosts = [torch.empty(o.shape, dtype=o.dtype).pin_memory() for o in outs]
    resident = dict(w1=to_dev(inp["w1"]), w2=to_dev(inp["w2"]), kc=kp, vc=vp)  # the graphs hold addresses only
    ps = PipelinedSteps(vs, dev, resident, outs, hosts)
    staged, views = ps.host_staging()
    for k in names:
        views[k].copy_(dev[k])
    torch.cuda.synchronize()
    for turn in range(4):
        if turn == 2:  # other pages for every row
            table = table[:, ::-1][[1, 2, 0]].copy()
            vs.page_table.copy_(dev_ints(table))
            for p, x in zip((kp, vp), pools(table)):
                p.copy_(x)
            torch.cuda.synchronize()
        for h in hosts:
            h.zero_()
        ps.step(staged)
        torch.cuda.synchronize()
        assert np.array_equal(to_host(hosts[0]), flat["accept_len"]) and np.array_equal(to_host(hosts[2]), flat["new_len"])
        assert np.array_equal(to_host(hosts[1]), flat["next_tok"])
        assert rel_err(host64(hosts[3]), flat["attn_out"]) <= TOL["bf16"]
        for b in range(B):
            n = int(flat["new_len"][b])
            assert np.array_equal(gathered(kp, table, b, n), flat["kc"][:, b, :n])
    assert vs.check() == 0


def test_a_step_refuses_what_does_not_fit(mg):
    c = wl.config("tiny")
    inp = make_step_inputs(c)
    B = len(inp["rows"])
    with pytest.raises(ValueError, match="page_table"):
        paged_step(mg, c, inp, np.zeros((B + 1, 4), np.int32), 16)
    vs = paged_step(mg, c, inp, np.zeros((B, 40), np.int32), 16)
    with pytest.raises(ValueError, match="RopeSpec"):
        vs.rope(to_dev(inp["q"]), to_dev(inp["kt"]))


def test_the_binding_refuses_tensors_that_do_not_fit(mg):
    """Types, shapes, strides and places, each named in the error; what is not refused runs."""
    i32, bf, f32 = torch.int32, torch.bfloat16, torch.float32
    z = lambda *s, dt=bf, dev="cuda": torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
    attn = dict(q=z(2, 5, 4, 64), k_pages=z(2, 6, 16, 2, 64), v_pages=z(2, 6, 16, 2, 64), page_table=z(2, 3, dt=i32), q_start=dev_ints([0, 2, 5]), prefix_len=dev_ints([0, 4]))
    tree = dict(q=z(2, 2, 3, 4, 64), k_pages=attn["k_pages"], v_pages=attn["v_pages"], page_table=attn["page_table"], kt=z(2, 2, 3, 2, 64), vt=z(2, 2, 3, 2, 64),
                mask=z(3, 1, dt=i32), prefix_len=attn["prefix_len"])
    entry = dict(k=z(2, 5, 2, 64), v=z(2, 5, 2, 64), k_pages=attn["k_pages"], v_pages=attn["v_pages"], page_table=attn["page_table"], q_start=attn["q_start"],
                 prefix_len=attn["prefix_len"])
    pack = dict(k_pages=attn["k_pages"], v_pages=attn["v_pages"], page_table=attn["page_table"], kt=tree["kt"], vt=tree["vt"], path_nodes=z(2, 3, dt=i32),
                accept_len=dev_ints([1, 2]), prefix_len=attn["prefix_len"])
    turn = dict(q=z(2, 5, 4, 64), k=z(2, 5, 2, 64), pos=z(5, dt=i32), rope=mg.RopeSpec(64))
    calls = {mg.medusa_paged_attention: attn, mg.medusa_paged_tree_attention: tree, mg.medusa_paged_append: entry, mg.medusa_paged_compact: pack, mg.medusa_rope: turn}
    for call, args in calls.items():
        call(**args)
    bad = [(mg.medusa_paged_attention, dict(q=z(2, 5, 4, 64, dt=f32)), "k_pages"), (mg.medusa_paged_attention, dict(q=z(1, 5, 4, 64)), "q"),
           (mg.medusa_paged_attention, dict(v_pages=z(2, 6, 16, 2, 32)), "v_pages"), (mg.medusa_paged_attention, dict(k_pages=z(2, 6, 16, 64)), "k_pages"),
           (mg.medusa_paged_attention, dict(k_pages=z(2, 6, 16, 4, 64)[:, :, :, :2]), "k_pages"), (mg.medusa_paged_attention, dict(page_table=z(2, 3, dt=torch.int64)), "page_table"),
           (mg.medusa_paged_attention, dict(page_table=z(2, 3, dt=i32, dev="cpu")), "page_table"), (mg.medusa_paged_attention, dict(q_start=dev_ints([0, 5])), "q_start"),
           (mg.medusa_paged_attention, dict(prefix_len=dev_ints([0, 1, 2])), "prefix_len"), (mg.medusa_paged_attention, dict(out=z(2, 5, 4, 64, dt=f32)), "out"),
           (mg.medusa_paged_attention, dict(lse=z(2, 5, 4)), "lse"), (mg.medusa_paged_attention, dict(ws=z(8, dt=torch.uint8)), "workspace"),
           (mg.medusa_paged_attention, dict(d_status=z(1)), "d_status"), (mg.medusa_paged_attention, dict(q=z(2, 4, 5, 64).transpose(1, 2)), "q"),
           (mg.medusa_paged_tree_attention, dict(q=z(2, 2, 3, 64)), "q"), (mg.medusa_paged_tree_attention, dict(kt=z(2, 2, 4, 2, 64)), "kt"),
           (mg.medusa_paged_tree_attention, dict(mask=z(3, 2, dt=i32)), "mask"), (mg.medusa_paged_append, dict(v=z(2, 4, 2, 64)), "v"),
           (mg.medusa_paged_append, dict(q_out=z(2, 5, 4, 64)), "q_out"), (mg.medusa_paged_append, dict(pos=z(4, dt=i32)), "pos"), (mg.medusa_paged_append, dict(q=z(2, 5, 4, 32)), "q"),
           (mg.medusa_paged_compact, dict(path_nodes=z(3, 3, dt=i32)), "path_nodes"), (mg.medusa_paged_compact, dict(new_len=z(2)), "new_len"),
           (mg.medusa_paged_compact, dict(vt=z(2, 2, 3, 2, 64, dt=f32)), "vt"), (mg.medusa_rope, dict(k=None, k_out=z(2, 5, 2, 64)), "k_out"),
           (mg.medusa_rope, dict(pos=z(5)), "pos"), (mg.medusa_rope, dict(q_out=z(2, 5, 6, 64)[:, :, :4]), "q_out"), (mg.medusa_rope, dict(k=z(2, 6, 2, 64)), "k")]
    for call, change, name in bad:
        with pytest.raises(ValueError, match=f"{call.__name__}.*{name}"):
            call(**{**calls[call], **change})
    with pytest.raises(TypeError, match="float16"):
        mg.medusa_paged_attention(**{**attn, "q": z(2, 5, 4, 64, dt=torch.float16)})
    with pytest.raises(TypeError, match="prefix_len"):
        mg.medusa_paged_attention(**{**attn, "prefix_len": [0, 4]})
    with pytest.raises(mg.MedusaError):  # the library's own: 3 q heads over 2 kv heads
        mg.medusa_paged_attention(**{**attn, "q": z(2, 5, 3, 64)})
    with pytest.raises(mg.MedusaError):  # and no tokens
        mg.medusa_paged_attention(**{**attn, "k_pages": z(1, 6, 16, 2, 64), "v_pages": z(1, 6, 16, 2, 64), "q": z(1, 0, 4, 64)})
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,nl,hkv,d", [("bf16", 1, 64, 128), ("f32", 1, 64, 128), ("bf16", 3, 24, 128), ("bf16", 1, 40, 256)])
def test_pools_whose_offsets_pass_32_bits(mg, dtype, nl, hkv, d):
    """The same calls on a small pool and on one of 2.6e9 elements with the pages at its end
    (the second layer of three passes 2^31 by itself): the same bits."""
    rng = np.random.default_rng(hkv)
    tt, page, B, G, N = (torch.bfloat16 if dtype == "bf16" else torch.float32), 16, 2, 2, 9
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("two pools of up to 10 GB")
    big_pages = int(2.6e9) // (nl * page * hkv * d)
    assert nl * big_pages * page * hkv * d > 2 ** 31
    few = 10
    small_table = rng.permutation(few).reshape(B, few // B).astype(np.int32)
    big_table = small_table + np.int32(big_pages - few)
    prefix, chunk = [0, 33], [37, 3]
    q0 = starts(chunk)
    T = int(q0[-1])
    q, k, v = (to_dev(values(rng, (nl, T, h, d), dtype)) for h in (G * hkv, hkv, hkv))
    kt, vt, tq = (to_dev(values(rng, (nl, B, N, h, d), dtype)) for h in (hkv, hkv, G * hkv))
    mask = dev_ints(np.array([[(2 << i) - 1] for i in range(N)]))
    first = [to_dev(values(rng, (nl, few, page, hkv, d), dtype)) for _ in range(2)]
    spec = mg.RopeSpec(d)
    results = []
    for n_pages, table in ((few, small_table), (big_pages, big_table)):
        pools = [torch.empty((nl, n_pages, page, hkv, d), dtype=tt, device="cuda") for _ in range(2)]
        for p, f in zip(pools, first):
            p[:, n_pages - few:] = f
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        tab, lens = dev_ints(table), dev_ints(prefix)
        turned = mg.medusa_paged_append(k, v, *pools, tab, dev_ints(q0), lens, q=q, rope=spec, d_status=st)
        out, lse = mg.medusa_paged_attention(turned, *pools, tab, dev_ints(q0), lens, want_lse=True, d_status=st)
        held = dev_ints(np.add(prefix, chunk))
        tree, tree_lse = mg.medusa_paged_tree_attention(tq, *pools, tab, kt, vt, mask, held, want_lse=True, d_status=st)
        new = mg.medusa_paged_compact(*pools, tab, kt, vt, dev_ints([[0, 2, 5], [0, 1, 8]]), dev_ints([3, 2]), held, d_status=st)
        assert mg.medusa_status_check(st) == 0
        results.append([turned, out, lse, tree, tree_lse, new] + [p[:, n_pages - few:].clone() for p in pools])
        del pools
        torch.cuda.empty_cache()
    for a, b in zip(*results):
        assert torch.equal(a, b)
