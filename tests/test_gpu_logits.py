"""medusa_logits_process and the counting calls against the float64 oracle (bounds: tests/verify.py)."""
import numpy as np
import pytest

import workloads as wl
from oracle import topology as otopo
from oracle import verify as ov
from tests.helpers import to_dev, to_host
from tests.verify import U, dev_words, host_words, value

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


def upload(mg, t):
    return mg.Topology.from_paths([list(p) for p in t.paths[1:]]).upload()


def tree(n, seed=0):
    """A tree of n nodes, up to 16 deep, some of them in one long branch."""
    rng = np.random.default_rng(seed)
    paths, kids = [()], {(): 0}
    while len(paths) < n:
        p = paths[-1] if rng.random() < 0.5 else paths[rng.integers(len(paths))]
        if len(p) < 16 and kids[p] < 30:
            q = p + (kids[p],)
            kids[p] += 1
            kids[q] = 0
            paths.append(q)
    return otopo.from_paths([list(p) for p in paths[1:]]) if n > 1 else otopo.from_paths([])


def inputs(rng, B, N, V, *, dtype="f32", pad=0, penalties=True, bias="each", masks=3, topo=None, rows=True):
    z = (rng.standard_normal((B, N, V + pad)) * 3).astype(np.float32)
    bits = wl.to_bf16_bits(z) if dtype == "bf16" else z
    z = ov.bf16_value(bits) if dtype == "bf16" else z.astype(np.float64)
    host, dev = dict(logits=z[..., :V]), dict(logits=to_dev(bits)[..., :V])
    if penalties:
        host["counts"] = np.where(rng.random((B, V)) < 0.2, rng.integers(1, 9, (B, V)), 0).astype(np.int32)
        host["prompt"] = ov.words_of(rng.random((B, V)) < 0.3)
        host["repetition"] = (1 + rng.random(B)).astype(np.float32)
        host["frequency"], host["presence"] = (rng.standard_normal(B).astype(np.float32) for _ in range(2))
    if bias:
        host["bias"] = (rng.standard_normal((B, V) if bias == "each" else V) * 4).astype(np.float32)
    if masks:
        host["mask"] = ov.words_of(rng.random((masks, V)) < 0.6)
        host["mask"][0] = 0                            # leaves nothing
        host["mask"][..., -1] |= np.uint32(0xffffffff) << np.uint32((V - 1) % 32) << np.uint32(1) if V % 32 else 0  # bits behind the last token
        if rows:
            host["mask_row"] = rng.integers(-1, masks, (B, N)).astype(np.int32)
    if topo is not None:
        host["tokens"] = rng.integers(0, min(V, 40), (B, N)).astype(np.int32) * max(1, V // 40) % V  # some of them again and again
        host["parent"] = topo.parent
    for k, v in host.items():
        if k not in ("logits", "parent"):
            dev["prompt_bits" if k == "prompt" else k] = dev_words(v) if v.dtype == np.uint32 else to_dev(v)
    return host, dev


def check(got, host):
    want, size = ov.process(**host)
    g = value(got)
    assert g.shape == want.shape
    ok = np.isfinite(want)
    np.testing.assert_array_equal(g[~ok], want[~ok])
    off = np.abs(g - want)[ok]
    assert np.all(off <= 6 * U * size[ok]), float(np.max(off / np.maximum(size[ok], 1e-30)) / U)


CASES = [  # B, N, V, dtype, pad, tree
    (1, 1, 1, "f32", 0, False), (1, 1, 5, "bf16", 3, True), (2, 7, 33, "f32", 0, True), (3, 30, 1000, "bf16", 24, True), (1, 64, 2052, "f32", 0, True),
    (2, 57, 1023, "bf16", 1, True), (2, 256, 516, "bf16", 0, True), (5, 3, 4100, "f32", 4, False), (70, 1, 257, "bf16", 63, False), (2, 300, 64, "f32", 0, False),
    (1, 33, 5000, "f32", 6, True)]


@pytest.mark.parametrize("B,N,V,dtype,pad,with_tree", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_parity(mg, B, N, V, dtype, pad, with_tree):
    rng = np.random.default_rng(B * 1000 + N + V)
    t = tree(N, V) if with_tree else None
    host, dev = inputs(rng, B, N, V, dtype=dtype, pad=pad, topo=t)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if with_tree:
        dev["topo"] = upload(mg, t)
    got = mg.medusa_logits_process(**dev, d_status=st)
    assert mg.medusa_status_check(st) == 0
    check(got, host)


@pytest.mark.parametrize("V", [400, 401])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_every_part_alone_and_left_out(mg, V, dtype):
    rng = np.random.default_rng(V)
    t = tree(12)
    host, dev = inputs(rng, 2, 12, V, dtype=dtype, topo=t)
    topo = upload(mg, t)
    name = {"prompt": "prompt_bits"}
    for keep in ([], ["repetition"], ["repetition", "prompt"], ["repetition", "counts"], ["frequency", "counts"], ["presence"], ["bias"], ["mask", "mask_row"],
                 ["counts", "prompt"], ["frequency", "presence", "bias"]):
        for with_tree in (False, True):
            h = {k: host[k] for k in ["logits"] + keep + (["tokens", "parent"] if with_tree else [])}
            d = {name.get(k, k): dev[name.get(k, k)] for k in ["logits"] + keep + (["tokens"] if with_tree else [])}
            if with_tree:
                d["topo"] = topo
            check(mg.medusa_logits_process(**d), h)
    host["bias"], dev["bias"] = host["bias"][0], dev["bias"][0].contiguous()  # one for all
    check(mg.medusa_logits_process(**dev, topo=topo), host)


@pytest.mark.parametrize("V", [512, 515])
def test_in_place_captured_on_another_stream_and_twice(mg, V):
    rng = np.random.default_rng(V)
    t = tree(20)
    host, dev = inputs(rng, 3, 20, V, topo=t)
    dev["topo"] = upload(mg, t)
    before = dev["logits"].clone()
    want = mg.medusa_logits_process(**dev)
    assert torch.equal(dev["logits"], before)
    same = mg.medusa_logits_process(**dev, out=dev["logits"])
    assert same.data_ptr() == dev["logits"].data_ptr() and torch.equal(same, want)
    dev["logits"].copy_(before)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mg.medusa_logits_process(**dev, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        mg.medusa_logits_process(**dev, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    check(want, host)


def test_masks_of_a_row_each_and_masked_places_that_are_not_numbers(mg):
    rng = np.random.default_rng(5)
    host, dev = inputs(rng, 2, 3, 100, masks=6, rows=False)
    host["logits"] = host["logits"].copy()
    host["logits"][0, 1, 7], host["logits"][1, 0, 8], host["logits"][1, 1, 9], host["logits"][1, 2, 10] = np.nan, np.inf, -np.inf, np.finfo(np.float32).min
    for n, place in ((1, 7), (3, 8), (4, 9)):
        host["mask"][n, 0] &= ~np.uint32(1 << place)
    host["bias"][:, 7:11] = 0
    dev["logits"], dev["mask"], dev["bias"] = to_dev(host["logits"].astype(np.float32)), dev_words(host["mask"]), to_dev(host["bias"])
    host["repetition"][:] = 1.0
    dev["repetition"] = to_dev(host["repetition"])
    check(mg.medusa_logits_process(**dev), host)
    dev["mask"].fill_(-1)  # nothing is masked: what is not a number stays so
    out = value(mg.medusa_logits_process(**dev))
    assert np.isnan(out[0, 1, 7]) and out[1, 0, 8] == np.inf and out[1, 1, 9] == -np.inf and np.isnan(out).sum() == 1


@pytest.mark.parametrize("V", [64, 67])
def test_bad_tokens_masks_and_trees_are_reported(mg, V):
    rng = np.random.default_rng(V)
    t = tree(9)
    host, dev = inputs(rng, 2, 9, V, topo=t)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    host["tokens"][1, 4] = V
    host["tokens"][0, 2] = -1
    dev["tokens"] = to_dev(host["tokens"])
    check(mg.medusa_logits_process(**dev, topo=upload(mg, t), d_status=st), host)  # passed over
    assert mg.medusa_status_check(st) == 1
    mg.medusa_logits_process(**dev, topo=upload(mg, t))  # and without a status word
    host["tokens"][:] = 3
    dev["tokens"] = to_dev(host["tokens"])
    host["mask_row"][1, 3], host["mask_row"][0, 0] = 3, -2
    dev["mask_row"] = to_dev(host["mask_row"])
    got = mg.medusa_logits_process(**dev, topo=upload(mg, t), d_status=st)
    assert mg.medusa_status_check(st) == 1
    host["mask_row"][1, 3] = host["mask_row"][0, 0] = -1
    check(got, host)
    dev["mask_row"] = to_dev(host["mask_row"])
    for node, parent in ((5, 5), (5, 200), (5, -1), (0, 0), (0, 3)):
        topo = upload(mg, t)
        topo.buf[node] = parent
        got = mg.medusa_logits_process(**dev, topo=topo, d_status=st)
        assert mg.medusa_status_check(st) == 4
        assert got.shape == (2, 9, V)


def test_refusals(mg):
    rng = np.random.default_rng(0)
    t = tree(6)
    _, dev = inputs(rng, 2, 6, 50, topo=t)
    topo = upload(mg, t)
    z = dev["logits"]

    def refused(match, kind=ValueError, **over):
        d = {**dev, "topo": topo, **over}
        with pytest.raises(kind, match=match):
            mg.medusa_logits_process(**d)

    refused("counts", counts=dev["counts"][:, :49])
    refused("counts", counts=dev["counts"].long())
    refused("prompt_bits", prompt_bits=dev["prompt_bits"][:, :1])
    refused("repetition", repetition=dev["repetition"][:1])
    refused("bias", bias=dev["bias"][:1])
    refused("mask_row", mask_row=dev["mask_row"][:1])
    refused("mask_row needs mask", mask=None)
    refused("mask", mask_row=None)  # three rows for twelve nodes
    refused("topo needs tokens", tokens=None)
    refused("tokens need topo", topo=None)
    refused("nodes", topo=upload(mg, tree(7)))
    refused("evenly spaced", logits=z.transpose(0, 1).contiguous().transpose(0, 1))
    refused("out", out=torch.empty((2, 6, 50), dtype=torch.bfloat16, device="cuda"))
    buf = torch.zeros(601, device="cuda")
    refused("ALIAS", mg.MedusaError, logits=buf[:600].view(2, 6, 50), out=buf[1:].view(2, 6, 50))
    with pytest.raises(ValueError, match="empty"):
        mg.medusa_logits_process(torch.empty((2, 0, 50), device="cuda"))


# ----------------------------------------------------------------- counting

@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 17, 40), (2, 1000, 33), (70, 300, 5000), (1, 4099, 64)])
def test_counting_tokens(mg, B, S, V):
    rng = np.random.default_rng(S)
    tokens = rng.integers(-2, V, (B, S)).astype(np.int32)
    counts, bits = rng.integers(0, 5, (B, V)).astype(np.int32), ov.words_of(rng.random((B, V)) < 0.1)
    want = ov.count_tokens(tokens, V, counts, bits)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for which in ((True, True), (True, False), (False, True)):
        c, p = (to_dev(counts) if which[0] else None), (dev_words(bits) if which[1] else None)
        rc, rp = mg.medusa_count_tokens(to_dev(tokens), V, counts=c, prompt_bits=p, d_status=st)
        assert rc is c and rp is p
        if c is not None:
            np.testing.assert_array_equal(to_host(c), want[0])
        if p is not None:
            np.testing.assert_array_equal(host_words(p), want[1])
    assert mg.medusa_status_check(st) == 0
    tokens[0, 0] = V
    c = to_dev(counts)
    mg.medusa_count_tokens(to_dev(tokens), V, counts=c, d_status=st)
    assert mg.medusa_status_check(st) == 1
    np.testing.assert_array_equal(to_host(c), ov.count_tokens(tokens, V, counts)[0])


def test_counting_no_tokens(mg):
    c = torch.ones((2, 9), dtype=torch.int32, device="cuda")
    mg.medusa_count_tokens(torch.empty((2, 0), dtype=torch.int32, device="cuda"), 9, counts=c)
    assert (c == 1).all()


@pytest.mark.parametrize("B,N,D1,V", [(1, 1, 1, 1), (5, 12, 6, 50), (300, 64, 17, 999)])
def test_counting_accepted_paths(mg, B, N, D1, V):
    rng = np.random.default_rng(B)
    tokens = rng.integers(0, V, (B, N)).astype(np.int32)
    tokens[0] = 0  # the same token all along a path
    acc = rng.integers(1, D1 + 1, B).astype(np.int32)
    path = np.where(np.arange(D1) < acc[:, None], rng.integers(0, N, (B, D1)), -1).astype(np.int32)
    counts = rng.integers(0, 5, (B, V)).astype(np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run():
        c = to_dev(counts)
        assert mg.medusa_count_accepted(c, to_dev(tokens), to_dev(path), to_dev(acc), d_status=st) is c
        np.testing.assert_array_equal(to_host(c), ov.count_accepted(counts, tokens, path, acc))
        return mg.medusa_status_check(st)

    assert run() == 0
    if B > 4:
        for what in ("long", "none", "node", "token"):
            a, p, t = acc.copy(), path.copy(), tokens.copy()
            if what == "long":
                acc[1] = D1 + 1
            elif what == "none":
                acc[2] = 0
            elif what == "node":
                path[3, acc[3] - 1] = N
            else:
                tokens[4, path[4, 0]] = V
            assert run() == 1, what
            acc, path, tokens = a, p, t


@pytest.mark.parametrize("N,V", [(64, 32016), (1, 32016), (64, 32001)])
def test_logits_past_32_bits(mg, N, V):
    B = 70400 // N
    rng = np.random.default_rng(N + V)
    rows = [0, 35000 // N, 67085 // N, B - 1]
    part = wl.to_bf16_bits(rng.standard_normal((len(rows), N, V)).astype(np.float32))
    counts, frequency = rng.integers(0, 3, (len(rows), V)).astype(np.int32), np.array([0.5, 1.0, -0.5, 0.25], np.float32)
    z, c, f = torch.zeros((B, N, V), dtype=torch.bfloat16, device="cuda"), torch.zeros((B, V), dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda")
    z[rows], c[rows], f[rows] = to_dev(part), to_dev(counts), to_dev(frequency)
    got = mg.medusa_logits_process(z, c, frequency=f)
    want, size = ov.process(ov.bf16_value(part), counts, frequency=frequency)
    assert np.all(np.abs(value(got[rows]) - want) <= 6 * U * size)
    assert not got[rows[1] + 1:rows[2]].any() and not got[rows[2] + 1:rows[3]].any()
