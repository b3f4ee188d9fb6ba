"""The operators at the output of a verify pass as they are measured: their plain
forms in elementary torch operations, and the calls a user makes of the library.

A server of Medusa steps keeps the backbone in 4 bits and lets requests ask for
penalties, biases and grammars.  Next to the bf16 linear layer and the acceptance
it then needs the product with 4-bit weights, the processing of the logits of all
tree nodes, each with the sequence and its own ancestors as its context, and the
counts of the tokens that the penalties go by.

4-bit weights: qweight [Nout, K / 8] int32, element 2i of a word in its nibble i and
element 2i + 1 in nibble i + 4; scales [K / G, Nout] bf16, zeros [K / G, Nout] uint8
(none: 8).  A weight stands for the bf16 nearest to scale * (q - zero).
Counts: [B, V] int32, the tokens a sequence has generated; prompt bits [B, ceil(V / 32)]
int32, bit v % 32 of word v / 32: token v is in the prompt.  Grammar masks [M, ceil(V / 32)]:
the bits of the tokens that may follow.
"""
import math
import random

import torch

own = False

GPU = "cuda"


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one layer's output projection for one decoded token (7B shape): latency counts
        dict(name="w4_decode_proj", op="linear", tokens=1, k=4096, n=4096, group=128, zeros=True, out="bf16", gap=0),
        # the output head for one decoded token (7B shape), logits in fp32
        dict(name="w4_decode_head", op="linear", tokens=1, k=4096, n=32000, group=128, zeros=False, out="f32", gap=0),
        # a few sequences decoding one token each, small groups, an odd number of outputs, rows of a wider buffer
        dict(name="w4_few_odd", op="linear", tokens=7, k=5120, n=13825, group=32, zeros=True, out="bf16", gap=64),
        # a verify pass of 64 tree tokens, gate and up projections in one (7B shape)
        dict(name="w4_tree_gate_up", op="linear", tokens=64, k=4096, n=22016, group=128, zeros=True, out="bf16", gap=0),
        # three trees of 57 nodes, down projection (7B shape)
        dict(name="w4_trees_down", op="linear", tokens=171, k=11008, n=4096, group=64, zeros=True, out="bf16", gap=0),
        # a prompt of odd length: compute counts
        dict(name="w4_prompt", op="linear", tokens=2311, k=4096, n=11008, group=128, zeros=True, out="bf16", gap=0),
        # the fp32 logits of one 64-node tree: everything asked for
        dict(name="logits_tree", op="logits", batch=1, nodes=64, tree=True, vocab=32000, dtype="f32", pad=0, penalties=True,
             bias="each", masks=9),
        # 16 trees of an odd size, bf16 logits
        dict(name="logits_trees", op="logits", batch=16, nodes=57, tree=True, vocab=32000, dtype="bf16", pad=0, penalties=True,
             bias="one", masks=40),
        # 64 sequences decoding without trees, an odd vocabulary in rows padded by the output head
        dict(name="logits_decode", op="logits", batch=64, nodes=1, tree=False, vocab=50257, dtype="bf16", pad=47, penalties=True,
             bias="none", masks=3),
        # the accepted paths of 64 sequences: the smallest call
        dict(name="count_accepted", op="accepted", batch=64, nodes=64, vocab=32000),
        # prompts of ragged lengths
        dict(name="count_prompts", op="tokens", batch=7, most=4099, vocab=32000, counts=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "logits", "logits", "accepted", "tokens"])
    if op == "linear":
        c = dict(op=op, group=rng.choice([32, 64, 128, 128]), zeros=rng.random() < 0.6, out=rng.choice(["bf16", "bf16", "f32"]),
                 gap=rng.choice([0, 0, 8, 40]))
        c["tokens"] = rng.choice([1, _log(rng, 1, 16), _log(rng, 2, 256), _log(rng, 16, 2200)])
        c["k"] = c["group"] * _log(rng, 1, 11008 // c["group"])
        c["n"] = _log(rng, 16, 32000)
        while c["tokens"] * c["k"] * c["n"] > 90e9 or c["k"] * c["n"] > 128e6:
            if c["tokens"] > 512:
                c["tokens"] = (c["tokens"] + 1) // 2
            else:
                c["n"] = (c["n"] + 1) // 2
        return c
    vocab = rng.choice([32000, 32000, 50257, _log(rng, 100, 130000)])
    if op == "logits":
        tree = rng.random() < 0.7
        c = dict(op=op, tree=tree, nodes=_log(rng, 1, 256) if tree else _log(rng, 1, 8), vocab=vocab, dtype=rng.choice(["f32", "bf16"]),
                 pad=rng.choice([0, 0, 64 - vocab % 64]), penalties=rng.random() < 0.75, bias=rng.choice(["none", "one", "each"]),
                 masks=rng.choice([0, 1, _log(rng, 1, 64)]))
        c["batch"] = _log(rng, 1, max(1, min(128, 28_000_000 // (c["nodes"] * vocab))))
        while c["batch"] * c["nodes"] * vocab > 29e6:
            c["nodes"] = (c["nodes"] + 1) // 2
        return c
    c = dict(op=op, batch=_log(rng, 1, 128), vocab=vocab)
    if op == "accepted":
        c["nodes"] = _log(rng, 1, 256)
    else:
        c["most"], c["counts"] = _log(rng, 1, 8192), rng.random() < 0.5
    while c["batch"] * vocab > 8e6:
        c["batch"] = (c["batch"] + 1) // 2
    return c


def work(case):
    op = case["op"]
    if op == "linear":
        T, K, N, G = case["tokens"], case["k"], case["n"], case["group"]
        w = N * K // 2 + N * (K // G) * (3 if case["zeros"] else 2)
        return {"bytes": w + 2 * T * K + (2 if case["out"] == "bf16" else 4) * T * N, "flops": 2 * T * K * N}
    B, V = case["batch"], case["vocab"]
    if op == "logits":
        N = case["nodes"]
        b = B * N * V * (4 + (4 if case["dtype"] == "f32" else 2))
        if case["penalties"]:
            b += B * V * 4 + B * ((V + 31) // 32) * 4
        b += {"none": 0, "one": 4 * V, "each": 4 * B * V}[case["bias"]] + min(case["masks"], B * N) * ((V + 31) // 32) * 4
        return {"bytes": b + (4 * B * N if case["masks"] else 0), "flops": 4 * B * N * V}
    if op == "accepted":
        return {"bytes": B * 4 * 5 * 4, "flops": B * 3}
    n = sum(_lengths(case))
    return {"bytes": 4 * B * case["most"] + n * (8 if not case["counts"] else 16), "flops": n}


def _lengths(case):
    rng = random.Random(case["most"])
    return [rng.randrange(case["most"] // 4, case["most"] + 1) if case["batch"] > 1 else case["most"] for _ in range(case["batch"])]


# ----------------------------------------------------------------- the inputs

def _tree(n, deepest, seed):
    """A random candidate tree as rank paths in the canonical order (length, then ranks), and every node's parent."""
    rng = random.Random(seed)
    paths, children = [()], {(): 0}
    while len(paths) < n:
        p = rng.choice(paths)
        if len(p) < deepest and children[p] < 10:
            q = p + (children[p],)
            children[p] += 1
            children[q] = 0
            paths.append(q)
    paths.sort(key=lambda p: (len(p), p))
    at = {p: i for i, p in enumerate(paths)}
    return paths, [-1] + [at[p[:-1]] for p in paths[1:]]


def _words(bits):
    """bits [..., V] -> int32 words [..., ceil(V / 32)]."""
    v = bits.shape[-1]
    b = torch.zeros(*bits.shape[:-1], (v + 31) // 32 * 32, dtype=torch.int64, device=bits.device)
    b[..., :v] = bits
    w = (b.unflatten(-1, (-1, 32)) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _zipf(g, vocab, *shape):
    """Token ids as texts have them: a few often, most of them rarely."""
    u = torch.rand(*shape, device=GPU, generator=g)
    return ((vocab + 1.0) ** u - 1.0).long().clamp_(0, vocab - 1).mul_(7919).remainder_(vocab).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=GPU).manual_seed(seed)
    host = random.Random(seed)
    op, st = case["op"], dict(case=dict(case))

    def normal(*shape):
        return torch.randn(*shape, device=GPU, generator=g)

    if op == "linear":
        T, K, N, G = case["tokens"], case["k"], case["n"], case["group"]
        st["x"] = normal(T, K + case["gap"]).to(torch.bfloat16)[:, :K]
        q = torch.zeros(N, K // 8, dtype=torch.int32, device=GPU)
        for shift in range(0, 32, 4):  # nibble by nibble
            q |= (normal(N, K // 8) * 2.6 + 7.5).round_().clamp_(0, 15).to(torch.int32) << shift
        st["qweight"] = q
        st["scales"] = (0.008 + 0.004 * torch.rand(K // G, N, device=GPU, generator=g)).to(torch.bfloat16)
        st["zeros"] = torch.randint(6, 10, (K // G, N), device=GPU, generator=g, dtype=torch.uint8) if case["zeros"] else None
        return st
    B, V = case["batch"], case["vocab"]
    if op == "tokens":
        tokens = _zipf(g, V, B, case["most"])
        length = torch.tensor(_lengths(case), device=GPU)
        st["tokens"] = torch.where(torch.arange(case["most"], device=GPU) < length[:, None], tokens, -1).to(torch.int32)
        st["counts"] = torch.zeros(B, V, dtype=torch.int32, device=GPU) if case["counts"] else None
        st["bits"] = torch.zeros(B, (V + 31) // 32, dtype=torch.int32, device=GPU)
        return st
    N = case["nodes"]
    st["tokens"] = _zipf(g, V, B, N)
    paths, parent = _tree(N, 8, N) if op == "accepted" or case["tree"] else (None, None)
    if op == "accepted":
        ends = [host.randrange(N) for _ in range(B)]
        rows = []
        for e in ends:
            row = []
            while e >= 0:
                row.insert(0, e)
                e = parent[e]
            rows.append(row)
        st["accept_len"] = torch.tensor([len(r) for r in rows], dtype=torch.int32, device=GPU)
        st["path_nodes"] = torch.tensor([r + [-1] * (9 - len(r)) for r in rows], dtype=torch.int32, device=GPU)
        st["counts"] = torch.zeros(B, V, dtype=torch.int32, device=GPU)
        return st
    row = V + case["pad"]
    z = normal(B, N, row) * 2.5
    st["logits"] = (z if case["dtype"] == "f32" else z.to(torch.bfloat16))[..., :V]
    st["out"] = torch.empty(B, N, V, dtype=torch.float32, device=GPU)
    if case["tree"]:
        st["parent"] = parent
        seen = torch.zeros(N, N, dtype=torch.int64)
        for n in range(N):
            if n:
                seen[n] = seen[parent[n]]
            seen[n, n] = 1
        st["ancestors"] = seen.to(GPU)
        if own:
            import medusa_head_speculative_heads_gb300 as mg
            st["topo"] = mg.Topology.from_paths([list(p) for p in paths[1:]]).upload()
    if case["penalties"]:
        said = torch.zeros(B, V, dtype=torch.int32, device=GPU)
        st["counts"] = said.scatter_add_(1, _zipf(g, V, B, 500).long(), torch.ones(B, 500, dtype=torch.int32, device=GPU))
        asked = torch.zeros(B, V, dtype=torch.bool, device=GPU).scatter_(1, _zipf(g, V, B, 1000).long(), True)
        st["bits"] = _words(asked)
        st["repetition"] = 1.0 + 0.5 * torch.rand(B, device=GPU, generator=g)
        st["frequency"], st["presence"] = (torch.rand(B, device=GPU, generator=g) * 0.6 for _ in range(2))
    if case["bias"] != "none":
        b = normal(*((V,) if case["bias"] == "one" else (B, V)))
        st["bias"] = torch.where(torch.rand(b.shape, device=GPU, generator=g) < 0.01, b * 4.0, 0.0)
    if case["masks"]:
        M = case["masks"]  # one lets everything pass but a few, others little
        share = torch.rand(M, 1, device=GPU, generator=g) ** 3
        st["mask"] = torch.cat([_words(torch.rand(1, V, device=GPU, generator=g) > share[i:i + 1]) for i in range(M)])
        st["mask_row"] = torch.randint(-1, M, (B, N), device=GPU, generator=g, dtype=torch.int32)
    return st


# ----------------------------------------------------------------- plain forms

def _bits(words, vocab):
    """int32 words [..., W] -> truth values [..., vocab]."""
    v = torch.arange(vocab, device=GPU)
    return (words[..., v // 32] >> (v % 32)) & 1 == 1


def _plain_linear(st):
    c = st["case"]
    place = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=GPU, dtype=torch.int32)  # bits before element 0 .. 7 of a word
    q = ((st["qweight"][:, :, None] >> place) & 15).flatten(1).float()
    scale = st["scales"].float().t().repeat_interleave(c["group"], 1)
    zero = 8.0 if st["zeros"] is None else st["zeros"].float().t().repeat_interleave(c["group"], 1)
    w = (scale * (q - zero)).to(torch.bfloat16).float()
    y = torch.matmul(st["x"].float(), w.t())
    return y.to(torch.bfloat16) if c["out"] == "bf16" else y


def _plain_logits(st):
    c = st["case"]
    z = st["logits"].float()
    if c["penalties"]:
        n = st["counts"][:, None].long().expand(z.shape)
        if c["tree"]:
            tokens = st["tokens"][:, None].long().expand(c["batch"], c["nodes"], c["nodes"])
            n = n.clone().scatter_add_(2, tokens, st["ancestors"].expand(tokens.shape))
        seen = (n > 0) | _bits(st["bits"], c["vocab"])[:, None]
        r, f, p = (st[k][:, None, None] for k in ("repetition", "frequency", "presence"))
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - f * n - p * (n > 0)
    if "bias" in st:
        z = z + (st["bias"] if c["bias"] == "one" else st["bias"][:, None])
    if c["masks"]:
        row = st["mask_row"].long()
        z = torch.where(_bits(st["mask"], c["vocab"])[row.clamp_min(0)] | (row < 0)[..., None], z, -math.inf)
    return z


def _plain_tokens(st):
    tokens, there = st["tokens"].clamp_min(0).long(), st["tokens"] >= 0
    if st["counts"] is not None:
        st["counts"].scatter_add_(1, tokens, there.to(torch.int32))
    V = st["case"]["vocab"]
    hit = torch.zeros(tokens.shape[0], V, dtype=torch.int32, device=GPU).scatter_add_(1, tokens, there.to(torch.int32)) > 0
    st["bits"] |= _words(hit)
    return st["counts"], st["bits"]


def _plain_accepted(st):
    keep = torch.arange(st["path_nodes"].shape[1], device=GPU) < st["accept_len"][:, None]
    tokens = st["tokens"].long().gather(1, st["path_nodes"].clamp_min(0).long())
    return st["counts"].scatter_add_(1, tokens, keep.to(torch.int32))


def run(st):
    op = st["case"]["op"]
    if own:
        import medusa_head_speculative_heads_gb300 as mg
        if op == "linear":
            return mg.medusa_linear_w4(st["x"], st["qweight"], st["scales"], st["zeros"],
                                       out_dtype=torch.bfloat16 if st["case"]["out"] == "bf16" else torch.float32)
        if op == "logits":
            return mg.medusa_logits_process(st["logits"], counts=st.get("counts"), prompt_bits=st.get("bits"), repetition=st.get("repetition"),
                                            frequency=st.get("frequency"), presence=st.get("presence"), bias=st.get("bias"), mask=st.get("mask"),
                                            mask_row=st.get("mask_row"), tokens=st["tokens"] if "topo" in st else None, topo=st.get("topo"),
                                            out=st["out"])
        if op == "accepted":
            return mg.medusa_count_accepted(st["counts"], st["tokens"], st["path_nodes"], st["accept_len"])
        return mg.medusa_count_tokens(st["tokens"], st["case"]["vocab"], counts=st["counts"], prompt_bits=st["bits"])
    if op == "linear":
        return _plain_linear(st)
    if op == "logits":
        return st["out"].copy_(_plain_logits(st))
    return _plain_accepted(st) if op == "accepted" else _plain_tokens(st)


# ----------------------------------------------------------------- in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        N, K, G = case["n"], case["k"], case["group"]
        w = torch.empty(N, K // 8, 8, dtype=torch.float64, device=GPU)
        words = st["qweight"].long() & 0xffffffff
        for i in range(4):
            w[..., 2 * i] = ((words >> (4 * i)) % 16).double()
            w[..., 2 * i + 1] = ((words >> (16 + 4 * i)) % 16).double()
        w = w.view(N, K // G, G)
        w -= 8.0 if st["zeros"] is None else st["zeros"].t().double()[..., None]
        w *= st["scales"].t().double()[..., None]
        part, _ = torch.frexp(w)  # to 8 significant bits, ties to even: part is 0.5 .. 1, w / part a power of two
        w = torch.where(w == 0, w, (part * 256.0).round() / 256.0 * (w / part))
        return st["x"].double() @ w.view(N, K).t()
    if op == "logits":
        B, N, V = case["batch"], case["nodes"], case["vocab"]
        out = st["logits"].double()
        v = torch.arange(V, device=GPU)
        rows = st["mask_row"].tolist() if case["masks"] else None
        for b in range(B):
            if case["penalties"]:
                asked = (st["bits"][b].long() & 0xffffffff).repeat_interleave(32)[:V] >> (v % 32) & 1
            for n in range(N):
                z = out[b, n]
                if case["penalties"]:
                    c = st["counts"][b].double()
                    e = n if case["tree"] else -1
                    while e >= 0:
                        c[st["tokens"][b, e].long()] += 1.0
                        e = st["parent"][e]
                    r = st["repetition"][b].double()
                    z[:] = z * torch.where((c + asked) > 0, torch.where(z > 0, 1.0 / r, r), 1.0)
                    z -= st["frequency"][b].double() * c + st["presence"][b].double() * c.sign()
                if case["bias"] != "none":
                    z += (st["bias"] if case["bias"] == "one" else st["bias"][b]).double()
                if rows and rows[b][n] >= 0:
                    m = (st["mask"][rows[b][n]].long() & 0xffffffff).repeat_interleave(32)[:V] >> (v % 32) & 1
                    z[m == 0] = -math.inf
        return out
    return None
