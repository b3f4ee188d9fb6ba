"""The paged-cache operators as they are measured: their plain forms in
elementary torch operations, and the calls a user makes of the library.

A verify step whose caches live in pages needs five operators next to the ones
over contiguous caches: the rotary embedding in the forms backbones use, the
append of a chunk of new tokens to the pages (with that embedding on the way),
causal attention of the chunk over the pages, tree attention over the pages,
and the append of an accepted path to the pages.

Caches: k_pages, v_pages [nl, n_pages, page_size, Hkv, d]; row r of sequence b
is row r % page_size of page page_table[b, r // page_size], in every layer.
Chunks: the T new tokens of all sequences back to back, sequence b's at
q_start[b] .. q_start[b + 1] - 1, after the prefix_len[b] rows it has already.
"""
import math
import random

import torch

own = False

GPU = "cuda"


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # rotation of the 64 tree tokens of one verify pass, all 32 layers (7B shape)
        dict(name="rope_verify_7b", op="rope", dtype="bf16", nl=32, tokens=64, hq=32, hkv=32, d=128, rotary=128,
             interleaved=False, scaling="none", inverse=False, max_pos=1100),
        # gradient of the rotation of a long training sequence: fp32, adjacent pairs,
        # half of each head, frequencies scaled by wavelength
        dict(name="rope_grad_long", op="rope", dtype="f32", nl=1, tokens=16384, hq=32, hkv=8, d=128, rotary=64,
             interleaved=True, scaling="bands", inverse=True, max_pos=131072),
        # one decoding step of 64 sequences in one layer: the smallest append
        dict(name="append_decode", op="append", dtype="bf16", nl=1, batch=64, chunk_max=1, prefix_max=2047, hq=32,
             hkv=8, d=128, rotary=128, interleaved=False, scaling="none", page=16, lens=1),
        # prompts of odd lengths entering the cache, frequencies scaled by a ramp over the pairs
        dict(name="append_prefill", op="append", dtype="bf16", nl=1, batch=7, chunk_max=2311, prefix_max=512, hq=32,
             hkv=8, d=128, rotary=128, interleaved=False, scaling="ramp", page=64, lens=2),
        # one decoding step of one sequence, MHA (7B shape): latency counts
        dict(name="attn_decode_one", op="attn", dtype="bf16", nl=1, batch=1, chunk_max=1, prefix_max=1024, hq=32,
             hkv=32, d=128, page=64, lens=3),
        # one decoding step of 64 sequences of ragged lengths, grouped heads
        dict(name="attn_decode_batch", op="attn", dtype="bf16", nl=1, batch=64, chunk_max=1, prefix_max=8191, hq=32,
             hkv=8, d=128, page=16, lens=4),
        # a long prompt's second half over its first: compute counts
        dict(name="attn_prefill", op="attn", dtype="bf16", nl=1, batch=1, chunk_max=8192, prefix_max=8192, hq=32,
             hkv=8, d=128, page=64, lens=0),
        # chunks of odd lengths in fp32, small heads
        dict(name="attn_ragged_f32", op="attn", dtype="f32", nl=1, batch=5, chunk_max=333, prefix_max=1501, hq=8,
             hkv=4, d=64, page=16, lens=6),
        # the verify pass of a 64-node tree over a 1024-row prefix, all layers (7B shape)
        dict(name="tree_verify_7b", op="tree", dtype="bf16", nl=32, batch=1, nodes=64, prefix_max=1024, hq=32, hkv=32,
             d=128, page=64, lens=0),
        # 16 sequences verified at once, grouped heads, ragged prefixes, an odd tree
        dict(name="tree_verify_batch", op="tree", dtype="bf16", nl=4, batch=16, nodes=57, prefix_max=4096, hq=32,
             hkv=8, d=128, page=32, lens=8),
        # the accepted paths of four sequences, all layers (7B shape)
        dict(name="compact_7b", op="compact", dtype="bf16", nl=32, batch=4, nodes=64, depth=4, prefix_max=300, hkv=32,
             d=128, page=64, lens=9),
        # one accepted path of a small fp32 model
        dict(name="compact_small_f32", op="compact", dtype="f32", nl=2, batch=1, nodes=7, depth=2, prefix_max=128,
             hkv=2, d=64, page=16, lens=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "tree", "compact"])
    c = dict(op=op, dtype="f32" if rng.random() < 0.25 else "bf16")
    es = 2 if c["dtype"] == "bf16" else 4
    hkv, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 7, 8])
    d = rng.choice([64, 128, 128, 96])
    if op in ("rope", "append"):
        c.update(rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "bands", "ramp"]))
    if op == "rope":
        d = c["d"] = rng.choice([64, 128, 96, 80, 256])
        c.update(rotary=rng.choice([d, d, d // 2]), nl=_log(rng, 1, 32), hq=hkv * group, hkv=hkv,
                 inverse=rng.random() < 0.4, max_pos=_log(rng, 64, 1 << 20))
        c["tokens"] = _log(rng, 1, max(2, min(20000, (300 << 20) // (c["nl"] * (c["hq"] + hkv) * d * es))))
        return c
    c.update(nl=1, hkv=hkv, d=d, page=rng.choice([8, 16, 24, 32, 64, 128, 256]), lens=rng.randrange(1, 1 << 30))
    if op == "append":
        c.update(hq=hkv * group, batch=_log(rng, 1, 128), prefix_max=_log(rng, 1, 2048))
        most = (200 << 20) // (hkv * d * es * c["batch"])  # rows of one sequence
        c["chunk_max"] = _log(rng, 1, max(2, min(2048, most // 2)))
        c["prefix_max"] = min(c["prefix_max"], max(1, most - c["chunk_max"]))
    elif op == "attn":
        # decoding, short chunks, prompts; what a pass costs stays below the listed prompt
        c.update(hq=hkv * group, batch=_log(rng, 1, 64), chunk_max=rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 64, 4096)]),
                 prefix_max=_log(rng, 1, 8192))
        most = (2 << 20) if c["dtype"] == "f32" else (48 << 20)  # pairs of (row, key) over all heads, in units of 64
        while c["batch"] * c["hq"] * c["chunk_max"] * (c["prefix_max"] + c["chunk_max"]) > 64 * most or \
                c["batch"] * hkv * d * (c["prefix_max"] + c["chunk_max"]) > (1 << 29):
            if c["batch"] > 1:
                c["batch"] = (c["batch"] + 1) // 2
            elif c["chunk_max"] > 1:
                c["chunk_max"] = (c["chunk_max"] + 1) // 2
            else:
                c["prefix_max"] = (c["prefix_max"] + 1) // 2
    elif op == "tree":
        c.update(hq=hkv * group, batch=_log(rng, 1, 16), nodes=_log(rng, 1, 256), prefix_max=_log(rng, 1, 4096), nl=_log(rng, 1, 8))
        most = (1 << 20) if c["dtype"] == "f32" else (16 << 20)
        while c["nl"] * c["batch"] * c["hq"] * c["nodes"] * (c["prefix_max"] + c["nodes"]) > 64 * most or \
                c["nl"] * c["batch"] * hkv * d * (c["prefix_max"] + c["nodes"]) > (1 << 28):
            k = "nl" if c["nl"] > 1 else "batch" if c["batch"] > 1 else "nodes" if c["nodes"] > 64 else "prefix_max"
            c[k] = (c[k] + 1) // 2
    else:
        c.update(nl=_log(rng, 1, 32), batch=_log(rng, 1, 32), nodes=_log(rng, 2, 256), depth=rng.randrange(1, 9),
                 prefix_max=_log(rng, 1, 512))
        while c["nl"] * c["batch"] * hkv * d * es * (c["prefix_max"] + 64) > (256 << 20):
            k = "nl" if c["nl"] > 1 else "batch" if c["batch"] > 1 else "prefix_max"
            c[k] = (c[k] + 1) // 2
    return c


def _lengths(case):
    """(prefix, chunk) lengths of the sequences: from the case alone.  lens = 0: the largest."""
    rng = random.Random(case["lens"])
    prefix, chunk = [], []
    for _ in range(case["batch"]):
        if case["lens"]:
            prefix.append(rng.randrange(case["prefix_max"] // 4, case["prefix_max"] + 1))
            chunk.append(rng.randrange((case.get("chunk_max", 1) + 3) // 4, case.get("chunk_max", 1) + 1))
        else:
            prefix.append(case["prefix_max"])
            chunk.append(case.get("chunk_max", 1))
    return prefix, chunk


def _accepted(case):
    rng = random.Random(case["lens"] + 1)
    most = min(case["depth"] + 1, case["nodes"])
    return [rng.randrange(1, most + 1) for _ in range(case["batch"])]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op, nl, d = case["op"], case["nl"], case["d"]
    if op == "rope":
        heads = case["tokens"] * (case["hq"] + case["hkv"]) * nl
        return {"bytes": 2 * heads * d * es + 4 * case["tokens"], "flops": 3 * heads * case["rotary"]}
    prefix, chunk = _lengths(case)
    row = case["hkv"] * d * es
    if op == "append":
        tokens = sum(chunk) * nl
        # q and the new rows read; q and the cache rows written
        return {"bytes": 2 * tokens * (case["hq"] * d * es + 2 * row), "flops": 3 * tokens * (case["hq"] + case["hkv"]) * case["rotary"]}
    if op == "compact":
        return {"bytes": 4 * nl * sum(_accepted(case)) * row, "flops": 0}
    if op == "attn":
        keys = sum(p + c for p, c in zip(prefix, chunk))
        pairs = sum(c * p + c * (c + 1) // 2 for p, c in zip(prefix, chunk))
        rows = sum(chunk)
    else:
        keys = sum(p + case["nodes"] for p in prefix)
        _, _, seen = _tree(case["nodes"], case["lens"])
        pairs = sum(case["nodes"] * p for p in prefix) + case["batch"] * int(seen)
        rows = case["batch"] * case["nodes"]
    q = rows * case["hq"] * d * es
    return {"bytes": nl * (2 * q + 2 * keys * row + 4 * rows * case["hq"]), "flops": 4 * nl * pairs * case["hq"] * d}


# ----------------------------------------------------------------- the inputs

def _tree(n, seed):
    """A random candidate tree: depth [n], ancestor table [n][n], visible pairs."""
    rng = random.Random(1000 + seed)
    depth, seen = [0] * n, [[False] * n for _ in range(n)]
    seen[0][0] = True
    for i in range(1, n):
        p = rng.randrange(max(0, i - 12), i)
        depth[i] = depth[p] + 1
        seen[i] = list(seen[p])
        seen[i][i] = True
    return depth, seen, sum(map(sum, seen))


def _mask_words(seen):
    n = len(seen)
    words = [[0] * ((n + 31) // 32) for _ in range(n)]
    for i in range(n):
        for j in range(n):
            if seen[i][j]:
                words[i][j // 32] |= 1 << (j % 32)
    return [[w - (1 << 32) if w >> 31 else w for w in row] for row in words]


def _rope_args(case):
    """The rotation's description, as plain values."""
    a = dict(rotary_dim=case["rotary"], interleaved=case["interleaved"], base=10000.0, scaling=case["scaling"])
    if case["scaling"] == "linear":
        a.update(factor=4.0)
    elif case["scaling"] == "bands":
        a.update(base=500000.0, factor=8.0, low=1.0, high=4.0, original_len=8192)
    elif case["scaling"] == "ramp":
        a.update(factor=16.0, low=1.0, high=32.0, original_len=4096, magnitude=0.1 * math.log(16.0) + 1.0)
    return a


def prepare(case, seed):
    g = torch.Generator(device=GPU).manual_seed(seed)
    host = random.Random(seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    op, nl, d = case["op"], case["nl"], case["d"]

    def normal(*shape):
        return torch.randn(*shape, device=GPU, dtype=dt, generator=g)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=GPU)

    st = dict(op=op, case=dict(case))
    if op in ("rope", "append"):
        st["rope"] = _rope_args(case)
        if own:
            import medusa_head_speculative_heads_gb300 as mg
            st["spec"] = mg.RopeSpec(**st["rope"])
    if op == "rope":
        st["q"], st["k"] = normal(nl, case["tokens"], case["hq"], d), normal(nl, case["tokens"], case["hkv"], d)
        first = host.randrange(0, max(1, case["max_pos"] - case["tokens"]))
        st["pos"] = ints([min(first + i, case["max_pos"] - 1) for i in range(case["tokens"])])
        return st
    prefix, chunk = _lengths(case)
    B, ps, hkv = case["batch"], case["page"], case["hkv"]
    more = case["depth"] + 1 if op == "compact" else 0
    need = [-(-(p + (c if op != "compact" and op != "tree" else 0) + more) // ps) for p, c in zip(prefix, chunk)]
    n_pages, wide = sum(need) + 3, max(max(need), 1)
    order = list(range(n_pages))
    host.shuffle(order)
    table, at = [], 0
    for n in need:  # pages in no order; entries behind a sequence's last page are never read
        table.append(order[at:at + n] + [-1] * (wide - n))
        at += n
    st["k_pages"], st["v_pages"] = normal(nl, n_pages, ps, hkv, d), normal(nl, n_pages, ps, hkv, d)
    st["page_table"], st["prefix_len"] = ints(table), ints(prefix)
    if op in ("append", "attn"):
        start = [0]
        for c in chunk:
            start.append(start[-1] + c)
        st["q_start"], st["max_q"], T = ints(start), max(chunk), start[-1]
        st["max_kv"] = max(p + c for p, c in zip(prefix, chunk))
    if op == "append":  # q, k and v as one projection leaves them
        qkv = normal(nl, T, case["hq"] + 2 * hkv, d)
        st["q"], st["k"], st["v"] = qkv[:, :, :case["hq"]], qkv[:, :, case["hq"]:case["hq"] + hkv], qkv[:, :, case["hq"] + hkv:]
    elif op == "attn":
        st["q"] = normal(nl, T, case["hq"], d)
    else:
        N = case["nodes"]
        st["kt"], st["vt"] = normal(nl, B, N, hkv, d), normal(nl, B, N, hkv, d)
        st["max_kv"] = max(prefix)
        if op == "tree":
            st["q"] = normal(nl, B, N, case["hq"], d)
            _, seen, _ = _tree(N, case["lens"])
            st["mask"] = ints(_mask_words(seen))
        else:
            acc = _accepted(case)
            paths = [[0] + sorted(host.sample(range(1, N), a - 1)) + [-1] * (case["depth"] + 1 - a) for a in acc]
            st["path_nodes"], st["accept_len"] = ints(paths), ints(acc)
    return st


# ----------------------------------------------------------------- plain forms

def _frequencies(a):
    """Radians a position of every pair, in 64 bits."""
    i = torch.arange(a["rotary_dim"] // 2, dtype=torch.float64, device=GPU)
    f = a["base"] ** (-2.0 * i / a["rotary_dim"])
    if a["scaling"] == "linear":
        f = f / a["factor"]
    elif a["scaling"] == "bands":  # by the turns a pair makes over the original length
        turns = a["original_len"] * f / (2.0 * math.pi)
        keep = ((turns - a["low"]) / (a["high"] - a["low"])).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / a["factor"]
    elif a["scaling"] == "ramp":  # by the pair's index, between the pairs that make `high` and `low` turns
        def pair(turns):
            return a["rotary_dim"] * math.log(a["original_len"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(a["base"]))
        lo, hi = max(math.floor(pair(a["high"])), 0), min(math.ceil(pair(a["low"])), a["rotary_dim"] - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / a["factor"]
    return f


def _rotate(x, pos, a, inverse=False, wide=torch.float32):
    """x [nl, T, H, d] at positions pos [T]: the leading rotary_dim elements of every head turn."""
    angle = pos.to(torch.float64)[:, None] * _frequencies(a)
    mag = a.get("magnitude", 1.0)
    c, s = (angle.cos() * mag).to(wide)[:, None], (angle.sin() * mag).to(wide)[:, None]
    if inverse:
        s = -s
    r = a["rotary_dim"]
    y = x.to(wide)
    if a["interleaved"]:
        x0, x1 = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack((x0 * c - x1 * s, x1 * c + x0 * s), -1).flatten(-2)
    else:
        x0, x1 = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat((x0 * c - x1 * s, x1 * c + x0 * s), -1)
    return torch.cat((turned, y[..., r:]), -1)


def _rows(table, rows, page):
    """Pool rows of the sequences' rows: rows [B, n]."""
    return table.long().gather(1, rows // page).clamp_min(0) * page + rows % page


def _token_of(st, T):
    t = torch.arange(T, device=GPU)
    b = torch.searchsorted(st["q_start"][1:].long(), t, right=True)
    return b, t - st["q_start"].long()[b]


def _softmax_product(s, visible, v):
    """s [..., rows, keys] (overwritten), visible broadcastable, v [..., keys, d] -> product, log of the sum."""
    s.masked_fill_(~visible, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v)
    return torch.where(l > 0, o / l, 0.0), (l.log() + m)[..., 0]


def _gathered(st, most):
    """Keys and values of the cache rows 0 .. most - 1 of every sequence, fp32: [nl, B, Hkv, most, d]."""
    c = st["case"]
    j = torch.arange(most, device=GPU).expand(c["batch"], most)
    j = j.minimum((st["page_table"].shape[1] * c["page"] - 1) * torch.ones_like(j))
    at = _rows(st["page_table"], j, c["page"])
    k = st["k_pages"].flatten(1, 2)[:, at].float().transpose(2, 3)
    v = st["v_pages"].flatten(1, 2)[:, at].float().transpose(2, 3)
    return k, v


def _plain_attention(st):
    c = st["case"]
    nl, B, hkv, d = c["nl"], c["batch"], c["hkv"], c["d"]
    G, mq, mk, T = c["hq"] // hkv, st["max_q"], st["max_kv"], st["q"].shape[1]
    start, prefix = st["q_start"].long(), st["prefix_len"].long()
    i = torch.arange(mq, device=GPU)
    tok = (start[:-1, None] + i).clamp_max(T - 1)
    q = st["q"][:, tok].float().view(nl, B, mq, hkv, G, d).permute(0, 1, 3, 4, 2, 5).reshape(nl, B, hkv, G * mq, d)
    k, v = _gathered(st, mk)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).view(nl, B, hkv, G, mq, mk)
    j = torch.arange(mk, device=GPU)
    visible = j < (prefix[:, None] + i + 1)[:, :, None]
    live = (j < (prefix + start[1:] - start[:-1])[:, None])[:, None, :, None]
    v = torch.where(live, v, 0.0)
    o, lse = _softmax_product(s, visible[:, None, None], v[:, :, :, None])
    b, r = _token_of(st, T)
    out = o.permute(1, 4, 0, 2, 3, 5)[b, r].transpose(0, 1).reshape(nl, T, c["hq"], d)
    return out.to(st["q"].dtype), lse.permute(1, 4, 0, 2, 3)[b, r].transpose(0, 1).reshape(nl, T, c["hq"])


def _plain_tree(st):
    c = st["case"]
    nl, B, hkv, d, N = c["nl"], c["batch"], c["hkv"], c["d"], c["nodes"]
    G, mk = c["hq"] // hkv, st["max_kv"]
    q = st["q"].float().view(nl, B, N, hkv, G, d).permute(0, 1, 3, 4, 2, 5).reshape(nl, B, hkv, G * N, d)
    k, v = _gathered(st, mk)
    j = torch.arange(mk, device=GPU)
    live = j < st["prefix_len"].long()[:, None]
    v = torch.where(live[:, None, :, None], v, 0.0)
    k = torch.cat((k, st["kt"].float().transpose(2, 3)), -2)
    v = torch.cat((v, st["vt"].float().transpose(2, 3)), -2)
    n = torch.arange(N, device=GPU)
    seen = (st["mask"][:, n // 32] >> (n % 32)) & 1 == 1
    visible = torch.cat((live[:, None].expand(B, N, mk), seen.expand(B, N, N)), -1)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(d ** -0.5).view(nl, B, hkv, G, N, mk + N)
    o, lse = _softmax_product(s, visible[:, None, None], v[:, :, :, None])
    out = o.permute(0, 1, 4, 2, 3, 5).reshape(nl, B, N, c["hq"], d).to(st["q"].dtype)
    return out, lse.permute(0, 1, 4, 2, 3).reshape(nl, B, N, c["hq"])


def _plain_append(st):
    T, page = st["q"].shape[1], st["case"]["page"]
    b, r = _token_of(st, T)
    row = st["prefix_len"].long()[b] + r
    at = st["page_table"].long()[b, row // page] * page + row % page
    st["k_pages"].flatten(1, 2)[:, at] = _rotate(st["k"], row, st["rope"]).to(st["k"].dtype)
    st["v_pages"].flatten(1, 2)[:, at] = st["v"]
    return _rotate(st["q"], row, st["rope"]).to(st["q"].dtype)


def _plain_compact(st):
    c = st["case"]
    nl, B = c["nl"], c["batch"]
    i = torch.arange(c["depth"] + 1, device=GPU)
    acc, prefix = st["accept_len"].long(), st["prefix_len"].long()
    keep = i < acc[:, None]
    at = _rows(st["page_table"], prefix[:, None] + i.minimum(acc[:, None] - 1), c["page"])
    node = st["path_nodes"].long().clamp_min(0)
    b = torch.arange(B, device=GPU)[:, None]
    for pool, tree in ((st["k_pages"], st["kt"]), (st["v_pages"], st["vt"])):
        flat = pool.flatten(1, 2)
        flat[:, at] = torch.where(keep[:, :, None, None], tree[:, b, node], flat[:, at])
        # a slot past the path points at its last row, which the line above may have left as it was
        last = (acc - 1)[:, None]
        flat[:, at.gather(1, last)] = tree[:, b, node.gather(1, last)]
    return (prefix + acc).to(torch.int32)


def run(st):
    op = st["op"]
    if own:
        import medusa_head_speculative_heads_gb300 as mg
        if op == "rope":
            return mg.medusa_rope(st["q"], st["k"], st["pos"], st["spec"], inverse=st["case"]["inverse"])
        cache = (st["k_pages"], st["v_pages"], st["page_table"])
        if op == "append":
            q = mg.medusa_paged_append(st["k"], st["v"], *cache, st["q_start"], st["prefix_len"], q=st["q"], rope=st["spec"])
            return q, st["k_pages"], st["v_pages"]
        if op == "attn":
            return mg.medusa_paged_attention(st["q"], *cache, st["q_start"], st["prefix_len"], want_lse=True)
        if op == "tree":
            return mg.medusa_paged_tree_attention(st["q"], *cache, st["kt"], st["vt"], st["mask"], st["prefix_len"], want_lse=True)
        n = mg.medusa_paged_compact(*cache, st["kt"], st["vt"], st["path_nodes"], st["accept_len"], st["prefix_len"])
        return n, st["k_pages"], st["v_pages"]
    if op == "rope":
        a, inv, dt = st["rope"], st["case"]["inverse"], st["q"].dtype
        return _rotate(st["q"], st["pos"], a, inv).to(dt), _rotate(st["k"], st["pos"], a, inv).to(dt)
    if op == "append":
        q = _plain_append(st)
        return q, st["k_pages"], st["v_pages"]
    if op == "attn":
        return _plain_attention(st)
    if op == "tree":
        return _plain_tree(st)
    n = _plain_compact(st)
    return n, st["k_pages"], st["v_pages"]


# ----------------------------------------------------------------- in 64 bits

def _exact_turn(x, pos, a, inverse):
    """The rotation as a product of complex numbers."""
    r = a["rotary_dim"]
    h = r // 2
    f = []
    for i in range(h):
        w = a["base"] ** (-2.0 * i / r)
        if a["scaling"] == "linear":
            w /= a["factor"]
        elif a["scaling"] == "bands":
            wave = 2.0 * math.pi / w
            if wave > a["original_len"] / a["low"]:
                w /= a["factor"]
            elif wave >= a["original_len"] / a["high"]:
                t = (a["original_len"] / wave - a["low"]) / (a["high"] - a["low"])
                w = (1.0 - t) * w / a["factor"] + t * w
        elif a["scaling"] == "ramp":
            edge = [r * math.log(a["original_len"] / (2.0 * math.pi * t)) / (2.0 * math.log(a["base"])) for t in (a["high"], a["low"])]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), r - 1)
            t = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            w = w / a["factor"] * t + w * (1.0 - t)
        f.append(w)
    angle = torch.outer(pos.double(), torch.tensor(f, dtype=torch.float64, device=GPU)) * (-1.0 if inverse else 1.0)
    z = torch.polar(torch.full_like(angle, a.get("magnitude", 1.0)), angle)[None, :, None]
    out = x.double().clone()
    if a["interleaved"]:
        p = torch.view_as_complex(out[..., :r].unflatten(-1, (h, 2)).contiguous()) * z
        out[..., :r] = torch.view_as_real(p).flatten(-2)
    else:
        p = torch.complex(out[..., :h].contiguous(), out[..., h:r].contiguous()) * z
        out[..., :h], out[..., h:r] = p.real, p.imag
    return out


def exact(case, seed):
    w = work(case)
    if w["flops"] > 2.5e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return tuple(_exact_turn(st[x], st["pos"], st["rope"], case["inverse"]) for x in ("q", "k"))
    prefix, chunk = _lengths(case)
    nl, ps, d, hkv = case["nl"], case["page"], case["d"], case["hkv"]
    table = st["page_table"].tolist()

    def at(b, n, first=0):
        return torch.tensor([table[b][r // ps] * ps + r % ps for r in range(first, first + n)], dtype=torch.long, device=GPU)

    kf, vf = st["k_pages"].flatten(1, 2), st["v_pages"].flatten(1, 2)
    if op == "append":
        k2, v2, q2, t = kf.double(), vf.double(), [], 0
        for b, (p, c) in enumerate(zip(prefix, chunk)):
            pos, rows = torch.arange(p, p + c, device=GPU), at(b, c, p)
            k2[:, rows] = _exact_turn(st["k"][:, t:t + c], pos, st["rope"], False)
            v2[:, rows] = st["v"][:, t:t + c].double()
            q2.append(_exact_turn(st["q"][:, t:t + c], pos, st["rope"], False))
            t += c
        return torch.cat(q2, 1), k2.view(st["k_pages"].shape), v2.view(st["v_pages"].shape)
    if op == "compact":
        k2, v2, acc = kf.double(), vf.double(), _accepted(case)
        paths = st["path_nodes"].tolist()
        for b, p in enumerate(prefix):
            rows = at(b, acc[b], p)
            k2[:, rows], v2[:, rows] = st["kt"][:, b, paths[b][:acc[b]]].double(), st["vt"][:, b, paths[b][:acc[b]]].double()
        n = torch.tensor([p + a for p, a in zip(prefix, acc)], dtype=torch.int32)
        return n, k2.view(st["k_pages"].shape), v2.view(st["v_pages"].shape)
    G, out = case["hq"] // hkv, torch.zeros(st["q"].shape, dtype=torch.float64, device=GPU)
    lses = torch.zeros(st["q"].shape[:-1], dtype=torch.float64, device=GPU)
    if op == "tree":
        _, seen, _ = _tree(case["nodes"], case["lens"])
        seen = torch.tensor(seen, device=GPU)
    t = 0
    for b, (p, c) in enumerate(zip(prefix, chunk)):
        n = case["nodes"] if op == "tree" else c
        rows = at(b, p if op == "tree" else p + c)
        for l in range(nl):
            for g in range(hkv):
                k, v = kf[l, rows, g].double(), vf[l, rows, g].double()
                if op == "tree":
                    k, v = torch.cat((k, st["kt"][l, b, :, g].double())), torch.cat((v, st["vt"][l, b, :, g].double()))
                    see = torch.cat((torch.ones(n, p, dtype=torch.bool, device=GPU), seen), 1)
                else:
                    see = torch.ones(n, p + n, dtype=torch.bool, device=GPU).tril(p)
                for h in range(g * G, (g + 1) * G):
                    q = (st["q"][l, b, :, h] if op == "tree" else st["q"][l, t:t + n, h]).double()
                    e = (q @ k.T / math.sqrt(d)).masked_fill(~see, -math.inf)
                    z = torch.logsumexp(e, -1)
                    o = torch.exp(e - z[:, None]) @ v
                    if op == "tree":
                        out[l, b, :, h], lses[l, b, :, h] = o, z
                    else:
                        out[l, t:t + n, h], lses[l, t:t + n, h] = o, z
        t += c
    return out, lses
