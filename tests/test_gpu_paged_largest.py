"""Paged compaction of as many rows as its checks let through, attention of very many sequences."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_compaction_of_almost_two_to_the_31_rows():
    """A path slot of K or V is a row of work: 2 x 17 of them for each of 63161283 sequences, 25 short of 2^31."""
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    B = 63161283
    assert 2 ** 31 - 2432 < B * 34 < 2 ** 31
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(B - 1, -1, -1, **i32).view(B, 1)
    tree = torch.arange(B, **i32).to(torch.int16).view(torch.bfloat16).view(1, B, 1, 1, 1)  # any bits: rows are moved, not computed
    k, v = (torch.zeros((1, B, 1, 1, 1), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    acc, prefix, path, st = torch.ones(B, **i32), torch.zeros(B, **i32), torch.zeros((B, 17), **i32), torch.zeros(1, **i32)
    other = (tree.view(torch.int16) ^ 1).view(torch.bfloat16)
    n = mg.medusa_paged_compact(k, v, table, tree, other, path, acc, prefix, d_status=st)
    assert mg.medusa_status_check(st) == 0
    assert torch.all(n == 1)
    assert torch.equal(k.view(torch.int16).flip(1), tree.view(torch.int16)) and torch.equal(v.view(torch.int16).flip(1), other.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_three_million_sequences_without_tokens(dtype):
    """Two have some, the first and the last, and one CTA works on both: nobody gives up waiting for it."""
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    B, rows, dt = 3000001, 60000, torch.bfloat16 if dtype == "bf16" else torch.float32
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((1, 64, 1024, 1, 64), generator=g, device="cuda").to(dt) for _ in range(2))
    q = torch.randn((1, 2, 1, 64), generator=g, device="cuda").to(dt)
    q0 = torch.ones(B + 1, **i32)
    q0[0], q0[B] = 0, 2
    prefix, table, st = torch.zeros(B, **i32), torch.full((B, 64), -1, **i32), torch.zeros(1, **i32)
    prefix[0], prefix[B - 1] = 5, rows
    table[0, 0] = 63
    table[B - 1, :60] = torch.arange(60, **i32)
    many, lse = mg.medusa_paged_attention(q, k, v, table, q0, prefix, want_lse=True, d_status=st)
    assert mg.medusa_status_check(st) == 0
    two = torch.tensor([0, B - 1], device="cuda")
    few, lse2 = mg.medusa_paged_attention(q, k, v, table[two].contiguous(), q0[[0, 1, B]].contiguous(), prefix[two].contiguous(), want_lse=True, d_status=st)
    assert mg.medusa_status_check(st) == 0
    assert torch.equal(many, few) and torch.equal(lse, lse2)
