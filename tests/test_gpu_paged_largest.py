"""Paged compaction of as many rows as its checks let through."""
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
