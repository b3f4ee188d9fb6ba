"""The paged calls refuse numbers of sequences that a block's threads cannot count past, and status words
that lie across words (no GPU needed)."""
import ctypes

import pytest

import medusa_head_speculative_heads_gb300 as mg

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("made-up device addresses: only where no GPU could be launched on them", allow_module_level=True)

INVALID = 1


def at(n):
    return n << 44  # far apart: nothing overlaps


def calls(B, status=None):
    L, F = mg.lib(), ctypes.c_float(0.1)
    yield L.medusa_paged_append(None, 0, at(2), 64, at(3), 64, None, None, at(4), at(5), at(6), 1, 4, B, 0, 1, 64, 9, 16, 1, 1, None, at(7), at(8), status, None)
    yield L.medusa_paged_attention(at(1), 64, at(2), at(3), at(4), at(5), at(6), 1, 4, B, 1, 1, 64, 9, 16, 1, F, 1, at(7), None, at(8), 1 << 40, status, None)
    yield L.medusa_paged_tree_attention(at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), 1, B, 1, 1, 1, 64, 9, 16, 1, F, 1, at(9), None, at(10), 1 << 40, status, None)
    yield L.medusa_paged_compact(at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), 1, B, 1, 1, 64, 9, 16, 1, 0, 1, status, None)


@pytest.mark.parametrize("B", [2 ** 31 - 1, 2 ** 31 - 300, 2 ** 31 - 2 ** 16 - 1])
def test_too_many_sequences_are_refused(B):
    mg.build()
    assert list(calls(B)) == [INVALID] * 4


def test_fewer_are_not():
    """Nothing is launched here: without a GPU the calls end at their first CUDA call."""
    mg.build()
    assert INVALID not in list(calls(2 ** 31 - 2 ** 16 - 2))[:3]
    assert INVALID not in list(calls(2 ** 30 - 1))[3:]  # rows of work: B x 2 < 2^31


@pytest.mark.parametrize("off", [1, 2, 3])
def test_a_status_word_across_words_is_refused(off):
    mg.build()
    assert list(calls(3, at(12) + off)) == [INVALID] * 4
    assert INVALID not in list(calls(3, at(12)))
