"""Sizes near 2^31 of the calls around a verify pass's output, on the host: refused from 2^31 - 2^16 on, as the header says, and not
below (where a call without a GPU fails otherwise).  Made-up device addresses: only where no GPU could be launched on them."""
import ctypes

import pytest

import medusa_head_speculative_heads_gb300 as mg
from medusa_head_speculative_heads_gb300 import binding as B_

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    pytest.skip("made-up device addresses", allow_module_level=True)

INVALID = 1
LIMIT = 2 ** 31 - 2 ** 16
SIZES = [LIMIT - 1, LIMIT, 2 ** 31 - 1]


@pytest.fixture(scope="module", autouse=True)
def built():
    mg.build()


def at(n):
    return (n + 1) << 52


@pytest.mark.parametrize("n", SIZES)
def test_features_and_tokens_of_the_vocabulary(n):
    refused = n >= LIMIT
    L, rules = mg.lib(), ctypes.byref(B_.medusa_logits_rules())
    assert (L.medusa_linear_w4(at(0), 32, at(1), at(2), None, 1, 32, n, 32, at(3), 0, None, None) == INVALID) == refused
    assert (L.medusa_w4_quantize(at(0), n, 32, 32, 1, 0, at(1), at(2), None, None) == INVALID) == refused
    assert (L.medusa_logits_process(at(0), n, 0, rules, None, None, 1, 1, n, at(1), None, None) == INVALID) == refused
    assert (L.medusa_count_tokens(at(0), 1, 1, n, at(1), at(2), None, None) == INVALID) == refused
    assert (L.medusa_count_tokens(at(0), 1, n, 1, at(1), at(2), None, None) == INVALID) == refused
    assert (L.medusa_count_accepted(at(0), at(1), at(2), n, 1, 0, 1, at(3), None, None) == INVALID) == refused
    assert (L.medusa_count_accepted(at(0), at(1), at(2), 1, 1, 0, n, at(3), None, None) == INVALID) == refused


@pytest.mark.parametrize("B", SIZES)
@pytest.mark.parametrize("S", [0, 1])
def test_sequences_whose_tokens_are_counted(B, S):
    """The kernel goes through sequences in steps of up to 65535: behind more than these an index would wrap below zero."""
    assert (mg.lib().medusa_count_tokens(at(0), B, S, 1, at(1), at(2), None, None) == INVALID) == (B >= LIMIT)
