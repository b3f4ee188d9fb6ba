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


def division(T, K, N):
    """(kernel, CTAs that share a tile, tokens and features of a tile, tiles, CTAs)"""
    d = (ctypes.c_int32 * 6)()
    assert mg.lib().medusa_linear_w4_test_division(T, K, N, d) == 0
    return list(d)


@pytest.mark.parametrize("T", [65, 10 ** 6 + 1, 2113929153, 2113929217, 2130706433, 2139095041, LIMIT - 65, LIMIT - 1])
@pytest.mark.parametrize("K,N", [(32, 1), (64, 20), (32, 130)])
def test_tokens_of_a_linear_layer(T, K, N):
    """Tiles of the tokens of the longest inputs: as high as the others', and covering all of them."""
    kernel, share, tokens, features, tiles, ctas = division(T, K, N)
    assert kernel in (1, 2) and share in (1, 2, 4, 8) and 1 <= ctas <= 152 * 8 and ctas % share == 0
    assert 16 <= tokens <= (64 if kernel == 1 else 128) and tokens % 16 == 0 and 16 <= features <= (128 if kernel == 1 else 256)
    across = -(-T // tokens)
    assert tiles == across * -(-N // features) and 0 <= across * tokens - T < 16 * across + tokens


def test_a_linear_layer_refuses_more_tokens():
    L = mg.lib()
    for T in SIZES:
        assert (L.medusa_linear_w4(at(0), 32, at(1), at(2), None, T, 32, 1, 32, at(3), 1, None, None) == INVALID) == (T >= LIMIT)
