"""The bounds of the paged attention's waits, from its source, and the refusals of its failure test."""
import ctypes
import os
import re

import pytest

import medusa_head_speculative_heads_gb300 as mg
from medusa_head_speculative_heads_gb300.build import CSRC

# Measured on a GB300: a try that sleeps takes 1.3 us (it wakes by itself), a poll of a warp's lanes 108 ns
# (2^26 of them 7.26 s).
TRY_S, POLL_S = 1.3e-6, 108e-9


def test_waits_end_within_two_seconds():
    src = open(os.path.join(CSRC, "paged_attention_tc.cu")).read()
    n = {k: 1 << int(v) for k, v in re.findall(r"constexpr int (kTries|kPolls) = 1 << (\d+);", src)}
    assert 0.5 < n["kTries"] * TRY_S < 2.0 and 0.5 < n["kPolls"] * POLL_S < 2.0
    loops = re.findall(r"for \(int n = ([^;]+); n > 0; --n\)", src)
    assert sorted(loops) == ["kPolls", "kTries"]


def test_the_stalled_call_is_of_tensor_core_shapes():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("made-up device addresses: only where no GPU could be launched on them")
    mg.build()
    at = lambda n: (n + 1) << 28  # noqa: E731

    def call(d=64, page=16, dt=1, q=at(0)):
        return mg.lib().medusa_paged_attention_test_stall(q, 2 * d, at(1), at(2), at(3), at(4), at(5), 1, 4, 1, 2, 1, d, 9, page, 4, ctypes.c_float(0.1), dt, at(6),
                                                          None, at(7), 1 << 27, None, None)
    for bad in (dict(d=256), dict(page=5), dict(dt=0), dict(q=None), dict(q=at(0) + 8)):
        assert call(**bad) == 1
