"""The division by a reciprocal that the rotation splits its work with (csrc/divide.h),
compiled for the host: equal to a division wherever x n < 2^31."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from medusa_head_speculative_heads_gb300.build import CSRC

SOURCE = """
#include "divide.h"
extern "C" uint32_t divided(uint32_t x, uint32_t n) { return medusa::quotient(x, medusa::reciprocal(n)); }
"""


@pytest.fixture(scope="module")
def divided(tmp_path_factory):
    at = tmp_path_factory.mktemp("divide")
    src, out = at / "divided.cpp", at / "divided.so"
    src.write_text(SOURCE)
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(out)], check=True)
    f = ctypes.CDLL(str(out)).divided
    f.argtypes, f.restype = [ctypes.c_uint32] * 2, ctypes.c_uint32
    return f


def test_tasks_of_a_cta(divided):
    """Up to 128 tasks of several tokens, for every number of tasks a token can have: one, too."""
    for n in range(1, 129):
        assert [divided(x, n) for x in range(128)] == [x // n for x in range(128)], n


def test_up_to_the_stated_limit(divided):
    rng = np.random.default_rng(1)
    for n in (1, 2, 3, 5, 7, 16, 40, 100, 127, 128, 65535, 65536, (1 << 31) - 1):
        most = ((1 << 31) - 1) // n
        for x in {0, 1, most, max(most - 1, 0), min(n - 1, most), *(int(v) for v in rng.integers(0, most + 1, 200))}:
            assert divided(x, n) == x // n, (x, n)
