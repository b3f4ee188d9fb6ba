"""The paged kernels start before the kernel in front of them has ended and wait for it then: what
it may have written (lengths, starts, tables, masks, paths) is not read as data that stays the
same while a kernel lives."""
import glob
import os
import re

from medusa_head_speculative_heads_gb300.build import CSRC


def test_no_load_is_declared_read_only():
    files = glob.glob(os.path.join(CSRC, "paged*.cu")) + glob.glob(os.path.join(CSRC, "paged*.cuh"))
    assert len(files) >= 6
    for f in files:
        code = re.sub(r"//.*", "", open(f).read())
        assert not re.findall(r"__ldg|__ldcs|ld\.global\.nc|__restrict__", code), f
