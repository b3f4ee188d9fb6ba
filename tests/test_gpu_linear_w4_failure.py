"""A wait of the 4-bit linear layer that runs out is reported and ends the kernel; the next call is right."""
import time

import numpy as np
import pytest

from tests.helpers import to_dev
from tests.verify import bf16, check_linear, dev_matrix, matrix

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N", [(64, 512, 300), (200, 2048, 256), (9, 4096, 4100), (40, 1088, 200), (300, 8192, 4096)])
def test_tokens_that_never_come(T, K, N):
    import medusa_head_speculative_heads_gb300 as mg
    from medusa_head_speculative_heads_gb300 import binding as B_
    mg.build()
    rng = np.random.default_rng(0)
    host = bf16(rng, T, K)
    m = matrix(rng, N, K, 64)
    x, (q, s, z) = to_dev(host), dev_matrix(m)
    st, y = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    mg.medusa_linear_w4(x, q, s, z, y=y)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    code = mg.lib().medusa_linear_w4_test_stall(B_._ptr(x), K, B_._ptr(q), B_._ptr(s), B_._ptr(z), T, K, N, 64, B_._ptr(y), 1, B_._ptr(st), B_._stream(None))
    assert code == 0 and mg.medusa_status_check(st) == 3  # TIMEOUT
    assert 0.3 < time.monotonic() - t0 < 5.0
    y.zero_()
    check_linear(mg.medusa_linear_w4(x, q, s, z, y=y, d_status=st), host, m, "bf16")
    assert mg.medusa_status_check(st) == 0
