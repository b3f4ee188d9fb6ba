"""Failure detection of the paged attention on tensor cores, without a fault: its values are
never loaded, its bounded waits run out, every role stops, and the context stays usable."""
import ctypes
import time

import numpy as np
import pytest

from oracle import paged as ref
from tests.helpers import bf16_to_f64, to_dev, to_host
from tests.paged import dev_ints, pool, starts, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TIMEOUT = 3


@pytest.fixture(scope="module")
def mg():
    import medusa_head_speculative_heads_gb300 as m
    m.build()
    return m


# blocks of one row tile (64 and 128 columns), and of two
@pytest.mark.parametrize("c", [dict(hq=4, hkv=2, d=128, prefix=[300, 7], chunk=[1, 1]), dict(hq=2, hkv=1, d=64, prefix=[130], chunk=[2]),
                               dict(hq=4, hkv=1, d=128, prefix=[200], chunk=[150])], ids=lambda c: f"d{c['d']}-{max(c['chunk'])}")
def test_waits_run_out_and_the_next_call_is_right(mg, c):
    rng = np.random.default_rng(5)
    kp, vp, table = pool(rng, [p + n for p, n in zip(c["prefix"], c["chunk"])], nl=1, page=16, hkv=c["hkv"], d=c["d"], dtype="bf16")
    q0 = starts(c["chunk"])
    T, B, d = int(q0[-1]), len(c["chunk"]), c["d"]
    q = values(rng, (1, T, c["hq"], d), "bf16")
    dq, dk, dv, ints = to_dev(q), to_dev(kp), to_dev(vp), [dev_ints(x) for x in (table, q0, c["prefix"])]
    n = mg.lib().medusa_paged_attention_workspace_size(1, T, B, c["hq"], c["hkv"], d, 16, 1)
    ws, out = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.empty_like(dq)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    code = mg.lib().medusa_paged_attention_test_stall(
        dq.data_ptr(), c["hq"] * d, dk.data_ptr(), dv.data_ptr(), *(x.data_ptr() for x in ints), 1, T, B, c["hq"], c["hkv"], d, kp.shape[1], 16,
        table.shape[1], ctypes.c_float(d ** -0.5), 1, out.data_ptr(), None, ws.data_ptr(), n, st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    assert code == 0 and mg.medusa_status_check(st) == TIMEOUT
    assert 0.04 < waited < 5.0  # the waits' own bound: neither at once nor a hang
    got, _ = mg.medusa_paged_attention(dq, dk, dv, *ints, d_status=st)
    assert mg.medusa_status_check(st) == 0
    want, _, _ = ref.paged_attention(q, kp, vp, table, q0, c["prefix"])
    g = bf16_to_f64(to_host(got))
    assert np.linalg.norm(g - want) <= 2.0 ** -8 * np.linalg.norm(want)
