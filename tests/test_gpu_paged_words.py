"""Calls in a row on one stream, each of which reads the lengths, the paths or the mask that the one in
front of it writes: as when each is waited for."""
import numpy as np
import pytest

from oracle import paged as ref
from tests.helpers import to_dev, to_host
from tests.paged import dev_ints, pool, values

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_whose_lengths_the_step_before_writes(dtype):
    import medusa_head_speculative_heads_gb300 as mg
    mg.build()
    rng = np.random.default_rng(3)
    B, N, steps, d, first = 3, 12, 50, 64, [5, 0, 17]
    kp, vp, table = pool(rng, [n + 4 * steps for n in first], nl=2, page=16, hkv=1, d=d, dtype=dtype)
    kp, vp = values(rng, kp.shape, dtype), values(rng, vp.shape, dtype)
    q, kt, vt = (to_dev(values(rng, (2, B, N, h, d), dtype)) for h in (2, 1, 1))
    mask = torch.zeros((N, 1), dtype=torch.int32, device="cuda")
    seen = dev_ints([[(1 << (i + 1)) - 1] for i in range(N)])
    paths = [dev_ints([rng.choice(N, 4, replace=False) for _ in range(B)]) for _ in range(steps)]
    accepted = [dev_ints(rng.integers(1, 5, B)) for _ in range(steps)]

    def run(wait):
        k, v, prefix, outs = to_dev(kp), to_dev(vp), dev_ints(first), []
        path, acc, tab, st = dev_ints(np.zeros((B, 4))), dev_ints(np.zeros(B)), dev_ints(table), torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(steps):
            mask.zero_()
            mask.copy_(seen)
            path.copy_(paths[i])
            acc.copy_(accepted[i])
            for call in (lambda: outs.append(mg.medusa_paged_tree_attention(q, k, v, tab, kt, vt, mask, prefix, d_status=st)[0]),
                         lambda: mg.medusa_paged_compact(k, v, tab, kt, vt, path, acc, prefix, new_len=prefix, d_status=st),
                         lambda: outs.append(mg.medusa_paged_tree_attention(q, k, v, tab, kt, vt, mask, prefix, d_status=st)[0])):
                call()
                if wait:
                    torch.cuda.synchronize()
        assert mg.medusa_status_check(st) == 0
        return k, v, prefix, outs

    a, b = run(True), run(False)
    assert a[2].tolist() == [n + sum(int(x[i]) for x in accepted) for i, n in enumerate(first)] == b[2].tolist()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(a[3], b[3]):
        assert torch.equal(x, y)
    want, _, _ = ref.paged_tree_attention(to_host(q), to_host(b[0]), to_host(b[1]), table, to_host(kt), to_host(vt), to_host(seen), b[2].tolist())
    g = b[3][-1].double().cpu().numpy()
    assert np.linalg.norm(g - want) <= (2.0 ** -8 if dtype == "bf16" else 2e-6) * np.linalg.norm(want)
